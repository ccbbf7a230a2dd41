// 8-bit integer products with a scale for each token and each channel:
//
//   y[t][n] = s_t s_n (sum_k q[t][k] w[n][k] - z_n sum_k q[t][k]) + b_n
//
// and the gated pair act(gate) * up of two such products over the same
// tokens.  The sums are exact 32-bit integers (in <= 32768, so the largest is
// below 1.7e9); one conversion to fp32, three fp32 operations and the output
// conversion are the only roundings.
//
// split kernel: the weights' channels are the tensor core's 128 rows (tensor-
// memory lanes), the tokens its columns (16 to 256, gated to 128), so a handful
// of tokens still streams the weights through full-height MMAs.  The CTAs of a
// cluster split k; each pushes its partial sums through distributed shared memory to
// the CTA that adds and writes that share of the tokens.  Integer addition makes
// the result independent of the split, and no workspace or atomic is needed.
//   warp 0     TMA producer
//   warp 1     tensor memory, tcgen05.mma.kind::i8
//   warps 2-9  epilogue, or their partial sums into the shared memory of the
//              rank that finishes the token, then that rank's epilogue
// Every wait is bounded; a wait that gives up raises ST_TIMEOUT in the
// library's int8 status word, and the CTA drains and leaves.
//
// What bounds it: for a few tokens the weights' way from memory and, in short
// products, the fixed parts (set-up and first load 2.5 us, epilogue 1.3 to 2).
// So the weights' first stages are on their way before anything else, and
// behind the quantizer while that still runs.  24 tokens of 11008 > 4096 from
// fp16 take 13.5 us with the quantizer, the weights' bytes alone 7.  For a few
// hundred tokens what one SM takes in, 171 GB/s, on fewer SMs than there are:
// 333 tokens of 4096 > 4096, 11.1 us, run on 96 CTAs that load 0.98 MB each,
// 5.8 us of it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "gemm.cuh"
#include "int8.cuh"
#include "internal.cuh"

namespace gptq {
namespace {

constexpr int kEpilogue = 256;           // threads of the epilogue: two warps a tensor-memory quarter
constexpr int kThreads = 64 + kEpilogue;
constexpr int kBK = 128;                 // int8 elements of k per stage row (128-byte swizzle)
constexpr int kTileM = 128;              // channels of a tile
constexpr int kTileBytes = kTileM * kBK;
constexpr int kMaxSplit = 8;             // portable cluster size
constexpr int kMaxNTile = 256;           // tokens of a tile
constexpr int kSmem = 232448, kSmemFixed = 1024 + 2 * 4 * kMaxNTile + 256;

// Raised by bounded waits that gave up, read and cleared by gptq_int8_status.
__device__ uint32_t g_int8_status;

struct MmParams {
  const float* tscale;
  const int32_t* tsum;
  const float* wscale[2];  // [1]: the up projection of a gated pair
  const int32_t* wzero[2];
  const float* bias;
  void* Y;
  int64_t ldy;
  int tokens, out, in;
  int act;
  int vec;  // rows of Y start on 16-byte boundaries
  int ktiles, split, ntile, stages, stage_bytes, push_bytes, tmem_cols, ctiles;
};

struct SplitMaps {
  CUtensorMap w[2];
  CUtensorMap x;
};

// ----------------------------------------------------------------- pieces
__device__ __forceinline__ void st_cluster(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// ------------------------------------------------------------ split kernel
template <int G, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    int8_split_kernel(const __grid_constant__ SplitMaps maps, const __grid_constant__ MmParams kp) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  // partial sums pushed by the cluster, [source rank][g][token of this rank's share][channel]
  int* pushed = (int*)(smem + (size_t)kp.stages * kp.stage_bytes);
  float* tscale = (float*)((uint8_t*)pushed + kp.push_bytes);  // [ntile]
  int* tsum = (int*)(tscale + kMaxNTile);
  uint64_t* full = (uint64_t*)(tsum + kMaxNTile);
  uint64_t* empty = full + kp.stages;
  uint64_t* acc_full = empty + kp.stages;
  uint64_t* drain = acc_full + 1;
  uint32_t* tmem_slot = (uint32_t*)(drain + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);

  const int warp = uniform_warp();
  const int lane = threadIdx.x & 31;
  const int split = kp.split;
  const int rank = split > 1 ? (int)cluster_rank() : 0;
  const int tile = (int)blockIdx.x / split;
  const int n0 = (tile % kp.ctiles) * kTileM;
  const int t0 = (tile / kp.ctiles) * kp.ntile;
  const int kt0 = (int)((int64_t)kp.ktiles * rank / split), kt1 = (int)((int64_t)kp.ktiles * (rank + 1) / split);
  const int ntile = kp.ntile;

  const int ahead = min(kp.stages, kt1 - kt0);  // k-tiles that need not wait for a free stage
  const uint32_t bytes = (uint32_t)(G * kTileBytes + ntile * kBK);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kp.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    // The weights do not come from the kernel before this one: the first
    // stages' are on their way while the rest is set up and the tokens are
    // quantized.
    for (int i = 0; i < ahead; ++i) {
      mbar_arrive_expect_tx(&full[i], bytes);
#pragma unroll
      for (int g = 0; g < G; ++g)
        tma_load_2d(smem + (size_t)i * kp.stage_bytes + g * kTileBytes, &maps.w[g], &full[i], (kt0 + i) * kBK, n0);
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, (uint32_t)kp.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  // first phase of the cluster's barrier: every CTA has begun, its shared
  // memory can be written to
  if (split > 1) cluster_arrive();

  const uint32_t stage0 = smem_u32(smem), full0 = smem_u32(full), empty0 = smem_u32(empty);
  if (warp == 0) {
    const uint32_t leader = elect_lane();
    const int stages = kp.stages, stage_bytes = kp.stage_bytes;
    grid_dependency_wait();
    for (int i = 0; i < ahead; ++i)
      tma_load_at(leader, stage0 + i * stage_bytes + G * kTileBytes, &maps.x, full0 + 8 * i, (kt0 + i) * kBK, t0);
    int stage = 0;
    uint32_t phase = 0, at = stage0;
    for (int x = (kt0 + ahead) * kBK; x < kt1 * kBK; x += kBK) {
      if (!wait_at(empty0 + 8 * stage, phase)) {
        raise_status(&g_int8_status, ST_TIMEOUT);
        *abort_flag = 1;
        break;
      }
      expect_at(leader, full0 + 8 * stage, bytes);
#pragma unroll
      for (int g = 0; g < G; ++g) tma_load_at(leader, at + g * kTileBytes, &maps.w[g], full0 + 8 * stage, x, n0);
      tma_load_at(leader, at + G * kTileBytes, &maps.x, full0 + 8 * stage, x, t0);
      at += stage_bytes;
      if (++stage == stages) {
        stage = 0;
        at = stage0;
        phase ^= 1;
      }
    }
    __syncwarp();
    if (split > 1) cluster_wait();
  } else if (warp == 1) {
    const uint32_t leader = elect_lane();
    const int stages = kp.stages;
    const uint32_t idesc = idesc_i8(kTileM, (uint32_t)ntile);
    const uint32_t a0 = desc_low(stage0), b0 = desc_low(stage0 + G * kTileBytes);
    const uint32_t desc_step = (uint32_t)kp.stage_bytes >> 4;
    int stage = 0;
    uint32_t phase = 0, at = 0;
    bool ok = true;
    for (int kt = kt0; kt < kt1; ++kt) {
      if (!wait_at(full0 + 8 * stage, phase)) {
        raise_status(&g_int8_status, ST_TIMEOUT);
        *abort_flag = 1;
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < kBK / 32; ++kk)
#pragma unroll
        for (int g = 0; g < G; ++g)
          umma_i8<1>(leader, tbase + (uint32_t)(g * ntile), a0 + at + g * (kTileBytes >> 4) + 2 * kk, b0 + at + 2 * kk, idesc,
                     kk > 0 ? 1u : (uint32_t)(kt > kt0));
      commit_at(leader, empty0 + 8 * stage);
      at += desc_step;
      if (++stage == stages) {
        stage = 0;
        at = 0;
        phase ^= 1;
      }
    }
    if (ok) commit_at(leader, smem_u32(acc_full));
    __syncwarp();
    if (split > 1) cluster_wait();
  } else {
    const int quarter = warp & 3, second = (warp - 2) / 4, e = threadIdx.x - 64;
    const int c = quarter * 32 + lane;
    const uint32_t tmem = tbase + ((uint32_t)(quarter * 32) << 16);
    // Everything the epilogue reads from memory is fetched under the main
    // loop.  A thread's channels: its lane of tensor memory, or four of a
    // row where the sums come from shared memory.
    constexpr int V = 4;
    const int n = n0 + (split > 1 ? V * lane : c);
    float ws[G][V], bias[V];
    int wz[G][V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool in = n + i < kp.out && (split > 1 || i == 0);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        ws[g][i] = in ? __ldg(kp.wscale[g] + n + i) : 0.f;
        wz[g][i] = in && kp.wzero[g] ? __ldg(kp.wzero[g] + n + i) : 0;
      }
      bias[i] = G == 1 && in && kp.bias ? __ldg(kp.bias + n + i) : 0.f;
    }
    grid_dependency_wait();
    for (int j = e; j < ntile; j += kEpilogue) {
      const bool in = t0 + j < kp.tokens;
      tscale[j] = in ? kp.tscale[t0 + j] : 0.f;
      tsum[j] = in ? kp.tsum[t0 + j] : 0;
    }
    named_bar_sync(1, kEpilogue);
    const int live = min(ntile, kp.tokens - t0);  // tokens of the tile inside the result
    if (!mbar_wait_sleep(acc_full, 0)) {
      raise_status(&g_int8_status, ST_TIMEOUT);
      *abort_flag = 1;
    }
    __syncwarp();
    tc_fence_after();
    // sixteen tokens at a time, the quarter's two warps in turn
    if (split == 1) {
      // a token at a time, 32 neighbouring channels a warp
      const bool zeros = kp.wzero[0] || (G == 2 && kp.wzero[1]);
      const Pair w0(ws[0][0]), w1(ws[G - 1][0]), b(bias[0]);
      auto scale = [&](const float* v, const Pair& w, int z, int j, Pair* y) {  // four tokens
        int a[4] = {__float_as_int(v[0]), __float_as_int(v[1]), __float_as_int(v[2]), __float_as_int(v[3])};
        if (zeros) {
          const int4 sum = *reinterpret_cast<const int4*>(tsum + j);
          a[0] -= z * sum.x;
          a[1] -= z * sum.y;
          a[2] -= z * sum.z;
          a[3] -= z * sum.w;
        }
        const float4 t = *reinterpret_cast<const float4*>(tscale + j);
        y[0] = mul2(mul2(Pair((float)a[0], (float)a[1]), Pair(t.x, t.y)), w);
        y[1] = mul2(mul2(Pair((float)a[2], (float)a[3]), Pair(t.z, t.w)), w);
      };
#pragma unroll 1
      for (int j0 = 16 * second; j0 < live; j0 += 32) {
        float v[G][16];
        Pair y[8];
#pragma unroll
        for (int g = 0; g < G; ++g) tmem_ld16(tmem + (uint32_t)(g * ntile + j0), v[g]);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          scale(v[0] + i, w0, wz[0][0], j0 + i, y + i / 2);
          if (G == 2) {
            Pair u[2];
            scale(v[G - 1] + i, w1, wz[G - 1][0], j0 + i, u);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float2 f = y[i / 2 + k].f();
              y[i / 2 + k] = mul2(Pair(activate(f.x, kp.act), activate(f.y, kp.act)), u[k]);
            }
          } else {
            y[i / 2] = add2(y[i / 2], b);
            y[i / 2 + 1] = add2(y[i / 2 + 1], b);
          }
        }
        T* col = (T*)kp.Y + (int64_t)(t0 + j0) * kp.ldy + n;
        const int left = n < kp.out ? live - j0 : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = y[i].f();
          if (2 * i < left) col[0] = from_f32<T>(f.x);
          if (2 * i + 1 < left) col[kp.ldy] = from_f32<T>(f.y);
          col += 2 * kp.ldy;
        }
      }
      tc_fence_before();
    } else {
      // each token's sums go to the rank that finishes it
      cluster_wait();
      const int share = ntile / split;
#pragma unroll 1
      for (int j0 = 16 * second; j0 < ntile; j0 += 32) {
        int owner = j0 / share, j = j0 - owner * share;
        uint32_t at = map_to_rank(smem_u32(pushed + (rank * G * share) * kTileM + c), (uint32_t)owner);
        float v[G][16];
#pragma unroll
        for (int g = 0; g < G; ++g) tmem_ld16(tmem + (uint32_t)(g * ntile + j0), v[g]);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
#pragma unroll
          for (int g = 0; g < G; ++g)
            st_cluster(at + (uint32_t)((g * share + j) * kTileM * 4), __float_as_int(v[g][i]));
          if (++j == share) {
            j = 0;
            at = map_to_rank(smem_u32(pushed + (rank * G * share) * kTileM + c), (uint32_t)min(++owner, split - 1));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      cluster_arrive();  // second phase: all partial sums are in place
      cluster_wait();
#pragma unroll 1
      for (int j = warp - 2; j < share; j += kEpilogue / 32) {
        const int at = rank * share + j;
        if (at >= live) break;
        int4 part[G][kMaxSplit];
#pragma unroll
        for (int r = 0; r < kMaxSplit; ++r)
#pragma unroll
          for (int g = 0; g < G; ++g)
            part[g][r] = r < split ? *reinterpret_cast<const int4*>(pushed + ((r * G + g) * share + j) * kTileM + V * lane)
                                   : make_int4(0, 0, 0, 0);
        int acc[G][V];
#pragma unroll
        for (int g = 0; g < G; ++g) {
          int4 sum = part[g][0];
#pragma unroll
          for (int r = 1; r < kMaxSplit; ++r) {
            sum.x += part[g][r].x;
            sum.y += part[g][r].y;
            sum.z += part[g][r].z;
            sum.w += part[g][r].w;
          }
          acc[g][0] = sum.x;
          acc[g][1] = sum.y;
          acc[g][2] = sum.z;
          acc[g][3] = sum.w;
        }
        alignas(16) T o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float y = scaled(acc[0][i], wz[0][i], tsum[at], tscale[at], ws[0][i]);
          if (G == 2)
            y = activate(y, kp.act) * scaled(acc[G - 1][i], wz[G - 1][i], tsum[at], tscale[at], ws[G - 1][i]);
          else
            y += bias[i];
          o[i] = from_f32<T>(y);
        }
        T* dst = (T*)kp.Y + (int64_t)(t0 + at) * kp.ldy + n;
        if (kp.vec && n + V <= kp.out) {
          if (sizeof(T) == 2)
            *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(o);
          else
            *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(o);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (n + i < kp.out) dst[i] = o[i];
        }
      }
    }
  }
  if (split > 1 && warp < 2) {
    cluster_arrive();
    cluster_wait();
  }
  grid_dependency_wait();
  __syncthreads();
  if (*abort_flag) {
    // let copies and MMAs already issued finish before the memory goes away
    if (warp == 1) {
      commit_at(elect_lane(), smem_u32(drain));
      mbar_wait(drain, 0);
    }
    if (threadIdx.x == 0) let_copies_land();
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, (uint32_t)kp.tmem_cols);
  }
}

// ------------------------------------------------------------------- plan
// Which kernel takes a product, and in which tiles.
struct Plan {
  bool pair;
  int bn;            // pair kernel: channels of a tile
  int ntile, split;  // split kernel: tokens of a tile, CTAs that share its k
};

// The estimates below choose among the tilings of both kernels.  Microseconds,
// from 220 products of 3 to 2600 tokens with in and out from 300 to 20000,
// each timed in up to 30 tilings: the tiling they choose takes on average
// 1.008 times the best one's time (at worst 1.24), one fixed tiling 1.2 to 2
// times.  G: products that share the tokens.
//
// A pair's k-tile takes the larger of its MMAs (0.30, or 0.25 with 128
// channels) and its share of what L2 delivers (16 TB/s); only the last tile's
// epilogue shows, unless a tile's main loop is shorter.
float pair_us(int G, int64_t tokens, int64_t ktiles, int64_t out, int bn, int sms) {
  const int64_t tiles = (tokens + 255) / 256 * ((out + bn / G - 1) / (bn / G));
  const int64_t pairs = std::min<int64_t>(tiles, sms / 2), waves = (tiles + sms / 2 - 1) / (sms / 2);
  const float ktile = std::max(bn == 256 ? 0.30f : 0.25f, 2.f * (16384 + bn * 64) * pairs / 16e6f);
  const float epilogue = bn == 256 ? 5.5f : 3.5f;
  return 2.9f + epilogue + waves * ktiles * ktile + (waves - 1) * std::max(0.f, epilogue - ktiles * ktile);
}

// A CTA's k-tile: issuing it (0.11), its MMAs, its share of L2, or what one SM
// takes in (171 GB/s).  Clusters of four and eight cannot fill every GPC: 132
// and 104 of their CTAs fit at once.  Partial sums cost their way to the other
// CTAs.
float split_us(int G, int64_t tokens, int64_t ktiles, int64_t out, int ntile, int split, int sms) {
  const int64_t ctas = (out + kTileM - 1) / kTileM * ((tokens + ntile - 1) / ntile) * split;
  const int64_t fit = split == 4 ? sms * 132 / 148 : split == 8 ? sms * 104 / 148 : sms;
  const int64_t waves = (ctas + fit - 1) / fit, k = (ktiles + split - 1) / split;
  const float bytes = (float)(G * kTileBytes + ntile * kBK);
  const float ktile = std::max(std::max(0.11f, G * ntile * 1.4e-3f),
                               bytes * std::max(std::min<int64_t>(ctas, sms) / 16e6f, 1 / 171e3f));
  const float epilogue = split == 1 ? 1.6f + 0.011f * ntile * (G == 2 ? 2.5f : 1.f)
                                    : 2.6f + 0.024f * ntile * (G == 2 ? 1.3f : 1.f);
  return 2.6f + waves * (k * ktile + epilogue);
}

int stages_of(int G, int ntile, int split) {
  return (kSmem - kSmemFixed - (split > 1 ? G * ntile * kTileM * 4 : 0)) / (G * kTileBytes + ntile * kBK);
}

Plan make_plan(int G, int64_t tokens, int64_t in, int64_t out, int sms) {
  const int64_t ktiles = (in + kBK - 1) / kBK;
  const int most = kMaxNTile / G;  // tokens of a tile that tensor memory and registers take
  Plan best = {};
  float best_us = 1e30f;
  auto offer = [&](const Plan& p, float us) {
    if (us < best_us) best = p, best_us = us;
  };
  // tiles of 64, 128 and 256 tokens, and those that divide the tokens evenly
  // into up to four
  const int64_t round = (tokens + 15) / 16 * 16;
  for (int i = 0; i < 7; ++i) {
    const int64_t ntile = i < 3 ? std::min<int64_t>(round, 64 << i) : ((tokens + i - 3) / (i - 2) + 15) / 16 * 16;
    if (ntile > most) continue;
    for (int split = 1; split <= kMaxSplit; split *= 2) {
      if (split > 1 && (ktiles < 2 * split || stages_of(G, (int)ntile, split) < 3)) break;
      offer({false, 0, (int)ntile, split}, split_us(G, tokens, ktiles, out, (int)ntile, split, sms));
    }
  }
  if (tokens > 64)  // a pair's tile has 256 tokens
    for (int bn = 128; bn <= 256; bn *= 2) offer({true, bn, 0, 0}, pair_us(G, tokens, ktiles, out, bn, sms));
  return best;
}

// ------------------------------------------------------------------- host
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = (EncodeTiledFn)p;
  });
  return fn;
}

}  // namespace

// A K-major int8 operand (rows x in, row stride ld bytes) in boxes of
// box_rows rows by 128 bytes; what lies past the matrix reads as zero.
bool int8_map(CUtensorMap* m, const int8_t* base, int64_t rows, int64_t in, int64_t ld, int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t gdim[2] = {(cuuint64_t)in, (cuuint64_t)rows};
  cuuint64_t gstride[1] = {(cuuint64_t)ld};
  cuuint32_t box[2] = {(cuuint32_t)kBK, (cuuint32_t)box_rows};
  cuuint32_t estride[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(base), gdim, gstride, box, estride,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

template <int G, typename T>
cudaError_t launch_split(const SplitMaps& maps, const MmParams& kp, int64_t tiles, bool follows, cudaStream_t st) {
  const void* f = (const void*)int8_split_kernel<G, T>;
  cudaError_t e = ensure_smem_limit(f, 232448);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * kp.split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)kSmemFixed + (size_t)kp.stages * kp.stage_bytes + kp.push_bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)kp.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.numAttrs = kp.split > 1 ? 1 : 0;
  cfg.attrs = attr;
  if (follows) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  e = cudaLaunchKernelEx(&cfg, int8_split_kernel<G, T>, maps, kp);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int G>
cudaError_t run_split(MmParams kp, const gptq_int8_tokens_t* x, const gptq_int8_layer_t* const (&w)[2],
                      gptq_dtype_t yt, const Plan& plan, bool follows, cudaStream_t st) {
  kp.ntile = plan.ntile;
  kp.split = plan.split;
  kp.ctiles = (kp.out + kTileM - 1) / kTileM;
  kp.ktiles = (kp.in + kBK - 1) / kBK;
  const int64_t tiles = (int64_t)kp.ctiles * ((kp.tokens + kp.ntile - 1) / kp.ntile);
  kp.stage_bytes = G * kTileBytes + kp.ntile * kBK;
  kp.push_bytes = kp.split > 1 ? G * kp.ntile * kTileM * 4 : 0;
  kp.tmem_cols = 32;
  while (kp.tmem_cols < G * kp.ntile) kp.tmem_cols *= 2;
  // The stages fill shared memory, so no two CTAs of these kernels share an
  // SM: a CTA that waits for tensor memory held by another could otherwise
  // hold up that one's cluster.
  kp.stages = std::min(12, stages_of(G, kp.ntile, kp.split));
  SplitMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  for (int g = 0; g < G; ++g)
    if (!int8_map(&maps.w[g], w[g]->w, kp.out, kp.in, w[g]->ldw, kTileM)) return cudaErrorInvalidValue;
  if (!int8_map(&maps.x, x->q, kp.tokens, kp.in, x->ldq, kp.ntile)) return cudaErrorInvalidValue;
  switch (yt) {
    case GPTQ_F16:
      return launch_split<G, __half>(maps, kp, tiles, follows, st);
    case GPTQ_BF16:
      return launch_split<G, __nv_bfloat16>(maps, kp, tiles, follows, st);
    default:
      return launch_split<G, float>(maps, kp, tiles, follows, st);
  }
}

template <int G>
cudaError_t run(const gptq_int8_tokens_t* x, int64_t tokens, int64_t in, const gptq_int8_layer_t* const (&w)[2],
                int64_t out, const float* bias, int act, void* Y, gptq_dtype_t yt, int64_t ldy, const Plan& plan,
                bool follows, cudaStream_t st) {
  MmParams kp = {};
  kp.tscale = x->scale;
  kp.tsum = x->sum;
  for (int g = 0; g < G; ++g) {
    kp.wscale[g] = w[g]->scale;
    kp.wzero[g] = w[g]->zero;
  }
  kp.bias = bias;
  kp.Y = Y;
  kp.ldy = ldy;
  kp.tokens = (int)tokens;
  kp.out = (int)out;
  kp.in = (int)in;
  kp.act = act;
  kp.vec = (uintptr_t)Y % 16 == 0 && (ldy * (yt == GPTQ_F32 ? 4 : 2)) % 16 == 0;
  return run_split<G>(kp, x, w, yt, plan, follows, st);
}

// follows: the kernel launched before on st is the quantizer that wrote x, and
// this one may be set up while it runs.
cudaError_t multiply(const gptq_int8_tokens_t* x, int64_t tokens, int64_t in, const gptq_int8_layer_t* const (&w)[2],
                     int64_t out, const float* bias, int act, void* Y, gptq_dtype_t yt, int64_t ldy, bool follows,
                     cudaStream_t st) {
  if (rows_int8_takes(tokens, in)) return rows_int8(nullptr, 0, 0, x, tokens, in, w, out, bias, act, Y, yt, ldy, st);
  const Plan plan = make_plan(w[1] ? 2 : 1, tokens, in, out, device_info().sms);
  if (plan.pair) {
    uint32_t* status = nullptr;
    const cudaError_t e = int8_status_word(&status);
    if (e != cudaSuccess) return e;
    return pair_int8(x, tokens, in, w, out, bias, act, Y, yt, ldy, plan.bn, follows, status, st);
  }
  if (w[1]) return run<2>(x, tokens, in, w, out, bias, act, Y, yt, ldy, plan, follows, st);
  return run<1>(x, tokens, in, w, out, bias, act, Y, yt, ldy, plan, follows, st);
}

// The workspace of a product that quantizes its tokens: codes, scales, sums.
struct TokenScratch {
  gptq_int8_tokens_t x;
  size_t bytes;
  TokenScratch(void* ws, int64_t tokens, int64_t in) {
    const int64_t ldq = round_up(in, 16), codes = round_up(tokens * ldq, 256), vec = round_up(tokens * 4, 256);
    x = {(const int8_t*)ws, ldq, (const float*)((uintptr_t)ws + codes), (const int32_t*)((uintptr_t)ws + codes + vec)};
    bytes = (size_t)(codes + 2 * vec);
  }
};

}  // namespace

gptq_status_t matmul_int8(const gptq_int8_tokens_t* x, int64_t tokens, int64_t in, const gptq_int8_layer_t* w,
                          int64_t out, const float* bias, void* Y, gptq_dtype_t yt, int64_t ldy, cudaStream_t st) {
  const gptq_int8_layer_t* const ws[2] = {w, nullptr};
  CUDA_TRY(multiply(x, tokens, in, ws, out, bias, 0, Y, yt, ldy, false, st));
  return GPTQ_OK;
}

gptq_status_t matmul_int8_gated(const gptq_int8_tokens_t* x, int64_t tokens, int64_t in, const gptq_int8_layer_t* gate,
                                const gptq_int8_layer_t* up, int64_t out, int act, void* Y, gptq_dtype_t yt,
                                int64_t ldy, cudaStream_t st) {
  const gptq_int8_layer_t* const ws[2] = {gate, up};
  CUDA_TRY(multiply(x, tokens, in, ws, out, nullptr, act, Y, yt, ldy, false, st));
  return GPTQ_OK;
}

size_t linear_int8_ws_bytes(int64_t tokens, int64_t in) {
  return rows_int8_takes(tokens, in) ? 0 : TokenScratch(nullptr, tokens, in).bytes;
}

gptq_status_t linear_int8(const void* X, gptq_dtype_t xt, int64_t tokens, int64_t in, int64_t ldx,
                          const gptq_int8_layer_t* w, const gptq_int8_layer_t* up, int64_t out, const float* bias,
                          int act, void* Y, gptq_dtype_t yt, int64_t ldy, void* ws, cudaStream_t st) {
  const gptq_int8_layer_t* const layers[2] = {w, up};
  if (rows_int8_takes(tokens, in)) {
    CUDA_TRY(rows_int8(X, xt, ldx, nullptr, tokens, in, layers, out, bias, act, Y, yt, ldy, st));
    return GPTQ_OK;
  }
  const TokenScratch q(ws, tokens, in);
  const gptq_status_t s = quantize_tokens(X, xt, tokens, in, ldx, const_cast<int8_t*>(q.x.q), q.x.ldq,
                                          const_cast<float*>(q.x.scale), const_cast<int32_t*>(q.x.sum), st);
  if (s != GPTQ_OK) return s;
  CUDA_TRY(multiply(&q.x, tokens, in, layers, out, bias, act, Y, yt, ldy, true, st));
  return GPTQ_OK;
}

cudaError_t int8_status_word(uint32_t** word) { return cudaGetSymbolAddress((void**)word, g_int8_status); }

gptq_status_t int8_status(cudaStream_t st) {
  uint32_t status = 0;
  uint32_t* at = nullptr;
  CUDA_TRY(int8_status_word(&at));
  CUDA_TRY(cudaMemcpyAsync(&status, at, sizeof(status), cudaMemcpyDeviceToHost, st));
  CUDA_TRY(cudaStreamSynchronize(st));
  if (status == 0) return GPTQ_OK;  // and nothing to clear: a flag that another stream raises by now stays
  CUDA_TRY(cudaMemsetAsync(at, 0, sizeof(status), st));
  CUDA_TRY(cudaStreamSynchronize(st));
  if (status & ST_TIMEOUT) return fail(GPTQ_ERR_TIMEOUT, "a bounded device-side wait gave up in an int8 kernel");
  return GPTQ_OK;
}

}  // namespace gptq
