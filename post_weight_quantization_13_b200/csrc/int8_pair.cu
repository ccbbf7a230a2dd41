// 8-bit integer products for many tokens, plain and gated.
//
// Bound by the tensor cores, and close behind by the operands' way from L2:
// an SM multiplies 128 x 256 x 128 bytes in 512 cycles, and a CTA on its own
// would have to load 48 KB for that.  So two CTAs on neighbouring SMs work as
// one (cta_group::2): the pair owns 256 tokens x up to 256 channels, each CTA
// loads its 128 tokens and half of the channels, and one tcgen05.mma reads
// both halves from both shared memories: 32 KB per CTA and 512 cycles.  In
// the gated form the first CTA's half are gate channels and the second's the
// same up channels, so a thread finds both factors of an output in its own
// tensor-memory lane.
//
// Persistent pairs, one per two SMs, warp-specialised in each CTA:
//   warp 0     TMA producer: its own operand halves; the transactions of both
//              CTAs are counted on the first CTA's barrier
//   warp 1     (in the first CTA) issues the pair's MMAs and commits them to both
//   warps 2-9  epilogue: scales, bias or activation, then whole sectors of a
//              row from each thread, or 64-byte row pieces through shared
//              memory to coalesced stores.  Two warps share a
//              quarter of tensor memory and halve its columns between them:
//              the last tile's epilogue has nothing to hide under, and with
//              four warps it took 4.9 of the 19 us of a product of one tile
//              (256 x 256, k 4096).
// Two 256-column accumulators in tensor memory let a tile's epilogue run
// under the next tile's main loop.  Every wait is bounded; one that gives up
// raises ST_TIMEOUT in the int8 status word, and both CTAs drain and leave.
//
// Measured, with the quantizer: 16384 tokens of 4096 > 11008 494 us in a burst
// (3.0e15 operations a second, 0.89 of twice the measured bf16 rate), 555 to 567
// call after call, where the power limit holds the clock down; gated 4096 tokens
// of 4096 > 11008 233 us and 263 to 268.
#include <algorithm>
#include <cstring>

#include "gemm.cuh"
#include "int8.cuh"
#include "internal.cuh"

namespace gptq {
namespace {

constexpr int kEpilogue = 256;               // threads of the epilogue: two warps a tensor-memory quarter
constexpr int kThreads = 64 + kEpilogue;
constexpr int kBK = 128;                     // bytes of k per stage
constexpr int kATile = 128 * kBK;            // a CTA's tokens of one stage
constexpr int kStageOut = 8 * 32 * 64;       // epilogue staging: 32 rows x 64 bytes a warp
constexpr int kVectors = 256 * 3 * 4;        // a tile's scales, zeros, bias
constexpr int kGroup = 8;                    // token tiles that walk the channels together

struct PairParams {
  const float* tscale;
  const int32_t* tsum;
  const float* wscale[2];
  const int32_t* wzero[2];
  const float* bias;
  void* Y;
  int64_t ldy;
  int tokens, out, act, vec, vec32;
  int ktiles, bn, stages, stage_bytes;
  int mtiles, ntiles, tiles, pairs;
  uint32_t* status;
};

struct PairMaps {
  CUtensorMap x;
  CUtensorMap w[2];
};

// A tile into this CTA's shared memory, counted on a barrier of the pair
// given by its cluster address.
__device__ __forceinline__ void load_pair(uint32_t leader, uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                          int y) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "@p cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(leader)
      : "memory");
}
// Arrive on a barrier of the pair.  What it orders are reads of tensor memory,
// complete behind tcgen05.wait and fenced: the release is block-wide, for a
// cluster-wide one would wait for the epilogue's global stores.
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The tile's first token and first channel.  kGroup token tiles walk the
// channel tiles side by side, so the pairs at work share both operands in L2.
__device__ __forceinline__ void tile_at(const PairParams& kp, int tile, int* mt, int* nt) {
  const int group = tile / (kGroup * kp.ntiles), rest = tile - group * kGroup * kp.ntiles;
  const int rows = min(kGroup, kp.mtiles - group * kGroup);
  *mt = group * kGroup + rest % rows;
  *nt = rest / rows;
}

// Byte offset of 16-byte unit u (0..3) of row r of a 64-byte-wide staging tile.
__device__ __forceinline__ uint32_t sw64(int r, int u) { return (uint32_t)(r * 64 + ((u ^ (r >> 1 & 3)) << 4)); }

// N columns of sums (32-bit integers in v) to the product's values; zeros:
// some channel has one.
template <int N>
__device__ __forceinline__ void scale_columns(const float (&v)[N], Pair (&y)[N / 2], const float* scale,
                                              const int* zero, bool zeros, int sum, float ts) {
  const Pair t(ts);
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    int a[4] = {__float_as_int(v[i]), __float_as_int(v[i + 1]), __float_as_int(v[i + 2]), __float_as_int(v[i + 3])};
    if (zeros) {
      const int4 z = *reinterpret_cast<const int4*>(zero + i);
      a[0] -= z.x * sum;
      a[1] -= z.y * sum;
      a[2] -= z.z * sum;
      a[3] -= z.w * sum;
    }
    const float4 s = *reinterpret_cast<const float4*>(scale + i);
    y[i / 2] = mul2(mul2(Pair((float)a[0], (float)a[1]), t), Pair(s.x, s.y));
    y[i / 2 + 1] = mul2(mul2(Pair((float)a[2], (float)a[3]), t), Pair(s.z, s.w));
  }
}

// Eight 32-bit words to a 32-byte boundary.
__device__ __forceinline__ void store_sector(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <int G, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    int8_pair_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ PairParams kp) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* staging = smem + (size_t)kp.stages * kp.stage_bytes;
  float* vectors = (float*)(staging + kStageOut);
  uint64_t* full = (uint64_t*)((uint8_t*)vectors + kVectors);
  uint64_t* empty = full + kp.stages;
  uint64_t* acc_full = empty + kp.stages;  // [2]
  uint64_t* acc_empty = acc_full + 2;      // [2], the first CTA's count
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = (uint32_t*)(drain + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  volatile int* epilogue_abort = abort_flag + 1;  // written and read between the epilogue warps' barriers only

  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int half = kp.bn / 2;  // channels a CTA loads

  if (threadIdx.x == 64) {
    tma_prefetch_desc(&maps.x);
    tma_prefetch_desc(&maps.w[G == 2 ? rank : 0]);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kp.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpilogue / 32);  // the epilogue warps of both CTAs
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *epilogue_abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const int pair = (int)blockIdx.x / 2;
  grid_dependency_wait();  // what came before ran beside the set-up above

  const uint32_t stage0 = smem_u32(smem), full0 = smem_u32(full), empty0 = smem_u32(empty);
  if (warp == 0) {
    const uint32_t leader = elect_lane();
    const int stages = kp.stages, stage_bytes = kp.stage_bytes, ktiles = kp.ktiles;
    const uint32_t bytes = 2u * (uint32_t)(kATile + half * kBK);  // of both CTAs
    const uint32_t pair_full0 = map_to_rank(full0, 0);
    const CUtensorMap* wmap = &maps.w[G == 2 ? rank : 0];
    int stage = 0;
    uint32_t phase = 1, at = stage0;
    bool ok = true;
    for (int tile = pair; tile < kp.tiles && ok; tile += kp.pairs) {
      int mt, nt;
      tile_at(kp, tile, &mt, &nt);
      const int t0 = mt * 256 + rank * 128;
      const int n0 = G == 2 ? nt * half : nt * kp.bn + rank * half;
      for (int x = 0; x < ktiles * kBK; x += kBK) {
        if (!wait_at(empty0 + 8 * stage, phase)) {
          raise_status(kp.status, ST_TIMEOUT);
          *abort_flag = 1;
          ok = false;
          break;
        }
        if (rank == 0) expect_at(leader, full0 + 8 * stage, bytes);
        load_pair(leader, at, &maps.x, pair_full0 + 8 * stage, x, t0);
        load_pair(leader, at + kATile, wmap, pair_full0 + 8 * stage, x, n0);
        at += stage_bytes;
        if (++stage == stages) {
          stage = 0;
          at = stage0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t leader = elect_lane();
      const int stages = kp.stages, ktiles = kp.ktiles;
      const uint32_t idesc = idesc_i8(256, (uint32_t)kp.bn);
      const uint32_t a0 = desc_low(stage0), b0 = desc_low(stage0 + kATile), desc_step = (uint32_t)kp.stage_bytes >> 4;
      int stage = 0, step = 0;
      uint32_t phase = 0, at = 0;
      bool ok = true;
      for (int tile = pair; tile < kp.tiles && ok; tile += kp.pairs, ++step) {
        const int buf = step & 1, use = step >> 1;
        if (use > 0 && !mbar_wait(&acc_empty[buf], (use - 1) & 1)) {
          raise_status(kp.status, ST_TIMEOUT);
          *abort_flag = 1;
          break;
        }
        tc_fence_after();
        const uint32_t d = tbase + (uint32_t)buf * 256u;
        for (int kt = 0; kt < ktiles; ++kt) {
          if (!wait_at(full0 + 8 * stage, phase)) {
            raise_status(kp.status, ST_TIMEOUT);
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          umma_i8<2>(leader, d, a0 + at, b0 + at, idesc, kt > 0);
#pragma unroll
          for (int kk = 1; kk < kBK / 32; ++kk) umma_i8<2>(leader, d, a0 + at + 2 * kk, b0 + at + 2 * kk, idesc, 1u);
          commit_pair_at(leader, empty0 + 8 * stage);
          at += desc_step;
          if (++stage == stages) {
            stage = 0;
            at = 0;
            phase ^= 1;
          }
        }
        if (ok) commit_pair_at(leader, smem_u32(&acc_full[buf]));
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    constexpr int CW = 64 / (int)sizeof(T);  // columns of a 64-byte row piece
    constexpr int STEP = 16;                 // columns of a step, see below
    const int quarter = warp & 3, e = threadIdx.x - 64;
    const int bn = kp.bn, width = G == 2 ? half : bn;  // channels of the tile's output
    const int c_begin = (warp - 2) / 4 * (width / 2), c_end = c_begin + width / 2;  // this warp's
    uint8_t* mine = staging + (warp - 2) * (32 * 64);
    float* const vscale = vectors;                 // [bn]: gated, gate then up
    int* const vzero = (int*)(vectors + 256);      // [bn]
    float* const vbias = vectors + 512;            // [bn]
    const bool zeros = kp.wzero[0] || (G == 2 && kp.wzero[1]), biased = G == 1 && kp.bias;
    int step = 0;
    for (int tile = pair; tile < kp.tiles; tile += kp.pairs, ++step) {
      int mt, nt;
      tile_at(kp, tile, &mt, &nt);
      const int n0 = nt * width;
      const int t = mt * 256 + rank * 128 + quarter * 32 + lane;
      // the tile's vectors, while its main loop runs
      named_bar_sync(1, kEpilogue);  // the previous tile's are no longer read
      for (int i = e; i < bn; i += kEpilogue) {
        const int g = G == 2 ? i / half : 0, n = n0 + (G == 2 ? i % half : i);
        const bool in = n < kp.out;
        vscale[i] = in ? __ldg(kp.wscale[g] + n) : 0.f;
        vzero[i] = in && kp.wzero[g] ? __ldg(kp.wzero[g] + n) : 0;
        vbias[i] = in && biased ? __ldg(kp.bias + n) : 0.f;
      }
      // (not through the read-only path: the quantizer may have written them since
      // this kernel began)
      const float ts = t < kp.tokens ? kp.tscale[t] : 0.f;
      const int sum = t < kp.tokens ? kp.tsum[t] : 0;
      named_bar_sync(1, kEpilogue);
      const int buf = step & 1, use = step >> 1;
      if (!mbar_wait_sleep(&acc_full[buf], use & 1)) {
        raise_status(kp.status, ST_TIMEOUT);
        *abort_flag = 1;
      }
      if (*abort_flag) *epilogue_abort = 1;
      // all warps leave together: they share barrier 1
      named_bar_sync(1, kEpilogue);
      if (*epilogue_abort) break;
      tc_fence_after();
      const uint32_t tmem = tbase + (uint32_t)buf * 256u + ((uint32_t)(quarter * 32) << 16);
      T* const rows = (T*)kp.Y + (int64_t)(t - lane) * kp.ldy;
      const int live = min(32, kp.tokens - (t - lane));  // rows of this warp inside the result
      for (int c0 = c_begin; c0 < c_end; c0 += CW) {
        // Rows on 32-byte boundaries are written by whole sectors without the
        // way through shared memory (4096 x 4096, k 1024: 24.7 us, so 23.2;
        // the gated form, short of instruction cache, 40.4 and 43.1).
        const bool direct = G == 1 && kp.vec32 && n0 + c0 + CW <= kp.out;
        // sixteen columns a step, not unrolled further: the loop has to stay
        // in the instruction cache (unrolled over 64 columns, the gated form
        // waited for instructions most of the time and took 1.4 times as long)
#pragma unroll 1
        for (int p = 0; p < CW / STEP; ++p) {
          const int c = c0 + STEP * p;
          float a[STEP];
          Pair y[STEP / 2];
          tmem_ld16(tmem + (uint32_t)c, a);
          scale_columns<STEP>(a, y, vscale + c, vzero + c, zeros, sum, ts);
          if (G == 2) {
            float b[STEP];
            Pair u[STEP / 2];
            tmem_ld16(tmem + (uint32_t)(half + c), b);
            scale_columns<STEP>(b, u, vscale + half + c, vzero + half + c, zeros, sum, ts);
            if (kp.act == GPTQ_ACT_GELU) {
#pragma unroll
              for (int i = 0; i < STEP / 2; ++i) {
                const float2 f = y[i].f();
                y[i] = mul2(Pair(activate(f.x, GPTQ_ACT_GELU), activate(f.y, GPTQ_ACT_GELU)), u[i]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < STEP / 2; ++i) {
                const float2 f = y[i].f();
                y[i] = mul2(Pair(activate(f.x, kp.act), activate(f.y, kp.act)), u[i]);
              }
            }
          } else if (biased) {
#pragma unroll
            for (int i = 0; i < STEP; i += 4) {
              const float4 b = *reinterpret_cast<const float4*>(vbias + c + i);
              y[i / 2] = add2(y[i / 2], Pair(b.x, b.y));
              y[i / 2 + 1] = add2(y[i / 2 + 1], Pair(b.z, b.w));
            }
          }
          alignas(16) T o[STEP];
#pragma unroll
          for (int i = 0; i < STEP / 2; ++i) {
            const float2 f = y[i].f();
            const float v[2] = {f.x, f.y};
            round_n<2>(v, o + 2 * i);
          }
          if (direct) {
            if (lane < live)
#pragma unroll
              for (int u = 0; u < STEP * (int)sizeof(T) / 32; ++u)
                store_sector((uint8_t*)(rows + lane * kp.ldy + n0 + c) + 32 * u,
                             reinterpret_cast<const uint32_t*>(o) + 8 * u);
            continue;
          }
          // 16-byte unit u of row r sits at unit u ^ (r / 2 & 3): neither the
          // row owner's writes nor the row-wise reads below meet in a bank
#pragma unroll
          for (int u = 0; u < STEP * (int)sizeof(T) / 16; ++u)
            *reinterpret_cast<uint4*>(mine + sw64(lane, p * (STEP * (int)sizeof(T) / 16) + u)) =
                reinterpret_cast<const uint4*>(o)[u];
        }
        if (c0 + CW >= c_end) {
          // the accumulator is read: the next tile but one may have it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_remote(map_to_rank(smem_u32(&acc_empty[buf]), 0));
        }
        if (direct) continue;
        __syncwarp();
        if (kp.vec && n0 + c0 + CW <= kp.out) {
#pragma unroll
          for (int r0 = 0; r0 < 32; r0 += 8) {
            const int r = r0 + (lane >> 2);
            if (r < live)
              *reinterpret_cast<uint4*>((uint8_t*)(rows + r * kp.ldy + n0 + c0) + 16 * (lane & 3)) =
                  *reinterpret_cast<const uint4*>(mine + sw64(r, lane & 3));
          }
        } else {
          const int c = lane % CW, cols = min(CW, kp.out - n0 - c0);
          const int byte = c * (int)sizeof(T);
          if (c < cols)
            for (int r = lane / CW; r < live; r += 32 / CW)
              rows[r * kp.ldy + n0 + c0 + c] = *reinterpret_cast<const T*>(mine + sw64(r, byte >> 4) + (byte & 15));
        }
        __syncwarp();
      }
    }
  }

  __syncwarp();
  if (*abort_flag && warp == 1 && rank == 0) {
    // let the MMAs already issued finish before the memory goes away
    commit_pair_at(elect_lane(), smem_u32(drain));
    mbar_wait(drain, 0);
  }
  if (*abort_flag && threadIdx.x == 0) let_copies_land();
  __syncwarp();
  // neither CTA leaves while the other's MMAs, commits or arrivals reach it
  cluster_arrive();
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(512u) : "memory");
  }
}

template <int G, typename T>
cudaError_t launch(const PairMaps& maps, const PairParams& kp, bool follows, cudaStream_t st) {
  const void* f = (const void*)int8_pair_kernel<G, T>;
  cudaError_t e = ensure_smem_limit(f, 232448);
  if (e != cudaSuccess) return e;
  const size_t smem = 1024 + (size_t)kp.stages * kp.stage_bytes + kStageOut + kVectors + 256;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * kp.pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = follows ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, int8_pair_kernel<G, T>, maps, kp);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t pair_int8(const gptq_int8_tokens_t* x, int64_t tokens, int64_t in, const gptq_int8_layer_t* const (&w)[2],
                      int64_t out, const float* bias, int act, void* Y, gptq_dtype_t yt, int64_t ldy, int bn,
                      bool follows, uint32_t* status, cudaStream_t st) {
  const int G = w[1] ? 2 : 1;
  PairParams kp = {};
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
  kp.act = act;
  kp.vec = (uintptr_t)Y % 16 == 0 && (ldy * (yt == GPTQ_F32 ? 4 : 2)) % 16 == 0;
  kp.vec32 = (uintptr_t)Y % 32 == 0 && (ldy * (yt == GPTQ_F32 ? 4 : 2)) % 32 == 0;
  kp.status = status;
  kp.ktiles = (int)((in + kBK - 1) / kBK);
  kp.bn = bn;
  kp.stage_bytes = kATile + kp.bn / 2 * kBK;
  kp.stages = std::min(12, (232448 - 1024 - kStageOut - kVectors - 256) / kp.stage_bytes);
  kp.mtiles = (int)((tokens + 255) / 256);
  const int width = kp.bn / G;
  kp.ntiles = (int)((out + width - 1) / width);
  kp.tiles = kp.mtiles * kp.ntiles;
  kp.pairs = std::min(kp.tiles, device_info().sms / 2);
  PairMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  if (!int8_map(&maps.x, x->q, tokens, in, x->ldq, 128)) return cudaErrorInvalidValue;
  for (int g = 0; g < G; ++g)
    if (!int8_map(&maps.w[g], w[g]->w, out, in, w[g]->ldw, kp.bn / 2)) return cudaErrorInvalidValue;
  if (G == 2)
    return yt == GPTQ_F16    ? launch<2, __half>(maps, kp, follows, st)
           : yt == GPTQ_BF16 ? launch<2, __nv_bfloat16>(maps, kp, follows, st)
                             : launch<2, float>(maps, kp, follows, st);
  return yt == GPTQ_F16    ? launch<1, __half>(maps, kp, follows, st)
         : yt == GPTQ_BF16 ? launch<1, __nv_bfloat16>(maps, kp, follows, st)
                           : launch<1, float>(maps, kp, follows, st);
}

}  // namespace gptq
