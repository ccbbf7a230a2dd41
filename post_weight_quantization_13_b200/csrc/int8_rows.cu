// 8-bit integer products for one or two tokens (decode), the plain one and
// the gated pair, taking the tokens in 8 bits or in 16/32 (then each block
// quantizes them itself: one launch, no scratch).
//
// What bounds it: the weights, in * out bytes once.  So they stream through a
// ring of shared memory, a few rows a slot, by bulk copies that a warp of its
// own issues from the first cycles on: some 180 KB are in flight on every SM
// whatever the rest of the block does.  (With rows loaded straight to
// registers, two blocks an SM and 64 KB in flight, one token of 11008 x 4096
// took 13.9 us, now 10.8; of the gated 4096 x 11008 20.4, now 18.0, where the
// bytes alone take 14.)  A block owns a contiguous range of channels, which
// divide evenly over the SMs whatever their number.  Two groups of 256 threads
// take batches of eight rows in turn, each from a ring of its own (rows_ring.cuh
// says why), one at its sums while the other multiplies.  A group's threads
// split k: each multiplies (dp4a) its own columns of the rows with its own
// columns of the tokens.  A row's sum then costs its share of one transposed
// warp reduction for the batch (N values in N - 1 + log2(32 / N) exchanges) and
// of one exchange between the warps.
#include "gemm.cuh"
#include "int8.cuh"
#include "internal.cuh"
#include "rows_ring.cuh"

namespace gptq {
namespace {

using namespace rows;
constexpr int kWarps = kThreads / 32;

struct RowsParams {
  const void* x;
  int xt;  // gptq_dtype_t, or -1: int8 tokens with tscale and tsum
  int64_t ldx;
  const float* tscale;
  const int32_t* tsum;
  const int8_t* w[2];
  int64_t ldw[2];
  const float* wscale[2];
  const int32_t* wzero[2];
  const float* bias;
  void* Y;
  int yt;
  int64_t ldy;
  int tokens, out, in, act;
  Plan plan;
  uint32_t* status;
  int vec;  // x's rows start on 16-byte boundaries
};

// 16 int8 from p, of which the first `left` (>= 1) lie inside the row; a
// partial vector is read by bytes, since nothing promises that the last
// row's storage goes on behind it.
__device__ __forceinline__ int4 load16(const int8_t* __restrict__ p, int left) {
  if (left >= 16) return __ldg(reinterpret_cast<const int4*>(p));
  uint32_t v[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < left) v[i >> 2] |= (uint32_t)(uint8_t)p[i] << (8 * (i & 3));
  return make_int4((int)v[0], (int)v[1], (int)v[2], (int)v[3]);
}

__device__ __forceinline__ int dot16(const int4& a, const int4& b, int c) {
  c = __dp4a(a.x, b.x, c);
  c = __dp4a(a.y, b.y, c);
  c = __dp4a(a.z, b.z, c);
  return __dp4a(a.w, b.w, c);
}

// Sums v[0..N) over the warp.  Each step halves the values a lane keeps: it
// hands one half to its partner and adds the partner's share of the other.
// Returns the sum of value lane / (32 / N).
template <int N>
__device__ __forceinline__ int warp_sums(int (&v)[N]) {
  const int lane = threadIdx.x & 31;
  int offset = 16;
#pragma unroll
  for (int n = N; n > 1; n >>= 1) {
    const bool upper = lane & offset;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const int give = upper ? v[i] : v[i + n / 2];
      const int keep = upper ? v[i + n / 2] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, offset);
    }
    offset >>= 1;
  }
  for (; offset > 0; offset >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], offset);
  return v[0];
}

// Eight columns from c of a token's row; columns past `in` are zero.
template <typename X>
__device__ __forceinline__ Raw8<X> load_columns(const X* __restrict__ row, int c, int in, bool vec) {
  return c < in ? load8(row + c, in - c, vec) : zero8<X>();
}

// The block's T tokens into codes (each thread its own columns), their scales
// and sums into tscale and tsum.  The loads are issued before `start` lets the
// weights flow, behind whose 180 KB per SM they would queue for microseconds.
template <typename X, int T, typename Start>
__device__ __forceinline__ void quantize_block(const RowsParams& kp, int4* codes, int steps, float* tscale, int* tsum,
                                               uint32_t (*exchange)[T], Start start) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Raw8<X> raw[T][2 * kMaxSteps];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int s = 0; s < 2 * kMaxSteps; ++s)
      raw[t][s] = t < kp.tokens ? load_columns((const X*)kp.x + t * kp.ldx,
                                               (s >> 1) * kSlice + 16 * (int)threadIdx.x + 8 * (s & 1), kp.in, kp.vec)
                                : zero8<X>();
  if (threadIdx.x < T) tsum[threadIdx.x] = 0;
  start();
#pragma unroll
  for (int t = 0; t < T; ++t) {
    uint32_t top = 0u;
#pragma unroll
    for (int s = 0; s < 2 * kMaxSteps; ++s) top = magnitude(raw[t][s], top);
    top = __reduce_max_sync(0xffffffffu, magnitude_bits<X>(top));
    if (lane == 0) exchange[warp][t] = top;
  }
  named_bar_sync(1, kThreads);
#pragma unroll
  for (int t = 0; t < T; ++t) {
    uint32_t top = 0u;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = max(top, exchange[w][t]);
    const TokenScale scale(top);
    int total = 0;
#pragma unroll
    for (int s = 0; s < kMaxSteps; ++s) {
      if (s >= steps) break;
      uint2 c[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        Pair f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = get2(raw[t][2 * s + h], i);
        c[h] = scale.codes(f);
        total = __dp4a((int)c[h].x, 0x01010101, __dp4a((int)c[h].y, 0x01010101, total));
      }
      codes[(t * steps + s) * kThreads + threadIdx.x] = make_int4((int)c[0].x, (int)c[0].y, (int)c[1].x, (int)c[1].y);
    }
    total = __reduce_add_sync(0xffffffffu, total);
    if (lane == 0) atomicAdd(&tsum[t], total);
    if (threadIdx.x == 0) tscale[t] = scale.scale;
  }
}

template <int G, int T>
__global__ void __launch_bounds__(kGroups * kThreads + 32, 1) int8_rows_kernel(const __grid_constant__ RowsParams kp) {
  constexpr int R = kBatch / G;  // channels of a batch
  constexpr int N = kBatch * T;  // sums of a batch, [g][channel][token]
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float tscale[T];
  __shared__ int tsum[T];
  __shared__ uint32_t exchange[kWarps][T];
  __shared__ int sums[kGroups][2][kWarps][N];
  __shared__ uint64_t full[kGroups * kMaxSlots], empty[kGroups * kMaxSlots];
  static_assert(sizeof(tscale) + sizeof(tsum) + sizeof(exchange) + sizeof(sums) + sizeof(full) + sizeof(empty) <= kStatic,
                "static arrays");

  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  const int steps = (kp.in + kSlice - 1) / kSlice;
  const int slots = kp.plan.slots, slot_bytes = kp.plan.slot_bytes, own = kp.plan.rows;
  uint8_t* const ring = smem;                                                // [group][slots][slot_bytes]
  int4* const codes = (int4*)(smem + (size_t)kGroups * slots * slot_bytes);  // [T][steps][thread]
  // the block's channels' scales, zeros and (plain) bias: fetched once up front,
  // since a load in a batch's epilogue would hold up the whole block for its
  // latency
  float* const wscale = (float*)(codes + (size_t)T * steps * kThreads);  // [G][own]
  int* const wzero = (int*)(wscale + G * own);                           // [G][own]
  float* const bias = (float*)(wzero + G * own);                         // [own]
  const int n_begin = (int)((int64_t)kp.out * blockIdx.x / gridDim.x);
  const int n_end = (int)((int64_t)kp.out * (blockIdx.x + 1) / gridDim.x);
  const int batches = (n_end - n_begin + R - 1) / R;

  // A slot: `group` rows of each of the batch's projections, one after another
  // at row_bytes.
  const int group = kp.plan.group, row_bytes = kp.plan.row_bytes, dense = kp.plan.dense;
  if (warp == kGroups * kWarps) {
    // ------------------------------------------------------------ producer
    for (int s = lane; s < kGroups * slots; s += 32) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarps);
    }
    fence_mbar_init();
    __syncwarp();
    named_bar_sync(2, kThreads + 32);
    const uint32_t leader = elect_lane();
    const uint32_t ring0 = smem_u32(ring), full0 = smem_u32(full), empty0 = smem_u32(empty);
    Cursor at, other;  // in this batch's ring and in the other one
    at.phase = other.phase = 1;
    int base = 0;
    for (int c = 0; c < n_end - n_begin; c += group) {
      if (c > 0 && c % R == 0) {
        const Cursor next = other;
        other = at;
        at = next;
        base = slots - base;
      }
      const int slot = base + at.slot;
      if (!wait_at(empty0 + 8 * slot, at.phase)) {
        raise_status(kp.status, ST_TIMEOUT);
        let_copies_land();
        break;
      }
      const int n = n_begin + c, rows = min(group, n_end - n);
      // whole 16-byte units of each row; the last row's storage may end inside one
      const bool last = n + rows == kp.out;
      const uint32_t row16 = (uint32_t)(kp.in + 15) & ~15u, tail = last ? (uint32_t)kp.in & ~15u : row16;
      expect_at(leader, full0 + 8 * slot,
                dense ? G * ((rows - 1) * (uint32_t)row_bytes + tail) : G * ((rows - 1) * row16 + tail));
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const uint32_t to = ring0 + slot * slot_bytes + g * group * row_bytes;
        const int8_t* from = kp.w[g] + n * kp.ldw[g];
        if (dense) {  // rows follow one another as the slot wants them
          bulk_load_at(leader, to, from, (rows - 1) * (uint32_t)row_bytes + tail, full0 + 8 * slot);
        } else {
          for (int r = 0; r < rows; ++r)
            bulk_load_at(leader, to + r * row_bytes, from + r * kp.ldw[g], r + 1 < rows ? row16 : tail,
                         full0 + 8 * slot);
        }
      }
      at.advance(1, slots);
    }
    __syncwarp();
  } else {
    const int who = warp / kWarps, tid = (int)threadIdx.x & (kThreads - 1);
    auto start = [&] { named_bar_sync(2, kThreads + 32); };
    auto vectors = [&] {
      for (int i = threadIdx.x; i < n_end - n_begin; i += kGroups * kThreads) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          wscale[g * own + i] = __ldg(kp.wscale[g] + n_begin + i);
          wzero[g * own + i] = kp.wzero[g] ? __ldg(kp.wzero[g] + n_begin + i) : 0;
        }
        if (G == 1) bias[i] = kp.bias ? __ldg(kp.bias + n_begin + i) : 0.f;
      }
    };
    if (who > 0) {
      // the first group brings the tokens
    } else if (kp.xt < 0) {
      if (threadIdx.x < T) {
        tscale[threadIdx.x] = threadIdx.x < kp.tokens ? kp.tscale[threadIdx.x] : 0.f;
        tsum[threadIdx.x] = threadIdx.x < kp.tokens ? kp.tsum[threadIdx.x] : 0;
      }
      int4 x[T][kMaxSteps];
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int s = 0; s < kMaxSteps; ++s) {
          const int k = s * kSlice + 16 * (int)threadIdx.x;
          x[t][s] = t < kp.tokens && k < kp.in ? load16((const int8_t*)kp.x + t * kp.ldx + k, kp.in - k)
                                               : make_int4(0, 0, 0, 0);
        }
      start();
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int s = 0; s < kMaxSteps; ++s)
          if (s < steps) codes[(t * steps + s) * kThreads + threadIdx.x] = x[t][s];
    } else if (kp.xt == GPTQ_F16) {
      quantize_block<__half, T>(kp, codes, steps, tscale, tsum, exchange, start);
    } else if (kp.xt == GPTQ_BF16) {
      quantize_block<__nv_bfloat16, T>(kp, codes, steps, tscale, tsum, exchange, start);
    } else {
      quantize_block<float, T>(kp, codes, steps, tscale, tsum, exchange, start);
    }
    vectors();
    named_bar_sync(3, kGroups * kThreads);

    uint8_t* const mine = ring + (size_t)who * slots * slot_bytes;  // the group's ring
    uint64_t* const my_empty = empty + who * slots;
    const uint32_t my_full = smem_u32(full + who * slots);
    Cursor at;
    bool gave_up = false;  // after a wait that gave up the block runs on without waiting, on whatever is there
    int half = 0;
    for (int batch = who; batch < batches; batch += kGroups, half ^= 1) {
      int acc[N];
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = 0;
      // the batch's slots; its rows' places in them (rows past the range
      // repeat its last one: their sums are not used)
      const int first = batch * R, rows = min(R, n_end - n_begin - first);
      const int4* row[kBatch];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int in_slot = r & (group - 1);  // a batch is whole slots
        if (in_slot == 0 && r < rows) {
          if (r > 0) at.advance(1, slots);
          if (!gave_up && !wait_at(my_full + 8 * at.slot, at.phase)) {
            gave_up = true;
            raise_status(kp.status, ST_TIMEOUT);
          }
        }
#pragma unroll
        for (int g = 0; g < G; ++g)
          row[g * R + r] =
              r < rows ? (const int4*)(mine + (size_t)at.slot * slot_bytes + (g * group + in_slot) * row_bytes) + tid
                       : row[g * R + r - 1];
      }
      for (int step = 0; step < steps; ++step) {
        const int k = step * kSlice + 16 * tid;
        if (k >= kp.in) break;
        int4 w[kBatch], x[T];
#pragma unroll
        for (int t = 0; t < T; ++t) x[t] = codes[(t * steps + step) * kThreads + tid];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) w[i] = row[i][step * kThreads];
        if (k + 16 > kp.in && n_begin + first + rows == kp.out)  // the last row's tail was not copied
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const int4 tail = load16(kp.w[g] + (int64_t)(kp.out - 1) * kp.ldw[g] + k, kp.in - k);
#pragma unroll
            for (int r = 0; r < R; ++r)
              if (r >= rows - 1) w[g * R + r] = tail;
          }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
          for (int t = 0; t < T; ++t) acc[i * T + t] = dot16(w[i], x[t], acc[i * T + t]);
      }
      __syncwarp();
      // back from the batch's last slot to its first
      const int held = (rows + group - 1) / group;
      for (int j = 0; j < held; ++j) {
        const int s = at.slot - j + (at.slot < j ? slots : 0);
        if (lane == 0) mbar_arrive(&my_empty[s]);
      }
      at.advance(1, slots);
      const int sum = warp_sums<N>(acc);
      if (lane % (32 / N) == 0) sums[who][half][warp % kWarps][lane / (32 / N)] = sum;
      // The other half of sums is written before the group's next barrier, this
      // one after it, when its readers below are done.
      named_bar_sync(4 + who, kThreads);
      if (tid < R * T) {
        const int t = tid % T, c = batch * R + tid / T, n = n_begin + c;
        if (t < kp.tokens && n < n_end) {
          float y[G];
#pragma unroll
          for (int g = 0; g < G; ++g) {
            int total = 0;
#pragma unroll
            for (int v = 0; v < kWarps; ++v) total += sums[who][half][v][g * R * T + tid];
            y[g] = scaled(total, wzero[g * own + c], tsum[t], tscale[t], wscale[g * own + c]);
          }
          float o = y[0];
          if (G == 2)
            o = activate(y[0], kp.act) * y[G - 1];
          else
            o += bias[c];
          const int64_t to = t * kp.ldy + n;
          if (kp.yt == GPTQ_F16)
            ((__half*)kp.Y)[to] = from_f32<__half>(o);
          else if (kp.yt == GPTQ_BF16)
            ((__nv_bfloat16*)kp.Y)[to] = from_f32<__nv_bfloat16>(o);
          else
            ((float*)kp.Y)[to] = o;
        }
      }
    }
    if (gave_up) let_copies_land();
  }
}

template <int G, int T>
cudaError_t launch(RowsParams& kp, cudaStream_t st, int sms) {
  const bool same = G == 1 || kp.ldw[0] == kp.ldw[1];
  kp.plan = plan(G, T, kp.in, kp.out, same ? kp.ldw[0] : 0, sms);
  const void* f = (const void*)int8_rows_kernel<G, T>;
  cudaError_t e = ensure_smem_limit(f, kSmem);
  if (e != cudaSuccess) return e;
  int8_rows_kernel<G, T><<<kp.plan.grid, kGroups * kThreads + 32, kp.plan.smem, st>>>(kp);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

bool rows_int8_takes(int64_t tokens, int64_t in) { return tokens <= 2 && in <= kMaxSteps * kSlice; }

cudaError_t rows_int8(const void* x, int xt, int64_t ldx, const gptq_int8_tokens_t* tokens8, int64_t tokens, int64_t in,
                      const gptq_int8_layer_t* const (&w)[2], int64_t out, const float* bias, int act, void* Y,
                      gptq_dtype_t yt, int64_t ldy, cudaStream_t st) {
  RowsParams kp = {};
  const cudaError_t e = int8_status_word(&kp.status);
  if (e != cudaSuccess) return e;
  kp.x = tokens8 ? tokens8->q : x;
  kp.xt = tokens8 ? -1 : xt;
  kp.ldx = tokens8 ? tokens8->ldq : ldx;
  if (tokens8) {
    kp.tscale = tokens8->scale;
    kp.tsum = tokens8->sum;
  }
  for (int g = 0; g < 2; ++g) {
    if (!w[g]) continue;
    kp.w[g] = w[g]->w;
    kp.ldw[g] = w[g]->ldw;
    kp.wscale[g] = w[g]->scale;
    kp.wzero[g] = w[g]->zero;
  }
  kp.bias = bias;
  kp.Y = Y;
  kp.yt = yt;
  kp.ldy = ldy;
  kp.tokens = (int)tokens;
  kp.out = (int)out;
  kp.in = (int)in;
  kp.act = act;
  kp.vec = (uintptr_t)kp.x % 16 == 0 && (kp.ldx * (xt == GPTQ_F32 ? 4 : 2)) % 16 == 0;
  const int sms = device_info().sms;
  if (w[1]) return tokens == 1 ? launch<2, 1>(kp, st, sms) : launch<2, 2>(kp, st, sms);
  return tokens == 1 ? launch<1, 1>(kp, st, sms) : launch<1, 2>(kp, st, sms);
}

}  // namespace gptq
