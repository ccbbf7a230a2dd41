// 8-bit integer products for one or two tokens (decode), the plain one and
// the gated pair, taking the tokens in 8 bits or in 16/32 (then each block
// quantizes them itself: one launch, no scratch).
//
// What bounds it: the weights, in * out bytes once; arithmetic is a fifth of
// what the SMs can do at that rate.  So the kernel keeps as many weight bytes
// in flight as it can.  A block owns a contiguous range of channels and its
// 256 threads split k: a thread's 16 columns of up to eight weight rows are
// one batch of eight independent 16-byte loads, and the next batch is loaded
// while this one is multiplied (dp4a) against the thread's own columns of the
// tokens, which it keeps in shared memory for itself.  Every row of a batch
// is read by the block as one contiguous run, the channels divide evenly over
// the SMs whatever their number, and a channel's sum needs no more than a
// transposed warp reduction (N values in N - 1 + log2(32 / N) exchanges) and
// one exchange between the eight warps.
#include <algorithm>

#include "gemm.cuh"
#include "int8.cuh"
#include "internal.cuh"

namespace gptq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kLoads = 8;              // weight vectors a thread has in flight per step
constexpr int kSlice = kThreads * 16;  // columns of one step

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
  int rows;  // the most channels a block owns
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
// and sums into tscale and tsum.
template <typename X, int T>
__device__ __forceinline__ void quantize_block(const RowsParams& kp, int4* codes, int steps, float* tscale, int* tsum,
                                               uint32_t (*exchange)[T]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = 2 * steps;  // of eight columns
#pragma unroll
  for (int t = 0; t < T; ++t) {
    uint32_t top = 0u;
    if (t < kp.tokens) {
#pragma unroll 4
      for (int s = 0; s < chunks; ++s)
        top = magnitude(load_columns((const X*)kp.x + t * kp.ldx, (s >> 1) * kSlice + 16 * (int)threadIdx.x + 8 * (s & 1),
                                     kp.in, kp.vec), top);
    }
    top = __reduce_max_sync(0xffffffffu, magnitude_bits<X>(top));
    if (lane == 0) exchange[warp][t] = top;
  }
  if (threadIdx.x < T) tsum[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int t = 0; t < T; ++t) {
    uint32_t top = 0u;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = max(top, exchange[w][t]);
    const TokenScale scale(top);
    int total = 0;
#pragma unroll 2
    for (int s = 0; s < chunks; ++s) {  // the second reading hits L1
      uint2 c = make_uint2(0u, 0u);
      if (t < kp.tokens) {
        const Raw8<X> r = load_columns((const X*)kp.x + t * kp.ldx,
                                       (s >> 1) * kSlice + 16 * (int)threadIdx.x + 8 * (s & 1), kp.in, kp.vec);
        Pair f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = get2(r, i);
        c = scale.codes(f);
        total = __dp4a((int)c.x, 0x01010101, __dp4a((int)c.y, 0x01010101, total));
      }
      reinterpret_cast<uint2*>(codes + (t * steps + (s >> 1)) * kThreads + threadIdx.x)[s & 1] = c;
    }
    total = __reduce_add_sync(0xffffffffu, total);
    if (lane == 0) atomicAdd(&tsum[t], total);
    if (threadIdx.x == 0) tscale[t] = scale.scale;
  }
}

template <int G, int T>
__global__ void __launch_bounds__(kThreads, 2) int8_rows_kernel(const __grid_constant__ RowsParams kp) {
  constexpr int R = kLoads / G;       // channels of a batch
  constexpr int N = kLoads * T;       // sums of a batch, [g][channel][token]
  extern __shared__ int4 codes[];     // [T][steps][thread]
  __shared__ float tscale[T];
  __shared__ int tsum[T];
  __shared__ uint32_t exchange[kWarps][T];
  __shared__ int sums[2][kWarps][N];
  // the block's channels' scales, zeros and bias: fetched once up front, since
  // a load in a batch's epilogue would hold up the whole block for its latency
  float* const wscale = (float*)(codes + (size_t)T * ((kp.in + kSlice - 1) / kSlice) * kThreads);  // [G][rows]
  int* const wzero = (int*)(wscale + G * kp.rows);                                                  // [G][rows]
  float* const bias = (float*)(wzero + G * kp.rows);                                                // [rows]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int steps = (kp.in + kSlice - 1) / kSlice;
  const int n_begin = (int)((int64_t)kp.out * blockIdx.x / gridDim.x);
  const int n_end = (int)((int64_t)kp.out * (blockIdx.x + 1) / gridDim.x);
  const int batches = (n_end - n_begin + R - 1) / R;

  // The loads of one step: a batch's rows at the thread's columns.  Rows past
  // the range repeat its last one; their sums are not used.
  auto load = [&](int4 (&w)[kLoads], int batch, int step) {
    const int k = step * kSlice + 16 * (int)threadIdx.x;
    const int n0 = n_begin + batch * R;
    const int left = kp.in - k;
    if (left >= 16 && n0 + R <= n_end) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int8_t* p = kp.w[g] + n0 * kp.ldw[g] + k;
#pragma unroll
        for (int i = 0; i < R; ++i, p += kp.ldw[g]) w[g * R + i] = __ldg(reinterpret_cast<const int4*>(p));
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        w[i] = left > 0 ? load16(kp.w[i / R] + min(n0 + i % R, n_end - 1) * kp.ldw[i / R] + k, left)
                        : make_int4(0, 0, 0, 0);
    }
  };

  int4 w[kLoads];
  load(w, 0, 0);  // in flight while the tokens are quantized
  for (int i = threadIdx.x; i < n_end - n_begin; i += kThreads) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      wscale[g * kp.rows + i] = __ldg(kp.wscale[g] + n_begin + i);
      wzero[g * kp.rows + i] = kp.wzero[g] ? __ldg(kp.wzero[g] + n_begin + i) : 0;
    }
    bias[i] = G == 1 && kp.bias ? __ldg(kp.bias + n_begin + i) : 0.f;
  }
  if (kp.xt < 0) {
    if (threadIdx.x < T) {
      tscale[threadIdx.x] = threadIdx.x < kp.tokens ? kp.tscale[threadIdx.x] : 0.f;
      tsum[threadIdx.x] = threadIdx.x < kp.tokens ? kp.tsum[threadIdx.x] : 0;
    }
    for (int t = 0; t < T; ++t)
      for (int s = 0; s < steps; ++s) {
        const int k = s * kSlice + 16 * (int)threadIdx.x;
        codes[(t * steps + s) * kThreads + threadIdx.x] =
            t < kp.tokens && k < kp.in ? load16((const int8_t*)kp.x + t * kp.ldx + k, kp.in - k)
                                       : make_int4(0, 0, 0, 0);
      }
  } else if (kp.xt == GPTQ_F16) {
    quantize_block<__half, T>(kp, codes, steps, tscale, tsum, exchange);
  } else if (kp.xt == GPTQ_BF16) {
    quantize_block<__nv_bfloat16, T>(kp, codes, steps, tscale, tsum, exchange);
  } else {
    quantize_block<float, T>(kp, codes, steps, tscale, tsum, exchange);
  }

  for (int batch = 0; batch < batches; ++batch) {
    int acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0;
    for (int step = 0; step < steps; ++step) {
      int4 next[kLoads];
      const bool last = step + 1 == steps;
      if (!last || batch + 1 < batches) load(next, batch + (last ? 1 : 0), last ? 0 : step + 1);
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const int4 x = codes[(t * steps + step) * kThreads + threadIdx.x];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) acc[i * T + t] = dot16(w[i], x, acc[i * T + t]);
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) w[i] = next[i];
    }
    const int sum = warp_sums<N>(acc);
    if (lane % (32 / N) == 0) sums[batch & 1][warp][lane / (32 / N)] = sum;
    // Also orders the tokens' scales and sums before their first use.  The
    // other half of sums is written before the next barrier, this one after
    // it, when its readers below are done.
    __syncthreads();
    if (threadIdx.x < R * T) {
      const int t = threadIdx.x % T, n = n_begin + batch * R + (int)threadIdx.x / T;
      if (t < kp.tokens && n < n_end) {
        float y[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
          int total = 0;
#pragma unroll
          for (int v = 0; v < kWarps; ++v) total += sums[batch & 1][v][g * R * T + threadIdx.x];
          y[g] = scaled(total, wzero[g * kp.rows + n - n_begin], tsum[t], tscale[t], wscale[g * kp.rows + n - n_begin]);
        }
        float o = y[0];
        if (G == 2)
          o = activate(y[0], kp.act) * y[G - 1];
        else
          o += bias[n - n_begin];
        const int64_t at = t * kp.ldy + n;
        if (kp.yt == GPTQ_F16)
          ((__half*)kp.Y)[at] = from_f32<__half>(o);
        else if (kp.yt == GPTQ_BF16)
          ((__nv_bfloat16*)kp.Y)[at] = from_f32<__nv_bfloat16>(o);
        else
          ((float*)kp.Y)[at] = o;
      }
    }
  }
}

template <int G, int T>
cudaError_t launch(RowsParams& kp, cudaStream_t st, int sms) {
  // two blocks an SM, none without a batch of its own
  const int grid = std::min(2 * sms, (kp.out + kLoads / G - 1) / (kLoads / G));
  kp.rows = (kp.out + grid - 1) / grid;
  const int steps = (kp.in + kSlice - 1) / kSlice;
  const int smem = T * steps * kThreads * 16 + (2 * G + 1) * kp.rows * 4;
  const void* f = (const void*)int8_rows_kernel<G, T>;
  cudaError_t e = ensure_smem_limit(f, smem);
  if (e != cudaSuccess) return e;
  int8_rows_kernel<G, T><<<grid, kThreads, smem, st>>>(kp);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t rows_int8(const void* x, int xt, int64_t ldx, const gptq_int8_tokens_t* tokens8, int64_t tokens, int64_t in,
                      const gptq_int8_layer_t* const (&w)[2], int64_t out, const float* bias, int act, void* Y,
                      gptq_dtype_t yt, int64_t ldy, cudaStream_t st) {
  RowsParams kp = {};
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
