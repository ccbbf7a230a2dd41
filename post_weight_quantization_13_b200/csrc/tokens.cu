// The 8-bit serving path's memory-bound kernels: the int8 weight layout, the
// per-token quantizer, and the norms around a block fused with its gate,
// residual and the quantizer.
//
// A token's row stays in registers from its one load to its one store, so
// every operand crosses HBM once: a thread owns NV chunks of eight
// consecutive elements (one 16-byte load for 16-bit types), a row is owned
// by one warp where 32 * 8 * NV elements hold it and by one block otherwise,
// and the two or three statistics of a row (sums of squares, means, the
// largest magnitude) are reduced by warp shuffles and one shared-memory
// exchange each.  All statistics are fp32; a mean is subtracted before the
// squares are summed, so a layer norm loses nothing to cancellation.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "gemm.cuh"
#include "int8.cuh"
#include "internal.cuh"

namespace gptq {
namespace {

// ------------------------------------------------------------ row reductions
// Reductions over the threads of one row (blockDim.x of them).  Successive
// reductions of a wide row alternate between two exchange buffers, so one
// barrier each is enough: a buffer is written again only after the barrier of
// the reduction in between.
struct RowReduce {
  uint32_t* buf;  // [2][32]
  int parity;
  __device__ __forceinline__ RowReduce(uint32_t* b) : buf(b), parity(0) {}
  template <typename V, typename F>
  __device__ __forceinline__ V exchange(V warp_value, V identity, F combine) {
    if (blockDim.x <= 32) return warp_value;
    V* b = reinterpret_cast<V*>(buf + 32 * parity);
    parity ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0) b[threadIdx.x >> 5] = warp_value;
    __syncthreads();
    return combine(lane < (int)(blockDim.x >> 5) ? b[lane] : identity);
  }
  static __device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  __device__ __forceinline__ float sum(float v) {
    return exchange(warp_sum(v), 0.f, [](float x) { return warp_sum(x); });
  }
  __device__ __forceinline__ uint32_t max_u32(uint32_t v) {
    return exchange(__reduce_max_sync(0xffffffffu, v), 0u,
                    [](uint32_t x) { return __reduce_max_sync(0xffffffffu, x); });
  }
  __device__ __forceinline__ int sum_s32(int v) {
    return exchange(__reduce_add_sync(0xffffffffu, v), 0, [](int x) { return __reduce_add_sync(0xffffffffu, x); });
  }
};

// The token quantizer on a row in registers (TokenScale holds its arithmetic).  The largest magnitude is taken on the bit patterns, where
// NaN and infinity sort above every finite value; such a row gets s = NaN and
// codes of zero, so its product row is NaN and no other row is touched.
template <int NV>
__device__ __forceinline__ void quantize_row(const float (&v)[NV][8], int d, RowReduce& red, int8_t* __restrict__ q,
                                             float* __restrict__ scale, int32_t* __restrict__ sum) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int u = 0; u < 8; ++u) top = max(top, __float_as_uint(v[i][u]) & 0x7fffffffu);
  top = red.max_u32(top);
  const TokenScale s(top);
  int total = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c0 = 8 * (threadIdx.x + i * blockDim.x);
    if (c0 >= d) continue;
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int code = s.code(v[i][u]);
      total += code;
      w[u >> 2] |= (uint32_t)(code & 0xff) << (8 * (u & 3));
    }
    if (c0 + 8 <= d) {
      *reinterpret_cast<uint2*>(q + c0) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (c0 + u < d) q[c0 + u] = (int8_t)(w[u >> 2] >> (8 * (u & 3)));
    }
  }
  total = red.sum_s32(total);
  if (threadIdx.x == 0) {
    *scale = s.scale;
    *sum = total;
  }
}

template <typename T, int NV>
__global__ void __launch_bounds__(1024) quantize_tokens_kernel(const T* __restrict__ X, int64_t tokens, int d,
                                                               int64_t ldx, int8_t* __restrict__ q, int64_t ldq,
                                                               float* __restrict__ scale, int32_t* __restrict__ sum,
                                                               bool vec) {
  __shared__ uint32_t buf[64];
  grid_launch_dependents();  // a product behind this kernel sets up beside it
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= tokens) return;  // whole warps: rows of several per block are one warp wide
  RowReduce red(buf);
  float v[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c0 = 8 * (threadIdx.x + i * blockDim.x);
    Raw8<T> r;
    if (c0 < d) r = load8(X + t * ldx + c0, d - c0, vec);
#pragma unroll
    for (int u = 0; u < 8; ++u) v[i][u] = c0 < d ? to_f32(r.v[u]) : 0.f;
  }
  quantize_row<NV>(v, d, red, q + t * ldq, scale + t, sum + t);
}

// ------------------------------------------------------------------- norms
struct NormParams {
  int64_t tokens;
  int d;
  const void *h, *y, *post_weight, *post_bias, *gate, *weight, *bias;
  void *h_out, *x;
  int64_t ldh, ldy, ldgate, ldh_out, ldx, ldq;
  int8_t* q;
  float* scale;
  int32_t* sum;
  float alpha, beta, eps;
  int layer;
  // 16-byte access per operand
  int vec_h, vec_y, vec_post_weight, vec_post_bias, vec_gate, vec_weight, vec_bias, vec_h_out, vec_x;
};

// v <- norm(v) * weight (+ bias) over the row's d elements.
template <typename T, int NV>
__device__ __forceinline__ void norm_row(float (&v)[NV][8], const NormParams& p, RowReduce& red,
                                         const T* __restrict__ w, const T* __restrict__ b, int vec_w, int vec_b) {
  const int d = p.d;
  const float inv_d = 1.f / (float)d;
  if (p.layer) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[i][u];
    const float mean = red.sum(s) * inv_d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c0 = 8 * (threadIdx.x + i * blockDim.x);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (c0 + u < d) v[i][u] -= mean;  // elements past the end stay zero
    }
  }
  float s2 = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int u = 0; u < 8; ++u) s2 = fmaf(v[i][u], v[i][u], s2);
  const float r = rsqrtf(fmaf(red.sum(s2), inv_d, p.eps));
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c0 = 8 * (threadIdx.x + i * blockDim.x);
    if (c0 >= d) continue;
    const Raw8<T> rw = load8(w + c0, d - c0, vec_w);
#pragma unroll
    for (int u = 0; u < 8; ++u) v[i][u] = v[i][u] * r * to_f32(rw.v[u]);
    if (b) {
      const Raw8<T> rb = load8(b + c0, d - c0, vec_b);
#pragma unroll
      for (int u = 0; u < 8; ++u) v[i][u] += to_f32(rb.v[u]);
    }
  }
}

// h' = alpha h + beta gate * post(y);  x = pre(h') in 16/32 bits and/or int8.
// The pre-norm works on h' before it is rounded to its stored type.
template <typename T, typename H, int NV>
__global__ void __launch_bounds__(1024) norm_tokens_kernel(const __grid_constant__ NormParams p) {
  __shared__ uint32_t buf[64];
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= p.tokens) return;
  const int d = p.d;
  RowReduce red(buf);
  float v[NV][8];
  Raw8<H> hr[NV];
  const H* __restrict__ h = (const H*)p.h + t * p.ldh;
#pragma unroll
  for (int i = 0; i < NV; ++i) {  // both operands' loads are in flight together
    const int c0 = 8 * (threadIdx.x + i * blockDim.x);
    if (c0 < d) {
      hr[i] = load8(h + c0, d - c0, p.vec_h);
    } else {
#pragma unroll
      for (int u = 0; u < 8; ++u) hr[i].v[u] = from_f32<H>(0.f);
    }
  }
  if (p.y) {
    const T* __restrict__ y = (const T*)p.y + t * p.ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c0 = 8 * (threadIdx.x + i * blockDim.x);
      Raw8<T> r;
      if (c0 < d) r = load8(y + c0, d - c0, p.vec_y);
#pragma unroll
      for (int u = 0; u < 8; ++u) v[i][u] = c0 < d ? to_f32(r.v[u]) : 0.f;
    }
    if (p.post_weight)
      norm_row<T, NV>(v, p, red, (const T*)p.post_weight, (const T*)p.post_bias, p.vec_post_weight, p.vec_post_bias);
    if (p.gate) {
      const T* __restrict__ g = (const T*)p.gate + t * p.ldgate;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c0 = 8 * (threadIdx.x + i * blockDim.x);
        if (c0 >= d) continue;
        const Raw8<T> r = load8(g + c0, d - c0, p.vec_gate);
#pragma unroll
        for (int u = 0; u < 8; ++u) v[i][u] *= to_f32(r.v[u]);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int u = 0; u < 8; ++u) v[i][u] = fmaf(p.alpha, to_f32(hr[i].v[u]), p.beta * v[i][u]);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int u = 0; u < 8; ++u) v[i][u] = p.alpha * to_f32(hr[i].v[u]);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c0 = 8 * (threadIdx.x + i * blockDim.x);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (c0 + u >= d) v[i][u] = 0.f;  // a bias or 0 * inf must not reach the statistics
    if (p.h_out && c0 < d) store8((H*)p.h_out + t * p.ldh_out + c0, v[i], d - c0, p.vec_h_out);
  }
  if (!p.weight) return;
  norm_row<T, NV>(v, p, red, (const T*)p.weight, (const T*)p.bias, p.vec_weight, p.vec_bias);
  if (p.x) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c0 = 8 * (threadIdx.x + i * blockDim.x);
      if (c0 < d) store8((T*)p.x + t * p.ldx + c0, v[i], d - c0, p.vec_x);
    }
  }
  if (p.q) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c0 = 8 * (threadIdx.x + i * blockDim.x);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (c0 + u >= d) v[i][u] = 0.f;
    }
    quantize_row<NV>(v, d, red, p.q + t * p.ldq, p.scale + t, p.sum + t);
  }
}

// ------------------------------------------------------------ weight layout
// bits 8: w = code - 128, zero = zeros - 128; fewer bits: w = code - zeros,
// zero = 0.  One thread turns sixteen columns of one row into one 16-byte
// store; their fields lie in the 32 * bits / 16 <= 4 words from bit 16 bits c.
__global__ void __launch_bounds__(256) layout_int8_kernel(const uint32_t* __restrict__ qweight,
                                                          const int32_t* __restrict__ zeros, int64_t out, int64_t in,
                                                          int bits, int8_t* __restrict__ w, int64_t ldw,
                                                          int32_t* __restrict__ zero) {
  const int64_t words = in * bits / 32;
  const int64_t hexes = (in + 15) / 16;
  const uint32_t mask = (1u << bits) - 1u;
  for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < out * hexes;
       e += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = e / hexes, c0 = (e % hexes) * 16;
    const int z = __ldg(zeros + r);
    const int shift = bits == 8 ? 128 : z;
    const uint32_t* qrow = qweight + r * words;
    alignas(16) int8_t o[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      o[u] = 0;
      if (c0 + u >= in) continue;
      const int64_t bit = (c0 + u) * bits;
      const int64_t w0 = bit >> 5;
      const int sh = (int)(bit & 31);
      uint32_t f = __ldg(qrow + w0) >> sh;
      if (sh + bits > 32) f |= __ldg(qrow + w0 + 1) << (32 - sh);
      o[u] = (int8_t)((int)(f & mask) - shift);
    }
    int8_t* dst = w + r * ldw + c0;
    if (c0 + 16 <= in) {
      *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(o);
    } else {
#pragma unroll
      for (int u = 0; u < 16; ++u)
        if (c0 + u < in) dst[u] = o[u];
    }
    if (c0 == 0 && zero) zero[r] = bits == 8 ? z - 128 : 0;
  }
}

// Threads of a row and rows of a block for rows of d elements at NV chunks a
// thread: one warp where it can hold the row (four rows a block), else one
// block.
dim3 row_block(int d, int nv) {
  const int lanes = (d + 8 * nv - 1) / (8 * nv);
  return lanes <= 32 ? dim3(32, 4) : dim3((unsigned)((lanes + 31) / 32 * 32), 1);
}

// Chunks a thread: two, so that a row of 4096 is a block of 256; four beyond
// 16384 elements, where 1024 threads hold no more with two.
int row_chunks(int d) { return d > 1024 * 16 ? 4 : 2; }

template <typename T>
cudaError_t launch_quantize(const T* X, int64_t tokens, int d, int64_t ldx, int8_t* q, int64_t ldq, float* scale,
                            int32_t* sum, cudaStream_t st) {
  const bool vec = (uintptr_t)X % 16 == 0 && (ldx * (int64_t)sizeof(T)) % 16 == 0;
  const int nv = row_chunks(d);
  const dim3 block = row_block(d, nv);
  const unsigned grid = (unsigned)((tokens + block.y - 1) / block.y);
  if (nv == 2)
    quantize_tokens_kernel<T, 2><<<grid, block, 0, st>>>(X, tokens, d, ldx, q, ldq, scale, sum, vec);
  else
    quantize_tokens_kernel<T, 4><<<grid, block, 0, st>>>(X, tokens, d, ldx, q, ldq, scale, sum, vec);
  note_launch();
  return cudaGetLastError();
}

template <typename T, typename H>
cudaError_t launch_norm(const NormParams& p, cudaStream_t st) {
  const int nv = row_chunks(p.d);
  const dim3 block = row_block(p.d, nv);
  const unsigned grid = (unsigned)((p.tokens + block.y - 1) / block.y);
  if (nv == 2)
    norm_tokens_kernel<T, H, 2><<<grid, block, 0, st>>>(p);
  else
    norm_tokens_kernel<T, H, 4><<<grid, block, 0, st>>>(p);
  note_launch();
  return cudaGetLastError();
}

int aligned_rows(const void* p, int64_t ld, gptq_dtype_t t) {
  return (uintptr_t)p % 16 == 0 && (ld * (t == GPTQ_F32 ? 4 : 2)) % 16 == 0;
}

}  // namespace

gptq_status_t layout_int8(const uint32_t* qweight, const int32_t* zeros, int64_t out, int64_t in, int bits, int8_t* w,
                          int64_t ldw, int32_t* zero, cudaStream_t st) {
  const DeviceInfo& dev = device_info();
  const int64_t work = out * ((in + 15) / 16);
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>((work + 255) / 256, (int64_t)dev.sms * 16));
  layout_int8_kernel<<<grid, 256, 0, st>>>(qweight, zeros, out, in, bits, w, ldw, zero);
  note_launch();
  CUDA_TRY(cudaGetLastError());
  return GPTQ_OK;
}

gptq_status_t quantize_tokens(const void* X, gptq_dtype_t xt, int64_t tokens, int64_t in, int64_t ldx, int8_t* q,
                              int64_t ldq, float* scale, int32_t* sum, cudaStream_t st) {
  const int d = (int)in;
  if (xt == GPTQ_F16)
    CUDA_TRY(launch_quantize((const __half*)X, tokens, d, ldx, q, ldq, scale, sum, st));
  else if (xt == GPTQ_BF16)
    CUDA_TRY(launch_quantize((const __nv_bfloat16*)X, tokens, d, ldx, q, ldq, scale, sum, st));
  else
    CUDA_TRY(launch_quantize((const float*)X, tokens, d, ldx, q, ldq, scale, sum, st));
  return GPTQ_OK;
}

gptq_status_t norm_tokens(const gptq_norm_t* a, cudaStream_t st) {
  NormParams p = {};
  p.tokens = a->tokens;
  p.d = (int)a->d;
  p.h = a->h;
  p.y = a->y;
  p.post_weight = a->post_weight;
  p.post_bias = a->post_bias;
  p.gate = a->gate;
  p.weight = a->weight;
  p.bias = a->bias;
  p.h_out = a->h_out;
  p.x = a->x;
  p.ldh = a->ldh;
  p.ldy = a->ldy;
  p.ldgate = a->ldgate;
  p.ldh_out = a->ldh_out;
  p.ldx = a->ldx;
  p.ldq = a->ldq;
  p.q = a->q;
  p.scale = a->scale;
  p.sum = a->sum;
  p.alpha = a->alpha;
  p.beta = a->beta;
  p.eps = a->eps;
  p.layer = a->kind == GPTQ_NORM_LAYER;
  p.vec_h = aligned_rows(a->h, a->ldh, a->ht);
  p.vec_y = aligned_rows(a->y, a->ldy, a->yt);
  p.vec_post_weight = aligned_rows(a->post_weight, 0, a->yt);
  p.vec_post_bias = aligned_rows(a->post_bias, 0, a->yt);
  p.vec_gate = aligned_rows(a->gate, a->ldgate, a->yt);
  p.vec_weight = aligned_rows(a->weight, 0, a->yt);
  p.vec_bias = aligned_rows(a->bias, 0, a->yt);
  p.vec_h_out = aligned_rows(a->h_out, a->ldh_out, a->ht);
  p.vec_x = aligned_rows(a->x, a->ldx, a->yt);
  if (a->yt == GPTQ_F16)
    CUDA_TRY((a->ht == GPTQ_F32 ? launch_norm<__half, float>(p, st) : launch_norm<__half, __half>(p, st)));
  else if (a->yt == GPTQ_BF16)
    CUDA_TRY((a->ht == GPTQ_F32 ? launch_norm<__nv_bfloat16, float>(p, st)
                                : launch_norm<__nv_bfloat16, __nv_bfloat16>(p, st)));
  else
    CUDA_TRY((launch_norm<float, float>(p, st)));
  return GPTQ_OK;
}

}  // namespace gptq
