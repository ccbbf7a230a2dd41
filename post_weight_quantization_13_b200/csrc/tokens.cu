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

constexpr int kMaxStages = 8;            // of a streaming kernel's ring
constexpr int kStreamChunks = 2;         // chunks of eight elements a thread of the streaming norm has
constexpr int kStreamMin = 1024;         // elements of the narrowest rows the streaming kernels take
constexpr int kSmemPerSm = 227 * 1024;

// Chunk i of the thread's share of a row of d elements; zero past the end.
template <typename T>
__device__ __forceinline__ Raw8<T> load_chunk(const T* __restrict__ row, int i, int d, bool vec) {
  const int c0 = 8 * (threadIdx.x + i * blockDim.x);
  return c0 < d ? load8(row + c0, d - c0, vec) : zero8<T>();
}

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
  __device__ __forceinline__ float sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return exchange(v, 0.f, [](float x) {
      // the warps' sums are in the first lanes: as many steps as they need
      // leave the total in all of those
      const int warps = blockDim.x >> 5;
      if (warps <= 4) {
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        return __shfl_sync(0xffffffffu, x, 0);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      return x;
    });
  }
  __device__ __forceinline__ uint32_t max_u32(uint32_t v) {
    return exchange(__reduce_max_sync(0xffffffffu, v), 0u,
                    [](uint32_t x) { return __reduce_max_sync(0xffffffffu, x); });
  }
  __device__ __forceinline__ int sum_s32(int v) {
    return exchange(__reduce_add_sync(0xffffffffu, v), 0, [](int x) { return __reduce_add_sync(0xffffffffu, x); });
  }
};

// A row in registers, top its largest magnitude (fp32 bits) over this thread's
// elements, to codes, scale and sum.
template <int NV>
__device__ __forceinline__ void quantize_row(const Pair (&v)[NV][4], uint32_t top, int d, RowReduce& red,
                                             int8_t* __restrict__ q, float* __restrict__ scale,
                                             int32_t* __restrict__ sum) {
  const TokenScale s(red.max_u32(top));
  int total = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c0 = 8 * (threadIdx.x + i * blockDim.x);
    if (c0 >= d) continue;
    const uint2 w = s.codes(v[i]);
    total = __dp4a((int)w.x, 0x01010101, __dp4a((int)w.y, 0x01010101, total));
    if (c0 + 8 <= d) {
      *reinterpret_cast<uint2*>(q + c0) = w;
    } else {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (c0 + u < d) q[c0 + u] = (int8_t)((u < 4 ? w.x : w.y) >> (8 * (u & 3)));
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
  Raw8<T> r[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) r[i] = load_chunk(X + t * ldx, i, d, vec);
  Pair v[NV][4];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    top = magnitude(r[i], top);
#pragma unroll
    for (int u = 0; u < 4; ++u) v[i][u] = get2(r[i], u);
  }
  quantize_row<NV>(v, magnitude_bits<T>(top), d, red, q + t * ldq, scale + t, sum + t);
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
  int stages, stage_bytes;  // of the streaming kernel
  uint32_t* status;
  // 16-byte access per operand
  int vec_h, vec_y, vec_post_weight, vec_post_bias, vec_gate, vec_weight, vec_bias, vec_h_out, vec_x;
};

// A norm's weight and bias (or a gate) at the thread's columns.  kEarly: held
// in registers from the start, so that no load waits behind a statistic; else
// fetched where they are used, for want of registers.
template <typename T, int NV, bool kEarly>
struct Vector {
  const T* p;
  int d, vec;
  Raw8<T> r[kEarly ? NV : 1];
  __device__ __forceinline__ Vector(const void* p_, int d_, int vec_) : p((const T*)p_), d(d_), vec(vec_) {
    if (kEarly && p) {
#pragma unroll
      for (int i = 0; i < NV; ++i) r[kEarly ? i : 0] = load_chunk(p, i, d, vec);
    }
  }
  __device__ __forceinline__ explicit operator bool() const { return p != nullptr; }
  __device__ __forceinline__ Raw8<T> chunk(int i) const {
    return kEarly ? r[kEarly ? i : 0] : load_chunk(p, i, d, vec);
  }
};

// Zero past the row's end, so that nothing there reaches a statistic.
template <int NV>
__device__ __forceinline__ void clear_past(Pair (&v)[NV][4], int d) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c0 = 8 * (threadIdx.x + i * blockDim.x);
    if (c0 + 8 <= d) continue;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float2 f = v[i][u].f();
      v[i][u] = Pair(c0 + 2 * u < d ? f.x : 0.f, c0 + 2 * u + 1 < d ? f.y : 0.f);
    }
  }
}

// The row without its mean where that is asked for, and 1 / sqrt(mean v^2 +
// eps).  kTail: rows may end inside a chunk or leave threads without one.
template <int NV, bool kTail>
__device__ __forceinline__ float norm_statistic(Pair (&v)[NV][4], const NormParams& p, RowReduce& red) {
  const float inv_d = 1.f / (float)p.d;
  if (p.layer) {
    Pair s(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) s = add2(s, v[i][u]);
    const Pair mean(-red.sum(s.f().x + s.f().y) * inv_d);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) v[i][u] = add2(v[i][u], mean);
    clear_past(v, p.d);
  }
  Pair s2(0.f);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int u = 0; u < 4; ++u) s2 = fma2(v[i][u], v[i][u], s2);
  return rsqrtf(fmaf(red.sum(s2.f().x + s2.f().y), inv_d, p.eps));
}

// v * r * weight (+ bias)
template <int NV, typename V, typename B>
__device__ __forceinline__ void norm_apply(Pair (&v)[NV][4], float r, const V& w, const B& b) {
  const Pair rr(r);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const auto rw = w.chunk(i);
#pragma unroll
    for (int u = 0; u < 4; ++u) v[i][u] = mul2(mul2(v[i][u], rr), get2(rw, u));
    if (b) {
      const auto rb = b.chunk(i);
#pragma unroll
      for (int u = 0; u < 4; ++u) v[i][u] = add2(v[i][u], get2(rb, u));
    }
  }
}

template <int NV, bool kTail, typename T>
__device__ __forceinline__ void store_row(T* __restrict__ row, const Pair (&v)[NV][4], int d, bool vec) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c0 = 8 * (threadIdx.x + i * blockDim.x);
    if (c0 < d) store8(row + c0, v[i], kTail ? d - c0 : 8, kTail ? vec : true);
  }
}

// One token: h' = alpha h + beta gate * post(y);  x = pre(h') in 16/32 bits
// and/or int8.  The pre-norm works on h' before it is rounded to its stored
// type.  h(i), y(i) and gate(i) give the operands' chunks; release() is called
// once by every thread when the whole row has been read by all of them.
template <typename T, typename H, int NV, bool kTail, typename LoadH, typename LoadY, typename LoadGate, typename V,
          typename B, typename Release>
__device__ __forceinline__ void norm_token(const NormParams& p, int64_t t, RowReduce& red, LoadH h, LoadY y,
                                           LoadGate gate, const V& post_weight, const B& post_bias, const V& weight,
                                           const B& bias, Release release) {
  const int d = p.d;
  const Pair alpha(p.alpha);
  Pair v[NV][4];
  if (p.y) {
    const Pair beta(p.beta);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Raw8<T> r = y(i);
#pragma unroll
      for (int u = 0; u < 4; ++u) v[i][u] = get2(r, u);
    }
    if (post_weight) norm_apply<NV>(v, norm_statistic<NV, kTail>(v, p, red), post_weight, post_bias);
    if (p.gate) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const Raw8<T> r = gate(i);
#pragma unroll
        for (int u = 0; u < 4; ++u) v[i][u] = mul2(v[i][u], get2(r, u));
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Raw8<H> r = h(i);
#pragma unroll
      for (int u = 0; u < 4; ++u) v[i][u] = fma2(v[i][u], beta, mul2(alpha, get2(r, u)));
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Raw8<H> r = h(i);
#pragma unroll
      for (int u = 0; u < 4; ++u) v[i][u] = mul2(alpha, get2(r, u));
    }
  }
  clear_past(v, d);
  if (p.h_out) store_row<NV, kTail>((H*)p.h_out + t * p.ldh_out, v, d, p.vec_h_out);
  if (!p.weight) return;
  const float r = norm_statistic<NV, kTail>(v, p, red);
  release();
  norm_apply<NV>(v, r, weight, bias);
  if (p.x) store_row<NV, kTail>((T*)p.x + t * p.ldx, v, d, p.vec_x);
  if (p.q) {
    clear_past(v, d);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 f = v[i][u].f();
        top = max(max(top, __float_as_uint(f.x) & 0x7fffffffu), __float_as_uint(f.y) & 0x7fffffffu);
      }
    quantize_row<NV>(v, top, d, red, p.q + t * p.ldq, p.scale + t, p.sum + t);
  }
}

// A row a warp or a block, every operand straight to registers: few tokens,
// narrow rows, unaligned rows.
template <typename T, typename H, int NV>
__global__ void __launch_bounds__(1024) norm_tokens_kernel(const __grid_constant__ NormParams p) {
  __shared__ uint32_t buf[64];
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= p.tokens) return;
  const int d = p.d;
  RowReduce red(buf);
  using V = Vector<T, NV, NV == 1>;
  Raw8<H> h[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) h[i] = load_chunk((const H*)p.h + t * p.ldh, i, d, p.vec_h);
  const Vector<T, NV, true> y(p.y ? (const T*)p.y + t * p.ldy : nullptr, d, p.vec_y);
  const V gate(p.gate ? (const T*)p.gate + t * p.ldgate : nullptr, d, p.vec_gate);
  const V post_weight(p.post_weight, d, p.vec_post_weight), post_bias(p.post_bias, d, p.vec_post_bias);
  const V weight(p.weight, d, p.vec_weight), bias(p.bias, d, p.vec_bias);
  norm_token<T, H, NV, true>(
      p, t, red, [&](int i) { return h[i]; }, [&](int i) { return y.chunk(i); }, [&](int i) { return gate.chunk(i); },
      post_weight, post_bias, weight, bias, [] {});
}

// ------------------------------------------------------- streaming kernels
// Many tokens of wide, aligned rows: persistent blocks whose rows arrive in a
// ring of shared-memory stages by bulk copies, the next rows' while this one
// is worked on, so memory never waits for a statistic.
struct Ring {
  uint8_t* at;
  uint64_t* full;
  int stages, stage_bytes, s;
  uint32_t phase;
  bool gave_up;  // after a wait that gave up the block runs on without waiting, on whatever is there
  uint32_t* status;
  __device__ __forceinline__ Ring(uint8_t* at_, uint64_t* full_, int stages_, int stage_bytes_, uint32_t* status_)
      : at(at_), full(full_), stages(stages_), stage_bytes(stage_bytes_), s(0), phase(0), gave_up(false),
        status(status_) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
      fence_mbar_init();
    }
    __syncthreads();
  }
  __device__ __forceinline__ uint8_t* stage() const { return at + (size_t)s * stage_bytes; }
  __device__ __forceinline__ void wait() {
    if (!gave_up && !mbar_wait(&full[s], phase)) {
      gave_up = true;
      raise_status(status, ST_TIMEOUT);
    }
  }
  __device__ __forceinline__ void advance() {
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
  }
};

template <typename T>
__device__ __forceinline__ Raw8<T> read8(const void* row, int c) {
  return load8((const T*)row + 8 * c, 8, true);
}

template <typename T>
__global__ void __launch_bounds__(1024) quantize_stream_kernel(const T* __restrict__ X, int64_t tokens, int d,
                                                               int64_t ldx, int8_t* __restrict__ q, int64_t ldq,
                                                               float* __restrict__ scale, int32_t* __restrict__ sum,
                                                               int stages, uint32_t* status) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t buf[64];
  __shared__ uint64_t full[kMaxStages];
  grid_launch_dependents();
  const int chunks = d / 8;
  const uint32_t bytes = (uint32_t)(d * sizeof(T));
  Ring ring(smem, full, stages, (int)bytes, status);
  auto fetch = [&](int64_t t, int s) {  // one thread
    mbar_arrive_expect_tx(&full[s], bytes);
    bulk_load(smem + (size_t)s * bytes, X + t * ldx, bytes, &full[s]);
  };
  if (threadIdx.x == 0)
    for (int s = 0; s < stages && blockIdx.x + (int64_t)s * gridDim.x < tokens; ++s)
      fetch(blockIdx.x + (int64_t)s * gridDim.x, s);
  RowReduce red(buf);
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    ring.wait();
    const uint8_t* row = ring.stage();
    uint32_t top = 0;
#pragma unroll 2
    for (int c = threadIdx.x; c < chunks; c += blockDim.x) top = magnitude(read8<T>(row, c), top);
    const TokenScale ts(red.max_u32(magnitude_bits<T>(top)));
    int total = 0;
#pragma unroll 2
    for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
      const Raw8<T> r = read8<T>(row, c);
      Pair v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = get2(r, u);
      const uint2 w = ts.codes(v);
      total = __dp4a((int)w.x, 0x01010101, __dp4a((int)w.y, 0x01010101, total));
      *reinterpret_cast<uint2*>(q + t * ldq + 8 * c) = w;
    }
    total = red.sum_s32(total);  // its barrier lies behind every read of the stage
    if (threadIdx.x == 0) {
      scale[t] = ts.scale;
      sum[t] = total;
      const int64_t next = t + (int64_t)stages * gridDim.x;
      if (next < tokens) fetch(next, ring.s);
    }
    ring.advance();
  }
}

// A thread has 16 elements of the row: with 8, what a row costs beside its
// elements (reductions, addresses) bound the kernel; unrolled over 32 the code
// left the instruction cache; and in loops over shared memory the weights had
// to come from L2 for every row, where here they stay in registers for all of
// a block's rows (8192 rows of 4096 bf16 with both norms and a gate: 87, 68
// and 76 us).
template <typename T, typename H, int MaxThreads>
__global__ void __launch_bounds__(MaxThreads, 1) norm_stream_kernel(const __grid_constant__ NormParams p) {
  constexpr int NV = kStreamChunks;
  using V = Vector<T, NV, true>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t buf[64];
  __shared__ uint64_t full[kMaxStages];
  const int d = p.d, stages = p.stages;
  const uint32_t hb = (uint32_t)(d * sizeof(H)), tb = (uint32_t)(d * sizeof(T));
  const bool gates = p.gate && p.ldgate;  // a gate for each token comes with the row
  const uint32_t bytes = hb + (p.y ? tb : 0u) + (gates ? tb : 0u);
  Ring ring(smem, full, stages, p.stage_bytes, p.status);
  auto fetch = [&](int64_t t, int s) {  // one thread
    uint8_t* at = smem + (size_t)s * p.stage_bytes;
    mbar_arrive_expect_tx(&full[s], bytes);
    bulk_load(at, (const H*)p.h + t * p.ldh, hb, &full[s]);
    at += hb;
    if (p.y) {
      bulk_load(at, (const T*)p.y + t * p.ldy, tb, &full[s]);
      at += tb;
    }
    if (gates) bulk_load(at, (const T*)p.gate + t * p.ldgate, tb, &full[s]);
  };
  if (threadIdx.x == 0)
    for (int s = 0; s < stages && blockIdx.x + (int64_t)s * gridDim.x < p.tokens; ++s)
      fetch(blockIdx.x + (int64_t)s * gridDim.x, s);
  RowReduce red(buf);
  const V post_weight(p.post_weight, d, 1), weight(p.weight, d, 1), gate(gates ? nullptr : p.gate, d, 1);
  const Vector<T, NV, false> post_bias(p.post_bias, d, 1), bias(p.bias, d, 1);  // no registers left for these
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    ring.wait();
    const H* const h = (const H*)ring.stage();
    const T* const y = (const T*)(h + d);
    const T* const g = y + (p.y ? d : 0);
    norm_token<T, H, NV, false>(
        p, t, red, [&](int i) { return load_chunk(h, i, d, true); }, [&](int i) { return load_chunk(y, i, d, true); },
        [&](int i) { return gates ? load_chunk(g, i, d, true) : gate.chunk(i); }, post_weight, post_bias, weight, bias,
        [&] {
          // the barrier of the pre-norm's statistic lies behind every read
          const int64_t next = t + (int64_t)stages * gridDim.x;
          if (threadIdx.x == 0 && next < p.tokens) fetch(next, ring.s);
        });
    ring.advance();
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

// Chunks a thread for rows straight to registers.  A few rows are a matter of
// latency: the fewest chunks with which 1024 threads hold one.  Many are a
// matter of instructions and bytes in flight: four, in whole warps up to 1024
// elements.
int row_chunks(int d, int64_t tokens, int sms) {
  if (tokens > 4 * sms) return d <= 256 ? 1 : d <= 512 ? 2 : 4;
  return d <= 1024 * 8 ? 1 : d <= 1024 * 16 ? 2 : 4;
}

// Whether the streaming kernel takes the call: rows a block wide whose bytes
// bulk copies can move (16-byte addresses and sizes; a vector's loads too),
// and enough of them to fill every block's ring more than once.
bool streams(const NormParams& p, int sms) {
  return p.weight && p.d >= kStreamMin && p.d <= 1024 * 8 * kStreamChunks && p.d % 8 == 0 && p.tokens > 4 * sms && p.vec_h && (!p.y || p.vec_y) &&
         (!p.gate || p.vec_gate) && p.vec_weight && (!p.bias || p.vec_bias) && (!p.post_weight || p.vec_post_weight) &&
         (!p.post_bias || p.vec_post_bias) && (!p.h_out || p.vec_h_out) && (!p.x || p.vec_x);
}

// The streaming kernels' blocks: threads for `each` elements of a row of d,
// as many blocks as `warps` warps an SM make, and the stages that then fit
// (0: not two).
struct StreamShape {
  int threads, blocks, stages;
  StreamShape(int d, int each, int warps, int stage_bytes) {
    threads = std::min(1024, ((d + each - 1) / each + 31) / 32 * 32);
    blocks = std::max(1, warps * 32 / threads);
    for (;; --blocks) {  // fewer blocks where their rings do not fit
      stages = std::min(kMaxStages, (kSmemPerSm / blocks - 2048) / stage_bytes);
      if (stages >= 2) break;
      stages = 0;
      if (blocks == 1) break;
    }
  }
};

template <typename T>
cudaError_t launch_quantize(const T* X, int64_t tokens, int d, int64_t ldx, int8_t* q, int64_t ldq, float* scale,
                            int32_t* sum, cudaStream_t st) {
  const bool vec = (uintptr_t)X % 16 == 0 && (ldx * (int64_t)sizeof(T)) % 16 == 0;
  const int sms = device_info().sms;
  if (d >= kStreamMin && d % 8 == 0 && tokens > 4 * sms && vec) {
    const StreamShape shape(d, 32, 32, d * (int)sizeof(T));
    if (shape.stages) {
      uint32_t* status = nullptr;
      cudaError_t e = int8_status_word(&status);
      const int smem = shape.stages * d * (int)sizeof(T);
      if (e == cudaSuccess) e = ensure_smem_limit((const void*)quantize_stream_kernel<T>, smem);
      if (e != cudaSuccess) return e;
      const unsigned grid = (unsigned)std::min<int64_t>(tokens, (int64_t)shape.blocks * sms);
      quantize_stream_kernel<T><<<grid, shape.threads, smem, st>>>(X, tokens, d, ldx, q, ldq, scale, sum, shape.stages,
                                                                    status);
      note_launch();
      return cudaGetLastError();
    }
  }
  const int nv = row_chunks(d, tokens, sms);
  const dim3 block = row_block(d, nv);
  const unsigned grid = (unsigned)((tokens + block.y - 1) / block.y);
  if (nv == 1)
    quantize_tokens_kernel<T, 1><<<grid, block, 0, st>>>(X, tokens, d, ldx, q, ldq, scale, sum, vec);
  else if (nv == 2)
    quantize_tokens_kernel<T, 2><<<grid, block, 0, st>>>(X, tokens, d, ldx, q, ldq, scale, sum, vec);
  else
    quantize_tokens_kernel<T, 4><<<grid, block, 0, st>>>(X, tokens, d, ldx, q, ldq, scale, sum, vec);
  note_launch();
  return cudaGetLastError();
}

template <typename T, typename H, int MaxThreads>
cudaError_t launch_stream(const NormParams& p, const StreamShape& shape, cudaStream_t st) {
  const int smem = p.stages * p.stage_bytes;
  const cudaError_t e = ensure_smem_limit((const void*)norm_stream_kernel<T, H, MaxThreads>, smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)std::min<int64_t>(p.tokens, (int64_t)shape.blocks * device_info().sms);
  norm_stream_kernel<T, H, MaxThreads><<<grid, shape.threads, smem, st>>>(p);
  note_launch();
  return cudaGetLastError();
}

template <typename T, typename H, int NV>
cudaError_t launch_rows(const NormParams& p, cudaStream_t st) {
  const dim3 block = row_block(p.d, NV);
  norm_tokens_kernel<T, H, NV><<<(unsigned)((p.tokens + block.y - 1) / block.y), block, 0, st>>>(p);
  note_launch();
  return cudaGetLastError();
}

template <typename T, typename H>
cudaError_t launch_norm(NormParams& p, cudaStream_t st) {
  const int sms = device_info().sms;
  if (streams(p, sms)) {
    p.stage_bytes = (int)round_up(p.d * (int)(sizeof(H) + (p.y ? sizeof(T) : 0) + (p.gate && p.ldgate ? sizeof(T) : 0)),
                                  128);
    const StreamShape shape(p.d, 8 * kStreamChunks, 24, p.stage_bytes);
    p.stages = shape.stages;
    // 768 threads leave each 85 registers, which the vectors need; wider rows
    // have to do with 64
    if (p.stages)
      return shape.threads <= 768 ? launch_stream<T, H, 768>(p, shape, st) : launch_stream<T, H, 1024>(p, shape, st);
  }
  const int nv = row_chunks(p.d, p.tokens, sms);
  return nv == 1 ? launch_rows<T, H, 1>(p, st) : nv == 2 ? launch_rows<T, H, 2>(p, st) : launch_rows<T, H, 4>(p, st);
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
  CUDA_TRY(int8_status_word(&p.status));
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
