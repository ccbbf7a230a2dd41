// The 8-bit serving path's memory-bound kernels: the int8 weight layout, the
// per-token quantizer, and the norms around a block fused with its gate,
// residual and the quantizer.
//
// Every operand crosses HBM once.  A token's row stays in registers from its
// one load to its one store, or, in the streaming kernels, waits for its turn in
// shared memory: a thread owns NV chunks of eight consecutive elements (one
// 16-byte load for 16-bit types), a row is owned by one warp where 32 * 8 * NV
// elements hold it and by one block otherwise, and the statistics of a row (sums
// of squares, means, the largest magnitude) are reduced by warp shuffles and one
// shared-memory exchange each.  All statistics are fp32; a mean is subtracted before the
// squares are summed, and what its rounding left is taken off after
// (norm_statistic), so that rows far from zero keep their accuracy.
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
constexpr int kStreamMin = 8192;         // elements of rows from which the streaming kernels take them
constexpr int kSmemPerSm = 227 * 1024;
constexpr int kExchange = 2 * 64;        // words of a row's reductions

// A thread's chunks of a row: eight neighbouring elements each.  Rows on 16-byte
// boundaries are cut at multiples of eight.  Else (kShift: odd sizes, where
// successive rows have every alignment) the cuts move to the row's 16-byte
// boundaries, m elements before those multiples, so that all but a row's two
// ends still go by 16-byte accesses for every operand aligned like the one m
// was taken from, as contiguous tensors of one size are.  (Norms of
// 8000 rows of 4001 bf16 by single elements: 120 to 150 us, now 81; 8192 rows
// of 4096: 57.)
template <bool kShift>
struct Cut {
  int m;
  // For rows of d elements like this one, on threads that hold `slots`; 0 in
  // the few cases where they do not hold the shift.
  template <typename T>
  __device__ __forceinline__ Cut(const T* row, int d, int slots) : m(kShift ? (int)((uintptr_t)row / sizeof(T)) & 7 : 0) {
    if (d + m > slots) m = 0;
  }
  __device__ __forceinline__ int start(int i) const {
    return 8 * (int)(threadIdx.x + i * blockDim.x) - (kShift ? m : 0);
  }
  static __device__ __forceinline__ bool inside(int e, int d) { return (!kShift || e >= 0) && e + 8 <= d; }
  // Whether this operand's chunks lie on 16-byte boundaries.
  template <typename T>
  __device__ __forceinline__ bool fits(const T* row) const {
    return !kShift || (((uintptr_t)row - m * sizeof(T)) & 15) == 0;
  }
};
// The chunk that starts at element e (from -7 on) of a row of d elements, in
// global or shared memory; zero outside the row.
template <bool kShift, typename T>
__device__ __forceinline__ Raw8<T> load_chunk(const Cut<kShift>& cut, const T* __restrict__ row, int e, int d) {
  if constexpr (!kShift) {
    return e < d ? load8(row + e, d - e, true) : zero8<T>();
  } else {
    if (cut.fits(row) && cut.inside(e, d)) return load8(row + e, 8, true);
    Raw8<T> r = zero8<T>();
    if (e >= d) return r;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (e + u < 0 || e + u >= d) continue;
      if constexpr (sizeof(T) == 4)
        r.w[u] = reinterpret_cast<const uint32_t*>(row)[e + u];
      else
        r.w[u / 2] |= (uint32_t)reinterpret_cast<const unsigned short*>(row)[e + u] << (16 * (u & 1));
    }
    return r;
  }
}
// The same of a vector in global memory, whose own alignment seldom is the
// rows': two 16-byte loads and a shift by the elements between.
template <bool kShift, typename T>
__device__ __forceinline__ Raw8<T> load_vector(const Cut<kShift>& cut, const T* __restrict__ p, int e, int d) {
  if constexpr (kShift && sizeof(T) == 2) {
    const int r = e & 7, at = e - r;
    if (r && ((uintptr_t)p & 15) == 0 && at >= 0 && at + 16 <= d) {
      const Raw8<T> a = load8(p + at, 8, true), b = load8(p + at + 8, 8, true);
      uint32_t v[8] = {a.w[0], a.w[1], a.w[2], a.w[3], b.w[0], b.w[1], b.w[2], b.w[3]};
#pragma unroll
      for (int j = 0; j < 6; ++j) v[j] = r & 4 ? v[j + 2] : v[j];
#pragma unroll
      for (int j = 0; j < 5; ++j) v[j] = r & 2 ? v[j + 1] : v[j];
      Raw8<T> o;
#pragma unroll
      for (int j = 0; j < 4; ++j) o.w[j] = __funnelshift_r(v[j], v[j + 1], (r & 1) * 16);
      return o;
    }
  }
  return load_chunk<kShift>(cut, p, e, d);
}
template <bool kShift, typename T>
__device__ __forceinline__ void store_chunk(const Cut<kShift>& cut, T* __restrict__ row, int e, int d,
                                            const Pair (&v)[4]) {
  if constexpr (!kShift) {
    if (e < d) store8(row + e, v, d - e, true);
  } else {
    if (cut.fits(row) && cut.inside(e, d)) {
      store8(row + e, v, 8, true);
      return;
    }
    if (e >= d) return;
    alignas(16) T r[8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float2 f = v[u].f();
      const float a[2] = {f.x, f.y};
      round_n<2>(a, r + 2 * u);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (e + u >= 0 && e + u < d) row[e + u] = r[u];
  }
}
// Eight codes from element e, a multiple of eight; q's rows start on 16-byte
// boundaries.
__device__ __forceinline__ void store_codes(int8_t* __restrict__ q, int e, int d, uint2 w) {
  if (e + 8 <= d) {
    *reinterpret_cast<uint2*>(q + e) = w;
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (e + u < d) q[e + u] = (int8_t)((u < 4 ? w.x : w.y) >> (8 * (u & 3)));
  }
}
// Eight elements from e, a multiple of eight, of a row in shared memory that
// begins anywhere: the 16-byte units it touches, shifted (units around the row
// belong to its stage); zero past the row.
template <typename T>
__device__ __forceinline__ Raw8<T> read_across(const T* row, int e, int d) {
  Raw8<T> o = zero8<T>();
  if constexpr (sizeof(T) == 2) {
    if (e >= d) return o;
    const int r = (int)((uintptr_t)row / 2) & 7;
    const T* at = row + e - r;
    const Raw8<T> a = load8(at, 8, true), b = load8(at + 8, 8, true);
    uint32_t v[8] = {a.w[0], a.w[1], a.w[2], a.w[3], b.w[0], b.w[1], b.w[2], b.w[3]};
#pragma unroll
    for (int j = 0; j < 6; ++j) v[j] = r & 4 ? v[j + 2] : v[j];
#pragma unroll
    for (int j = 0; j < 5; ++j) v[j] = r & 2 ? v[j + 1] : v[j];
#pragma unroll
    for (int j = 0; j < 4; ++j) o.w[j] = __funnelshift_r(v[j], v[j + 1], (r & 1) * 16);
    if (e + 8 > d)
#pragma unroll
      for (int j = 0; j < 4; ++j) o.w[j] = e + 2 * j + 1 < d ? o.w[j] : e + 2 * j < d ? o.w[j] & 0xffffu : 0u;
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (e + u < d) o.w[u] = reinterpret_cast<const uint32_t*>(row)[e + u];
  }
  return o;
}

// ------------------------------------------------------------ row reductions
// Reductions over the threads of one row (blockDim.x of them).  Successive
// reductions of a wide row alternate between two exchange buffers, so one
// barrier each is enough: a buffer is written again only after the barrier of
// the reduction in between.
struct RowReduce {
  uint32_t* buf;  // [kExchange]: two buffers, each of two words for a warp
  int parity;
  __device__ __forceinline__ RowReduce(uint32_t* b) : buf(b), parity(0) {}
  template <typename V, typename F>
  __device__ __forceinline__ V exchange(V warp_value, V identity, F combine) {
    if (blockDim.x <= 32) return warp_value;
    V* b = reinterpret_cast<V*>(buf + kExchange / 2 * parity);
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
  // Two sums through one exchange.
  __device__ __forceinline__ float2 sum(float2 v) {
    const auto lanes = [](float2 x) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        x.x += __shfl_xor_sync(0xffffffffu, x.x, o);
        x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
      }
      return x;
    };
    return exchange(lanes(v), make_float2(0.f, 0.f), lanes);
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
// Shifted cuts: an aligned eight of codes comes from a chunk's last 8 - m and
// its right neighbour's first m; a warp's last lane gets those through shared
// memory (edge) behind the barrier of the codes' sum.
template <int NV, bool kShift>
__device__ __forceinline__ void quantize_row(const Cut<kShift>& cut, const Pair (&v)[NV][4], uint32_t top, int d,
                                             RowReduce& red, uint64_t (&edge)[kShift ? 32 * NV : 1],
                                             int8_t* __restrict__ q, float* __restrict__ scale,
                                             int32_t* __restrict__ sum) {
  const TokenScale s(red.max_u32(top));
  const int lane = threadIdx.x & 31, m = cut.m, warps = blockDim.x >> 5;
  const int warp = (threadIdx.x >> 5) + warps * threadIdx.y;  // (several rows of one warp, or one row)
  int total = 0;
  uint64_t last[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = cut.start(i);
    if (!kShift && e >= d) continue;
    const uint2 w = s.codes(v[i]);
    total = __dp4a((int)w.x, 0x01010101, __dp4a((int)w.y, 0x01010101, total));
    if (!kShift || m == 0) {
      if (e < d) store_codes(q, e, d, w);
    } else {
      const uint64_t own = (uint64_t)w.y << 32 | w.x, next = __shfl_down_sync(0xffffffffu, own, 1);
      const uint64_t eight = own >> (8 * m) | next << (64 - 8 * m);
      if (lane < 31 && e + m < d) store_codes(q, e + m, d, make_uint2((uint32_t)eight, (uint32_t)(eight >> 32)));
      if (lane == 0) edge[32 * i + warp] = own;
      last[i] = own;
    }
  }
  if (kShift && warps == 1) __syncwarp();
  total = red.sum_s32(total);
  if (kShift && m && lane == 31) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool inner = (threadIdx.x >> 5) + 1 < warps;
      const uint64_t next = inner        ? edge[32 * i + warp + 1]
                            : i + 1 < NV ? edge[32 * (i + 1 < NV ? i + 1 : i) + warp + 1 - warps]
                                         : 0;
      const uint64_t eight = last[i] >> (8 * m) | next << (64 - 8 * m);
      const int e = cut.start(i) + m;
      if (e < d) store_codes(q, e, d, make_uint2((uint32_t)eight, (uint32_t)(eight >> 32)));
    }
  }
  if (threadIdx.x == 0) {
    *scale = s.scale;
    *sum = total;
  }
}

template <typename T, int NV, bool kShift>
__global__ void __launch_bounds__(1024) quantize_tokens_kernel(const T* __restrict__ X, int64_t tokens, int d,
                                                               int64_t ldx, int8_t* __restrict__ q, int64_t ldq,
                                                               float* __restrict__ scale, int32_t* __restrict__ sum) {
  __shared__ __align__(8) uint32_t buf[kExchange];
  __shared__ uint64_t edge[kShift ? 32 * NV : 1];
  grid_launch_dependents();  // a product behind this kernel sets up beside it
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= tokens) return;  // whole warps: rows of several per block are one warp wide
  RowReduce red(buf);
  const Cut<kShift> cut(X + t * ldx, d, 8 * NV * (int)blockDim.x);
  Raw8<T> r[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) r[i] = load_chunk<kShift>(cut, X + t * ldx, cut.start(i), d);
  Pair v[NV][4];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    top = magnitude(r[i], top);
#pragma unroll
    for (int u = 0; u < 4; ++u) v[i][u] = get2(r[i], u);
  }
  quantize_row<NV, kShift>(cut, v, magnitude_bits<T>(top), d, red, edge, q + t * ldq, scale + t, sum + t);
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
  int stages, stage_bytes;  // of the streaming kernel
  int post_bias_at, bias_at;  // their places in its shared memory, 0: none
  uint32_t* status;
  int aligned;  // every operand's rows start on 16-byte boundaries
};

// A norm's weight and bias (or a gate) at the thread's columns.  kEarly: held
// in registers from the start, so that no load waits behind a statistic; else
// fetched where they are used, for want of registers.
template <typename T, int NV, bool kEarly, bool kShift>
struct Vector {
  const T* p;
  int d;
  Cut<kShift> cut;
  Raw8<T> r[kEarly ? NV : 1];
  __device__ __forceinline__ Vector(const Cut<kShift>& cut_, const void* p_, int d_) : p((const T*)p_), d(d_), cut(cut_) {
    if (kEarly && p) {
#pragma unroll
      for (int i = 0; i < NV; ++i) r[kEarly ? i : 0] = load_vector<kShift>(cut, p, cut.start(i), d);
    }
  }
  __device__ __forceinline__ explicit operator bool() const { return p != nullptr; }
  __device__ __forceinline__ Raw8<T> chunk(int i) const {
    return kEarly ? r[kEarly ? i : 0] : load_vector<kShift>(cut, p, cut.start(i), d);
  }
};

// A norm's bias in the streaming kernel, where the registers are full: in shared
// memory, each thread's chunks written and read by itself; where there is no
// room (at null), fetched when it is used.  (Two layer norms a row, 2000 x 14000:
// 91 us with both biases from L2 for every row, 80 from here.)
template <typename T, int NV, bool kShift>
struct SharedVector {
  Vector<T, NV, false, kShift> from;
  Raw8<T>* at;  // the thread's first chunk
  __device__ __forceinline__ SharedVector(const Cut<kShift>& cut, const void* p, int d, uint8_t* smem, int offset)
      : from(cut, p, d), at(p && offset ? (Raw8<T>*)(smem + offset) + threadIdx.x : nullptr) {
    if (at)
#pragma unroll
      for (int i = 0; i < NV; ++i) at[i * blockDim.x] = from.chunk(i);
  }
  __device__ __forceinline__ explicit operator bool() const { return (bool)from; }
  __device__ __forceinline__ Raw8<T> chunk(int i) const { return at ? at[i * blockDim.x] : from.chunk(i); }
};

// Zero outside the row, so that nothing there reaches a statistic.
template <int NV, bool kShift>
__device__ __forceinline__ void clear_past(const Cut<kShift>& cut, Pair (&v)[NV][4], int d) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = cut.start(i);
    if (cut.inside(e, d)) continue;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float2 f = v[i][u].f();
      const int a = e + 2 * u;
      v[i][u] = Pair(a >= 0 && a < d ? f.x : 0.f, a + 1 >= 0 && a + 1 < d ? f.y : 0.f);
    }
  }
}

// The row without its mean for a layer norm, and 1 / sqrt(mean v^2 + eps).  A
// mean in fp32 is off by a few roundings of its own size, which for rows far
// from zero is much beside their spread: a row of equal values around 1000 gave
// up to 1 for 0.  So the sum of what is left is taken with the sum of its
// squares, in one exchange, and its mean comes off the variance and the row.
// (Layer norms take 2 to 7 % longer for it: 8000 x 4096 before and after a
// block 65.3 us, so 68.4.  Only where the mean is large beside the spread, by
// a branch: 66.6, but 1001 x 11008 from the ring 47 us, so 39.7.)
template <bool kLayer, int NV, bool kShift>
__device__ __forceinline__ float norm_statistic(const Cut<kShift>& cut, Pair (&v)[NV][4], const NormParams& p,
                                                RowReduce& red) {
  const float inv_d = 1.f / (float)p.d;
  Pair s(0.f), s2(0.f);
  if (!kLayer) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) s2 = fma2(v[i][u], v[i][u], s2);
    return rsqrtf(fmaf(red.sum(s2.f().x + s2.f().y), inv_d, p.eps));
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int u = 0; u < 4; ++u) s = add2(s, v[i][u]);
  const Pair mean(-red.sum(s.f().x + s.f().y) * inv_d);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int u = 0; u < 4; ++u) v[i][u] = add2(v[i][u], mean);
  clear_past<NV, kShift>(cut, v, p.d);
  s = Pair(0.f);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      s = add2(s, v[i][u]);
      s2 = fma2(v[i][u], v[i][u], s2);
    }
  const float2 sums = red.sum(make_float2(s.f().x + s.f().y, s2.f().x + s2.f().y));
  const float left = sums.x * inv_d, var = fmaf(-left, left, sums.y * inv_d);
  const Pair minus(-left);  // (also outside the row, where weights, gates and biases are zero)
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int u = 0; u < 4; ++u) v[i][u] = add2(v[i][u], minus);
  return rsqrtf((var < 0.f ? 0.f : var) + p.eps);
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

template <int NV, bool kShift, typename T>
__device__ __forceinline__ void store_row(const Cut<kShift>& cut, T* __restrict__ row, const Pair (&v)[NV][4], int d) {
#pragma unroll
  for (int i = 0; i < NV; ++i) store_chunk<kShift>(cut, row, cut.start(i), d, v[i]);
}

// One token: h' = alpha h + beta gate * post(y);  x = pre(h') in 16/32 bits
// and/or int8.  The pre-norm works on h' before it is rounded to its stored
// type.  h(i), y(i) and gate(i) give the operands' chunks; release() is called
// once by every thread when the whole row has been read by all of them.
template <bool kLayer, typename T, typename H, int NV, bool kShift, typename LoadH, typename LoadY, typename LoadGate, typename V,
          typename B, typename Release>
__device__ __forceinline__ void norm_token(const Cut<kShift>& cut, const NormParams& p, int64_t t, RowReduce& red,
                                           uint64_t (&edge)[kShift ? 32 * NV : 1], LoadH h, LoadY y, LoadGate gate,
                                           const V& post_weight, const B& post_bias, const V& weight, const B& bias,
                                           Release release) {
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
    if (post_weight) norm_apply<NV>(v, norm_statistic<kLayer, NV, kShift>(cut, v, p, red), post_weight, post_bias);
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
  clear_past<NV, kShift>(cut, v, d);
  if (p.h_out) store_row<NV, kShift>(cut, (H*)p.h_out + t * p.ldh_out, v, d);
  if (!p.weight) return;
  const float r = norm_statistic<kLayer, NV, kShift>(cut, v, p, red);
  release();
  norm_apply<NV>(v, r, weight, bias);
  if (p.x) store_row<NV, kShift>(cut, (T*)p.x + t * p.ldx, v, d);
  if (p.q) {
    clear_past<NV, kShift>(cut, v, d);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 f = v[i][u].f();
        top = max(max(top, __float_as_uint(f.x) & 0x7fffffffu), __float_as_uint(f.y) & 0x7fffffffu);
      }
    quantize_row<NV, kShift>(cut, v, top, d, red, edge, p.q + t * p.ldq, p.scale + t, p.sum + t);
  }
}

// A row a warp or a block, every operand straight to registers: few tokens, or
// rows of which several blocks fit an SM, so that one's loads and reductions
// overlap the others'.  One token of 4096 takes 2.2 us, all latency.  8000 of
// them with one RMS norm take 42.8, the bytes alone 40.6; 8192 with both norms
// and a gate 55 (the bytes 41.6): a second statistic for each row, and
// three vectors that every row fetches from L2, not memory (issue slots 65 % used,
// DRAM 46 %).
template <bool kLayer, typename T, typename H, int NV, bool kShift>
__global__ void __launch_bounds__(1024) norm_tokens_kernel(const __grid_constant__ NormParams p) {
  __shared__ __align__(8) uint32_t buf[kExchange];
  __shared__ uint64_t edge[kShift ? 32 * NV : 1];
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= p.tokens) return;
  const int d = p.d;
  RowReduce red(buf);
  using V = Vector<T, NV, NV == 1, kShift>;
  const H* const hr = (const H*)p.h + t * p.ldh;
  const T* const yr = p.y ? (const T*)p.y + t * p.ldy : nullptr;
  const T* const gr = p.gate ? (const T*)p.gate + t * p.ldgate : nullptr;
  const int slots = 8 * NV * (int)blockDim.x;
  const Cut<kShift> cut = yr ? Cut<kShift>(yr, d, slots) : Cut<kShift>(hr, d, slots);
  Raw8<H> h[NV];
  Raw8<T> y[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) h[i] = load_chunk<kShift>(cut, hr, cut.start(i), d);
  if (yr) {
#pragma unroll
    for (int i = 0; i < NV; ++i) y[i] = load_chunk<kShift>(cut, yr, cut.start(i), d);
  }
  const V gate(cut, gr, d);
  const V post_weight(cut, p.post_weight, d), post_bias(cut, p.post_bias, d);
  const V weight(cut, p.weight, d), bias(cut, p.bias, d);
  norm_token<kLayer, T, H, NV, kShift>(
      cut, p, t, red, edge, [&](int i) { return h[i]; }, [&](int i) { return y[i]; }, [&](int i) { return gate.chunk(i); },
      post_weight, post_bias, weight, bias, [] {});
}

// ------------------------------------------------------- streaming kernels
// Many tokens of wide rows: persistent blocks whose rows arrive in a ring of
// shared-memory stages by bulk copies, the next rows' while this one is worked
// on, so memory does not wait for a statistic.  What bounds the norm is its four
// reductions a row, since one block fills an SM (1001 x 11008 layer norms: 44
// us, the bytes alone 24).
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

// One operand's rows on their way to a ring.  kShift: of any alignment.  A copy
// moves the whole 16-byte units that a row touches, so the row stands in its
// stage at its own offset from such a boundary; units that reach past the
// tensor's first or last element are not copied, patch() fills in what those
// two rows then miss.
template <typename T, bool kShift>
struct Source {
  const T* base;
  int64_t ld, tokens;
  int d;
  __device__ __forceinline__ uint32_t room() const {  // of a row in a stage
    return kShift ? ((uint32_t)(d * sizeof(T)) + 15 + 15) & ~15u : (uint32_t)(d * sizeof(T));
  }
  __device__ __forceinline__ uintptr_t row(int64_t t) const { return (uintptr_t)(base + t * ld); }
  __device__ __forceinline__ const T* at(const uint8_t* stage, int64_t t) const {
    return (const T*)(stage + (kShift ? row(t) & 15 : 0));
  }
  __device__ __forceinline__ void range(int64_t t, uintptr_t* from, uintptr_t* to) const {
    *from = row(t);
    *to = *from + d * sizeof(T);
    if (!kShift) return;
    const uintptr_t first = ((uintptr_t)base + 15) & ~(uintptr_t)15;
    const uintptr_t last = (row(tokens - 1) + d * sizeof(T)) & ~(uintptr_t)15;
    *from = max(*from & ~(uintptr_t)15, first);
    *to = min((*to + 15) & ~(uintptr_t)15, last);
  }
  __device__ __forceinline__ uint32_t bytes(int64_t t) const {
    uintptr_t from, to;
    range(t, &from, &to);
    return to > from ? (uint32_t)(to - from) : 0u;
  }
  __device__ __forceinline__ void fetch(uint8_t* stage, int64_t t, uint64_t* bar) const {
    uintptr_t from, to;
    range(t, &from, &to);
    if (to > from) bulk_load(stage + (from - (row(t) & ~(uintptr_t)15)), (const void*)from, (uint32_t)(to - from), bar);
  }
  __device__ __forceinline__ void patch(uint8_t* stage, int64_t t) const {
    uintptr_t from, to;
    range(t, &from, &to);
    T* const mine = const_cast<T*>(at(stage, t));
    const int head = (int)(((int64_t)from - (int64_t)row(t)) / (int64_t)sizeof(T));  // elements before the copy
    const int tail = (int)(((int64_t)to - (int64_t)row(t)) / (int64_t)sizeof(T));    // and its end
    const int i = threadIdx.x;
    if (i < head && i < d) mine[i] = base[t * ld + i];
    if (tail + i < d && i < 16) mine[max(tail, 0) + i] = base[t * ld + max(tail, 0) + i];
    fence_proxy_async_smem();  // a copy writes here next
  }
};

template <typename T, bool kShift>
__global__ void __launch_bounds__(1024) quantize_stream_kernel(const T* __restrict__ X, int64_t tokens, int d,
                                                               int64_t ldx, int8_t* __restrict__ q, int64_t ldq,
                                                               float* __restrict__ scale, int32_t* __restrict__ sum,
                                                               int stages, int stage_bytes, uint32_t* status) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint32_t buf[kExchange];
  __shared__ uint64_t full[kMaxStages];
  grid_launch_dependents();
  const int step = 8 * (int)blockDim.x;
  const Source<T, kShift> source = {X, ldx, tokens, d};
  const Cut<kShift> cut(X + (int64_t)blockIdx.x * ldx, d, d + 7);
  Ring ring(smem, full, stages, stage_bytes, status);
  auto fetch = [&](int64_t t, int s) {  // one thread
    mbar_arrive_expect_tx(&full[s], source.bytes(t));
    source.fetch(smem + (size_t)s * stage_bytes, t, &full[s]);
  };
  if (threadIdx.x == 0)
    for (int s = 0; s < stages && blockIdx.x + (int64_t)s * gridDim.x < tokens; ++s)
      fetch(blockIdx.x + (int64_t)s * gridDim.x, s);
  RowReduce red(buf);
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    ring.wait();
    if (kShift && (t == 0 || t == tokens - 1)) {
      source.patch(ring.stage(), t);
      __syncthreads();
    }
    const T* row = source.at(ring.stage(), t);
    uint32_t top = 0;
#pragma unroll 2
    for (int e = cut.start(0); e < d; e += step) top = magnitude(load_chunk<kShift>(cut, row, e, d), top);
    const TokenScale ts(red.max_u32(magnitude_bits<T>(top)));
    int total = 0;
#pragma unroll 2
    for (int e = 8 * (int)threadIdx.x; e < d; e += step) {
      const Raw8<T> r = kShift ? read_across(row, e, d) : load8(row + e, 8, true);
      Pair v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = get2(r, u);
      const uint2 w = ts.codes(v);
      total = __dp4a((int)w.x, 0x01010101, __dp4a((int)w.y, 0x01010101, total));
      store_codes(q + t * ldq, e, d, w);
    }
    total = red.sum_s32(total);  // its barrier lies behind every read of the stage
    if (threadIdx.x == 0) {
      scale[t] = ts.scale;
      sum[t] = total;
      const int64_t next = t + (int64_t)stages * gridDim.x;
      if (next < tokens && !ring.gave_up) fetch(next, ring.s);
    }
    ring.advance();
  }
  if (ring.gave_up) let_copies_land();
}

// A thread has 16 elements of the row: with 8, what a row costs beside its
// elements (reductions, addresses) bound the kernel; unrolled over 32 the code
// left the instruction cache; and in loops over shared memory the weights had
// to come from L2 for every row, where here they stay in registers for all of
// a block's rows.
template <bool kLayer, typename T, typename H, bool kShift, int MaxThreads>
__global__ void __launch_bounds__(MaxThreads, 1) norm_stream_kernel(const __grid_constant__ NormParams p) {
  constexpr int NV = kStreamChunks;
  using V = Vector<T, NV, true, kShift>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint32_t buf[kExchange];
  __shared__ uint64_t edge[kShift ? 32 * NV : 1];
  __shared__ uint64_t full[kMaxStages];
  const int d = p.d, stages = p.stages;
  const bool gates = p.gate && p.ldgate;  // a gate for each token comes with the row
  const Source<H, kShift> h = {(const H*)p.h, p.ldh, p.tokens, d};
  const Source<T, kShift> y = {(const T*)p.y, p.ldy, p.tokens, d}, g = {(const T*)p.gate, p.ldgate, p.tokens, d};
  const uint32_t y_at = h.room(), g_at = y_at + (p.y ? y.room() : 0u);
  Ring ring(smem, full, stages, p.stage_bytes, p.status);
  auto fetch = [&](int64_t t, int s) {  // one thread
    uint8_t* at = smem + (size_t)s * p.stage_bytes;
    mbar_arrive_expect_tx(&full[s], h.bytes(t) + (p.y ? y.bytes(t) : 0u) + (gates ? g.bytes(t) : 0u));
    h.fetch(at, t, &full[s]);
    if (p.y) y.fetch(at + y_at, t, &full[s]);
    if (gates) g.fetch(at + g_at, t, &full[s]);
  };
  if (threadIdx.x == 0)
    for (int s = 0; s < stages && blockIdx.x + (int64_t)s * gridDim.x < p.tokens; ++s)
      fetch(blockIdx.x + (int64_t)s * gridDim.x, s);
  RowReduce red(buf);
  // a shifted grid is a multiple of eight: all of a block's rows are aligned alike
  const int64_t t0 = blockIdx.x;
  const int slots = 8 * NV * (int)blockDim.x;
  const Cut<kShift> cut = p.y ? Cut<kShift>((const T*)p.y + t0 * p.ldy, d, slots)
                              : Cut<kShift>((const H*)p.h + t0 * p.ldh, d, slots);
  const V post_weight(cut, p.post_weight, d), weight(cut, p.weight, d), gate(cut, gates ? nullptr : p.gate, d);
  const SharedVector<T, NV, kShift> post_bias(cut, p.post_bias, d, smem, p.post_bias_at),
      bias(cut, p.bias, d, smem, p.bias_at);
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    ring.wait();
    uint8_t* const stage = ring.stage();
    if (kShift && (t == 0 || t == p.tokens - 1)) {
      h.patch(stage, t);
      if (p.y) y.patch(stage + y_at, t);
      if (gates) g.patch(stage + g_at, t);
      __syncthreads();
    }
    const H* const hr = h.at(stage, t);
    const T *const yr = y.at(stage + y_at, t), *const gr = g.at(stage + g_at, t);
    norm_token<kLayer, T, H, NV, kShift>(
        cut, p, t, red, edge, [&](int i) { return load_chunk<kShift>(cut, hr, cut.start(i), d); },
        [&](int i) { return load_chunk<kShift>(cut, yr, cut.start(i), d); },
        [&](int i) { return gates ? load_chunk<kShift>(cut, gr, cut.start(i), d) : gate.chunk(i); }, post_weight,
        post_bias, weight, bias, [&] {
          // the barrier of the pre-norm's statistic lies behind every read
          const int64_t next = t + (int64_t)stages * gridDim.x;
          if (threadIdx.x == 0 && next < p.tokens && !ring.gave_up) fetch(next, ring.s);
        });
    ring.advance();
  }
  if (ring.gave_up) let_copies_land();
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
  return lanes <= 32 ? dim3(32, 4) : dim3((unsigned)std::min(1024, (lanes + 31) / 32 * 32), 1);
}

// Chunks a thread for rows straight to registers.  A few rows are a matter of
// latency: the fewest chunks with which 1024 threads hold one.  Many are a
// matter of instructions: two, beside which a row's reductions and addresses
// count for less, up to 16384 elements.
int row_chunks(int d, int64_t tokens, int sms) {
  if (d > 1024 * 16) return 4;
  return tokens > 4 * sms ? (d <= 256 ? 1 : 2) : (d <= 1024 * 8 ? 1 : 2);
}

// Whether a streaming kernel takes the call: enough rows to fill every block's
// ring more than once, and of those the rows so wide that few of their blocks
// fit an SM.  Narrower rows overlap better as many blocks of one row each (norms
// of 8000 x 4096 bf16 and quantized: streaming 60.9 us, else 51.6; 2000 x 8192
// 41.3 and 32.6), but for some on an fp32 residual (both norms and a gate for
// each token, 2000 x 4096 20.7 and 24.7).  Of wider rows, in registers at 32
// elements a thread, those with a gate for each token lose (both norms, 2000 x
// 11008 45 and 54 to 61 us, 8000 x 11008 155 and 187), those that are quantized
// and layer norms without such a gate win (8000 x 11008: RMS and quantized 163
// and 132, two layer norms 205 and 173), which this rule leaves there.  The
// quantizer does so little for a row that of 16-bit types it streams from some
// size on (8000 x 4096: 23.6 us, else 27.7; 2000 x 4096: 7.6 and 7.4; fp32
// 8000 x 4096 29.8 and 28.3).
bool streams_norm(int d, int64_t tokens, int sms) { return d > kStreamMin && tokens > 4 * sms; }
bool streams_quantizer(int d, size_t size, int64_t tokens, int sms) {
  return tokens > 4 * sms && (d >= kStreamMin || (size == 2 && d >= 1024 && tokens * d > 12000000));
}

// Bytes of a row in a stage (Source::room).
int row_room(int d, size_t size, bool shift) {
  const int bytes = d * (int)size;
  return shift ? (bytes + 30) & ~15 : bytes;
}
// Elements that a thread count has to cover: shifted cuts start up to seven early.
int span(int d, bool shift) { return shift ? d + 7 : d; }
// A streaming kernel's grid; its blocks' rows are aligned alike (Cut) when it
// is a multiple of eight.
unsigned stream_grid(int64_t tokens, int blocks, bool shift) {
  const unsigned grid = (unsigned)std::min<int64_t>(tokens, (int64_t)blocks * device_info().sms);
  return shift ? grid & ~7u : grid;
}

// The streaming kernels' blocks: threads for `each` elements of a row of d,
// as many blocks as `warps` warps an SM make, and the stages that then fit
// (0: not two).
struct StreamShape {
  int threads, blocks, stages;
  StreamShape(int d, int each, int warps, int stage_bytes, int fixed_bytes = 0) {
    threads = std::min(1024, ((d + each - 1) / each + 31) / 32 * 32);
    blocks = std::max(1, warps * 32 / threads);
    for (;; --blocks) {  // fewer blocks where their rings do not fit
      stages = std::min(kMaxStages, (kSmemPerSm / blocks - 2048 - fixed_bytes) / stage_bytes);
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
  if (streams_quantizer(d, sizeof(T), tokens, sms)) {
    const bool whole = vec && d % 8 == 0;
    const int stage_bytes = (int)round_up(row_room(d, sizeof(T), !whole), 128);
    const StreamShape shape(span(d, !whole), 32, 32, stage_bytes);
    if (shape.stages) {
      uint32_t* status = nullptr;
      const auto kernel = whole ? quantize_stream_kernel<T, false> : quantize_stream_kernel<T, true>;
      cudaError_t e = int8_status_word(&status);
      const int smem = shape.stages * stage_bytes;
      if (e == cudaSuccess) e = ensure_smem_limit((const void*)kernel, smem);
      if (e != cudaSuccess) return e;
      const unsigned grid = stream_grid(tokens, shape.blocks, !whole);
      kernel<<<grid, shape.threads, smem, st>>>(X, tokens, d, ldx, q, ldq, scale, sum, shape.stages, stage_bytes,
                                                status);
      note_launch();
      return cudaGetLastError();
    }
  }
  const int nv = row_chunks(span(d, !vec), tokens, sms);
  const dim3 block = row_block(span(d, !vec), nv);
  const unsigned grid = (unsigned)((tokens + block.y - 1) / block.y);
  auto launch = [&](auto whole, auto strided) {
    (vec ? whole : strided)<<<grid, block, 0, st>>>(X, tokens, d, ldx, q, ldq, scale, sum);
  };
  if (nv == 1)
    launch(quantize_tokens_kernel<T, 1, false>, quantize_tokens_kernel<T, 1, true>);
  else if (nv == 2)
    launch(quantize_tokens_kernel<T, 2, false>, quantize_tokens_kernel<T, 2, true>);
  else
    launch(quantize_tokens_kernel<T, 4, false>, quantize_tokens_kernel<T, 4, true>);
  note_launch();
  return cudaGetLastError();
}

template <bool kLayer, typename T, typename H, bool kShift, int MaxThreads>
cudaError_t launch_stream(const NormParams& p, const StreamShape& shape, int bias_bytes, cudaStream_t st) {
  const int smem = p.stages * p.stage_bytes + bias_bytes;
  const auto kernel = norm_stream_kernel<kLayer, T, H, kShift, MaxThreads>;
  const cudaError_t e = ensure_smem_limit((const void*)kernel, smem);
  if (e != cudaSuccess) return e;
  kernel<<<stream_grid(p.tokens, shape.blocks, kShift), shape.threads, smem, st>>>(p);
  note_launch();
  return cudaGetLastError();
}

template <bool kLayer, typename T, typename H, int NV>
cudaError_t launch_rows(const NormParams& p, cudaStream_t st) {
  const dim3 block = row_block(span(p.d, !p.aligned), NV);
  const unsigned grid = (unsigned)((p.tokens + block.y - 1) / block.y);
  if (p.aligned)
    norm_tokens_kernel<kLayer, T, H, NV, false><<<grid, block, 0, st>>>(p);
  else
    norm_tokens_kernel<kLayer, T, H, NV, true><<<grid, block, 0, st>>>(p);
  note_launch();
  return cudaGetLastError();
}

template <bool kLayer, typename T, typename H>
cudaError_t launch_norm_kind(NormParams& p, cudaStream_t st) {
  const int sms = device_info().sms;
  const bool whole = p.aligned && p.d % 8 == 0;
  if (p.weight && span(p.d, !whole) <= 1024 * 8 * kStreamChunks && streams_norm(p.d, p.tokens, sms)) {
    p.stage_bytes = (int)round_up(row_room(p.d, sizeof(H), !whole) +
                                      ((p.y ? 1 : 0) + (p.gate && p.ldgate ? 1 : 0)) * row_room(p.d, sizeof(T), !whole),
                                  128);
    const int width = span(p.d, !whole);
    StreamShape shape(width, 8 * kStreamChunks, 24, p.stage_bytes);
    const int vector = shape.threads * kStreamChunks * 8 * (int)sizeof(T), biases = (p.post_bias ? 1 : 0) + (p.bias ? 1 : 0);
    int bias_bytes = 0;
    if (biases) {
      const StreamShape with(width, 8 * kStreamChunks, 24, p.stage_bytes, biases * vector);
      if (with.stages && with.blocks == shape.blocks) {
        shape = with;
        bias_bytes = biases * vector;
        p.post_bias_at = p.post_bias ? shape.stages * p.stage_bytes : 0;
        p.bias_at = p.bias ? shape.stages * p.stage_bytes + bias_bytes - vector : 0;
      }
    }
    p.stages = shape.stages;
    // 768 threads leave each 85 registers, which the vectors need; wider rows
    // have to do with 64
    if (p.stages && whole)
      return shape.threads <= 768 ? launch_stream<kLayer, T, H, false, 768>(p, shape, bias_bytes, st)
                                  : launch_stream<kLayer, T, H, false, 1024>(p, shape, bias_bytes, st);
    if (p.stages)
      return shape.threads <= 768 ? launch_stream<kLayer, T, H, true, 768>(p, shape, bias_bytes, st)
                                  : launch_stream<kLayer, T, H, true, 1024>(p, shape, bias_bytes, st);
  }
  const int nv = row_chunks(span(p.d, !p.aligned), p.tokens, sms);
  return nv == 1   ? launch_rows<kLayer, T, H, 1>(p, st)
         : nv == 2 ? launch_rows<kLayer, T, H, 2>(p, st)
                   : launch_rows<kLayer, T, H, 4>(p, st);
}

template <typename T, typename H>
cudaError_t launch_norm(NormParams& p, bool layer, cudaStream_t st) {
  return layer ? launch_norm_kind<true, T, H>(p, st) : launch_norm_kind<false, T, H>(p, st);
}

bool aligned_rows(const void* p, int64_t ld, gptq_dtype_t t) {  // NULL: it is not read
  return !p || (uintptr_t)p % 16 == 0 && (ld * (t == GPTQ_F32 ? 4 : 2)) % 16 == 0;
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
  const bool layer = a->kind == GPTQ_NORM_LAYER;
  p.aligned = aligned_rows(a->h, a->ldh, a->ht) && aligned_rows(a->y, a->ldy, a->yt) &&
              aligned_rows(a->post_weight, 0, a->yt) && aligned_rows(a->post_bias, 0, a->yt) &&
              aligned_rows(a->gate, a->ldgate, a->yt) && aligned_rows(a->weight, 0, a->yt) &&
              aligned_rows(a->bias, 0, a->yt) && aligned_rows(a->h_out, a->ldh_out, a->ht) &&
              aligned_rows(a->x, a->ldx, a->yt);
  if (a->yt == GPTQ_F16)
    CUDA_TRY((a->ht == GPTQ_F32 ? launch_norm<__half, float>(p, layer, st) : launch_norm<__half, __half>(p, layer, st)));
  else if (a->yt == GPTQ_BF16)
    CUDA_TRY((a->ht == GPTQ_F32 ? launch_norm<__nv_bfloat16, float>(p, layer, st)
                                : launch_norm<__nv_bfloat16, __nv_bfloat16>(p, layer, st)));
  else
    CUDA_TRY((launch_norm<float, float>(p, layer, st)));
  return GPTQ_OK;
}

}  // namespace gptq
