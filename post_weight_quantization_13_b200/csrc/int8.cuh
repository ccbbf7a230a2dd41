// Device code shared by the 8-bit serving kernels (tokens.cu, int8_mm.cu,
// int8_pair.cu, int8_rows.cu): typed element access, the loops that feed the
// tensor cores, the token quantizer's arithmetic, the products' epilogue.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"

namespace gptq {

// ------------------------------------------------------------ element access
template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Two fp32 values in one 64-bit register pair: an operation on both is one
// instruction (f32x2, sm_100), and these kernels are bound by issuing them.
struct Pair {
  uint64_t v;
  Pair() = default;
  __device__ __forceinline__ Pair(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
  __device__ __forceinline__ explicit Pair(float a) : Pair(a, a) {}
  __device__ __forceinline__ float2 f() const {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
  }
};
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// N (even) values rounded to T, two at a time.
template <int N, typename T>
__device__ __forceinline__ void round_n(const float* v, T* r) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    if constexpr (std::is_same<T, __half>::value)
      *reinterpret_cast<__half2*>(r + i) = __floats2half2_rn(v[i], v[i + 1]);
    else if constexpr (std::is_same<T, __nv_bfloat16>::value)
      *reinterpret_cast<__nv_bfloat162*>(r + i) = __floats2bfloat162_rn(v[i], v[i + 1]);
    else
      r[i] = v[i], r[i + 1] = v[i + 1];
  }
}

// Eight consecutive elements as loaded, in 32-bit words.
template <typename T>
struct Raw8 {
  alignas(16) uint32_t w[2 * sizeof(T)];
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[i]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    } else {
      return __half2float(__ushort_as_half((unsigned short)(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu)));
    }
  }
};
// Elements 2i and 2i + 1.
template <typename T>
__device__ __forceinline__ Pair get2(const Raw8<T>& r, int i) {
  if constexpr (std::is_same<T, __half>::value) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
    return Pair(f.x, f.y);
  } else {
    return Pair(r.get(2 * i), r.get(2 * i + 1));
  }
}
template <typename T>
__device__ __forceinline__ Raw8<T> zero8() {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < 2 * (int)sizeof(T); ++i) r.w[i] = 0u;
  return r;
}
// The `left` (>= 1) first of eight elements lie inside the row, the others
// read as zero.  vec: the address is 16-byte aligned.
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* __restrict__ p, int left, bool vec) {
  Raw8<T> r;
  if (vec && left >= 8) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      reinterpret_cast<uint4*>(r.w)[i] = reinterpret_cast<const uint4*>(p)[i];
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = i < left ? reinterpret_cast<const uint32_t*>(p)[i] : 0u;
  } else {
    const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r.w[i] = (2 * i < left ? (uint32_t)h[2 * i] : 0u) | (2 * i + 1 < left ? (uint32_t)h[2 * i + 1] << 16 : 0u);
  }
  return r;
}
// Eight values rounded to T; those from `left` on lie past the row's end.
template <typename T>
__device__ __forceinline__ void store8(T* __restrict__ p, const Pair (&v)[4], int left, bool vec) {
  alignas(16) T r[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = v[i].f();
    const float a[2] = {f.x, f.y};
    round_n<2>(a, r + 2 * i);
  }
  if (vec && left >= 8) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(r)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = r[i];
  }
}

// ------------------------------------------------------------ tensor cores
// Instruction descriptor of kind::i8: 32-bit integer accumulator (bits 4-5 =
// 2), both operands signed (bits 7-9 and 10-12 = 1) and K-major, N >> 3 at
// bits 17-22, M >> 4 at bits 24-28.
__host__ __device__ constexpr uint32_t idesc_i8(uint32_t M, uint32_t N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// The loops that feed the tensor cores are run by whole warps, so that their
// addresses and descriptors are uniform values; each copy, MMA or arrival is
// done by one lane (`leader`, from elect_lane) under a predicate.  Run by a
// single thread, every tcgen05.mma first moved its operands to uniform
// registers: 58 cycles each, so that a k-tile of 128 bytes took 520 to 600
// cycles to issue where its MMAs take 512 at most.  Addresses are 32-bit and
// stepped by addition; the constant half of a descriptor is kept apart.
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0); }
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t leader;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(leader));
  return leader;
}
// As mbar_wait, false once the limit is past.
__device__ __forceinline__ bool wait_at(uint32_t bar, uint32_t parity, uint64_t limit_ns = kWaitLimitNs) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  if (ok) return true;
  const uint64_t start = globaltimer();
  while (globaltimer() - start <= limit_ns) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
  }
  return false;
}
__device__ __forceinline__ void expect_at(uint32_t leader, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t"
      "@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void tma_load_at(uint32_t leader, uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                            int y) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "@p cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(leader)
      : "memory");
}
// Untiled: bytes (a multiple of 16, possibly 0) from a 16-byte aligned address.
__device__ __forceinline__ void bulk_load_at(uint32_t leader, uint32_t dst, const void* src, uint32_t bytes,
                                             uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.and.b32 q, %2, 0, p;\n\t"
      "@q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "r"(leader)
      : "memory");
}
// K-major operand with 128-byte swizzling (see smem_desc_k_sw128): the low
// word holds the address >> 4, the high word is the same for all.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t smem_addr) { return ((smem_addr >> 4) & 0x3FFF) | (1u << 16); }

// D[tmem] (+)= A[smem] B[smem]^T, signed 8-bit inputs, 32-bit integers;
// kGroup CTAs (cta_group).
template <int kGroup>
__device__ __forceinline__ void umma_i8(uint32_t leader, uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t idesc,
                                        uint32_t accumulate) {
  if constexpr (kGroup == 1)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::i8 [%0], a, b, %4, p;\n\t}" ::"r"(d),
        "r"(a_low), "r"(b_low), "r"(kDescHigh), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::2.kind::i8 [%0], a, b, %4, p;\n\t}" ::"r"(d),
        "r"(a_low), "r"(b_low), "r"(kDescHigh), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void commit_at(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(leader)
      : "memory");
}
// Arrive on both CTAs' barrier at this offset once this thread's MMAs are done.
__device__ __forceinline__ void commit_pair_at(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t"
      "@p tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::
          "r"(bar),
      "h"((uint16_t)3), "r"(leader)
      : "memory");
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// A block that gave up a wait lets the copies it has under way land before its
// shared memory goes to another.
__device__ __forceinline__ void let_copies_land() {
  const uint64_t start = globaltimer();
  while (globaltimer() - start < 1000000ull) {
  }
}

// Lets the kernel behind this one (launched to overlap it) begin its set-up.
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ------------------------------------------------------------ token quantizer
// The largest magnitude of a row is taken on the bit patterns, where NaN and
// infinity sort above every finite value.  16-bit types: both halves of a
// word at once; magnitude_bits turns the running maximum into the bits of the
// fp32 value.
template <typename T>
__device__ __forceinline__ uint32_t magnitude(const Raw8<T>& r, uint32_t top) {
#pragma unroll
  for (int i = 0; i < 2 * (int)sizeof(T); ++i)
    top = sizeof(T) == 2 ? __vmaxu2(top, r.w[i] & 0x7fff7fffu) : max(top, r.w[i] & 0x7fffffffu);
  return top;
}
template <typename T>
__device__ __forceinline__ uint32_t magnitude_bits(uint32_t top) {
  if (sizeof(T) == 4) return top;
  const unsigned short h = (unsigned short)max(top & 0xffffu, top >> 16);
  return __float_as_uint(to_f32(*reinterpret_cast<const T*>(&h)));
}

// s = RN(max |x| RN(1/127)), code = clamp(rint(RN(x / s)), -127, 127), fp32.
// A row with NaN or an infinity gets s = NaN and codes of zero.
//
// Eight codes at a time: the quotient rounded to nearest by quot_rn's five
// operations (an x too small for its range has |x / s| < 1/2 either way, its
// code is 0), then rint by adding 1.5 2^23, which leaves the code in the sum's
// low byte; |x / s| stays below 127.5, so nothing needs clamping.  A cheaper
// rint(x RN(1/s)) with the exact quotient only near halfway cases does not
// pay: 16-bit values over a 16-bit maximum fall exactly on them too often
// (half a percent of bf16 values).
struct TokenScale {
  float scale, inv;
  bool some, fast;
  __device__ __forceinline__ explicit TokenScale(uint32_t top) {
    const bool finite = top < 0x7f800000u;
    scale = finite ? __uint_as_float(top) * (1.f / 127.f) : __uint_as_float(0x7fc00000u);
    some = finite && scale > 0.f;
    fast = scale >= 0x1p-60f && scale <= 0x1p60f;
    inv = fast ? __frcp_rn(scale) : 0.f;
  }
  static __device__ __forceinline__ uint32_t pack(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
  }
  __device__ __forceinline__ uint2 codes(const Pair (&x)[4]) const {
    uint32_t b[8];
    if (fast) {
      const Pair y(inv), minus_s(-scale), magic(12582912.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Pair q0 = mul2(x[i], y);
        const Pair q1 = fma2(fma2(q0, minus_s, x[i]), y, q0);
        const Pair q2 = fma2(fma2(q1, minus_s, x[i]), y, q1);
        const float2 m = add2(q2, magic).f();
        b[2 * i] = __float_as_uint(m.x);
        b[2 * i + 1] = __float_as_uint(m.y);
      }
    } else {
      if (!some) return make_uint2(0u, 0u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = x[i].f();
        b[2 * i] = (uint32_t)min(127, max(-127, __float2int_rn(__fdiv_rn(f.x, scale))));
        b[2 * i + 1] = (uint32_t)min(127, max(-127, __float2int_rn(__fdiv_rn(f.y, scale))));
      }
    }
    return make_uint2(pack(b[0], b[1], b[2], b[3]), pack(b[4], b[5], b[6], b[7]));
  }
};

// ------------------------------------------------------------------ epilogue
// g Phi(g), Phi the normal distribution.  0.5 (1 + erf(g / sqrt 2)) cancels where
// Phi vanishes (at g = -5 a tenth of the value was lost), so the smaller tail
// is taken from
//   Phi(-|g|) = exp(-g^2 / 2) t P(t),  t = 1 / (1 + 0.26 |g|),
// where t P(t) is half the scaled complementary error function of
// |g| / sqrt 2: smooth, so that a polynomial of degree 8 in t (least squares
// in the relative error, reweighted towards minimax, to |g| = 14.5, beyond which
// the product is below the normal range) is within 2.9e-8.  In fp32 the result
// is off by 12 roundings near zero and, from g^2's, by about g^2 of them in the
// tail.  (4096 tokens of 4096 > 11008: 243 us, with 1 + erff 242; CUDA's erfcf
// is as accurate and took 266 where 1 + erff took 246.)
__device__ __forceinline__ float gelu(float g) {
  const float t = __fdividef(1.f, fmaf(0.26f, fabsf(g), 1.f));
  float p = 0.030230144f;
  p = fmaf(p, t, -0.151493728f);
  p = fmaf(p, t, 0.248731837f);
  p = fmaf(p, t, -0.147787884f);
  p = fmaf(p, t, 0.158757821f);
  p = fmaf(p, t, 0.0519651882f);
  p = fmaf(p, t, 0.102788597f);
  p = fmaf(p, t, 0.103050984f);
  p = fmaf(p, t, 0.103757024f);
  const float tail = exp2f(g * g * -0.72134752044f) * (p * t);  // -log2(e) / 2
  return g * (g < 0.f ? tail : 1.f - tail);
}

// The gate's activation in fp32.  tanh's gelu is written through the logistic
// function, 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z)), so that silu and it need
// one exponential and one quotient (__expf and __fdividef: 2 + 1.173 |z| and 2
// units in the last place, so a relative error of 5e-7 near zero and 1e-5 at
// |z| = 80, far below a 16-bit result's step).
__device__ __forceinline__ float activate(float g, int act) {
  if (act == GPTQ_ACT_GELU) return gelu(g);
  const float z = act == GPTQ_ACT_SILU ? g : 1.5957691216057308f * fmaf(0.044715f * g * g, g, g);
  return __fdividef(g, 1.f + __expf(-z));
}

// One product's value from its exact integer sum.
__device__ __forceinline__ float scaled(int acc, int zero, int tsum, float tscale, float wscale) {
  return (float)(acc - zero * tsum) * tscale * wscale;
}

}  // namespace gptq
