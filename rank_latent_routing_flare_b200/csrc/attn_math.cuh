// Arithmetic of the attention kernels' softmax threads.  What bounds these
// threads is the FMA pipe (a paired instruction holds it as long as two
// single ones) and 2^x on the special-function unit (16 a clock and SM).  tanh
// by 2^x and a reciprocal would triple the load of the latter, so where the
// scores are at most half the cap it is a polynomial, s p(s^2), with the
// scale and the cap folded into its coefficients: five FMA slots.
#pragma once

#include "ptx.cuh"

namespace flare {

template <bool NAN_TOO>
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  if (NAN_TOO) asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  else asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float as_f(uint32_t x) { return __uint_as_float(x); }
__device__ __forceinline__ uint64_t f2(uint32_t lo, uint32_t hi) { return f2_pack(as_f(lo), as_f(hi)); }
__device__ __forceinline__ uint64_t f2_dup(float a) { return f2_pack(a, a); }
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Bits [first, last) of the 32 columns from `from` on.
__device__ __forceinline__ uint32_t column_bits(int first, int last, int from) {
  const int lo = max(first - from, 0), hi = min(last - from, 32);
  return lo >= hi ? 0u : (~0u >> (32 - (hi - lo))) << lo;
}

// Largest of N values (a multiple of 8): four chains.  NAN_TOO: NaN if one is
// (else NaN is passed over).
template <int N, bool NAN_TOO = false>
__device__ __forceinline__ float max_of(const uint32_t (&s)[N]) {
  float a[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) a[c] = max3<NAN_TOO>(as_f(s[2 * c]), as_f(s[2 * c + 1]), as_f(s[2 * c + 1]));
#pragma unroll
  for (int k = 8; k < N; k += 8)
#pragma unroll
    for (int c = 0; c < 4; ++c) a[c] = max3<NAN_TOO>(a[c], as_f(s[k + 2 * c]), as_f(s[k + 2 * c + 1]));
  return max3<NAN_TOO>(max3<NAN_TOO>(a[0], a[1], a[2]), a[3], a[3]);
}
// Smallest of N values, likewise.
template <int N>
__device__ __forceinline__ float min_of(const uint32_t (&s)[N]) {
  float a[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) a[c] = fminf(as_f(s[2 * c]), as_f(s[2 * c + 1]));
#pragma unroll
  for (int k = 8; k < N; k += 8)
#pragma unroll
    for (int c = 0; c < 4; ++c)
      asm("min.f32 %0, %1, %2, %3;" : "=f"(a[c]) : "f"(a[c]), "f"(as_f(s[k + 2 * c])), "f"(as_f(s[k + 2 * c + 1])));
  return fminf(fminf(a[0], a[1]), fminf(a[2], a[3]));
}
__device__ __forceinline__ void ex2_pair(uint64_t x, float& e0, float& e1) {
  float x0, x1;
  f2_unpack(x, x0, x1);
  e0 = ex2_mufu(x0);
  e1 = ex2_mufu(x1);
}

// tanh from 2^x and a reciprocal, any argument, given 2 u log2(e): 1 - 2 /
// (1 + e^(2u)).  Absolute error about 1e-7.
__device__ __forceinline__ float tanh_exp(float u2log2e) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2_mufu(u2log2e)));
  return fmaf(-2.f, r, 1.f);
}

// What turns raw products s into scores in log2 units.
struct ScoreOps {
  float c2;           // scale log2(e)
  float u;            // cap: scale / cap; 0 without a cap
  float most;         // products up to here in magnitude take the polynomial
  float out;          // cap log2(e)
  uint64_t k[4];      // f tanh(s u) = s (k0 + k1 w + k2 w^2 + k3 w^3), w = s^2, for |s u| <= 1/2
  __device__ __forceinline__ ScoreOps(float scale, float cap, bool times_out)
      : c2(scale * 1.4426950408889634f), u(cap > 0.f ? scale / cap : 0.f), out(cap * 1.4426950408889634f) {
    const float f = u * (times_out ? out : 1.f), w = u * u;
    k[0] = f2_dup(0x1.ffffeep-1f * f);
    k[1] = f2_dup(-0x1.5542f2p-2f * f * w);
    k[2] = f2_dup(0x1.0e2324p-3f * f * w * w);
    k[3] = f2_dup(-0x1.6bbe38p-5f * f * w * w * w);
    most = f * w * w * w < 1e38f ? (u >= 1e-5f ? 0.5f : 0.0625f) / u : -1.f;
  }
  // Whether products up to `top` in magnitude may take the polynomial: up to
  // half the cap.  Under a cap so large that u^7 may vanish from the
  // coefficients, up to a sixteenth, where its term is below a rounding; under
  // one so small that u^7 may overflow, none.  tanh_any's absolute error of 1e-7
  // cap is then at most 2e-6 of the largest score.
  __device__ __forceinline__ bool small(float top) const { return top <= most; }
  // f tanh(s u) of two products + c
  __device__ __forceinline__ uint64_t poly(uint64_t s, uint64_t c) const {
    const uint64_t w = f2_mul(s, s);
    return f2_fma(s, f2_fma(f2_fma(f2_fma(k[3], w, k[2]), w, k[1]), w, k[0]), c);
  }
  __device__ __forceinline__ float tanh_any(float s) const { return tanh_exp(s * (2.8853900817779268f * u)); }
  // the capped score of one product
  __device__ __forceinline__ float capped(float s) const {
    float a, b;
    f2_unpack(poly(f2_dup(s), f2_dup(0.f)), a, b);
    return small(fabsf(s)) ? a : tanh_any(s) * out;
  }
};

}  // namespace flare
