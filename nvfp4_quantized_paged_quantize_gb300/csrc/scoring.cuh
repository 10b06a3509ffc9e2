// scoring.cuh -- what the scored attention calls do to a score before the
// softmax: a cap through tanh, computed on the FMA pipe two scores at a time.
#pragma once

#include <cstdint>

namespace nvfp4kv {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Two fp32 -> two bf16 (round to nearest even), `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two fp32 products / fused multiply-adds per instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)),
        "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// tanh on |x| <= 1: x + x^3 P(x^2), P of degree 5, fitted here to tanh in the
// relative maximum norm (5.5e-8 before rounding; with fp32 steps within 1.5e-7
// of tanh over the whole interval).
__device__ __forceinline__ float2 tanh_unit(float2 x) {
  const float2 u = mul2(x, x);
  float2 p = both(0x1.156afp-10f);
  p = fma2(p, u, both(-0x1.9a364ap-8f));
  p = fma2(p, u, both(0x1.4d9306p-6f));
  p = fma2(p, u, both(-0x1.b642ecp-5f));
  p = fma2(p, u, both(0x1.10ecc4p-3f));
  p = fma2(p, u, both(-0x1.55546cp-2f));
  return fma2(mul2(x, u), p, x);
}

// tanh for |x| > 1: 1 - 2 / (e^{2|x|} + 1) with the sign of x; the value is
// above 0.76 there, so the error of the exponential and the quotient (a few
// 1e-7 of 2 / (e^2 + 1)) stays below fp32's last place of it.
__device__ __forceinline__ float tanh_outer(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fabsf(x) * (2.0f * kLog2e)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 1.0f));
  return copysignf(fmaf(-2.0f, r, 1.0f), x);
}

// x <- tanh(x) for N pairs per lane.  Scores beyond their cap (|x| > 1) are
// rare in practice, so the outer form (two special-function operations a
// score, against nine packed FMA-pipe ones a pair) runs only when some lane of
// the warp holds one.
template <int N>
__device__ __forceinline__ void tanh_warp(float2 (&x)[N]) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
  if (__any_sync(0xFFFFFFFFu, top > 1.0f)) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 t = tanh_unit(x[i]);
      x[i].x = fabsf(x[i].x) > 1.0f ? tanh_outer(x[i].x) : t.x;
      x[i].y = fabsf(x[i].y) > 1.0f ? tanh_outer(x[i].y) : t.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = tanh_unit(x[i]);
  }
}

// S -> tanh(c S) for many scores with one factor c.  While |c S| <= 0.6 (the
// usual case: scores well inside their cap) the factor is part of the
// polynomial's coefficients, S Q(S^2) with Q of degree 4, fitted here in the
// relative maximum norm (7.3e-8 before rounding): six packed operations a pair
// against ten with the separate product and the wider interval.
struct CapPoly {
  float scale;  // c
  float limit;  // the short form holds for |S| <= limit (-1: never)
  float k[5];
};

inline CapPoly cap_poly(double c) {
  constexpr double a[5] = {0x1.fffffep-1, -0x1.5552a6p-2, 0x1.1097a4p-3, -0x1.aad0b8p-5, 0x1.fb1946p-7};
  CapPoly p;
  p.scale = (float)c;
  // the coefficients' range: c^9 a_4 stays a normal number
  p.limit = c >= 0x1p-12 && c <= 0x1p+12 ? (float)(0.6 / c) : -1.0f;
  double f = c;
  for (int i = 0; i < 5; ++i, f *= c * c) p.k[i] = p.limit > 0.0f ? (float)(a[i] * f) : 0.0f;
  return p;
}

template <int N>
__device__ __forceinline__ void cap_scores(float2 (&x)[N], const CapPoly& p) {
  float top[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < N; ++i) top[i & 3] = fmaxf(top[i & 3], fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
  if (__all_sync(0xFFFFFFFFu, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) <= p.limit)) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 w = mul2(x[i], x[i]);
      float2 q = fma2(both(p.k[4]), w, both(p.k[3]));
      q = fma2(q, w, both(p.k[2]));
      q = fma2(q, w, both(p.k[1]));
      q = fma2(q, w, both(p.k[0]));
      x[i] = mul2(x[i], q);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = mul2(x[i], both(p.scale));
    tanh_warp(x);
  }
}

}  // namespace nvfp4kv
