// scoring.cuh -- what the scored attention calls do to a score before the
// softmax: a cap through tanh, computed on the FMA pipe two scores at a time.
#pragma once

#include <cstdint>

#include "nvfp4kv_device.cuh"

namespace nvfp4kv {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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
// A slope in base-2 units per token, kept finite: the query's own key lies at
// distance 0, and infinity times 0 would be NaN.
__device__ __forceinline__ float base2_slope(float slope) {
  constexpr float kMax = 0x1.fffffep+127f;
  return fminf(fmaxf(slope * kLog2e, -kMax), kMax);
}

// The largest and the smallest of three.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
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

// tanh away from 0: 1 - 2 / (e^{2|x|} + 1) with the sign of x.  For |x| > 1 the
// value is above 0.76, so the error of the exponential and the quotient (a few
// 1e-7 of 2 / (e^2 + 1)) stays below fp32's last place of it; for |x| > 0.6 it is
// above 0.53 and off by 2e-7 of it at most.
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

// a * tanh(c S) + add for many scores S with the same factors, in three forms.
//   far from the cap (|c S| <= 0.4, the usual case): a polynomial whose
//     coefficients hold both factors, S Q(S^2) with Q of degree 3: five packed
//     operations a pair, the last of which adds;
//   |c S| <= 0.6: x Q(x^2), x = c S, Q of degree 4: eight;
//   any: the second form where |c S| <= 0.6, elsewhere a (1 - 2 / (e^{2 |c S|} + 1))
//     with the sign of S, two special-function operations a score.
// Both Q were fitted here in the relative maximum norm (9.8e-8 and 7.3e-8 before
// rounding).  The exponential alone would do for the last form, but its error is
// one of a (2^-23 a): scores far from the cap, which take this form when another
// row of the warp needs it, would lose what a large cap leaves of them.  (A packed
// multiply-add reads three register pairs and takes 2.6 cycles of a scheduler, so
// a shorter form is worth a branch per tile.)
struct CapPoly {
  float c, a;
  float far, near;  // the first form holds for |S| <= far (-1: never), the second up to near
  float2 k[4];      // the first form's coefficients, each twice, as the packed operations take them
};

inline CapPoly cap_poly(double c, double a) {
  constexpr double fit[4] = {0x1.fffffcp-1, -0x1.55502ap-2, 0x1.0fca24p-3, -0x1.858f2p-5};
  if (c > 0x1p+100) c = 0x1p+100;  // finite: it may meet a zero
  CapPoly p;
  p.c = (float)c;
  p.a = (float)a;
  p.near = (float)(0.6 / c);
  // the last coefficient is the one that leaves fp32's range first
  const double c6 = c * c * c * c * c * c, last = a * c * c6;
  const bool fits = last > 0x1p-110 && last < 0x1p+110 && a * c > 0x1p-110 && a * c < 0x1p+110;
  p.far = fits ? (float)(0.4 / c) : -1.0f;
  double f = fits ? a * c : 0.0;
  for (int i = 0; i < 4; ++i, f *= c * c) {
    const float k = (float)(fit[i] * f);
    p.k[i] = make_float2(k, k);
  }
  return p;
}

__device__ __forceinline__ float2 cap_far(float2 S, const CapPoly& p, float2 add) {
  const float2 w = mul2(S, S);
  float2 q = fma2(p.k[3], w, p.k[2]);
  q = fma2(q, w, p.k[1]);
  q = fma2(q, w, p.k[0]);
  return fma2(S, q, add);
}
__device__ __forceinline__ float2 cap_near(float2 S, const CapPoly& p, float2 add) {
  const float2 x = mul2(S, both(p.c)), w = mul2(x, x);
  float2 q = fma2(both(0x1.fb1946p-7f), w, both(-0x1.aad0b8p-5f));
  q = fma2(q, w, both(0x1.1097a4p-3f));
  q = fma2(q, w, both(-0x1.5552a6p-2f));
  q = fma2(q, w, both(0x1.fffffep-1f));
  return fma2(mul2(x, both(p.a)), q, add);
}
__device__ __forceinline__ float2 cap_any(float2 S, const CapPoly& p, float2 add) {
  const float2 near = cap_near(S, p, add);
  const float2 far = fma2(make_float2(tanh_outer(S.x * p.c), tanh_outer(S.y * p.c)), both(p.a), add);
  return make_float2(fabsf(S.x) <= p.near ? near.x : far.x, fabsf(S.y) <= p.near ? near.y : far.y);
}

// S -> a * tanh(c S) in place.
template <int N>
__device__ __forceinline__ void cap_scores(float2 (&x)[N], const CapPoly& p) {
  float hi = x[0].x, lo = x[0].x;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    hi = max3(hi, x[i].x, x[i].y);
    lo = min3(lo, x[i].x, x[i].y);
  }
  if (__all_sync(0xFFFFFFFFu, hi <= p.near && lo >= -p.near)) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = cap_near(x[i], p, both(0.0f));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = cap_any(x[i], p, both(0.0f));
  }
}

}  // namespace nvfp4kv
