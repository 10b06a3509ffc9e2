// nvfp4_block.cuh -- one 16-value block of bf16 values to its E2M1 codes and
// E4M3 scale ("nvfp4-kv-cache-memory-wall", section 2, two-level scaling), for
// the kernels that append to the cache.
#pragma once

#include "nvfp4kv_device.cuh"

namespace nvfp4kv {

// What a tensor's global scale g gives all of its blocks.
struct GlobalScale {
  float g;
  float t6;    // 6 g: the block amax maps onto E2M1's 6
  float r6;    // 1 / t6
  bool t6_ok;  // t6 and 1 / t6 well inside the normal range
};

__device__ __forceinline__ GlobalScale global_scale(float g) {
  GlobalScale s;
  s.g = g;
  s.t6 = __fmul_rn(6.0f, g);
  s.r6 = __frcp_rn(s.t6);
  s.t6_ok = s.t6 >= 0x1p-100f && s.t6 <= 0x1p+100f;
  return s;
}

//   amax = max |x|                       (exact; inputs are bf16)
//   sb   = E4M3(amax / (6 g))            (correctly rounded quotient, RNE, saturating)
//   den  = E4M3val(sb) * g
//   code = E2M1(x / den)                 (correctly rounded quotient, RNE, saturating)
// A block with den == 0 stores signed zeros.
struct BlockScale {
  uint32_t sb;  // E4M3 block scale
  float den, rcp;
  bool fast;    // den, 1 / den and every quotient well inside the normal range
};

__device__ __forceinline__ void set_reciprocal(BlockScale& b, float amax) {
  b.rcp = __frcp_rn(b.den);
  b.fast = b.den >= 0x1p-100f && b.den <= 0x1p+100f && __fmul_rn(amax, b.rcp) < 0x1p+64f;
}

// kEarly: with its reciprocal, else block_codes makes it once the block is known not to be
// zeros.  Early, the appends with FP8 rows take 0.3 % and the normed one 0.7 % less time;
// the plain append takes 0.2 % less without.
template <bool kEarly>
__device__ __forceinline__ BlockScale block_scale(float amax, const GlobalScale& s) {
  // the block scale's quotient: Markstein while the first product stays far
  // from overflow (a quotient below 2^-11 encodes as 0 either way)
  const float sq =
      (s.t6_ok && __fmul_rn(amax, s.r6) < 0x1p+64f) ? div_markstein(amax, s.t6, s.r6) : __fdiv_rn(amax, s.t6);
  BlockScale b;
  b.sb = e4m3_from_f32(sq);
  b.den = __fmul_rn(e4m3_to_f32(b.sb), s.g);
  if constexpr (kEarly) set_reciprocal(b, amax);
  return b;
}

// The codes of 8 kWords of the block's values, value i in nibble i % 8 of word i / 8.
template <bool kEarly, int kWords>
__device__ __forceinline__ void block_codes(const float* f, float amax, BlockScale b, uint32_t (&c)[kWords]) {
  if (b.den == 0.0f) {
    // signed zeros: code 8 for negative inputs
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      c[w] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) c[w] |= (__float_as_uint(f[8 * w + i]) >> 31) << (4 * i + 3);
    }
    return;
  }
  if constexpr (!kEarly) set_reciprocal(b, amax);
  float y[8 * kWords];
  if (b.fast) {
    // a quotient that rounds to zero can come out as +0 for negative x;
    // the sign of x / den is the sign of x (den > 0)
#pragma unroll
    for (int i = 0; i < 8 * kWords; ++i) y[i] = copysignf(div_markstein(f[i], b.den, b.rcp), f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8 * kWords; ++i) y[i] = __fdiv_rn(f[i], b.den);
  }
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    c[w] = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) c[w] |= e2m1x2_from_f32(y[8 * w + 2 * k], y[8 * w + 2 * k + 1]) << (8 * k);
  }
}

struct BlockCodes {
  uint32_t lo, hi;  // codes of values 0-7 and 8-15, value i in nibble i % 8
  uint32_t sb;      // E4M3 block scale
};

template <bool kEarly>
__device__ __forceinline__ BlockCodes quantize_block(const float (&f)[16], const GlobalScale& s) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(f[i]));
  const BlockScale b = block_scale<kEarly>(amax, s);
  uint32_t c[2];
  block_codes<kEarly>(f, amax, b, c);
  return BlockCodes{c[0], c[1], b.sb};
}

// Eight packed bf16 (16 bytes) -> fp32.
__device__ __forceinline__ void unpack_bf16x8(const uint4& x, float* f) {
  f[0] = bf16_to_f32(x.x & 0xFFFFu); f[1] = bf16_to_f32(x.x >> 16);
  f[2] = bf16_to_f32(x.y & 0xFFFFu); f[3] = bf16_to_f32(x.y >> 16);
  f[4] = bf16_to_f32(x.z & 0xFFFFu); f[5] = bf16_to_f32(x.z >> 16);
  f[6] = bf16_to_f32(x.w & 0xFFFFu); f[7] = bf16_to_f32(x.w >> 16);
}

// FP8 workspace scales of K and V and what their quotients need.
struct WsScales {
  float sk, sv, rsk, rsv;  // s_ws and RN(1 / s_ws)
  bool sk_fast, sv_fast, unit;
};

inline WsScales ws_scales(float k_ws_scale, float v_ws_scale) {
  WsScales w;
  w.sk = k_ws_scale;
  w.sv = v_ws_scale;
  w.rsk = 1.0f / k_ws_scale;  // host IEEE division: RN(1 / s_ws)
  w.rsv = 1.0f / v_ws_scale;
  w.sk_fast = k_ws_scale >= 0x1p-100f && k_ws_scale <= 0x1p+100f;
  w.sv_fast = v_ws_scale >= 0x1p-100f && v_ws_scale <= 0x1p+100f;
  w.unit = k_ws_scale == 1.0f && v_ws_scale == 1.0f;
  return w;
}

}  // namespace nvfp4kv
