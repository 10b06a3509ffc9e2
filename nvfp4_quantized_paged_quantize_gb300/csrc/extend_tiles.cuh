// extend_tiles.cuh -- what the extend attention kernels share: the layout of
// f16 operand tiles in shared memory and the conversions into it.
#pragma once

#include "nvfp4kv_device.cuh"

namespace nvfp4kv {

constexpr uint32_t kLBO = 128;   // next core matrix along K
constexpr uint32_t kSBO = 2048;  // next 8-row (N) group: 16 core matrices of 128 B

// byte offset of element (row, k) in a K-major f16 tile / (mn, k) in an MN-major one
__device__ __forceinline__ uint32_t kmajor_off(int row, int k) {
  return (uint32_t)(row >> 3) * kSBO + (uint32_t)(k >> 3) * kLBO + (uint32_t)(row & 7) * 16 + (uint32_t)(k & 7) * 2;
}
__device__ __forceinline__ uint32_t mnmajor_off(int mn, int k) {
  return (uint32_t)(mn >> 3) * kSBO + (uint32_t)(k >> 3) * kLBO + (uint32_t)(k & 7) * 16 + (uint32_t)(mn & 7) * 2;
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t f16x2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 8 bf16 -> 8 f16 (round to nearest; exact for 2^-14 <= |x| <= 65504)
__device__ __forceinline__ uint4 bf16x8_to_f16x8(const uint4& x) {
  return make_uint4(f16x2_bits(bf16_to_f32(x.x & 0xFFFFu), bf16_to_f32(x.x >> 16)),
                    f16x2_bits(bf16_to_f32(x.y & 0xFFFFu), bf16_to_f32(x.y >> 16)),
                    f16x2_bits(bf16_to_f32(x.z & 0xFFFFu), bf16_to_f32(x.z >> 16)),
                    f16x2_bits(bf16_to_f32(x.w & 0xFFFFu), bf16_to_f32(x.w >> 16)));
}

// 8 E4M3 bytes (a uint2) -> 8 f16 (exact)
__device__ __forceinline__ uint4 e4m3x8_to_f16x8(uint32_t lo, uint32_t hi) {
  return make_uint4(e4m3x2_to_f16x2(lo & 0xFFFFu), e4m3x2_to_f16x2(lo >> 16), e4m3x2_to_f16x2(hi & 0xFFFFu),
                    e4m3x2_to_f16x2(hi >> 16));
}

}  // namespace nvfp4kv
