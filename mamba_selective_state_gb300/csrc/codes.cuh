// codes.cuh -- the 8-bit codes of a row with one scale (int8, or e4m3 where
// kFp8), as the state cache and the norm write them and the product reads them.
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

namespace ssd {

// The factor and the scale of a row whose largest value is `big`: products
// with the reciprocals 1 / big and 1 / top, each rounded by itself.
template <bool kFp8>
__device__ __forceinline__ float factor_of(float big) { return __frcp_rn(big) * (kFp8 ? 448.f : 127.f); }
template <bool kFp8>
__device__ __forceinline__ float scale_of(float big) { return big * (kFp8 ? 1.f / 448.f : 1.f / 127.f); }

// A row whose largest value is below this is zeros.  (Chosen for both formats: the
// factor is finite from about 2^-119.2 on for e4m3 and from 2^-121 for int8.)
constexpr float kTiny = 3.009265538105056e-36f;  // 2^-118

template <bool kFp8>
__device__ __forceinline__ uint8_t encode(float y) {
  if (kFp8) return (uint8_t)__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
  return (uint8_t)(int8_t)__float2int_rn(fminf(fmaxf(y, -127.f), 127.f));
}
template <bool kFp8>
__device__ __forceinline__ float decode(uint8_t v) {
  if (kFp8) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(v, __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half*>(&h));
  }
  return (float)(int8_t)v;
}

template <bool kFp8>
__device__ __forceinline__ uint32_t encode4(float4 v, float inv) {
  if (kFp8)
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v.x * inv, v.y * inv), __NV_SATFINITE, __NV_E4M3) |
           (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v.z * inv, v.w * inv), __NV_SATFINITE, __NV_E4M3) << 16;
  // |v inv| <= 127 (1 + 2^-22): the sum with 1.5 * 2^23 rounds it to an integer, ties to even, in its low byte
  // (float-to-integer conversions run at a quarter of the rate)
  const float magic = 12582912.f;
  const uint32_t x = __float_as_uint(__fadd_rn(__fmul_rn(v.x, inv), magic)),
                 y = __float_as_uint(__fadd_rn(__fmul_rn(v.y, inv), magic)),
                 z = __float_as_uint(__fadd_rn(__fmul_rn(v.z, inv), magic)),
                 w = __float_as_uint(__fadd_rn(__fmul_rn(v.w, inv), magic));
  return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
}

}  // namespace ssd
