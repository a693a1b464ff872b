// What the kernels of the page-scaled 8-bit cache share: the page scale's
// exponent and the recoding of e4m3 codes into a larger scale.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "pair_math.cuh"

namespace mla {

constexpr int kP8MinExp = -64, kP8MaxExp = 64;  // exponents a page scale can have

__host__ __device__ inline bool p8_aligned(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// 2^e, e the least integer in [kP8MinExp, kP8MaxExp] with amax <= 448 * 2^e.
// With amax = m * 2^x, m in [0.5, 1), and 448 = 0.875 * 2^9: e = x - 9 for
// m <= 0.875, else x - 8. amax >= 0 and not NaN.
__device__ __forceinline__ float p8_scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 126 - 9 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = min(max(e, kP8MinExp), kP8MaxExp);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Two packed fp32 products, as the pair_math.cuh ones.
__device__ __forceinline__ float2 mul_f32x2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(f32x2_pack(a.x, a.y)), "l"(f32x2_pack(b.x, b.y)));
  return f32x2_unpack(d);
}

// Four e4m3 codes times f <= 1, rounded to nearest even again (exact for a
// power of two unless the result is subnormal; NaN stays NaN).
__device__ __forceinline__ uint32_t p8_recode4(uint32_t c, float f) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((c >> (16 * i)) & 0xffffu), __NV_E4M3);
    const float2 v = __half22float2(__half2(h));
    r |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v.x * f, v.y * f), __NV_SATFINITE, __NV_E4M3)
         << (16 * i);
  }
  return r;
}

__device__ __forceinline__ uint4 p8_recode16(uint4 c, float f) {
  return make_uint4(p8_recode4(c.x, f), p8_recode4(c.y, f), p8_recode4(c.z, f), p8_recode4(c.w, f));
}

}  // namespace mla
