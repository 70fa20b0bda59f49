// fp8.cuh — E4M3 conversion helpers shared by the quantizing kernels.
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

namespace tp {

constexpr float kE4M3Max = 448.0f;

// Four E4M3 codes, round to nearest even, beyond ±448 saturated, NaN kept.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const __nv_fp8x2_storage_t lo =
      __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi =
      __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Block-scaled quantization: the largest magnitude of a block of 128 gives
// the factor r that codes are made with (q = e4m3(x·r)) and the scale s that
// a code is multiplied by to get its value back.  A block of zeros has s = 1;
// a largest magnitude below 2^-100 counts as 2^-100, so that r stays finite.
constexpr float kBlockAmaxFloor = 7.888609052210118e-31f;   // 2^-100
__device__ __forceinline__ float block_factor(float amax) {
  return __fdiv_rn(kE4M3Max, fmaxf(amax, kBlockAmaxFloor));
}
__device__ __forceinline__ float block_scale(float amax) {
  return amax == 0.0f ? 1.0f
                      : __fdiv_rn(fmaxf(amax, kBlockAmaxFloor), kE4M3Max);
}

}  // namespace tp
