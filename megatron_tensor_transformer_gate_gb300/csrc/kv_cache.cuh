// kv_cache.cuh — device helpers of the key-value cache's kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "kv_place.h"

namespace tp {

// Two neighbouring elements as fp32.
template <int DT>
__device__ __forceinline__ float2 pair_to_f32(uint32_t u) {
  if constexpr (DT == TP_BF16) return unpack_bf16x2(u);
  if constexpr (DT == TP_F16) return unpack_f16x2(u);
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)u, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// kv_page_of that says in the status word what it refuses.
__device__ __forceinline__ int64_t page_of(const tp_kv_cache& c, int seq,
                                           int pos, int* offset,
                                           unsigned* status) {
  const int64_t page = kv_page_of(c, seq, pos, offset);
  if (page < 0) record_error(status, kDevPage, 40);
  return page;
}

}  // namespace tp
