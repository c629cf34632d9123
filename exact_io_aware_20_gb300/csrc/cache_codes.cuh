// e4m3 codes of a paged cache for another scale (the device side shared by
// fa_cache_append.cu and fa_cache_pages.cu).
#pragma once

#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace fa {

// Sixteen codes for a scale `ratio` (<= 1) times their own.
__device__ __forceinline__ uint4 rescaled(uint4 v, float ratio) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t out = 0;
    #pragma unroll
    for (int j = 0; j < 2; ++j) {
      const __nv_fp8x2_storage_t two = static_cast<__nv_fp8x2_storage_t>(w[i] >> (16 * j));
      const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3)));
      out |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
                 make_float2(f.x * ratio, f.y * ratio), __NV_SATFINITE, __NV_E4M3))
             << (16 * j);
    }
    w[i] = out;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace fa
