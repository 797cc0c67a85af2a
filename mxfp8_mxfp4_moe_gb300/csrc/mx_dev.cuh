// MXFP8 element conversion shared by the quantisation and the norm kernels.
#pragma once
#include <cuda_fp8.h>

#include "common.cuh"

namespace kmoe {

__device__ __forceinline__ uint8_t e4m3_code(float x, float inv_scale) {
  if (isnan(x)) return 0;
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(x * inv_scale, __NV_SATFINITE, __NV_E4M3));
}

// 8 E4M3 codes, packed little-endian
__device__ __forceinline__ uint2 e4m3_chunk(const float (&v)[8], float inv_scale) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t p[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float a = v[4 * i + 2 * j], b = v[4 * i + 2 * j + 1];
      const float2 f = make_float2(isnan(a) ? 0.f : a * inv_scale, isnan(b) ? 0.f : b * inv_scale);
      p[j] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
    }
    w[i] = p[0] | (p[1] << 16);
  }
  return make_uint2(w[0], w[1]);
}

}  // namespace kmoe
