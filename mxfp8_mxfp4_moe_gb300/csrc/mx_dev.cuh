// MXFP8 element conversion shared by the quantisation and the norm kernels.
#pragma once
#include <cuda_fp8.h>

#include "common.cuh"

namespace kmoe {

__device__ __forceinline__ uint8_t e4m3_code(float x, float inv_scale) {
  if (isnan(x)) return 0;
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(x * inv_scale, __NV_SATFINITE, __NV_E4M3));
}

}  // namespace kmoe
