// MXFP8 element conversion shared by the quantisation and the norm kernels.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace kmoe {

__device__ __forceinline__ uint8_t e4m3_code(float x, float inv_scale) {
  if (isnan(x)) return 0;
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(x * inv_scale, __NV_SATFINITE, __NV_E4M3));
}

// ---------------------------------------------------------------- bf16 chunks
// The quantisation of 8 bf16 values held as packed pairs, with two-wide bf16
// instructions; the same codes and scales as the fp32 forms above (a power of
// two scales a bf16 value exactly, down to results that round to 0).

// Largest magnitude as bf16 bits; above infinity's (0x7F80) where one of the values is NaN.
__device__ __forceinline__ uint32_t bf16_amax_nan(const uint4& q) {
  auto b2 = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
  const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(__habs2(b2(q.x)), __habs2(b2(q.y))),
                                       __hmax2_nan(__habs2(b2(q.z)), __habs2(b2(q.w))));
  const uint32_t u = *reinterpret_cast<const uint32_t*>(&m);
  return max(u & 0x7FFFu, (u >> 16) & 0x7FFFu);
}
// The values with +0 for NaN, which neither counts in the scale nor has another code.
__device__ __forceinline__ uint4 bf16_drop_nan(uint4 q) {
  auto drop = [](uint32_t w) {
    if ((w & 0x7FFFu) > 0x7F80u) w &= 0xFFFF0000u;
    if ((w & 0x7FFF0000u) > 0x7F800000u) w &= 0xFFFFu;
    return w;
  };
  return make_uint4(drop(q.x), drop(q.y), drop(q.z), drop(q.w));
}

// e4m3_scale_exp + 127 of a bf16 magnitude: 448 = 1.75 * 2^8, so the exponent
// field less 8, one more where the fraction exceeds 0.75 (0x60 of 0x80).
__device__ __forceinline__ uint32_t e4m3_scale_byte(uint32_t amax) {
  const uint32_t e = (amax + 0x1Fu) >> 7;
  return amax == 0x7F80u ? 254u : (e > 8u ? e - 8u : 0u);
}

// The 8 codes for a scale byte, packed little-endian (no NaN).
__device__ __forceinline__ uint2 e4m3_chunk(const uint4& q, uint32_t scale) {
  // 2^(127 - scale); 2^-127 is subnormal
  const uint32_t inv = scale == 254u ? 0x0040u : (254u - scale) << 7;
  const uint32_t inv2 = inv | (inv << 16);
  const uint32_t in[4] = {q.x, q.y, q.z, q.w};
  uint32_t pair[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p =
        __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&in[i]), *reinterpret_cast<const __nv_bfloat162*>(&inv2));
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&p);
    const float2 f = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    pair[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(pair[0] | (pair[1] << 16), pair[2] | (pair[3] << 16));
}

}  // namespace kmoe
