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

// Largest magnitude as bf16 bits, NaN dropped.
__device__ __forceinline__ uint32_t bf16_amax(const uint4& q) {
  auto b2 = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
  const __nv_bfloat162 m = __hmax2(__hmax2(__habs2(b2(q.x)), __habs2(b2(q.y))),
                                   __hmax2(__habs2(b2(q.z)), __habs2(b2(q.w))));
  const uint32_t u = *reinterpret_cast<const uint32_t*>(&m);
  // a lane whose four values were all NaN is left with NaN: magnitude above infinity's bits
  const uint32_t lo = u & 0x7FFFu, hi = (u >> 16) & 0x7FFFu;
  return max(lo > 0x7F80u ? 0u : lo, hi > 0x7F80u ? 0u : hi);
}

// e4m3_scale_exp + 127 of a bf16 magnitude: 448 = 1.75 * 2^8, so the exponent
// field less 8, one more where the fraction exceeds 0.75 (0x60 of 0x80).
__device__ __forceinline__ uint32_t e4m3_scale_byte(uint32_t amax) {
  const uint32_t e = (amax + 0x1Fu) >> 7;
  return amax == 0x7F80u ? 254u : (e > 8u ? e - 8u : 0u);
}

// The 8 codes for a scale byte, packed little-endian.
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
  uint2 out = make_uint2(pair[0] | (pair[1] << 16), pair[2] | (pair[3] << 16));
  // NaN converts to the NaN code (0x7F, either sign); its code is +0.  No other value gives it.
  const uint32_t n0 = __vcmpeq4(out.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu), n1 = __vcmpeq4(out.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
  out.x &= ~n0;
  out.y &= ~n1;
  return out;
}

}  // namespace kmoe
