// Gradient of the combine with respect to the routing weights:
//   d_w[t, j] = rsf * sum_h d_out[t, h] * y[t*k + j, h]
// with y the per-slot FC2 outputs that the forward leaves in its workspace.
// Slots with an expert id outside [0, E) have no y row and get 0.
//
// The y rows are read once and nothing else comes near them in bytes (a d_out
// row is shared by k slots and stays in L2), so HBM bounds it: T = 8192, H =
// 7168, k = 16 reads 3.88 GB, 3.76 of them y, in 528 us, 7.3 TB/s (reads alone
// go faster than the copy that the peak is taken from).  A slot is one warp's
// dot product, eight 16-byte loads of y in flight a lane (4-byte loads: 594 us), or, where
// there are too few slots for their length to fill the SMs that way, four
// warps' (launch_combine_backward).
#include <cuda_bf16.h>

#include "common.cuh"

namespace kmoe {

template <int WPS>  // warps a slot
__global__ void __launch_bounds__(256) combine_backward_kernel(const __nv_bfloat16* __restrict__ d_out,
                                                               const float* __restrict__ y,
                                                               const int32_t* __restrict__ ids, int R, int H, int k,
                                                               int E, float rsf, float* __restrict__ d_w) {
  __shared__ float s_part[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = blockIdx.x * (8 / WPS) + warp / WPS;
  float acc = 0.f;
  if (s < R) {
    const int id = ids[s];
    if (id >= 0 && id < E) {
      const uint2* g = reinterpret_cast<const uint2*>(d_out + static_cast<size_t>(s / k) * H);
      const float4* row = reinterpret_cast<const float4*>(y + static_cast<size_t>(s) * H);
      float2 a = make_float2(0.f, 0.f), b = a;
#pragma unroll 8
      for (int i = lane + 32 * (warp % WPS); i < H / 4; i += 32 * WPS) {
        const float4 v = __ldcs(row + i);
        const uint2 u = __ldg(g + i);
        a = __ffma2_rn(make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u)),
                       make_float2(v.x, v.y), a);
        b = __ffma2_rn(make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u)),
                       make_float2(v.z, v.w), b);
      }
      acc = (a.x + a.y) + (b.x + b.y);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    }
  }
  if constexpr (WPS > 1) {  // the slot's warps in order
    if (lane == 0) s_part[warp] = acc;
    __syncthreads();
    acc = 0.f;
#pragma unroll
    for (int w = 0; w < WPS; ++w) acc += s_part[warp / WPS * WPS + w];
  }
  if (s < R && lane == 0 && warp % WPS == 0) d_w[s] = acc * rsf;
}

cudaError_t launch_combine_backward(const void* d_out, const float* y, const int32_t* ids, int T, int H, int k, int E,
                                    float rsf, float* d_w, cudaStream_t st) {
  const int R = T * k;
  const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(d_out);
  // us with four warps a slot / one: H = 7168, R = 16 slots 5.2 / 8.2, 1216 10.1 / 17.9, 4864 24.7 / 26.1,
  // 9728 45.0 / 44.5; H = 1024, R = 1216 4.2 / 4.1, 4864 8.2 / 7.5, 9728 12.4 / 10.0
  if (static_cast<long long>(R) * 2048 < 152LL * 16 * H)
    combine_backward_kernel<4><<<(R + 1) / 2, 256, 0, st>>>(g, y, ids, R, H, k, E, rsf, d_w);
  else
    combine_backward_kernel<1><<<(R + 7) / 8, 256, 0, st>>>(g, y, ids, R, H, k, E, rsf, d_w);
  return cudaGetLastError();
}

}  // namespace kmoe
