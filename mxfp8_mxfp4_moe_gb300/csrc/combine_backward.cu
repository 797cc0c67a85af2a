// Gradient of the combine with respect to the routing weights:
//   d_w[t, j] = rsf * sum_h d_out[t, h] * y[t*k + j, h]
// with y the per-slot FC2 outputs that the forward leaves in its workspace.
// Slots with an expert id outside [0, E) have no y row and get 0.
#include <cuda_bf16.h>

#include "common.cuh"

namespace kmoe {

// One warp per slot.
__global__ void __launch_bounds__(256) combine_backward_kernel(const __nv_bfloat16* __restrict__ d_out,
                                                               const float* __restrict__ y,
                                                               const int32_t* __restrict__ ids, int R, int H, int k,
                                                               int E, float rsf, float* __restrict__ d_w) {
  const int lane = threadIdx.x & 31;
  const int s = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (s >= R) return;
  const int id = ids[s];
  float acc = 0.f;
  if (id >= 0 && id < E) {
    const __nv_bfloat16* g = d_out + static_cast<size_t>(s / k) * H;
    const float* row = y + static_cast<size_t>(s) * H;
    for (int h = lane; h < H; h += 32) acc = fmaf(__bfloat162float(g[h]), row[h], acc);
    for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
  }
  if (lane == 0) d_w[s] = acc * rsf;
}

cudaError_t launch_combine_backward(const void* d_out, const float* y, const int32_t* ids, int T, int H, int k, int E,
                                    float rsf, float* d_w, cudaStream_t st) {
  const int R = T * k;
  combine_backward_kernel<<<(R + 7) / 8, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(d_out), y, ids, R, H, k, E,
                                                       rsf, d_w);
  return cudaGetLastError();
}

}  // namespace kmoe
