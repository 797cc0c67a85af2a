// Host interface of the norm kernels (norm.cu).
#pragma once
#include "common.cuh"

namespace kmoe {

constexpr int kMaxNormH = 32768;  // columns a block keeps on chip

// Partial rows of the weight gradient.  A function of the row count alone, so
// that the summation order is the same on every GPU.
__host__ inline int norm_parts(int T) { return T < 304 ? T : 304; }
__host__ inline size_t norm_part_bytes(int T, int H) { return static_cast<size_t>(norm_parts(T)) * H * 4; }

cudaError_t launch_rmsnorm(const void* x, const void* residual, const void* weight, int T, int H, float eps,
                           bool stream_f32, bool weight_f32, void* h, void* y, uint8_t* codes, uint8_t* scales,
                           cudaStream_t st);
cudaError_t launch_rmsnorm_backward(const void* dy, const void* h, const void* weight, const void* dh_in, int T, int H,
                                    float eps, bool stream_f32, bool weight_f32, void* dh, float* dweight, float* part,
                                    cudaStream_t st);

}  // namespace kmoe
