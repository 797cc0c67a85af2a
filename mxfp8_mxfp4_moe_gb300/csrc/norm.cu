// Root-mean-square norm of the rows that enter the expert layer, with the
// residual's addition in front and the MXFP8 quantisation behind it, and its
// gradient.
//   h = x + r,  y = bf16(h * rstd * w),  rstd = (mean(h^2) + eps)^-1/2,
// sums and products in fp32; y comes from the unrounded h, the stored h is
// rounded once to the stream's type.  The codes are those of the bf16 row y
// (not of the fp32 product), so that a layer fed with them gives what the
// layer fed with y gives, bit for bit.
#include <cuda_bf16.h>

#include "mx_dev.cuh"
#include "norm.cuh"

namespace kmoe {

__device__ __forceinline__ float load_f(const float* p, size_t i) { return p[i]; }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p, size_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ void store_f(float* p, size_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store_f(__nv_bfloat16* p, size_t i, float v) { p[i] = __float2bfloat16_rn(v); }

// Sum over the block, the same value on every thread.  Warps in order.
__device__ __forceinline__ float block_sum(float v, float* s_part) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) s += s_part[w];
  return s;
}

// One block per row.
template <class S, class W>
__global__ void __launch_bounds__(256) rmsnorm_kernel(const __nv_bfloat16* __restrict__ x, const S* residual,
                                                      const W* __restrict__ weight, int H, float eps, S* h,
                                                      __nv_bfloat16* __restrict__ y, uint8_t* __restrict__ codes,
                                                      uint8_t* __restrict__ scales) {
  extern __shared__ float s_h[];  // [H]
  __shared__ float s_part[8];
  const size_t base = static_cast<size_t>(blockIdx.x) * H;
  float sum = 0.f;
  for (int i = threadIdx.x; i < H; i += blockDim.x) {
    float v = load_f(x, base + i);
    if (residual) {
      v += load_f(residual, base + i);
      if (h) store_f(h, base + i, v);
    }
    s_h[i] = v;
    sum = fmaf(v, v, sum);
  }
  const float rstd = rsqrtf(block_sum(sum, s_part) / static_cast<float>(H) + eps);
  // 32 consecutive columns a warp: one scale group
  for (int i = threadIdx.x; i < H; i += blockDim.x) {
    const __nv_bfloat16 yb = __float2bfloat16_rn(s_h[i] * rstd * load_f(weight, i));
    if (y) y[base + i] = yb;
    if (codes) {
      const float v = __bfloat162float(yb);
      float a = isnan(v) ? 0.f : fabsf(v);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
      const int e = e4m3_scale_exp(a);
      codes[base + i] = e4m3_code(v, exp2i(-e));
      if ((i & 31) == 0) scales[(base + i) >> 5] = static_cast<uint8_t>(e + 127);
    }
  }
}

template <class S, class W>
cudaError_t rmsnorm_typed(const void* x, const void* residual, const void* weight, int T, int H, float eps, void* h,
                          void* y, uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  const size_t smem = static_cast<size_t>(H) * 4;
  const cudaError_t e = cudaFuncSetAttribute(rmsnorm_kernel<S, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  rmsnorm_kernel<S, W><<<T, 256, smem, st>>>(static_cast<const __nv_bfloat16*>(x), static_cast<const S*>(residual),
                                             static_cast<const W*>(weight), H, eps, static_cast<S*>(h),
                                             static_cast<__nv_bfloat16*>(y), codes, scales);
  return cudaGetLastError();
}

cudaError_t launch_rmsnorm(const void* x, const void* residual, const void* weight, int T, int H, float eps,
                           bool stream_f32, bool weight_f32, void* h, void* y, uint8_t* codes, uint8_t* scales,
                           cudaStream_t st) {
  if (stream_f32)
    return weight_f32 ? rmsnorm_typed<float, float>(x, residual, weight, T, H, eps, h, y, codes, scales, st)
                      : rmsnorm_typed<float, __nv_bfloat16>(x, residual, weight, T, H, eps, h, y, codes, scales, st);
  return weight_f32
             ? rmsnorm_typed<__nv_bfloat16, float>(x, residual, weight, T, H, eps, h, y, codes, scales, st)
             : rmsnorm_typed<__nv_bfloat16, __nv_bfloat16>(x, residual, weight, T, H, eps, h, y, codes, scales, st);
}

// ---------------------------------------------------------------- gradient
// With n = h * rstd, g = dy * w:
//   dh = dh_in + rstd * (g - n * mean(g * n)),  dw = sum over rows of dy * n.
// rstd is recomputed from h in the pass that reads it anyway.  Block b takes
// rows b, b + parts, ... and writes its own row of dw partial sums; a second
// kernel adds the parts in order, so dw does not depend on timing.
template <class S, class W>
__global__ void __launch_bounds__(256) rmsnorm_backward_kernel(const __nv_bfloat16* __restrict__ dy,
                                                               const S* __restrict__ h, const W* __restrict__ weight,
                                                               const S* dh_in, int T, int H, float eps, S* dh,
                                                               float* __restrict__ part) {
  extern __shared__ float s_dw[];  // [H]
  __shared__ float s_part[8];
  for (int i = threadIdx.x; i < H; i += blockDim.x) s_dw[i] = 0.f;
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    const size_t base = static_cast<size_t>(t) * H;
    float ss = 0.f, gh = 0.f;
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
      const float hv = load_f(h, base + i);
      ss = fmaf(hv, hv, ss);
      gh = fmaf(load_f(dy, base + i) * load_f(weight, i), hv, gh);
    }
    ss = block_sum(ss, s_part);
    gh = block_sum(gh, s_part);
    const float rstd = rsqrtf(ss / static_cast<float>(H) + eps);
    const float c = gh * rstd / static_cast<float>(H);
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
      const float n = load_f(h, base + i) * rstd;
      const float d = load_f(dy, base + i);
      s_dw[i] = fmaf(d, n, s_dw[i]);
      const float v = rstd * (d * load_f(weight, i) - n * c);
      store_f(dh, base + i, dh_in ? load_f(dh_in, base + i) + v : v);
    }
  }
  for (int i = threadIdx.x; i < H; i += blockDim.x) part[static_cast<size_t>(blockIdx.x) * H + i] = s_dw[i];
}

__global__ void __launch_bounds__(256) rmsnorm_dweight_kernel(const float* __restrict__ part, int parts, int H,
                                                              float* __restrict__ dweight) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= H) return;
  float s = 0.f;
  for (int p = 0; p < parts; ++p) s += part[static_cast<size_t>(p) * H + i];
  dweight[i] = s;
}

template <class S, class W>
cudaError_t rmsnorm_backward_typed(const void* dy, const void* h, const void* weight, const void* dh_in, int T, int H,
                                   float eps, void* dh, float* dweight, float* part, cudaStream_t st) {
  const size_t smem = static_cast<size_t>(H) * 4;
  const int parts = norm_parts(T);
  const cudaError_t e = cudaFuncSetAttribute(rmsnorm_backward_kernel<S, W>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  rmsnorm_backward_kernel<S, W><<<parts, 256, smem, st>>>(
      static_cast<const __nv_bfloat16*>(dy), static_cast<const S*>(h), static_cast<const W*>(weight),
      static_cast<const S*>(dh_in), T, H, eps, static_cast<S*>(dh), part);
  rmsnorm_dweight_kernel<<<(H + 255) / 256, 256, 0, st>>>(part, parts, H, dweight);
  return cudaGetLastError();
}

cudaError_t launch_rmsnorm_backward(const void* dy, const void* h, const void* weight, const void* dh_in, int T, int H,
                                    float eps, bool stream_f32, bool weight_f32, void* dh, float* dweight, float* part,
                                    cudaStream_t st) {
  if (T == 0) return cudaMemsetAsync(dweight, 0, static_cast<size_t>(H) * 4, st);
  if (stream_f32)
    return weight_f32
               ? rmsnorm_backward_typed<float, float>(dy, h, weight, dh_in, T, H, eps, dh, dweight, part, st)
               : rmsnorm_backward_typed<float, __nv_bfloat16>(dy, h, weight, dh_in, T, H, eps, dh, dweight, part, st);
  return weight_f32 ? rmsnorm_backward_typed<__nv_bfloat16, float>(dy, h, weight, dh_in, T, H, eps, dh, dweight, part,
                                                                  st)
                    : rmsnorm_backward_typed<__nv_bfloat16, __nv_bfloat16>(dy, h, weight, dh_in, T, H, eps, dh,
                                                                          dweight, part, st);
}

}  // namespace kmoe
