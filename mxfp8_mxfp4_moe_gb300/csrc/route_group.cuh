// Host interface of the grouped routing kernels (route_group.cu).
#pragma once
#include "common.cuh"

namespace kmoe {

constexpr int kMaxGroups = 32;  // one per lane

struct RouteGroupArgs {
  int T, E, k, n_group, topk_group;
  bool softmax, renormalize;
  float scale;
};

cudaError_t launch_route_grouped(const float* logits, const float* bias, const RouteGroupArgs& a, int32_t* ids,
                                 float* wts, cudaStream_t st);
cudaError_t launch_route_backward(const float* d_w, const float* logits, const int32_t* ids, const RouteGroupArgs& a,
                                  float* d_logits, cudaStream_t st);

}  // namespace kmoe
