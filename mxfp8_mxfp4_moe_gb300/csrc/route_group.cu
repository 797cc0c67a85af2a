// Expert routing with score functions, groups and renormalised weights, and
// its gradient with respect to the logits (definitions in include/kmoe.h).
#include "route_dev.cuh"
#include "route_group.cuh"

namespace kmoe {

constexpr int kRouteWarps = 4;  // tokens per block, one warp each

__device__ __forceinline__ float neg_inf_f() { return -__int_as_float(0x7f800000); }

__global__ void __launch_bounds__(32 * kRouteWarps) route_grouped_kernel(const float* __restrict__ logits,
                                                                         const float* __restrict__ bias,
                                                                         RouteGroupArgs a, int32_t* __restrict__ ids,
                                                                         float* __restrict__ wts) {
  extern __shared__ float s_all[];  // per warp: keys [E], scores [E]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouteWarps + warp;
  if (t >= a.T) return;
  float* key = s_all + static_cast<size_t>(warp) * 2 * a.E;
  float* score = key + a.E;
  const float* lg = logits + static_cast<size_t>(t) * a.E;
  const float NEG = neg_inf_f();
  float top = NEG;
  for (int e = lane; e < a.E; e += 32) top = fmaxf(top, lg[e]);
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  double total = 0.0;
  if (a.softmax) {
    for (int e = lane; e < a.E; e += 32) {
      const float l = lg[e];
      if (l > NEG) total += l == top ? 1.0 : exp(static_cast<double>(l) - top);
    }
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  }
  for (int e = lane; e < a.E; e += 32) {
    const float l = lg[e];
    float k = NEG, s = 0.f;
    if (l > NEG) {
      s = a.softmax ? static_cast<float>((l == top ? 1.0 : exp(static_cast<double>(l) - top)) / total)
                    : sigmoid_exact_f32(l);
      k = bias ? s + bias[e] : l;
      if (!(k > NEG)) k = NEG;
    }
    key[e] = k;
    score[e] = s;
  }
  __syncwarp();
  if (a.n_group > 1) {
    const int per = a.E / a.n_group;
    float gs = NEG;
    if (lane < a.n_group) {
      float k1 = NEG, k2 = NEG;
      for (int i = 0; i < per; ++i) {
        const float k = key[lane * per + i];
        k2 = fmaxf(k2, fminf(k, k1));
        k1 = fmaxf(k1, k);
      }
      gs = bias && k2 > NEG ? k1 + k2 : k1;
    }
    int better = 0;
    for (int g = 0; g < a.n_group; ++g) {
      const float o = __shfl_sync(0xffffffffu, gs, g);
      better += o > gs || (o == gs && g < lane);
    }
    const unsigned kept = __ballot_sync(0xffffffffu, lane < a.n_group && better < a.topk_group);
    for (int e = lane; e < a.E; e += 32)
      if (!((kept >> (e / per)) & 1u)) key[e] = NEG;
    __syncwarp();
  }
  int myid = -1;
  float mys = 0.f;
  for (int j = 0; j < a.k; ++j) {
    float bk = NEG;
    int bi = 0x7fffffff;
    for (int e = lane; e < a.E; e += 32) {
      const float k = key[e];
      if (k > bk) {
        bk = k;
        bi = e;
      }
    }
    warp_argmax(bk, bi);
    if (bk == NEG) break;
    if (lane == j) {
      myid = bi;
      mys = score[bi];
    }
    __syncwarp();
    if (lane == 0) key[bi] = NEG;
    __syncwarp();
  }
  double sum = mys;
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane < a.k) {
    const double p = !a.renormalize ? mys : (sum > 0.0 ? mys / sum : 0.0);
    ids[static_cast<size_t>(t) * a.k + lane] = myid;
    wts[static_cast<size_t>(t) * a.k + lane] = static_cast<float>(p * a.scale);
  }
}

cudaError_t launch_route_grouped(const float* logits, const float* bias, const RouteGroupArgs& a, int32_t* ids,
                                 float* wts, cudaStream_t st) {
  const size_t smem = static_cast<size_t>(kRouteWarps) * 2 * a.E * 4;
  route_grouped_kernel<<<(a.T + kRouteWarps - 1) / kRouteWarps, 32 * kRouteWarps, smem, st>>>(logits, bias, a, ids,
                                                                                             wts);
  return cudaGetLastError();
}

// One warp per token; lane j holds slot j.
__global__ void __launch_bounds__(32 * kRouteWarps) route_backward_kernel(const float* __restrict__ d_w,
                                                                          const float* __restrict__ logits,
                                                                          const int32_t* __restrict__ ids,
                                                                          RouteGroupArgs a,
                                                                          float* __restrict__ d_logits) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const float NEG = neg_inf_f();
  const float* lg = logits + static_cast<size_t>(t) * a.E;
  float* out = d_logits + static_cast<size_t>(t) * a.E;
  int id = lane < a.k ? ids[static_cast<size_t>(t) * a.k + lane] : -1;
  if (id < 0 || id >= a.E) id = -1;
  const float l = id >= 0 ? lg[id] : NEG;
  const float g = l > NEG ? a.scale * d_w[static_cast<size_t>(t) * a.k + lane] : 0.f;
  auto warp_sum = [](float v) {
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
  };
  float top = l, total = 1.f;
  if (a.softmax) {
    if (!a.renormalize)
      for (int e = lane; e < a.E; e += 32) top = fmaxf(top, lg[e]);
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (!a.renormalize) {
      total = 0.f;
      for (int e = lane; e < a.E; e += 32)
        if (lg[e] > NEG) total += lg[e] == top ? 1.f : expf(lg[e] - top);
      total = warp_sum(total);
    }
  }
  // the slot's score and, for the sigmoid, its complement, from one exponential of a negative number
  float s = 0.f, slope = 1.f;
  if (l > NEG) {
    if (a.softmax) {
      s = (l == top ? 1.f : expf(l - top)) / total;
    } else {
      const float q = expf(-fabsf(l)), r = 1.f / (1.f + q);
      s = l >= 0.f ? r : q * r;
      slope = l >= 0.f ? q * r : r;
    }
  }
  float d;
  if (a.renormalize) {
    const float sum = warp_sum(s);
    const float p = sum > 0.f ? s / sum : 0.f;
    d = p * (g - warp_sum(g * p)) * slope;
  } else {
    d = g * s * slope;
  }
  // slots of one expert (routing gives none) are added in slot order
  const unsigned same = __match_any_sync(0xffffffffu, id);
  float acc = 0.f;
  for (int j = 0; j < a.k; ++j) {
    const float o = __shfl_sync(0xffffffffu, d, j);
    if ((same >> j) & 1u) acc += o;
  }
  if (a.softmax && !a.renormalize) {
    const float dot = warp_sum(d);
    for (int e = lane; e < a.E; e += 32) {
      const float v = lg[e];
      out[e] = v > NEG ? -(v == top ? 1.f : expf(v - top)) / total * dot : 0.f;
    }
    __syncwarp();
    if (id >= 0 && l > NEG && lane == __ffs(same) - 1) out[id] = acc - s * dot;
  } else {
    for (int e = lane; e < a.E; e += 32) out[e] = 0.f;
    __syncwarp();
    if (id >= 0 && lane == __ffs(same) - 1) out[id] = acc;
  }
}

cudaError_t launch_route_backward(const float* d_w, const float* logits, const int32_t* ids, const RouteGroupArgs& a,
                                  float* d_logits, cudaStream_t st) {
  route_backward_kernel<<<(a.T + kRouteWarps - 1) / kRouteWarps, 32 * kRouteWarps, 0, st>>>(d_w, logits, ids, a,
                                                                                           d_logits);
  return cudaGetLastError();
}

}  // namespace kmoe
