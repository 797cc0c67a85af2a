// Expert routing with score functions, groups and renormalised weights, and
// its gradient with respect to the logits (definitions in include/kmoe.h).
#include "route_dev.cuh"
#include "route_group.cuh"

namespace kmoe {

constexpr int kRouteWarps = 4;  // tokens per block, one warp each

__device__ __forceinline__ float neg_inf_f() { return -__int_as_float(0x7f800000); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
// Warp maximum through the integer images (NaN never gets here).
__device__ __forceinline__ float warp_max(float v) {
  return order_key_inverse(__reduce_max_sync(0xffffffffu, order_key(v)));
}

// ---------------------------------------------------------------- weights of chosen experts
// What a chosen expert's logit l gives (lane j: slot j; -inf: an empty slot).
struct Share {
  float p;      // score, or with renormalisation its share of the chosen scores' sum
  float slope;  // d log(score) / d logit without the softmax's common term: 1, or 1 - sigmoid
};

// total: the softmax's denominator relative to exp(top), used without
// renormalisation only.  Shares do not change with a common factor of the
// scores, so softmax shares are taken relative to the largest chosen logit and
// sigmoid shares below -40 (where the sigmoid is its exponential to within
// e^-40) likewise: they stay right where the scores themselves underflow.  A
// row masked with the type's lowest values (below -700) has scores of 0.
__device__ __forceinline__ Share chosen_share(float l, const RouteGroupArgs& a, float top, float total) {
  Share r{0.f, 1.f};
  const bool live = l > neg_inf_f();
  float base = top;
  bool expo = a.softmax;
  if (a.renormalize) {
    base = warp_max(l);
    expo = expo || (base < -40.f && base > -700.f);
  }
  if (live) {
    if (expo) {
      r.p = l == base ? 1.f : expf(l - base);
    } else {
      const float q = expf(-fabsf(l)), s = 1.f / (1.f + q);  // of |l|
      r.p = l >= 0.f ? s : q * s;
      r.slope = l >= 0.f ? q * s : s;
    }
  }
  if (a.renormalize) {
    const float sum = warp_sum(r.p);
    r.p = sum > 0.f ? r.p / sum : 0.f;
  } else if (a.softmax) {
    r.p /= total;
  }
  return r;
}

// ---------------------------------------------------------------- choice
// The keys are compared as fp32 numbers whose scores are rounded once, which
// wants double precision, slow on this part.  So the choice is made on cheap
// fp32 keys first, and it stands if every comparison that decided it was wider
// than the cheap keys' error; otherwise only what is in doubt gets exact keys:
//   1. the k-th largest of the 32 lane maxima bounds the k-th largest key from
//      below; experts within the margin of it are the candidates, usually at
//      most one a lane.  More than 32 (k near 32, or many equal keys): the
//      bound is raised by bisection over the keys' integer images.
//   2. the candidates are sorted by (key, lower index).  Neighbours in the
//      chosen order, or at its end, closer than the margin: the candidates get
//      exact keys (sigmoid: one double evaluation a lane) and are sorted again.
//   3. a group at the cut closer than the margin, softmax scores in doubt, or
//      more than 32 candidates: all keys exactly, and the same steps without a
//      margin; if equal keys still leave more than 32 candidates, k rounds of
//      warp arg-max.
// Without a bias the logits are the keys and nothing is in doubt.
//
// Margin.  Sigmoid: the fast exponential is off by 2 + 1.16 |x| units in the
// last place, which the sigmoid damps to at most 0.62 units of 2^-23; the sum
// and the fast quotient add 2.5 more, the exact key's own two roundings one:
// 6e-7 * max(1, |key|).  Two keys: 1.2e-6; 2e-6 is used.  Softmax: the
// denominator's fp32 sum over up to 33 steps adds up to 2e-6; 1e-5 is used.
constexpr float kMarginSigmoid = 2e-6f;
constexpr float kMarginSoftmax = 1e-5f;

// Bitonic sort across the warp, lane 0 the largest.
template <class V>
__device__ __forceinline__ V warp_sort_desc(V v, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      const V o = __shfl_xor_sync(0xffffffffu, v, stride);
      const bool larger = ((lane & stride) == 0) == ((lane & size) == 0);
      v = larger == (v < o) ? o : v;
    }
  }
  return v;
}

// Where expert e's key lies in shared memory: groups start LPG banks apart
// (LPG lanes scan a group), so that the warp's scan of all groups has no bank
// conflicts.
struct GroupLayout {
  int per, lpg, stride;
  float inv;    // 1 / per
  float first;  // (0.5 - per / 2) / per
  // Group of expert e = lane + 32 i: the nearest integer to (e + 0.5) / per - 0.5, which is never
  // within 0.5 / per >= 2^-11 of half-way, read off the mantissa of its sum with 1.5 * 2^23.
  __device__ __forceinline__ int group(float lane_pos, int i) const {
    return static_cast<int>(__float_as_uint(fmaf(32.f * i, inv, lane_pos) + 12582912.f) & 63u);
  }
};

template <int KPL, bool BIAS>
__global__ void __launch_bounds__(32 * kRouteWarps, 5) route_grouped_kernel(const float* __restrict__ logits,
                                                                         const float* __restrict__ bias,
                                                                         const RouteGroupArgs a, GroupLayout gl,
                                                                         int warp_words, int32_t* __restrict__ ids,
                                                                         float* __restrict__ wts) {
  extern __shared__ float s_all[];  // per warp: candidates [32] (8 bytes each), keys
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + warp;
  if (t >= a.T) return;
  unsigned long long* s_cand = reinterpret_cast<unsigned long long*>(s_all + static_cast<size_t>(warp) * warp_words);
  float* s_key = reinterpret_cast<float*>(s_cand + 32);
  const float* lg = logits + static_cast<size_t>(t) * a.E;
  const float NEG = neg_inf_f();
  const unsigned kAll = 0xffffffffu;

  // the row's logits; what cannot be chosen is -inf
  float lv[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const int e = lane + 32 * i;
    lv[i] = e < a.E ? __ldg(lg + e) : NEG;
  }
  float top = NEG, total = 1.f;
  if (a.softmax && (BIAS || !a.renormalize)) {
#pragma unroll
    for (int i = 0; i < KPL; ++i) top = fmaxf(top, lv[i]);
    top = warp_max(top);
    total = 0.f;
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      if (lv[i] > NEG) total += lv[i] == top ? 1.f : __expf(lv[i] - top);
    total = warp_sum(total);
  }
  const float margin = BIAS ? (a.softmax ? kMarginSoftmax : kMarginSigmoid) : 0.f;
  const float inv_total = 1.f / total;

  uint32_t okey[KPL];  // integer images of the keys, 0: cannot be chosen
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const int e = lane + 32 * i;
    float k = lv[i];
    if (BIAS && k > NEG) {
      const float s = a.softmax ? (lv[i] == top ? 1.f : __expf(lv[i] - top)) * inv_total
                                : __fdividef(1.f, 1.f + __expf(-lv[i]));
      k = s + __ldg(bias + e);
    }
    okey[i] = k > NEG ? order_key(k) : 0u;
  }
  const float lane_pos = fmaf(static_cast<float>(lane), gl.inv, gl.first);
  unsigned long long best = 0;  // lane j: slot j as (image, ~expert)
  int kk = 0;                   // slots filled
  bool exact = !BIAS, redo = false;
  for (;;) {
    if (BIAS && redo) {  // all keys exactly
      exact = true;
      double sum = 0.0;
      if (a.softmax) {
#pragma unroll 1
        for (int e = lane; e < a.E; e += 32) {
          const float l = lg[e];
          if (l > NEG) sum += l == top ? 1.0 : exp(static_cast<double>(l) - top);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kAll, sum, off);
      }
#pragma unroll 1
      for (int e = lane; e < a.E; e += 32) {
        const float l = lg[e];
        float k = NEG;
        if (l > NEG) {
          const float s = a.softmax
                              ? static_cast<float>((l == top ? 1.0 : exp(static_cast<double>(l) - top)) / sum)
                              : sigmoid_exact_f32(l);
          k = s + bias[e];
        }
        s_key[e] = k > NEG ? k : NEG;
      }
      // a lane reads back what it wrote
#pragma unroll
      for (int i = 0; i < KPL; ++i) {
        const int e = lane + 32 * i;
        const float k = e < a.E ? s_key[e] : NEG;
        okey[i] = k > NEG ? order_key(k) : 0u;
      }
      __syncwarp();
    }
    // ---- groups
    bool doubt = false;
    if (a.n_group > 1) {
#pragma unroll
      for (int i = 0; i < KPL; ++i) {
        const int e = lane + 32 * i;
        if (e < a.E) s_key[e + gl.group(lane_pos, i) * (gl.stride - gl.per)] = okey[i] ? order_key_inverse(okey[i]) : NEG;
      }
      __syncwarp();
      const int g = lane / gl.lpg, sub = lane - g * gl.lpg;
      float k1 = NEG, k2 = NEG;
      if (g < a.n_group) {
        const float* row = s_key + g * gl.stride;
#pragma unroll 4
        for (int j = sub; j < gl.per; j += gl.lpg) {
          const float k = row[j];
          if (BIAS) k2 = fmaxf(k2, fminf(k, k1));
          k1 = fmaxf(k1, k);
        }
      }
      for (int off = gl.lpg >> 1; off > 0; off >>= 1) {
        const float o1 = __shfl_xor_sync(kAll, k1, off), o2 = __shfl_xor_sync(kAll, k2, off);
        k2 = fmaxf(fminf(k1, o1), fmaxf(k2, o2));
        k1 = fmaxf(k1, o1);
      }
      const float gs = BIAS && k2 > NEG ? k1 + k2 : k1;
      int better = 0;
      for (int q = 0; q < a.n_group; ++q) {
        const float o = __shfl_sync(kAll, gs, q * gl.lpg);
        better += o > gs || (o == gs && q < g);
      }
      const bool keep = better < a.topk_group;
      if (BIAS && !exact) {
        // the closest kept and dropped groups; a key's error grows with its size, so with the largest
        const bool live = g < a.n_group && k1 > NEG;
        float size = live ? fmaxf(1.f, fabsf(k1)) : 1.f;
        if (live && k2 > NEG) size = fmaxf(size, fabsf(k2));
        size = warp_max(size);
        const float in = -warp_max(live && keep ? -gs : NEG), out = warp_max(live && !keep ? gs : NEG);
        doubt = out > NEG && !(in - out > 2.f * margin * size);
      }
      const unsigned kept = __ballot_sync(kAll, g < a.n_group && keep);  // group q at bit q * lpg
      __syncwarp();
#pragma unroll
      for (int i = 0; i < KPL; ++i) {
        const int e = lane + 32 * i;
        if (e < a.E && !((kept >> (gl.group(lane_pos, i) * gl.lpg)) & 1u)) okey[i] = 0u;
      }
    }
    if (doubt) {
      redo = true;
      continue;
    }
    // ---- candidates
    uint32_t lmax = 0;
    unsigned alive = 0;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      lmax = max(lmax, okey[i]);
      alive += okey[i] != 0u;
    }
    kk = min(a.k, static_cast<int>(__reduce_add_sync(kAll, alive)));
    if (kk == 0) break;
    uint32_t lo = max(1u, __shfl_sync(kAll, warp_sort_desc(lmax, lane), kk - 1));  // at least kk images reach lo
    auto cut_of = [&](uint32_t image) {
      if (exact || image < 0x00800000u) return image;  // below: no number's image
      const float v = order_key_inverse(image);
      return order_key(v - margin * fmaxf(1.f, fabsf(v)));
    };
    auto candidates = [&](uint32_t cut, unsigned& mask) {
      mask = 0;
#pragma unroll
      for (int i = 0; i < KPL; ++i) mask |= static_cast<unsigned>(okey[i] >= cut) << i;
      return static_cast<int>(__reduce_add_sync(kAll, static_cast<unsigned>(__popc(mask))));
    };
    const uint32_t umax = __reduce_max_sync(kAll, lmax);
    if (!exact && umax >= 0xff800000u) {  // an infinite key has no margin
      redo = true;
      continue;
    }
    unsigned mask;
    int n = candidates(cut_of(lo), mask);
    if (n > 32) {
      uint32_t hi = umax + 1;  // fewer than kk images reach hi, or it is past them all
      while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        unsigned unused;
        const int c = candidates(mid, unused);
        if (c >= kk) {
          lo = mid;
          if (c <= 32 && candidates(cut_of(lo), unused) <= 32) break;
        } else {
          hi = mid;
        }
      }
      n = candidates(cut_of(lo), mask);
    }
    if (n > 32) {
      if (!exact) {
        redo = true;
        continue;
      }
      // more equal keys than lanes: one slot a round
      for (int j = 0; j < kk; ++j) {
        unsigned long long mine = 0;
#pragma unroll
        for (int i = 0; i < KPL; ++i) {
          const unsigned long long v =
              (static_cast<unsigned long long>(okey[i]) << 32) | (0xffffffffu - static_cast<unsigned>(lane + 32 * i));
          if (((mask >> i) & 1u) && v > mine) mine = v;
        }
        const uint32_t key = __reduce_max_sync(kAll, static_cast<uint32_t>(mine >> 32));
        const uint32_t low = __reduce_max_sync(kAll, static_cast<uint32_t>(mine >> 32) == key
                                                         ? static_cast<uint32_t>(mine) : 0u);
        const int e = static_cast<int>(0xffffffffu - low);
        if (lane == j) best = (static_cast<unsigned long long>(key) << 32) | low;
        if ((e & 31) == lane) mask &= ~(1u << (e >> 5));
      }
      break;
    }
    // ---- one candidate a lane, sorted
    int pos = __popc(mask);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(kAll, pos, off);
      if (lane >= off) pos += o;
    }
    pos -= __popc(mask);
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      if ((mask >> i) & 1u)
        s_cand[pos++] = (static_cast<unsigned long long>(okey[i]) << 32) | (0xffffffffu - static_cast<unsigned>(lane + 32 * i));
    __syncwarp();
    best = lane < n ? s_cand[lane] : 0ull;
    __syncwarp();
    best = warp_sort_desc(best, lane);
    if (exact) break;
    const float mine = order_key_inverse(static_cast<uint32_t>(best >> 32));
    const unsigned long long nb = __shfl_down_sync(kAll, best, 1);
    bool close = false;
    if (lane < kk && lane + 1 < n) {
      const float next = order_key_inverse(static_cast<uint32_t>(nb >> 32));
      close = !(mine - next > margin * fmaxf(1.f, fmaxf(fabsf(mine), fabsf(next))));
      if (close) {  // equal inputs have equal keys: their index decides, as it did
        const int e = static_cast<int>(0xffffffffu - static_cast<uint32_t>(best));
        const int f = static_cast<int>(0xffffffffu - static_cast<uint32_t>(nb));
        close = !(lg[e] == lg[f] && bias[e] == bias[f]);
      }
    }
    if (!__any_sync(kAll, close)) break;
    if (a.softmax) {
      redo = true;
      continue;
    }
    if (lane < n) {
      const int e = static_cast<int>(0xffffffffu - static_cast<uint32_t>(best));
      best = (static_cast<unsigned long long>(order_key(sigmoid_exact_f32(lg[e]) + bias[e])) << 32) |
             static_cast<uint32_t>(best);
    }
    best = warp_sort_desc(best, lane);
    break;
  }

  // ---- weights
  const int id = lane < kk ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(best)) : -1;
  const float p = chosen_share(id >= 0 ? lg[id] : NEG, a, top, total).p;
  if (lane < a.k) {
    ids[static_cast<size_t>(t) * a.k + lane] = id;
    wts[static_cast<size_t>(t) * a.k + lane] = p * a.scale;
  }
}

template <bool BIAS>
cudaError_t launch_route_bias(const float* logits, const float* bias, const RouteGroupArgs& a, int32_t* ids, float* wts,
                              cudaStream_t st) {
  GroupLayout gl{};
  gl.per = a.E / a.n_group;
  int lpg = 32;
  while (lpg * a.n_group > 32) lpg >>= 1;
  gl.lpg = lpg;
  gl.stride = gl.per + ((lpg - gl.per) % 32 + 32) % 32;
  gl.inv = 1.f / static_cast<float>(gl.per);
  gl.first = 0.5f * gl.inv - 0.5f;
  const int words = gl.stride * a.n_group > a.E ? gl.stride * a.n_group : a.E;
  const int warp_words = 64 + (words + 1) / 2 * 2;
  // few tokens: a warp a block, spread over the SMs
  const int warps = a.T <= 152 * kRouteWarps ? 1 : kRouteWarps;
  const size_t smem = static_cast<size_t>(warps) * warp_words * 4;
  const int blocks = (a.T + warps - 1) / warps;
  const int kpl = (a.E + 31) / 32;
#define KMOE_ROUTE(N)                                                                                             \
  if (kpl <= N) {                                                                                                 \
    route_grouped_kernel<N, BIAS><<<blocks, 32 * warps, smem, st>>>(logits, bias, a, gl, warp_words, ids, wts);   \
    return cudaGetLastError();                                                                                    \
  }
  KMOE_ROUTE(2)
  KMOE_ROUTE(4)
  KMOE_ROUTE(8)
  KMOE_ROUTE(16)
  KMOE_ROUTE(32)
#undef KMOE_ROUTE
  return cudaErrorInvalidValue;
}

cudaError_t launch_route_grouped(const float* logits, const float* bias, const RouteGroupArgs& a, int32_t* ids,
                                 float* wts, cudaStream_t st) {
  return bias ? launch_route_bias<true>(logits, bias, a, ids, wts, st)
              : launch_route_bias<false>(logits, bias, a, ids, wts, st);
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
  const float given = id >= 0 ? lg[id] : NEG;
  const float l = given > NEG ? given : NEG;  // NaN too
  const float g = l > NEG ? a.scale * d_w[static_cast<size_t>(t) * a.k + lane] : 0.f;
  float top = NEG, total = 1.f;
  if (a.softmax && !a.renormalize) {
    for (int e = lane; e < a.E; e += 32) top = fmaxf(top, lg[e]);
    top = warp_max(top);
    total = 0.f;
    for (int e = lane; e < a.E; e += 32)
      if (lg[e] > NEG) total += lg[e] == top ? 1.f : expf(lg[e] - top);
    total = warp_sum(total);
  }
  const Share sh = chosen_share(l, a, top, total);
  const float s = sh.p;
  const float d = a.renormalize ? s * (g - warp_sum(g * s)) * sh.slope : g * s * sh.slope;
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
