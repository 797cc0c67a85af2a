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
// One warp a token.  The keys are compared as fp32 numbers whose scores are
// rounded once, which wants double precision, slow on this part.  So the
// choice is made on cheap fp32 keys first, and it stands if every comparison
// that decided it was wider than the cheap keys' error; what is in doubt gets
// exact keys:
//   1. groups: the kept and the dropped group next to the cut closer than the
//      margin: the keys that can be among a group's two largest are evaluated
//      exactly and the groups ranked again.
//   2. the k-th largest of the 32 lane maxima bounds the k-th largest key from
//      below; experts within the margin of it are the candidates, usually at
//      most one a lane.  More than 32 (k near 32, or many equal keys): the
//      bound is raised by bisection over the keys' integer images.
//   3. the candidates are sorted by (key, lower index).  Neighbours in the
//      chosen order, or at its end, closer than the margin: the candidates get
//      exact keys, one a lane, and are sorted again.
//   4. softmax scores in doubt, infinite keys, or still more than 32
//      candidates: all keys exactly, and the same steps without a margin; if
//      equal keys leave more than 32 candidates even so, k rounds of arg-max.
// Without a bias the logits are the keys and nothing is in doubt.
//
// Margin.  Sigmoid: the fast exponential is off by 2 + 1.16 |x| units in the
// last place, which the sigmoid damps to at most 0.62 units of 2^-23; the sum
// and the fast quotient add 2.5 more, the exact key's own two roundings one:
// 6e-7 * max(1, |key|).  Two keys: 1.2e-6; 2e-6 is used.  Softmax: the
// denominator's fp32 sum over up to 37 steps adds up to 2.3e-6; 1e-5 is used.
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

// Groups in shared memory.  LPG lanes scan a group, VEC keys a lane and step;
// groups start LPG * VEC banks apart (modulo 32), so that the warp's scan of
// all groups has no bank conflicts.
struct GroupLayout {
  int per, lpg, stride;
  float inv;    // 1 / per
  float first;  // (0.5 - per / 2) / per
  // Group of expert e: the nearest integer to (e + 0.5) / per - 0.5, which is never within
  // 0.5 / per >= 2^-11 of half-way, read off the mantissa of its sum with 1.5 * 2^23.
  __device__ __forceinline__ int group(int e) const {
    return static_cast<int>(__float_as_uint(fmaf(static_cast<float>(e), inv, first) + 12582912.f) & 63u);
  }
};

struct Top2 {
  float k1, k2;
  __device__ __forceinline__ void add(float k) {
    k2 = fmaxf(k2, fminf(k, k1));
    k1 = fmaxf(k1, k);
  }
  // over the `lanes` lanes (a power of two) that hold a group
  __device__ __forceinline__ void merge(int lanes) {
    for (int off = lanes >> 1; off > 0; off >>= 1) {
      const float o1 = __shfl_xor_sync(0xffffffffu, k1, off), o2 = __shfl_xor_sync(0xffffffffu, k2, off);
      k2 = fmaxf(fminf(k1, o1), fmaxf(k2, o2));
      k1 = fmaxf(k1, o1);
    }
  }
};

__device__ __forceinline__ unsigned long long ranked(float key, int e) {
  return (static_cast<unsigned long long>(order_key(key)) << 32) | (0xffffffffu - static_cast<unsigned>(e));
}
__device__ __forceinline__ int expert_of(unsigned long long v) {
  return static_cast<int>(0xffffffffu - static_cast<uint32_t>(v));
}

// KPL keys a lane, VEC of them consecutive (one 16-byte load for VEC = 4).
template <int KPL, int VEC, bool BIAS>
__global__ void __launch_bounds__(32 * kRouteWarps, 5) route_grouped_kernel(const float* __restrict__ logits,
                                                                            const float* __restrict__ bias,
                                                                            const RouteGroupArgs a, GroupLayout gl,
                                                                            int warp_words, int32_t* __restrict__ ids,
                                                                            float* __restrict__ wts) {
  extern __shared__ uint4 s_all[];  // per warp: candidates [32] (8 bytes each), keys
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + warp;
  if (t >= a.T) return;
  unsigned long long* s_cand =
      reinterpret_cast<unsigned long long*>(reinterpret_cast<float*>(s_all) + static_cast<size_t>(warp) * warp_words);
  float* s_key = reinterpret_cast<float*>(s_cand + 32);
  const float* lg = logits + static_cast<size_t>(t) * a.E;
  const float NEG = neg_inf_f();
  const unsigned kAll = 0xffffffffu;
  constexpr int kChunks = KPL / VEC;
  auto first_of = [&](int q) { return VEC * (lane + 32 * q); };  // first expert of this lane's chunk q
  // chunk q of a row of E floats, -inf behind its end
  auto load = [&](const float* row, int q, float (&v)[VEC]) {
    const int e = first_of(q);
    if constexpr (VEC == 4) {
      const float4 f = e < a.E ? __ldg(reinterpret_cast<const float4*>(row + e)) : make_float4(NEG, NEG, NEG, NEG);
      v[0] = f.x;
      v[1] = f.y;
      v[2] = f.z;
      v[3] = f.w;
    } else {
      v[0] = e < a.E ? __ldg(row + e) : NEG;
    }
  };

  // the row's logits; what cannot be chosen is -inf
  float key[KPL];
#pragma unroll
  for (int q = 0; q < kChunks; ++q) {
    float v[VEC];
    load(lg, q, v);
#pragma unroll
    for (int j = 0; j < VEC; ++j) key[q * VEC + j] = fmaxf(v[j], NEG);  // NaN to -inf
  }
  float top = NEG, total = 1.f;
  if (a.softmax && (BIAS || !a.renormalize)) {
#pragma unroll
    for (int i = 0; i < KPL; ++i) top = fmaxf(top, key[i]);
    top = warp_max(top);
    total = 0.f;
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      if (key[i] > NEG) total += key[i] == top ? 1.f : __expf(key[i] - top);
    total = warp_sum(total);
  }
  const float margin = BIAS ? (a.softmax ? kMarginSoftmax : kMarginSigmoid) : 0.f;

  if constexpr (BIAS) {  // the cheap keys
    const float inv_total = 1.f / total;
#pragma unroll
    for (int q = 0; q < kChunks; ++q) {
      float b[VEC];
      load(bias, q, b);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float& k = key[q * VEC + j];
        const float s = a.softmax ? (k == top ? 1.f : __expf(k - top)) * inv_total
                                  : __fdividef(1.f, 1.f + __expf(-k));
        k = k > NEG ? fmaxf(s + b[j], NEG) : NEG;
      }
    }
  }
  unsigned long long best = 0;  // lane j: slot j
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
          k = fmaxf(s + bias[e], NEG);
        }
        s_key[e] = k;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < KPL; ++i) {
        const int e = first_of(i / VEC) + i % VEC;
        key[i] = e < a.E ? s_key[e] : NEG;
      }
      __syncwarp();
    }
    // ---- groups
    if (a.n_group > 1) {
      const int gap = gl.stride - gl.per;
#pragma unroll
      for (int q = 0; q < kChunks; ++q) {
        const int e = first_of(q);
        if (e < a.E) {
          float* at = s_key + e + gl.group(e) * gap;
          if constexpr (VEC == 4)
            *reinterpret_cast<float4*>(at) = make_float4(key[4 * q], key[4 * q + 1], key[4 * q + 2], key[4 * q + 3]);
          else
            *at = key[q];
        }
      }
      __syncwarp();
      const int g = lane / gl.lpg, sub = lane - g * gl.lpg;
      const bool mine = g < a.n_group;
      const float* row = s_key + g * gl.stride;
      Top2 two{NEG, NEG};
      if (mine) {
#pragma unroll 4
        for (int j = VEC * sub; j < gl.per; j += VEC * gl.lpg) {
          if constexpr (VEC == 4) {
            const float4 k = *reinterpret_cast<const float4*>(row + j);
            two.add(k.x);
            two.add(k.y);
            two.add(k.z);
            two.add(k.w);
          } else {
            two.add(row[j]);
          }
        }
      }
      two.merge(gl.lpg);
      float gs;
      bool keep;
      auto rank_groups = [&]() {
        gs = BIAS && two.k2 > NEG ? two.k1 + two.k2 : two.k1;
        int better = 0;
        for (int q = 0; q < a.n_group; ++q) {
          const float o = __shfl_sync(kAll, gs, q * gl.lpg);
          better += o > gs || (o == gs && q < g);
        }
        keep = better < a.topk_group;
      };
      rank_groups();
      if (BIAS && !exact) {
        // the closest kept and dropped groups; a key's error grows with its size, so with the largest
        const bool live = mine && two.k1 > NEG;
        float size = live ? fmaxf(1.f, fabsf(two.k1)) : 1.f;
        if (live && two.k2 > NEG) size = fmaxf(size, fabsf(two.k2));
        size = warp_max(size);
        const float in = -warp_max(live && keep ? -gs : NEG), out = warp_max(live && !keep ? gs : NEG);
        if (out > NEG && !(in - out > 2.f * margin * size)) {
          if (a.softmax || size > 1e30f) {
            redo = true;
            continue;
          }
          // exact keys of what can be among a group's two largest
          const float reach = (two.k2 > NEG ? two.k2 : two.k1) - margin * size;
          two = Top2{NEG, NEG};
          if (mine) {
#pragma unroll 1
            for (int j0 = sub; j0 < gl.per; j0 += 32 * gl.lpg) {
              unsigned todo = 0;
              for (int i = 0; i < 32 && j0 + i * gl.lpg < gl.per; ++i) {
                const float k = row[j0 + i * gl.lpg];
                todo |= static_cast<unsigned>(k > NEG && k >= reach) << i;
              }
#pragma unroll 1
              for (; todo != 0; todo &= todo - 1) {
                const int e = g * gl.per + j0 + (__ffs(todo) - 1) * gl.lpg;
                two.add(fmaxf(sigmoid_exact_f32(lg[e]) + bias[e], NEG));
              }
            }
          }
          __syncwarp();
          two.merge(gl.lpg);
          rank_groups();
        }
      }
      const unsigned kept = __ballot_sync(kAll, mine && keep);  // group q at bit q * lpg
#pragma unroll
      for (int q = 0; q < kChunks; ++q) {
        const int e = first_of(q);
        if (e < a.E && !((kept >> (gl.group(e) * gl.lpg)) & 1u)) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) key[q * VEC + j] = NEG;
        }
      }
      __syncwarp();
    }
    // ---- candidates
    float lmax = NEG;
#pragma unroll
    for (int i = 0; i < KPL; ++i) lmax = fmaxf(lmax, key[i]);
    const float sorted = warp_sort_desc(lmax, lane);
    float bound = __shfl_sync(kAll, sorted, a.k - 1);  // at least k keys reach it
    const float umax = __shfl_sync(kAll, sorted, 0);
    kk = a.k;
    if (!(bound > NEG)) {  // fewer lanes than slots have anything to choose from
      unsigned alive = 0;
#pragma unroll
      for (int i = 0; i < KPL; ++i) alive += key[i] > NEG;
      kk = min(a.k, static_cast<int>(__reduce_add_sync(kAll, alive)));
      if (kk == 0) break;
      bound = -3.402823466e38f;  // the lowest finite key
    }
    if (!exact && umax > 1e30f) {  // a key of such size, or infinite, has no margin
      redo = true;
      continue;
    }
    auto cut_of = [&](float v) { return exact ? v : fmaxf(v - margin * fmaxf(1.f, fabsf(v)), -3.402823466e38f); };
    auto candidates = [&](float cut, unsigned& mask) {
      mask = 0;
#pragma unroll
      for (int i = 0; i < KPL; ++i) mask |= static_cast<unsigned>(key[i] >= cut) << i;
      return static_cast<int>(__reduce_add_sync(kAll, static_cast<unsigned>(__popc(mask))));
    };
    unsigned mask;
    int n = candidates(cut_of(bound), mask);
    if (n > 32) {
      uint32_t lo = order_key(bound), hi = order_key(umax) + 1;  // kk keys reach lo; fewer reach hi, or none
      unsigned unused;
      while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        const float v = order_key_inverse(mid);
        const int c = candidates(v, unused);
        if (c >= kk) {
          lo = mid;
          if (c <= 32 && candidates(cut_of(v), unused) <= 32) break;
        } else {
          hi = mid;
        }
      }
      n = candidates(cut_of(order_key_inverse(lo)), mask);
    }
    if (n > 32) {
      if (!exact) {
        redo = true;
        continue;
      }
      // more equal keys than lanes: one slot a round
#pragma unroll 1
      for (int j = 0; j < kk; ++j) {
        unsigned long long v = 0;
        int slot = 0;
#pragma unroll
        for (int i = 0; i < KPL; ++i) {
          const unsigned long long o = ranked(key[i], first_of(i / VEC) + i % VEC);
          if (((mask >> i) & 1u) && o > v) {
            v = o;
            slot = i;
          }
        }
        const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(v >> 32));
        const uint32_t low =
            __reduce_max_sync(kAll, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
        const unsigned long long won = (static_cast<unsigned long long>(hi) << 32) | low;
        if (lane == j) best = won;
        if (v == won) mask &= ~(1u << slot);
      }
      break;
    }
    // ---- one candidate a lane, sorted
    const int own = __popc(mask);
    int pos = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(kAll, pos, off);
      if (lane >= off) pos += o;
    }
    pos -= own;
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      if ((mask >> i) & 1u) s_cand[pos++] = ranked(key[i], first_of(i / VEC) + i % VEC);
    __syncwarp();
    best = lane < n ? s_cand[lane] : 0ull;
    __syncwarp();
    best = warp_sort_desc(best, lane);
    if (exact) break;
    const float self = order_key_inverse(static_cast<uint32_t>(best >> 32));
    const unsigned long long nb = __shfl_down_sync(kAll, best, 1);
    bool close = false;
    if (lane < kk && lane + 1 < n) {
      const float next = order_key_inverse(static_cast<uint32_t>(nb >> 32));
      close = !(self - next > margin * fmaxf(1.f, fmaxf(fabsf(self), fabsf(next))));
      if (close) {  // equal inputs have equal keys: their index decides, as it did
        const int e = expert_of(best), f = expert_of(nb);
        close = !(lg[e] == lg[f] && bias[e] == bias[f]);
      }
    }
    if (!__any_sync(kAll, close)) break;
    if (a.softmax) {
      redo = true;
      continue;
    }
    if (lane < n) {
      const int e = expert_of(best);
      best = ranked(sigmoid_exact_f32(lg[e]) + bias[e], e);
    }
    best = warp_sort_desc(best, lane);
    break;
  }

  // ---- weights
  const int id = lane < kk ? expert_of(best) : -1;
  const float p = chosen_share(id >= 0 ? lg[id] : NEG, a, top, total).p;
  if (lane < a.k) {
    ids[static_cast<size_t>(t) * a.k + lane] = id;
    wts[static_cast<size_t>(t) * a.k + lane] = p * a.scale;
  }
}

template <int VEC, bool BIAS>
cudaError_t launch_route_vec(const float* logits, const float* bias, const RouteGroupArgs& a, int32_t* ids, float* wts,
                             cudaStream_t st) {
  GroupLayout gl{};
  gl.per = a.E / a.n_group;
  int lpg = 32;
  while (lpg * a.n_group > 32) lpg >>= 1;
  gl.lpg = lpg;
  gl.stride = gl.per + ((VEC * lpg - gl.per) % 32 + 32) % 32;
  gl.inv = 1.f / static_cast<float>(gl.per);
  gl.first = 0.5f * gl.inv - 0.5f;
  const int words = gl.stride * a.n_group > a.E ? gl.stride * a.n_group : a.E;
  const int warp_words = 64 + (words + 3) / 4 * 4;
  // few tokens: a warp a block, spread over the SMs
  const int warps = a.T <= 152 * kRouteWarps ? 1 : kRouteWarps;
  const size_t smem = static_cast<size_t>(warps) * warp_words * 4;
  const int blocks = (a.T + warps - 1) / warps;
  const int kpl = (a.E + 32 * VEC - 1) / (32 * VEC) * VEC;
#define KMOE_ROUTE(N)                                                                                                \
  if (kpl <= N) {                                                                                                    \
    route_grouped_kernel<N, VEC, BIAS><<<blocks, 32 * warps, smem, st>>>(logits, bias, a, gl, warp_words, ids, wts); \
    return cudaGetLastError();                                                                                       \
  }
  KMOE_ROUTE(4)
  KMOE_ROUTE(8)
  KMOE_ROUTE(16)
  KMOE_ROUTE(32)
#undef KMOE_ROUTE
  return cudaErrorInvalidValue;
}

cudaError_t launch_route_grouped(const float* logits, const float* bias, const RouteGroupArgs& a, int32_t* ids,
                                 float* wts, cudaStream_t st) {
  const uintptr_t both = reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(bias);
  // 16-byte loads where every row and every group starts on a 16-byte boundary
  if ((both & 15) == 0 && (a.E / a.n_group) % 4 == 0)
    return bias ? launch_route_vec<4, true>(logits, bias, a, ids, wts, st)
                : launch_route_vec<4, false>(logits, bias, a, ids, wts, st);
  return bias ? launch_route_vec<1, true>(logits, bias, a, ids, wts, st)
              : launch_route_vec<1, false>(logits, bias, a, ids, wts, st);
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
