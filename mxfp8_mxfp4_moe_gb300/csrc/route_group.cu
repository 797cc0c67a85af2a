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

// exp(x) and 1 / x from the hardware's approximations, results below 2^-126 as 0
__device__ __forceinline__ float fast_exp(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
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
      const float q = expf(-fabsf(l)), s = fast_rcp(1.f + q);  // of |l|
      r.p = l >= 0.f ? s : q * s;
      r.slope = l >= 0.f ? q * s : s;
    }
  }
  if (a.renormalize) {
    const float sum = warp_sum(r.p);
    r.p = sum > 0.f ? __fdividef(r.p, sum) : 0.f;
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
//      below (k > 16: or the k/2-th largest of the lanes' second keys, where
//      that is more); experts within the margin of it are the candidates, about
//      22 for k = 16.  More than 64 (many equal keys, mostly): the bound is
//      raised by bisection over the keys' integer images.
//   3. the candidates are sorted by (key, lower index).  Neighbours in the
//      chosen order, or at its end, closer than the margin: the candidates get
//      exact keys, one or two a lane, and are sorted again.
//   4. softmax scores in doubt, infinite keys, or still more than 64
//      candidates: all keys exactly, and the same steps without a margin; if
//      equal keys leave more than 64 candidates even so, k rounds of arg-max.
// Without a bias the logits are the keys and nothing is in doubt.
//
// Margin.  Sigmoid: the fast exponential is off by 2 + 1.16 |x| units in the
// last place, which the sigmoid damps to at most 0.62 units of 2^-23; the sum
// and the fast reciprocal add 1.5 more, the exact key's own two roundings one:
// 6e-7 * max(1, |key|).  Two keys: 1.2e-6; 2e-6 is used.  Softmax: the
// denominator's fp32 sum over up to 37 steps adds up to 2.3e-6; 1e-5 is used.
constexpr int kMaxCand = 64;  // two a lane
constexpr float kMarginSigmoid = 2e-6f;
constexpr float kMarginSoftmax = 1e-5f;

// Ranks by counting: a lane compares its value with all 32, read back from
// shared memory in 16-byte pieces: independent instructions, where a bitonic
// sort across the warp is a chain of 15 shuffles.
// Number of the 32 floats at s_val (no NaN) that are larger.
__device__ __forceinline__ int count_larger(float v, const float* s_val) {
  int r = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float4 o = reinterpret_cast<const float4*>(s_val)[q];
    r += (o.x > v) + (o.y > v) + (o.z > v) + (o.w > v);
  }
  return r;
}
// Sorts the n <= 64 candidates (key, expert) in place by (larger key, lower
// expert): a lane ranks numbers lane and lane + 32.
__device__ __forceinline__ void sort_candidates(float* s_ckey, int* s_ce, int n, int lane) {
  const bool two = n > 32, h0 = lane < n, h1 = lane + 32 < n;
  const float v0 = h0 ? s_ckey[lane] : neg_inf_f(), v1 = h1 ? s_ckey[lane + 32] : neg_inf_f();
  const int e0 = h0 ? s_ce[lane] : 0, e1 = h1 ? s_ce[lane + 32] : 0;
  if (!h0) s_ckey[lane] = v0;
  if (two && !h1) s_ckey[lane + 32] = v1;
  __syncwarp();
  int r0 = count_larger(v0, s_ckey), r1 = 0;
  if (two) {
    r0 += count_larger(v0, s_ckey + 32);
    r1 = count_larger(v1, s_ckey) + count_larger(v1, s_ckey + 32);
  }
  // equal keys have equal counts: then the index decides
  const unsigned low = (h0 && r0 < 32 ? 1u << (r0 & 31) : 0u) | (h1 && r1 < 32 ? 1u << (r1 & 31) : 0u);
  const unsigned high = (h0 && r0 >= 32 ? 1u << (r0 & 31) : 0u) | (h1 && r1 >= 32 ? 1u << (r1 & 31) : 0u);
  int distinct = __popc(__reduce_or_sync(0xffffffffu, low));
  if (two) distinct += __popc(__reduce_or_sync(0xffffffffu, high));
  if (distinct != n) {
#pragma unroll 1
    for (int q = 0; q < n; ++q) {
      r0 += s_ckey[q] == v0 && s_ce[q] < e0;
      r1 += s_ckey[q] == v1 && s_ce[q] < e1;
    }
  }
  __syncwarp();
  if (h0) {
    s_ckey[r0] = v0;
    s_ce[r0] = e0;
  }
  if (h1) {
    s_ckey[r1] = v1;
    s_ce[r1] = e1;
  }
  __syncwarp();
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
// Keys below this are below `v` beyond doubt.
__device__ __forceinline__ float margin_cut(float v, float margin) {
  return fmaxf(v - margin * fmaxf(1.f, fabsf(v)), -3.402823466e38f);
}
// ---- rare paths, kept out of the kernel's instruction stream: over the keys
// of a row in shared memory in expert order, -inf where nothing can be chosen.

// Candidates of the largest value that kk keys reach, less the margin, written
// to s_ckey and s_ce; returns their number, which is above 64 (and nothing
// written) where equal or close keys leave more.
__device__ __noinline__ int cold_candidates(const float* s_key, int E, int kk, float bound, float umax, float margin,
                                            float* s_ckey, int* s_ce) {
  const unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  auto count = [&](float cut) {
    unsigned c = 0;
#pragma unroll 4
    for (int e = lane; e < E; e += 32) c += s_key[e] >= cut;
    return static_cast<int>(__reduce_add_sync(kAll, c));
  };
  uint32_t lo = order_key(bound), hi = order_key(umax) + 1;  // kk keys reach lo; fewer reach hi, or none
  while (hi - lo > 1) {
    const uint32_t mid = lo + (hi - lo) / 2;
    const float v = order_key_inverse(mid);
    const int c = count(v);
    if (c >= kk) {
      lo = mid;
      if (c <= kMaxCand && count(margin_cut(v, margin)) <= kMaxCand) break;
    } else {
      hi = mid;
    }
  }
  const float cut = margin_cut(order_key_inverse(lo), margin);
  const int n = count(cut);
  if (n > kMaxCand) return n;
  int base = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    const float k = e < E ? s_key[e] : neg_inf_f();
    const unsigned m = __ballot_sync(kAll, k >= cut);
    if (k >= cut) {
      const int at = base + __popc(m & ((1u << lane) - 1u));
      s_ckey[at] = k;
      s_ce[at] = e;
    }
    base += __popc(m);
  }
  __syncwarp();
  return n;
}

// kk rounds of arg-max: more equal keys than lanes.  Lane j gets slot j.
__device__ __noinline__ int cold_argmax(float* s_key, int E, int kk) {
  const unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  int best = -1;
  for (int j = 0; j < kk; ++j) {
    unsigned long long v = 0;
    for (int e = lane; e < E; e += 32) {
      const unsigned long long o = s_key[e] > neg_inf_f() ? ranked(s_key[e], e) : 0ull;
      v = o > v ? o : v;
    }
    const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(v >> 32));
    const uint32_t low =
        __reduce_max_sync(kAll, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
    const unsigned long long won = (static_cast<unsigned long long>(hi) << 32) | low;
    const int e = static_cast<int>(0xffffffffu - low);
    if (lane == j) best = e;
    if (v == won) s_key[e] = neg_inf_f();
    __syncwarp();
  }
  return best;
}

// All keys exactly.
__device__ __noinline__ void cold_exact_keys(float* s_key, const float* lg, const float* bias, int E, bool softmax,
                                             float top) {
  const int lane = threadIdx.x & 31;
  double sum = 0.0;
  if (softmax) {
    for (int e = lane; e < E; e += 32) {
      const float l = lg[e];
      if (l > neg_inf_f()) sum += l == top ? 1.0 : exp(static_cast<double>(l) - top);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  }
  for (int e = lane; e < E; e += 32) {
    const float l = lg[e];
    float k = neg_inf_f();
    if (l > neg_inf_f()) {
      const float s = softmax ? static_cast<float>((l == top ? 1.0 : exp(static_cast<double>(l) - top)) / sum)
                              : sigmoid_exact_f32(l);
      k = fmaxf(s + bias[e], neg_inf_f());
    }
    s_key[e] = k;
  }
  __syncwarp();
}

// The two largest exact keys among a lane's share of a group (keys j = sub,
// sub + lpg, ... of `row`, experts from e0): those whose cheap key reaches
// `reach`.
__device__ __noinline__ Top2 cold_group_top2(const float* row, const float* lg, const float* bias, int e0, int sub,
                                             int lpg, int per, float reach) {
  Top2 two{neg_inf_f(), neg_inf_f()};
  for (int j0 = sub; j0 < per; j0 += 32 * lpg) {
    unsigned todo = 0;
    for (int i = 0; i < 32 && j0 + i * lpg < per; ++i) {
      const float k = row[j0 + i * lpg];
      todo |= static_cast<unsigned>(k > neg_inf_f() && k >= reach) << i;
    }
    for (; todo != 0; todo &= todo - 1) {
      const int e = e0 + j0 + (__ffs(todo) - 1) * lpg;
      two.add(fmaxf(sigmoid_exact_f32(lg[e]) + bias[e], neg_inf_f()));
    }
  }
  return two;
}

// KPL keys a lane, VEC of them consecutive (one 16-byte load for VEC = 4).
template <int KPL, int VEC, bool BIAS>
__global__ void __launch_bounds__(32 * kRouteWarps, 5) route_grouped_kernel(const float* __restrict__ logits,
                                                                            const float* __restrict__ bias,
                                                                            const RouteGroupArgs a, GroupLayout gl,
                                                                            int warp_words, int32_t* __restrict__ ids,
                                                                            float* __restrict__ wts) {
  extern __shared__ uint4 s_all[];  // per warp: candidate keys [64] and experts [64], all keys
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + warp;
  if (t >= a.T) return;
  float* s_ckey = reinterpret_cast<float*>(s_all) + static_cast<size_t>(warp) * warp_words;
  int* s_ce = reinterpret_cast<int*>(s_ckey + kMaxCand);
  float* s_key = s_ckey + 2 * kMaxCand;
  const float* lg = logits + static_cast<size_t>(t) * a.E;
  const float NEG = neg_inf_f();
  const unsigned kAll = 0xffffffffu;
  constexpr int kChunks = KPL / VEC;
  const int chunks = (a.E + 32 * VEC - 1) / (32 * VEC);  // chunks in use, the same for all lanes
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
    load(lg, q, v);  // without a branch: all loads are in flight together
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
      if (key[i] > NEG) total += key[i] == top ? 1.f : fast_exp(key[i] - top);
    total = warp_sum(total);
  }
  float margin = BIAS ? (a.softmax ? kMarginSoftmax : kMarginSigmoid) : 0.f;

  if constexpr (BIAS) {  // the cheap keys
    const float inv_total = 1.f / total;
    auto keys = [&](auto score) {
#pragma unroll
      for (int q = 0; q < kChunks; ++q) {
        float b[VEC];
        load(bias, q, b);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          float& k = key[q * VEC + j];
          k = k > NEG ? fmaxf(score(k) + b[j], NEG) : NEG;
        }
      }
    };
    if (a.softmax)
      keys([&](float l) { return (l == top ? 1.f : fast_exp(l - top)) * inv_total; });
    else
      keys([&](float l) { return fast_rcp(1.f + fast_exp(-l)); });
  }
  int group_at[kChunks];  // this lane's chunks: their groups
#pragma unroll
  for (int q = 0; q < kChunks; ++q) group_at[q] = a.n_group > 1 && q < chunks ? gl.group(first_of(q)) : 0;
  int id = -1;  // lane j: slot j
  int kk = 0;   // slots filled
  bool exact = !BIAS, redo = false;
  for (;;) {
    if (BIAS && redo) {  // all keys exactly
      exact = true;
      margin = 0.f;
      cold_exact_keys(s_key, lg, bias, a.E, a.softmax, top);
#pragma unroll
      for (int i = 0; i < KPL; ++i) {
        const int e = first_of(i / VEC) + i % VEC;
        key[i] = e < a.E ? s_key[e] : NEG;
      }
      __syncwarp();
    }
    // the keys into shared memory, groups apart
    const int gap = gl.stride - gl.per;
    auto to_smem = [&]() {
#pragma unroll
      for (int q = 0; q < kChunks; ++q) {
        if (q >= chunks) break;
        const int e = first_of(q);
        if (e < a.E) {
          float* at = s_key + e + group_at[q] * gap;
          if constexpr (VEC == 4)
            *reinterpret_cast<float4*>(at) = make_float4(key[4 * q], key[4 * q + 1], key[4 * q + 2], key[4 * q + 3]);
          else
            *at = key[q];
        }
      }
      __syncwarp();
    };
    bool in_smem = false;
    // ---- groups
    if (a.n_group > 1) {
      to_smem();
      in_smem = true;
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
      int better;
      auto rank_groups = [&]() {
        gs = BIAS && two.k2 > NEG ? two.k1 + two.k2 : two.k1;
        better = 0;
#pragma unroll 8
        for (int q = 0; q < a.n_group; ++q) {
          const float o = __shfl_sync(kAll, gs, q * gl.lpg);
          better += o > gs || (o == gs && q < g);
        }
      };
      rank_groups();
      if (BIAS && !exact && a.topk_group < a.n_group) {
        // the last kept and the first dropped group
        const float in = __shfl_sync(kAll, gs, __ffs(__ballot_sync(kAll, mine && better == a.topk_group - 1)) - 1);
        const float out = __shfl_sync(kAll, gs, __ffs(__ballot_sync(kAll, mine && better == a.topk_group)) - 1);
        // a key's error grows with its size: with the largest of all groups
        float size = mine && two.k1 > NEG ? fabsf(two.k1) : 0.f;
        if (mine && two.k2 > NEG) size = fmaxf(size, fabsf(two.k2));
        size = fmaxf(1.f, __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(size))));
        if (out > NEG && !(in - out > 2.f * margin * size)) {
          if (a.softmax || size > 1e30f) {
            redo = true;
            continue;
          }
          // exact keys of what can be among a group's two largest
          const float reach = (two.k2 > NEG ? two.k2 : two.k1) - margin * size;
          two = mine ? cold_group_top2(row, lg, bias, g * gl.per, sub, gl.lpg, gl.per, reach) : Top2{NEG, NEG};
          __syncwarp();
          two.merge(gl.lpg);
          rank_groups();
        }
      }
      const unsigned kept = __ballot_sync(kAll, mine && better < a.topk_group);  // group q at bit q * lpg
#pragma unroll
      for (int q = 0; q < kChunks; ++q) {
        if (q >= chunks) break;
        const float most = (kept >> (group_at[q] * gl.lpg)) & 1u ? -NEG : NEG;
#pragma unroll
        for (int j = 0; j < VEC; ++j) key[q * VEC + j] = fminf(key[q * VEC + j], most);
      }
      __syncwarp();
    }
    // ---- candidates
    float lmax = NEG;
#pragma unroll
    for (int i = 0; i < KPL; ++i) lmax = fmaxf(lmax, key[i]);
    s_ckey[lane] = lmax;
    __syncwarp();
    const int larger = count_larger(lmax, s_ckey);
    // the k-th largest lane maximum, which at least k keys reach, and the largest
    float bound = order_key_inverse(__reduce_min_sync(kAll, larger < a.k ? order_key(lmax) : 0xffffffffu));
    const float umax = __shfl_sync(kAll, lmax, __ffs(__ballot_sync(kAll, larger == 0)) - 1);
    __syncwarp();
    if (a.k > 16) {  // half as many lanes hold two keys that reach it
      Top2 two{NEG, NEG};
#pragma unroll
      for (int i = 0; i < KPL; ++i) two.add(key[i]);
      s_ckey[lane] = two.k2;
      __syncwarp();
      const int l2 = count_larger(two.k2, s_ckey);
      bound = fmaxf(bound, order_key_inverse(
                               __reduce_min_sync(kAll, l2 < (a.k + 1) / 2 ? order_key(two.k2) : 0xffffffffu)));
      __syncwarp();
    }
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
    const float cut = margin_cut(bound, margin);
    unsigned mask = 0;
#pragma unroll
    for (int i = 0; i < KPL; ++i) mask |= static_cast<unsigned>(key[i] >= cut) << i;
    const int own = __popc(mask);
    int pos = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(kAll, pos, off);
      if (lane >= off) pos += o;
    }
    int n = __shfl_sync(kAll, pos, 31);
    if (n <= kMaxCand) {
      pos -= own;
      // their keys are read where they lie: an index into registers is not possible
      if (!in_smem) to_smem();
#pragma unroll 1
      for (; mask != 0; mask &= mask - 1, ++pos) {
        const int i = __ffs(mask) - 1;
        const int e = VEC * (lane + 32 * (i / VEC)) + i % VEC;
        s_ckey[pos] = s_key[a.n_group > 1 ? e + gl.group(e) * gap : e];
        s_ce[pos] = e;
      }
      __syncwarp();
    } else {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < KPL; ++i) {
        const int e = first_of(i / VEC) + i % VEC;
        if (e < a.E) s_key[e] = key[i];
      }
      __syncwarp();
      n = cold_candidates(s_key, a.E, kk, bound, umax, margin, s_ckey, s_ce);
      if (n > kMaxCand) {
        if (!exact) {
          redo = true;
          continue;
        }
        id = cold_argmax(s_key, a.E, kk);
        break;
      }
    }
    sort_candidates(s_ckey, s_ce, n, lane);
    if (!exact) {
      bool close = false;
      if (lane < kk && lane + 1 < n) {
        const float k0 = s_ckey[lane], k1 = s_ckey[lane + 1];
        close = !(k0 - k1 > margin * fmaxf(1.f, fmaxf(fabsf(k0), fabsf(k1))));
        if (close) {  // equal inputs have equal keys: their index decides, as it did
          const int e = s_ce[lane], f = s_ce[lane + 1];
          close = !(lg[e] == lg[f] && bias[e] == bias[f]);
        }
      }
      if (__any_sync(kAll, close)) {
        if (a.softmax) {
          redo = true;
          continue;
        }
#pragma unroll 1
        for (int c = lane; c < n; c += 32) s_ckey[c] = sigmoid_exact_f32(lg[s_ce[c]]) + bias[s_ce[c]];
        __syncwarp();
        sort_candidates(s_ckey, s_ce, n, lane);
      }
    }
    id = s_ce[lane];
    break;
  }

  // ---- weights
  if (lane >= kk) id = -1;
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
  const int warp_words = 2 * kMaxCand + (words + 3) / 4 * 4;
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
