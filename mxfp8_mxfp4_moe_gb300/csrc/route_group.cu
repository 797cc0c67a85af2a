// Expert routing with score functions, groups and renormalised weights, and
// its gradient with respect to the logits (definitions in include/kmoe.h).
#include <cuda_bf16.h>

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

// top, total: the softmax's largest logit (-inf: not known, nor needed) and its
// denominator relative to exp(top), the latter used without renormalisation
// only.  Shares do not change with a common factor of the scores, so softmax
// shares are taken relative to the largest chosen logit, and sigmoid shares
// below -17 (where the sigmoid is its exponential to within e^-17, less than a
// rounding) likewise: they stay right where the scores themselves underflow.
// Scores below e^-700 are 0: experts masked with the type's lowest value weigh
// nothing, not even among themselves.
__device__ __forceinline__ Share chosen_share(float l, const RouteGroupArgs& a, float top, float total) {
  constexpr float kLeast = 700.f;
  Share r{0.f, 1.f};
  bool live = l > neg_inf_f();
  float base = top;
  bool expo = a.softmax;
  if (a.renormalize) {
    live = live && l >= (a.softmax ? top - kLeast : -kLeast);
    if (a.softmax || !__any_sync(0xffffffffu, l >= -17.f)) {
      base = warp_max(live ? l : neg_inf_f());
      expo = true;
    }
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
  } else if (a.softmax && live) {  // total >= exp(top - top); it is 0 where the row has no expert left
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
//      chosen order, or at its end, closer than the margin, with a different
//      logit or bias among them: the candidates get exact keys, one or two a
//      lane, and are sorted again.
//   4. softmax scores in doubt, infinite keys, or still more than 64
//      candidates: all keys exactly, and the same steps without a margin; if
//      equal keys leave more than 64 candidates even so, k rounds of arg-max.
// Without a bias the logits are the keys and nothing is in doubt.
//
// Margin.  Sigmoid: the fast exponential is off by 2 + 1.16 |x| units in the
// last place, which the sigmoid damps to at most 0.62 units of 2^-23; the sum
// and the fast reciprocal add 1.5 more, the exact key's own two roundings one:
// 6e-7 * max(1, |key|).  Two keys: 1.2e-6; 2e-6 is used.  Softmax: the
// denominator's fp32 sum over up to 37 steps adds up to 2.3e-6 of a score; 1e-5
// is used, of 1 as for a sigmoid.  That is safe, since no score exceeds 1, and
// wide: scores of many experts are about 1 / E, and where logits or biases
// differ little many rows hold closer neighbours and go through step 4.  T =
// 8192, E = 896, k = 16, 8 groups: 85 us for logits of deviation 1.7 and biases
// of deviation 0.1, 212 with biases of 0.01, 332 with 1.0 and 0.001, 628 with
// 0.3 and 0.001 (sigmoid with a bias 21, softmax without one 16).
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
// A lower bound of the k-th largest of the lanes' values: the k-th largest of
// them rounded down to bf16, compared and counted two at a time (counts up to
// 32 are exact in bf16).  -inf where fewer than k lanes have more.
__device__ __forceinline__ float kth_largest(float v, int k, float* s_val, int lane) {
  // down: towards zero for positive values, away from it for negative ones
  uint32_t u = __float_as_uint(v);
  if (v < 0.f && v > neg_inf_f()) u += 0xFFFFu;
  const uint16_t h = static_cast<uint16_t>(u >> 16);
  reinterpret_cast<uint16_t*>(s_val)[lane] = h;
  __syncwarp();
  const uint32_t twice = h | (static_cast<uint32_t>(h) << 16);
  const __nv_bfloat162 mine = *reinterpret_cast<const __nv_bfloat162*>(&twice);
  __nv_bfloat162 r = __float2bfloat162_rn(0.f);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint4 o = reinterpret_cast<const uint4*>(s_val)[q];
    const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) r = __hadd2(r, __hgt2(*reinterpret_cast<const __nv_bfloat162*>(&w[j]), mine));
  }
  __syncwarp();
  const float larger = __low2float(r) + __high2float(r);
  const float down = __uint_as_float(static_cast<uint32_t>(h) << 16);
  return order_key_inverse(
      __reduce_min_sync(0xffffffffu, larger < static_cast<float>(k) ? order_key(down) : 0xffffffffu));
}
// Sorts the n <= 64 candidates (key, expert) in place by (larger key, lower
// expert): a lane ranks numbers lane and lane + 32.
__device__ __noinline__ void cold_sort(float* s_ckey, int* s_ce, int n, int lane) {
  const bool h0 = lane < n, h1 = lane + 32 < n;
  const float v0 = h0 ? s_ckey[lane] : 0.f, v1 = h1 ? s_ckey[lane + 32] : 0.f;
  const int e0 = h0 ? s_ce[lane] : 0, e1 = h1 ? s_ce[lane + 32] : 0;
  int r0 = 0, r1 = 0;
#pragma unroll 4
  for (int q = 0; q < n; ++q) {
    const float o = s_ckey[q];
    const int f = s_ce[q];
    r0 += o > v0 || (o == v0 && f < e0);
    r1 += o > v1 || (o == v1 && f < e1);
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
__device__ __forceinline__ void sort_candidates(float* s_ckey, int* s_ce, int n, int lane) {
  if (n <= 32) {
    const bool have = lane < n;
    const float v = have ? s_ckey[lane] : neg_inf_f();
    const int e = s_ce[lane];
    s_ckey[lane] = v;
    __syncwarp();
    const int r = count_larger(v, s_ckey);
    // equal keys have equal counts: then the index has to decide
    if (__popc(__reduce_or_sync(0xffffffffu, have ? 1u << r : 0u)) == n) {
      __syncwarp();
      if (have) {
        s_ckey[r] = v;
        s_ce[r] = e;
      }
      __syncwarp();
      return;
    }
  }
  cold_sort(s_ckey, s_ce, n, lane);
}

// The row's keys in shared memory, and its groups: LPG lanes scan a group, VEC
// keys a lane and step.
struct KeyLayout {
  int E, per;    // experts, experts a group
  int lpg, mul;  // lanes a group, 2^20 / per (rounded down) + 1
  // floor(e / per): mul exceeds 2^20 / per by at most 1, times e < 1024 that is below 2^20 / per
  __device__ __forceinline__ int group(int e) const { return (e * mul) >> 20; }
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

// Keys below this are below `v` beyond doubt.
__device__ __forceinline__ float margin_cut(float v, float margin) {
  return fmaxf(v - margin * fmaxf(1.f, fabsf(v)), -3.402823466e38f);
}

// ---- rare paths, kept out of the kernel's instruction stream.  `kept` has the
// groups that experts are chosen from, group g at bit g * lpg.

// Candidates of the largest value that kk keys reach, less the margin, written
// to s_ckey and s_ce; returns their number, which is above 64 (and nothing
// written) where equal or close keys leave more.
__device__ __noinline__ int cold_candidates(const float* s_key, const KeyLayout& kl, unsigned kept, int kk, float bound,
                                            float umax, float margin, float* s_ckey, int* s_ce) {
  const unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  auto key = [&](int e) {
    return e < kl.E && ((kept >> (kl.group(e) * kl.lpg)) & 1u) ? s_key[e] : neg_inf_f();
  };
  auto count = [&](float cut) {
    unsigned c = 0;
#pragma unroll 4
    for (int e = lane; e < kl.E; e += 32) c += key(e) >= cut;
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
  for (int e0 = 0; e0 < kl.E; e0 += 32) {
    const float k = key(e0 + lane);
    const unsigned m = __ballot_sync(kAll, k >= cut);
    if (k >= cut) {
      const int at = base + __popc(m & ((1u << lane) - 1u));
      s_ckey[at] = k;
      s_ce[at] = e0 + lane;
    }
    base += __popc(m);
  }
  __syncwarp();
  return n;
}

// kk rounds of arg-max: more equal keys than candidates fit.  Lane j gets slot j.
__device__ __noinline__ int cold_argmax(float* s_key, const KeyLayout& kl, unsigned kept, int kk) {
  const unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  int best = -1;
  for (int j = 0; j < kk; ++j) {
    uint32_t key = 0, low = 0;  // the lane's best: its key's image, ~expert
    for (int e = lane; e < kl.E; e += 32) {
      const float k = (kept >> (kl.group(e) * kl.lpg)) & 1u ? s_key[e] : neg_inf_f();
      const uint32_t image = k > neg_inf_f() ? order_key(k) : 0u;
      if (image > key) {
        key = image;
        low = 0xffffffffu - static_cast<unsigned>(e);
      }
    }
    const uint32_t top = __reduce_max_sync(kAll, key);
    const int e = static_cast<int>(0xffffffffu - __reduce_max_sync(kAll, key == top ? low : 0u));
    if (lane == j) best = e;
    if ((e & 31) == lane) s_key[e] = neg_inf_f();
    __syncwarp();
  }
  return best;
}

// All keys exactly.
__device__ __noinline__ void cold_exact_keys(float* s_key, const KeyLayout& kl, const float* lg, const float* bias,
                                             bool softmax, float top) {
  const int lane = threadIdx.x & 31;
  double sum = 0.0;
  if (softmax) {
    for (int e = lane; e < kl.E; e += 32) {
      const float l = lg[e];
      if (l > neg_inf_f()) sum += l == top ? 1.0 : exp(static_cast<double>(l) - top);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  }
  for (int e = lane; e < kl.E; e += 32) {
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

// Whether the order of the sorted candidates around the kk chosen is in doubt:
// runs of neighbours closer than the margin that begin among the chosen, and
// hold two candidates of different inputs.  Equal inputs have equal keys, so
// among those the index has decided, however many there are; but a run of them
// can stand between a chosen expert and another that it is too close to.
__device__ __noinline__ bool cold_doubt(const float* s_ckey, const int* s_ce, int n, int kk, float margin,
                                        const float* lg, const float* bias) {
  const int lane = threadIdx.x & 31;
  unsigned long long near = 0, differ = 0;  // bit r: candidates r and r + 1
  for (int h = 0; h < 64; h += 32) {
    const int r = lane + h;
    bool close = false, other = false;
    if (r + 1 < n) {
      const float k0 = s_ckey[r], k1 = s_ckey[r + 1];
      close = !(k0 - k1 > margin * fmaxf(1.f, fmaxf(fabsf(k0), fabsf(k1))));
      other = close && !(lg[s_ce[r]] == lg[s_ce[r + 1]] && bias[s_ce[r]] == bias[s_ce[r + 1]]);
    }
    near |= static_cast<unsigned long long>(__ballot_sync(0xffffffffu, close)) << h;
    differ |= static_cast<unsigned long long>(__ballot_sync(0xffffffffu, other)) << h;
  }
  // pairs up to the chosen's end, and on while the run lasts
  int last = kk - 1;
  while (last < 63 && ((near >> last) & 1u)) ++last;
  return (differ & ((1ull << last) - 1u)) != 0;
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

// The keys live in shared memory and every pass over them is a short loop: few
// registers (so that many tokens share an SM) and little code, which matter
// more here than the loads saved by keeping them in registers (28 keys a lane
// in registers and unrolled passes: 20 warps an SM, a fifth of their cycles
// without an instruction to issue, 1.14 times the time).  T = 8192, E = 896, k =
// 16, sigmoid, bias, GPU time with the inputs in HBM: 21.3 us with 8 groups,
// 18.5 without; all keys in double precision: 365.  What bounds it is the issue
// of about 1500 instructions a token (two special-function operations a key);
// the logits' 29 MB are 4.4 us at the copy rate.  VEC keys are consecutive on a
// lane (16-byte loads).
// WPT warps load a token's row and make its keys; the first chooses.  One, four
// tokens a block, where tokens are many or rows short; four where a token's
// latency counts (launch_route_vec).
template <int VEC, bool BIAS, int WPT>
__global__ void __launch_bounds__(32 * kRouteWarps, 10) route_grouped_kernel(const float* __restrict__ logits,
                                                                             const float* __restrict__ bias,
                                                                             const RouteGroupArgs a, const KeyLayout kl,
                                                                             int warp_words, int32_t* __restrict__ ids,
                                                                             float* __restrict__ wts) {
  extern __shared__ uint4 s_all[];  // per warp: candidate keys [64] and experts [64], all keys
  const int warp = WPT > 1 ? 0 : threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = WPT > 1 ? blockIdx.x : blockIdx.x * kRouteWarps + warp;
  if (t >= a.T) return;
  float* s_ckey = reinterpret_cast<float*>(s_all) + static_cast<size_t>(warp) * warp_words;
  int* s_ce = reinterpret_cast<int*>(s_ckey + kMaxCand);
  float* s_key = s_ckey + 2 * kMaxCand;
  const float* lg = logits + static_cast<size_t>(t) * a.E;
  const float NEG = neg_inf_f();
  const unsigned kAll = 0xffffffffu;
  const int step = 32 * VEC;

  auto load = [&](const float* row, int e, float (&v)[VEC]) {
    if constexpr (VEC == 4) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(row + e));
      v[0] = f.x;
      v[1] = f.y;
      v[2] = f.z;
      v[3] = f.w;
    } else {
      v[0] = __ldg(row + e);
    }
  };
  auto put = [&](int at, const float (&v)[VEC]) {
    if constexpr (VEC == 4)
      *reinterpret_cast<float4*>(s_key + at) = make_float4(v[0], v[1], v[2], v[3]);
    else
      s_key[at] = v[0];
  };
  auto get = [&](int at, float (&v)[VEC]) {
    if constexpr (VEC == 4) {
      const float4 f = *reinterpret_cast<const float4*>(s_key + at);
      v[0] = f.x;
      v[1] = f.y;
      v[2] = f.z;
      v[3] = f.w;
    } else {
      v[0] = s_key[at];
    }
  };
  auto sigmoid_keys = [&](float (&v)[VEC], const float (&b)[VEC]) {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      v[j] = v[j] > NEG ? fmaxf(fast_rcp(1.f + fast_exp(-v[j])) + b[j], NEG) : NEG;
  };

  // ---- keys: cheap ones; what cannot be chosen is -inf
  float lmax = NEG;  // of this lane's keys
  const bool denominator = a.softmax && (BIAS || !a.renormalize);
  // the whole row in flight at once, without registers; a lane reads what it copied itself
  for (int e = VEC * (WPT > 1 ? threadIdx.x : lane); e < a.E; e += step * WPT)
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(s_key + e)), "l"(lg + e), "n"(4 * VEC)
                 : "memory");
  asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 2
  for (int e = VEC * (WPT > 1 ? threadIdx.x : lane); e < a.E; e += step * WPT) {
    float v[VEC], b[VEC];
    if (BIAS) load(bias, e, b);
    get(e, v);
    if (BIAS && !a.softmax) {
      sigmoid_keys(v, b);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = fmaxf(v[j], NEG);  // NaN to -inf
    }
    put(e, v);
    if (denominator || a.n_group == 1) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) lmax = fmaxf(lmax, v[j]);
    }
  }
  unsigned kept = kAll;  // groups that experts are chosen from, group g at bit g * lpg
  unsigned open = kAll;  // this lane's chunks in them, chunk q at bit q
  auto lane_max = [&]() {
    lmax = NEG;
    open = 0;
    unsigned bit = 1;
    for (int e = VEC * lane; e < a.E; e += step, bit <<= 1) {
      float v[VEC];
      get(e, v);
      if ((kept >> (kl.group(e) * kl.lpg)) & 1u) {
        open |= bit;
#pragma unroll
        for (int j = 0; j < VEC; ++j) lmax = fmaxf(lmax, v[j]);
      }
    }
  };
  if constexpr (WPT > 1) {
    __syncthreads();
    if (threadIdx.x >= 32) return;
    if (denominator || a.n_group == 1) lane_max();
  }
  float top = NEG, total = 1.f;
  if (denominator) {  // what is stored are logits
    top = warp_max(lmax);
    total = 0.f;
    for (int e = VEC * lane; e < a.E; e += step) {
      float v[VEC];
      get(e, v);
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (v[j] > NEG) total += v[j] == top ? 1.f : fast_exp(v[j] - top);
    }
    total = warp_sum(total);
    if (BIAS) {
      const float inv_total = 1.f / total;
      lmax = NEG;
      for (int e = VEC * lane; e < a.E; e += step) {
        float v[VEC], b[VEC];
        get(e, v);
        load(bias, e, b);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float s = (v[j] == top ? 1.f : fast_exp(v[j] - top)) * inv_total;
          v[j] = v[j] > NEG ? fmaxf(s + b[j], NEG) : NEG;
          lmax = fmaxf(lmax, v[j]);
        }
        put(e, v);
      }
    }
  }
  __syncwarp();

  float margin = BIAS ? (a.softmax ? kMarginSoftmax : kMarginSigmoid) : 0.f;
  int id = -1;  // lane j: slot j
  int kk = 0;   // slots filled
  bool exact = !BIAS, redo = false;
  for (;;) {
    if (BIAS && redo) {
      exact = true;
      margin = 0.f;
      cold_exact_keys(s_key, kl, lg, bias, a.softmax, top);
    }
    if (a.n_group > 1) {
      // ---- groups
      const int g = lane / kl.lpg, sub = lane - g * kl.lpg;
      const bool mine = g < a.n_group;
      const int row = g * kl.per;
      Top2 two{NEG, NEG};
      if (mine) {
#pragma unroll 2
        for (int j = VEC * sub; j < kl.per; j += VEC * kl.lpg) {
          float v[VEC];
          get(row + j, v);
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            if (BIAS)
              two.add(v[i]);
            else
              two.k1 = fmaxf(two.k1, v[i]);
          }
        }
      }
      two.merge(kl.lpg);
      float gs;
      int better;
      auto rank_groups = [&]() {
        gs = BIAS && two.k2 > NEG ? two.k1 + two.k2 : two.k1;
        better = 0;
#pragma unroll 4
        for (int q = 0; q < a.n_group; ++q) better += __shfl_sync(kAll, gs, q * kl.lpg) > gs;
        // equal groups have equal counts: then the index decides
        if (__popc(__reduce_or_sync(kAll, mine ? 1u << better : 0u)) != a.n_group) {
          for (int q = 0; q < a.n_group; ++q) better += __shfl_sync(kAll, gs, q * kl.lpg) == gs && q < g;
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
          two = mine ? cold_group_top2(s_key + row, lg, bias, g * kl.per, sub, kl.lpg, kl.per, reach) : Top2{NEG, NEG};
          __syncwarp();
          two.merge(kl.lpg);
          rank_groups();
        }
      }
      kept = __ballot_sync(kAll, mine && better < a.topk_group);
    }
    if (a.n_group > 1 || (BIAS && redo)) lane_max();
    // ---- candidates
    // the k-th largest lane maximum, which at least k keys reach (rounded down)
    float bound = kth_largest(lmax, a.k, s_ckey, lane);
    if (a.k > 16) {  // half as many lanes hold two keys that reach it
      Top2 two{NEG, NEG};
      unsigned left = open;
      for (int e = VEC * lane; e < a.E; e += step, left >>= 1) {
        float v[VEC];
        get(e, v);
        if (left & 1u) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) two.add(v[j]);
        }
      }
      bound = fmaxf(bound, kth_largest(two.k2, (a.k + 1) / 2, s_ckey, lane));
    }
    kk = a.k;
    if (!(bound > NEG)) {  // fewer lanes than slots have anything to choose from
      unsigned alive = 0;
      for (int e = lane; e < a.E; e += 32) alive += s_key[e] > NEG && ((kept >> (kl.group(e) * kl.lpg)) & 1u);
      kk = min(a.k, static_cast<int>(__reduce_add_sync(kAll, alive)));
      if (kk == 0) break;
      bound = -3.402823466e38f;  // the lowest finite key
    }
    if (!exact && __any_sync(kAll, lmax > 1e30f)) {  // a key of such size, or infinite, has no margin
      redo = true;
      continue;
    }
    const float cut = margin_cut(bound, margin);
    unsigned mask = 0;  // this lane's keys that reach it
    unsigned left = open;
    int bit = 0;
    for (int e = VEC * lane; e < a.E; e += step, bit += VEC, left >>= 1) {
      float v[VEC];
      get(e, v);
      const float least = left & 1u ? cut : __int_as_float(0x7fc00000);  // NaN: no key reaches it
      unsigned m = 0;
#pragma unroll
      for (int j = 0; j < VEC; ++j) m |= v[j] >= least ? 1u << j : 0u;
      mask |= m << bit;
    }
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
      for (; mask != 0; mask &= mask - 1, ++pos) {
        const int i = __ffs(mask) - 1;
        const int e = VEC * (lane + 32 * (i / VEC)) + i % VEC;
        s_ckey[pos] = s_key[e];
        s_ce[pos] = e;
      }
      __syncwarp();
    } else {
      n = cold_candidates(s_key, kl, kept, kk, bound, warp_max(lmax), margin, s_ckey, s_ce);
      if (n > kMaxCand) {
        if (!exact) {
          redo = true;
          continue;
        }
        id = cold_argmax(s_key, kl, kept, kk);
        break;
      }
    }
    sort_candidates(s_ckey, s_ce, n, lane);
    if (!exact) {
      bool close = false;
      if (lane < kk && lane + 1 < n) {
        const float k0 = s_ckey[lane], k1 = s_ckey[lane + 1];
        close = !(k0 - k1 > margin * fmaxf(1.f, fmaxf(fabsf(k0), fabsf(k1))));
      }
      if (__any_sync(kAll, close) && cold_doubt(s_ckey, s_ce, n, kk, margin, lg, bias)) {
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
  KeyLayout kl{};
  kl.E = a.E;
  kl.per = a.E / a.n_group;
  kl.lpg = 32;
  while (kl.lpg * a.n_group > 32) kl.lpg >>= 1;
  kl.mul = (1 << 20) / kl.per + 1;
  const int warp_words = 2 * kMaxCand + (a.E + 3) / 4 * 4;
  // E = 896, 8 groups, us with four warps a token / one: T = 16 6.2 / 7.2, 152 7.2 / 8.2, 1216 8.6 / 10.0,
  // 2432 13.0 / 11.0; E = 256: T = 16 4.2 / 4.2, 608 5.6 / 4.2
  if (a.E >= 512 && a.T <= 152 * 8)
    route_grouped_kernel<VEC, BIAS, kRouteWarps>
        <<<a.T, 32 * kRouteWarps, warp_words * 4, st>>>(logits, bias, a, kl, warp_words, ids, wts);
  else
    route_grouped_kernel<VEC, BIAS, 1><<<(a.T + kRouteWarps - 1) / kRouteWarps, 32 * kRouteWarps,
                                         static_cast<size_t>(kRouteWarps) * warp_words * 4, st>>>(
        logits, bias, a, kl, warp_words, ids, wts);
  return cudaGetLastError();
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

// ---------------------------------------------------------------- gradient
// One warp a token; lane j holds slot j.  With p the weights without `scale`
// and g = scale * d_w:
//   renormalised: d_logit = p (g - sum g p) * slope at the chosen experts, 0
//                 elsewhere (the softmax's common term cancels);
//   sigmoid:      d_logit = g s (1 - s) at the chosen experts;
//   softmax:      d_logit = p (g - sum g p) for all experts, g = 0 where not
//                 chosen.
// Softmax forms read the whole row: that one for its terms (kRowTerms), the
// renormalised one for its largest logit (kRowTop), which decides what weighs
// nothing (chosen_share) and which a bias can have kept out of the chosen.
// Memory bounds it: E floats are written a token, and read for a softmax.  The
// row goes out as 16-byte zeros (or softmax terms), then the chosen elements
// over them; a slot whose expert an earlier slot has too (routing gives none)
// is added there.
// T = 8192, E = 896, k = 16: sigmoid, 29 MB written in 10.3 us, about 4 of them
// launch and the dependent look-up of the slots' logits (zeros stored before
// the look-up: 2 us more); softmax, 59 MB, 14.4 us in both forms.
enum RowUse { kNoRow, kRowTop, kRowTerms };
template <int KPL, int VEC, RowUse ROW>
__global__ void __launch_bounds__(32 * kRouteWarps) route_backward_kernel(const float* __restrict__ d_w,
                                                                          const float* __restrict__ logits,
                                                                          const int32_t* __restrict__ ids,
                                                                          const RouteGroupArgs a,
                                                                          float* __restrict__ d_logits) {
  constexpr bool FULL = ROW == kRowTerms;
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const float NEG = neg_inf_f();
  const float* lg = logits + static_cast<size_t>(t) * a.E;
  float* out = d_logits + static_cast<size_t>(t) * a.E;
  constexpr int kChunks = KPL / VEC;
  float p_all[ROW != kNoRow ? KPL : 1];
  auto store_row = [&](float factor) {  // p_all * factor, or zeros
#pragma unroll
    for (int q = 0; q < kChunks; ++q) {
      const int e = VEC * (lane + 32 * q);
      if (e >= a.E) break;
      if constexpr (VEC == 4) {
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if constexpr (FULL)
          f = make_float4(p_all[4 * q] * factor, p_all[4 * q + 1] * factor, p_all[4 * q + 2] * factor,
                          p_all[4 * q + 3] * factor);
        *reinterpret_cast<float4*>(out + e) = f;
      } else {
        out[e] = FULL ? p_all[FULL ? q : 0] * factor : 0.f;
      }
    }
  };
  if constexpr (ROW != kNoRow) {  // in flight while the slots are looked up
#pragma unroll
    for (int q = 0; q < kChunks; ++q) {
      const int e = VEC * (lane + 32 * q);
      if constexpr (VEC == 4) {
        const float4 f = e < a.E ? __ldg(reinterpret_cast<const float4*>(lg + e)) : make_float4(NEG, NEG, NEG, NEG);
        p_all[4 * q] = f.x;
        p_all[4 * q + 1] = f.y;
        p_all[4 * q + 2] = f.z;
        p_all[4 * q + 3] = f.w;
      } else {
        p_all[q] = e < a.E ? __ldg(lg + e) : NEG;
      }
    }
  }
  int id = lane < a.k ? ids[static_cast<size_t>(t) * a.k + lane] : -1;
  const float given_w = lane < a.k ? d_w[static_cast<size_t>(t) * a.k + lane] : 0.f;
  if (id < 0 || id >= a.E) id = -1;
  const float given = id >= 0 ? __ldg(lg + id) : NEG;
  const float l = given > NEG ? given : NEG;  // NaN too
  const float g = l > NEG ? a.scale * given_w : 0.f;

  float top = NEG, total = 1.f;
  if constexpr (ROW != kNoRow) {
#pragma unroll
    for (int i = 0; i < KPL; ++i) top = fmaxf(top, p_all[i]);  // fmaxf drops NaN
    top = warp_max(top);
  }
  if constexpr (FULL) {
    total = 0.f;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      p_all[i] = p_all[i] > NEG ? (p_all[i] == top ? 1.f : expf(p_all[i] - top)) : 0.f;
      total += p_all[i];
    }
    total = warp_sum(total);
  }
  const Share sh = chosen_share(l, a, top, total);
  const float s = sh.p;
  const float d = a.renormalize ? s * (g - warp_sum(g * s)) * sh.slope : g * s * sh.slope;
  float common = 0.f, factor = 0.f;  // sum g p, and what turns p_all into its row's terms
  if constexpr (FULL) {
    common = warp_sum(d);
    factor = total > 0.f ? -common / total : 0.f;
  }
  store_row(factor);
  const unsigned same = __match_any_sync(0xffffffffu, id);
  float acc = d;
  if (__any_sync(0xffffffffu, id >= 0 && (same & (same - 1)) != 0)) {  // in slot order
    acc = 0.f;
    for (int j = 0; j < a.k; ++j) {
      const float o = __shfl_sync(0xffffffffu, d, j);
      if ((same >> j) & 1u) acc += o;
    }
  }
  __syncwarp();  // the row's stores come before these
  if (id >= 0 && l > NEG && lane == __ffs(same) - 1) out[id] = FULL ? fmaf(-s, common, acc) : acc;
}

template <int VEC>
cudaError_t launch_route_backward_vec(const float* d_w, const float* logits, const int32_t* ids,
                                      const RouteGroupArgs& a, float* d_logits, cudaStream_t st) {
  const RowUse row = !a.softmax ? kNoRow : (a.renormalize ? kRowTop : kRowTerms);
  const int warps = a.T <= 152 * kRouteWarps ? 1 : kRouteWarps;
  const int blocks = (a.T + warps - 1) / warps;
  const int kpl = (a.E + 32 * VEC - 1) / (32 * VEC) * VEC;
#define KMOE_ROUTE_ROW(N, ROW) \
  route_backward_kernel<N, VEC, ROW><<<blocks, 32 * warps, 0, st>>>(d_w, logits, ids, a, d_logits)
#define KMOE_ROUTE(N)                   \
  if (kpl <= N) {                       \
    if (row == kRowTerms)               \
      KMOE_ROUTE_ROW(N, kRowTerms);     \
    else if (row == kRowTop)            \
      KMOE_ROUTE_ROW(N, kRowTop);       \
    else                                \
      KMOE_ROUTE_ROW(N, kNoRow);        \
    return cudaGetLastError();          \
  }
  KMOE_ROUTE(4)
  KMOE_ROUTE(8)
  KMOE_ROUTE(16)
  KMOE_ROUTE(32)
#undef KMOE_ROUTE
#undef KMOE_ROUTE_ROW
  return cudaErrorInvalidValue;
}

cudaError_t launch_route_backward(const float* d_w, const float* logits, const int32_t* ids, const RouteGroupArgs& a,
                                  float* d_logits, cudaStream_t st) {
  const uintptr_t both = reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(d_logits);
  return (both & 15) == 0 && a.E % 4 == 0 ? launch_route_backward_vec<4>(d_w, logits, ids, a, d_logits, st)
                                          : launch_route_backward_vec<1>(d_w, logits, ids, a, d_logits, st);
}

}  // namespace kmoe
