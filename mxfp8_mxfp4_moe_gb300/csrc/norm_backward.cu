// Gradient of the norm (norm.cu).  With n = h * rstd, g = dy * w:
//   dh = dh_in + rstd * (g - n * mean(g * n)),  dw = sum over rows of dy * n.
// rstd is recomputed from h in the pass that reads it anyway.  Each block adds
// its rows' share of dw in fp32 and writes one partial row; a second kernel
// adds the partial rows in order, so dw does not depend on timing.
//
// Measured (GPU time, inputs from HBM): T = 8192, H = 7168, bf16: 470 MB in 76
// us, 6.2 TB/s, 0.93 of the copy rate, the second kernel (about 4 us, most of
// it hidden by its early launch) included; an fp32 stream: 822 MB in 183 us,
// 4.5 TB/s, 0.67 (one block an SM, three rows of 72 KB in its ring).  T = 333, H
// = 3584, fp32 stream: 12.6 us for both kernels.
#include "norm_dev.cuh"

namespace kmoe {

struct NormGradArgs {
  const __nv_bfloat16* dy;
  const void* h;
  const void* weight;
  bool weight_f32;
  const void* dh_in;  // of the stream's type, may be dh
  int T, H, stages;
  float eps;
  void* dh;
  float* part;  // [blocks, H]
};

// The row's two sums (h^2 and dy * w * h) come from a first read of its ring
// slot, dh and the dw terms from a second: shared memory keeps the row across
// the barrier, the registers hold weights and dw sums only.
template <class S, int NC, bool WARP, bool RAGGED>
__global__ void __launch_bounds__(512, NC == 4 ? 1 : 2) rmsnorm_backward_kernel(const NormGradArgs a) {
  extern __shared__ uint4 s_ring[];
  __shared__ float s_part[2 * 2 * 32];
  const int lane = threadIdx.x & 31;
  const int TS = WARP ? 32 : blockDim.x;
  const int rank = WARP ? lane : threadIdx.x;
  const int per_block = WARP ? blockDim.x >> 5 : 1;
  const int team = blockIdx.x * per_block + (WARP ? threadIdx.x >> 5 : 0);
  const int teams = gridDim.x * per_block;
  const int T = a.T, H = a.H, stages = a.stages;
  const int slots = TS * NC;
  constexpr int kS = sizeof(S) / 2;  // planes of a stream tensor
  constexpr int kPlanes = 1 + 2 * kS;
  uint4* ring = s_ring + (WARP ? (threadIdx.x >> 5) * stages * slots * kPlanes : 0);
  const int lead = RAGGED ? ((team & 7) * (H & 7)) & 7 : 0;
  const int nchunk = (lead + H + 7) >> 3;
  const size_t total = static_cast<size_t>(T) * H;
  const S* h = static_cast<const S*>(a.h);
  const S* dh_in = static_cast<const S*>(a.dh_in);

  auto issue = [&](int t, int s) {
    if (t < T) {
      const size_t first = static_cast<size_t>(t) * H - lead;
      uint4* slot = ring + s * slots * kPlanes;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = i * TS + rank;
        if (c >= nchunk) break;
        load_chunk<__nv_bfloat16, RAGGED>(slot + c, slots, a.dy, first + 8 * c, total);
        load_chunk<S, RAGGED>(slot + slots + c, slots, h, first + 8 * c, total);
        if (dh_in) load_chunk<S, RAGGED>(slot + (1 + kS) * slots + c, slots, dh_in, first + 8 * c, total);
      }
    }
    cp_async_commit();
  };
  for (int s = 0; s < stages; ++s) issue(team + s * teams, s);
  float2 w[NC][4], dw[NC][4];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = i * TS + rank;
    zero(w[i]);
    zero(dw[i]);
    if (c < nchunk) load_weight<RAGGED>(a.weight, a.weight_f32, 8 * c - lead, H, w[i]);
  }

  int s = 0, odd = 0;
  const float inv_h = 1.f / static_cast<float>(H);
  for (int t = team; t < T; t += teams) {
    const size_t base = static_cast<size_t>(t) * H;
    cp_async_wait(stages - 1);
    const uint4* slot = ring + s * slots * kPlanes;
    float2 ss = make_float2(0.f, 0.f), gh = ss;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = i * TS + rank;
      if (c >= nchunk) break;
      float2 d[4], v[4];
      read_chunk<__nv_bfloat16>(slot + c, slots, d);
      read_chunk<S>(slot + slots + c, slots, v);
      const int j0 = 8 * c - lead;
      if (RAGGED && (j0 < 0 || j0 + 8 > H)) {
        mask_edge(v, j0, H);
        mask_edge(d, j0, H);
      }
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        ss = __ffma2_rn(v[p], v[p], ss);
        gh = __ffma2_rn(__fmul2_rn(d[p], w[i][p]), v[p], gh);
      }
    }
    float sum[2] = {ss.x + ss.y, gh.x + gh.y};
    team_sum<2, WARP>(sum, s_part, odd);
    const float rstd = rsqrtf(sum[0] * inv_h + a.eps);
    const float nc1 = -sum[1] * rstd * inv_h;  // -mean(g * n)
    const float2 rstd2 = make_float2(rstd, rstd), nc2 = make_float2(nc1, nc1);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = i * TS + rank;
      if (c >= nchunk) break;
      float2 d[4], v[4], o[4];
      read_chunk<__nv_bfloat16>(slot + c, slots, d);
      read_chunk<S>(slot + slots + c, slots, v);
      zero(o);
      if (dh_in) read_chunk<S>(slot + (1 + kS) * slots + c, slots, o);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float2 n = __fmul2_rn(v[p], rstd2);
        dw[i][p] = __ffma2_rn(d[p], n, dw[i][p]);
        o[p] = __ffma2_rn(rstd2, __ffma2_rn(d[p], w[i][p], __fmul2_rn(n, nc2)), o[p]);
      }
      Vec8<S> q;
      pack(o, q);
      store_chunk<S, RAGGED>(static_cast<S*>(a.dh) + base, 8 * c - lead, H, q);
    }
    issue(t + stages * teams, s);
    s = s + 1 == stages ? 0 : s + 1;
    odd ^= 1;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!WARP) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = i * TS + rank;
      if (c >= nchunk) break;
      Vec8<float> q;
      pack(dw[i], q);
      store_chunk<float, RAGGED>(a.part + static_cast<size_t>(blockIdx.x) * H, 8 * c - lead, H, q);
    }
    return;
  }
  // the block's warps added in order, through the ring's memory
  float* s_dw = reinterpret_cast<float*>(s_ring);  // [warps][H]
  cp_async_wait(0);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = i * TS + rank;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int col = 8 * c - lead + 2 * p;
      float* row = s_dw + (threadIdx.x >> 5) * H;
      if (col >= 0 && col < H) row[col] = dw[i][p].x;
      if (col + 1 >= 0 && col + 1 < H) row[col + 1] = dw[i][p].y;
    }
  }
  __syncthreads();
  for (int col = threadIdx.x; col < H; col += blockDim.x) {
    float v = 0.f;
    for (int k = 0; k < per_block; ++k) v += s_dw[k * H + col];
    a.part[static_cast<size_t>(blockIdx.x) * H + col] = v;
  }
}

// Sum of the partial rows: 32 columns a block, 16 warps that take every 16th
// row, then the warps in order.
__global__ void __launch_bounds__(512) rmsnorm_dweight_kernel(const float* __restrict__ part, int parts, int H,
                                                              float* __restrict__ dweight) {
  __shared__ float s_sum[16][32];
  chain_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (col < H) {
#pragma unroll 8
    for (int p = warp; p < parts; p += 16) v += part[static_cast<size_t>(p) * H + col];
  }
  s_sum[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && col < H) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) sum += s_sum[k][lane];
    dweight[col] = sum;
  }
}

// Block b takes rows b, b + blocks, ...
template <class S>
__global__ void __launch_bounds__(256) rmsnorm_backward_elems_kernel(const NormGradArgs a) {
  extern __shared__ float s_dw[];  // [H]
  __shared__ float s_part[8];
  const int H = a.H;
  const S* h = static_cast<const S*>(a.h);
  const S* dh_in = static_cast<const S*>(a.dh_in);
  auto weight = [&](int i) {
    return a.weight_f32 ? load_f(static_cast<const float*>(a.weight), i)
                        : load_f(static_cast<const __nv_bfloat16*>(a.weight), i);
  };
  for (int i = threadIdx.x; i < H; i += blockDim.x) s_dw[i] = 0.f;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t base = static_cast<size_t>(t) * H;
    float ss = 0.f, gh = 0.f;
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
      const float hv = load_f(h, base + i);
      ss = fmaf(hv, hv, ss);
      gh = fmaf(load_f(a.dy, base + i) * weight(i), hv, gh);
    }
    ss = block_sum(ss, s_part);
    gh = block_sum(gh, s_part);
    const float rstd = rsqrtf(ss / static_cast<float>(H) + a.eps);
    const float c = gh * rstd / static_cast<float>(H);
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
      const float n = load_f(h, base + i) * rstd;
      const float d = load_f(a.dy, base + i);
      s_dw[i] = fmaf(d, n, s_dw[i]);
      const float v = rstd * (d * weight(i) - n * c);
      store_f(static_cast<S*>(a.dh), base + i, dh_in ? load_f(dh_in, base + i) + v : v);
    }
  }
  for (int i = threadIdx.x; i < H; i += blockDim.x) a.part[static_cast<size_t>(blockIdx.x) * H + i] = s_dw[i];
}

template <class S, int NC, bool WARP, bool RAGGED>
cudaError_t launch_rows(const NormGradArgs& a, const NormPlan& p, cudaStream_t st) {
  static int ready[kMaxDevices] = {};
  const cudaError_t e = allow_smem(rmsnorm_backward_kernel<S, NC, WARP, RAGGED>, ready);
  if (e != cudaSuccess) return e;
  // a warp's share of dw passes through the ring's memory
  const size_t own = p.warp ? static_cast<size_t>(p.threads / 32) * a.H * 4 : 0;
  rmsnorm_backward_kernel<S, NC, WARP, RAGGED><<<p.blocks, p.threads, p.smem > own ? p.smem : own, st>>>(a);
  return cudaGetLastError();
}
template <class S, int NC>
cudaError_t launch_nc(const NormGradArgs& a, const NormPlan& p, cudaStream_t st) {
  if (a.H % 8 == 0)
    return p.warp ? launch_rows<S, NC, true, false>(a, p, st) : launch_rows<S, NC, false, false>(a, p, st);
  return p.warp ? launch_rows<S, NC, true, true>(a, p, st) : launch_rows<S, NC, false, true>(a, p, st);
}
template <class S>
cudaError_t launch_stream(NormGradArgs a, float* dweight, cudaStream_t st) {
  constexpr uintptr_t kVec = 15;
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.h) |
                        reinterpret_cast<uintptr_t>(a.dh_in) | reinterpret_cast<uintptr_t>(a.dh) |
                        reinterpret_cast<uintptr_t>(a.weight);
  const NormPlan p = (all & kVec) == 0 ? plan_norm(a.T, a.H, 16 * (1 + sizeof(S)), true) : NormPlan{};
  a.stages = p.stages;
  const int parts = p.nc ? p.blocks : (a.T < kNormMaxParts ? a.T : kNormMaxParts);
  // one block's partial row is the sum
  const bool alone = parts == 1 && (reinterpret_cast<uintptr_t>(dweight) & kVec) == 0;
  if (alone) a.part = dweight;
  cudaError_t e;
  if (p.nc == 1) {
    e = launch_nc<S, 1>(a, p, st);
  } else if (p.nc == 2) {
    e = launch_nc<S, 2>(a, p, st);
  } else if (p.nc == 4) {
    e = launch_nc<S, 4>(a, p, st);
  } else {
    static int ready[kMaxDevices] = {};
    e = allow_smem(rmsnorm_backward_elems_kernel<S>, ready);
    if (e != cudaSuccess) return e;
    rmsnorm_backward_elems_kernel<S><<<parts, 256, static_cast<size_t>(a.H) * 4, st>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || alone) return e;
  return launch_chained(rmsnorm_dweight_kernel, dim3((a.H + 31) / 32), dim3(512), 0, st, true,
                        static_cast<const float*>(a.part), parts, a.H, dweight);
}

cudaError_t launch_rmsnorm_backward(const void* dy, const void* h, const void* weight, const void* dh_in, int T, int H,
                                    float eps, bool stream_f32, bool weight_f32, void* dh, float* dweight, float* part,
                                    cudaStream_t st) {
  if (T == 0) return cudaMemsetAsync(dweight, 0, static_cast<size_t>(H) * 4, st);
  const NormGradArgs a{static_cast<const __nv_bfloat16*>(dy), h, weight, weight_f32, dh_in, T, H, 0, eps, dh, part};
  return stream_f32 ? launch_stream<float>(a, dweight, st) : launch_stream<__nv_bfloat16>(a, dweight, st);
}

}  // namespace kmoe
