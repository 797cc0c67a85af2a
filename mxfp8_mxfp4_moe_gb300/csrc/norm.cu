// Root-mean-square norm of the rows that enter the expert layer, with the
// residual's addition in front and the MXFP8 quantisation behind it.
//   h = x + r,  y = bf16(h * rstd * w),  rstd = (mean(h^2) + eps)^-1/2,
// sums and products in fp32; y comes from the unrounded h, the stored h is
// rounded once to the stream's type.  The codes are those of the bf16 row y
// (not of the fp32 product), so that a layer fed with them gives what the
// layer fed with y gives, bit for bit.
//
// Measured (row layout and ring in norm_dev.cuh; GPU time, inputs from HBM): T =
// 8192, H = 7168, bf16 stream, with codes: 530 MB in 87 us, 6.1 TB/s, 0.91 of
// the copy rate; without codes 470 MB in 84 us.  HBM bounds it: a fifth fewer
// instructions left the time as it was.  An fp32 stream, with codes: 763 MB in
// 141 us, 5.4 TB/s, 0.81.  T = 1024, bf16: 16.5 us, of which about 5 are launch
// and the first rows' latency; one row: 4.1 us, a launch.
#include "norm_dev.cuh"

namespace kmoe {

struct NormArgs {
  const __nv_bfloat16* x;
  const void* residual;  // of the stream's type, may be h
  const void* weight;
  bool weight_f32;
  int T, H, stages;
  float eps;
  void* h;
  __nv_bfloat16* y;
  uint8_t* codes;
  uint8_t* scales;
};

// A quad of lanes holds a scale group of 32 columns.  The stored h, the sum of
// squares and y all come from one read of the row: its fp32 values stay in
// registers across the row's one barrier, and their ring slot is filled again
// before it.
template <class S, int NC, bool WARP, bool RAGGED>
__global__ void __launch_bounds__(512, NC == 4 ? 1 : 2) rmsnorm_kernel(const NormArgs a) {
  extern __shared__ uint4 s_ring[];
  __shared__ float s_part[2 * 32];
  const int lane = threadIdx.x & 31;
  const int TS = WARP ? 32 : blockDim.x;
  const int rank = WARP ? lane : threadIdx.x;
  const int per_block = WARP ? blockDim.x >> 5 : 1;
  const int team = blockIdx.x * per_block + (WARP ? threadIdx.x >> 5 : 0);
  const int teams = gridDim.x * per_block;
  const int T = a.T, H = a.H, stages = a.stages;
  const int slots = TS * NC;
  constexpr int kPlanes = 1 + sizeof(S) / 2;
  uint4* ring = s_ring + (WARP ? (threadIdx.x >> 5) * stages * slots * kPlanes : 0);
  const int lead = RAGGED ? ((team & 7) * (H & 7)) & 7 : 0;
  const int nchunk = (lead + H + 7) >> 3;
  const size_t total = static_cast<size_t>(T) * H;
  const S* residual = static_cast<const S*>(a.residual);

  auto issue = [&](int t, int s) {
    if (t < T) {
      const size_t first = static_cast<size_t>(t) * H - lead;
      uint4* slot = ring + s * slots * kPlanes;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = i * TS + rank;
        if (c >= nchunk) break;
        load_chunk<__nv_bfloat16, RAGGED>(slot + c, slots, a.x, first + 8 * c, total);
        if (residual) load_chunk<S, RAGGED>(slot + slots + c, slots, residual, first + 8 * c, total);
      }
    }
    cp_async_commit();
  };
  for (int s = 0; s < stages; ++s) issue(team + s * teams, s);
  float2 w[NC][4];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = i * TS + rank;
    if (c < nchunk) load_weight<RAGGED>(a.weight, a.weight_f32, 8 * c - lead, H, w[i]);
  }

  int s = 0, odd = 0;
  for (int t = team; t < T; t += teams) {
    const size_t base = static_cast<size_t>(t) * H;
    cp_async_wait(stages - 1);
    const uint4* slot = ring + s * slots * kPlanes;
    float2 v[NC][4], sq = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = i * TS + rank;
      zero(v[i]);
      if (c >= nchunk) continue;
      read_chunk<__nv_bfloat16>(slot + c, slots, v[i]);
      if (residual) {
        float2 r[4];
        read_chunk<S>(slot + slots + c, slots, r);
#pragma unroll
        for (int p = 0; p < 4; ++p) v[i][p] = __fadd2_rn(v[i][p], r[p]);
      }
      const int j0 = 8 * c - lead;
      if (RAGGED && (j0 < 0 || j0 + 8 > H)) mask_edge(v[i], j0, H);
      if (a.h) {
        Vec8<S> o;
        pack(v[i], o);
        store_chunk<S, RAGGED>(static_cast<S*>(a.h) + base, j0, H, o);
      }
#pragma unroll
      for (int p = 0; p < 4; ++p) sq = __ffma2_rn(v[i][p], v[i][p], sq);
    }
    issue(t + stages * teams, s);
    float sum[1] = {sq.x + sq.y};
    team_sum<1, WARP>(sum, s_part, odd);
    const float rstd = rsqrtf(sum[0] / static_cast<float>(H) + a.eps);
    const float2 rstd2 = make_float2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = i * TS + rank;
      const bool active = c < nchunk;
      Vec8<__nv_bfloat16> o;
      o.q[0] = make_uint4(0u, 0u, 0u, 0u);
      if (active) {
#pragma unroll
        for (int p = 0; p < 4; ++p) v[i][p] = __fmul2_rn(__fmul2_rn(v[i][p], rstd2), w[i][p]);
        pack(v[i], o);
        if (a.y) store_chunk<__nv_bfloat16, RAGGED>(a.y + base, 8 * c - lead, H, o);
      }
      if (!RAGGED && a.codes) {
        // the quad's largest magnitude; H is a multiple of 32, so whole quads are active or not
        uint32_t amax = bf16_amax_nan(o.q[0]);
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        if (__any_sync(0xffffffffu, amax > 0x7F80u)) {  // rare: without the NaN
          o.q[0] = bf16_drop_nan(o.q[0]);
          amax = bf16_amax_nan(o.q[0]);
          amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        }
        if (active) {
          const uint32_t scale = e4m3_scale_byte(amax);
          reinterpret_cast<uint2*>(a.codes + base)[c] = e4m3_chunk(o.q[0], scale);
          if ((c & 3) == 0) a.scales[(base >> 5) + (c >> 2)] = static_cast<uint8_t>(scale);
        }
      }
    }
    s = s + 1 == stages ? 0 : s + 1;
    odd ^= 1;
  }
}

// One block per row.
template <class S>
__global__ void __launch_bounds__(256) rmsnorm_elems_kernel(const NormArgs a) {
  extern __shared__ float s_h[];  // [H]
  __shared__ float s_part[8];
  const int H = a.H;
  const size_t base = static_cast<size_t>(blockIdx.x) * H;
  const S* residual = static_cast<const S*>(a.residual);
  float sum = 0.f;
  for (int i = threadIdx.x; i < H; i += blockDim.x) {
    float v = load_f(a.x, base + i);
    if (residual) v += load_f(residual, base + i);
    if (a.h) store_f(static_cast<S*>(a.h), base + i, v);
    s_h[i] = v;
    sum = fmaf(v, v, sum);
  }
  const float rstd = rsqrtf(block_sum(sum, s_part) / static_cast<float>(H) + a.eps);
  for (int i = threadIdx.x; i < H; i += blockDim.x) {
    const float w = a.weight_f32 ? load_f(static_cast<const float*>(a.weight), i)
                                 : load_f(static_cast<const __nv_bfloat16*>(a.weight), i);
    const __nv_bfloat16 yb = __float2bfloat16_rn(s_h[i] * rstd * w);
    if (a.y) a.y[base + i] = yb;
    if (a.codes) {  // 32 consecutive columns a warp: one scale group (H is a multiple of 32)
      const float v = __bfloat162float(yb);
      float amax = isnan(v) ? 0.f : fabsf(v);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
      const int e = e4m3_scale_exp(amax);
      a.codes[base + i] = e4m3_code(v, exp2i(-e));
      if ((i & 31) == 0) a.scales[(base + i) >> 5] = static_cast<uint8_t>(e + 127);
    }
  }
}

template <class S, int NC, bool WARP, bool RAGGED>
cudaError_t launch_rows(const NormArgs& a, const NormPlan& p, cudaStream_t st) {
  static int ready[kMaxDevices] = {};
  const cudaError_t e = allow_smem(rmsnorm_kernel<S, NC, WARP, RAGGED>, ready);
  if (e != cudaSuccess) return e;
  rmsnorm_kernel<S, NC, WARP, RAGGED><<<p.blocks, p.threads, p.smem, st>>>(a);
  return cudaGetLastError();
}
template <class S, int NC>
cudaError_t launch_nc(const NormArgs& a, const NormPlan& p, cudaStream_t st) {
  if (a.H % 8 == 0)
    return p.warp ? launch_rows<S, NC, true, false>(a, p, st) : launch_rows<S, NC, false, false>(a, p, st);
  return p.warp ? launch_rows<S, NC, true, true>(a, p, st) : launch_rows<S, NC, false, true>(a, p, st);
}
template <class S>
cudaError_t launch_stream(NormArgs a, cudaStream_t st) {
  constexpr uintptr_t kVec = 15;
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.residual) |
                        reinterpret_cast<uintptr_t>(a.h) | reinterpret_cast<uintptr_t>(a.y) |
                        reinterpret_cast<uintptr_t>(a.weight);
  const NormPlan p = (all & kVec) == 0 ? plan_norm(a.T, a.H, 16 * (1 + sizeof(S) / 2), false) : NormPlan{};
  a.stages = p.stages;
  if (p.nc == 1) return launch_nc<S, 1>(a, p, st);
  if (p.nc == 2) return launch_nc<S, 2>(a, p, st);
  if (p.nc == 4) return launch_nc<S, 4>(a, p, st);
  static int ready[kMaxDevices] = {};
  const cudaError_t e = allow_smem(rmsnorm_elems_kernel<S>, ready);
  if (e != cudaSuccess) return e;
  rmsnorm_elems_kernel<S><<<a.T, 256, static_cast<size_t>(a.H) * 4, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_rmsnorm(const void* x, const void* residual, const void* weight, int T, int H, float eps,
                           bool stream_f32, bool weight_f32, void* h, void* y, uint8_t* codes, uint8_t* scales,
                           cudaStream_t st) {
  const NormArgs a{static_cast<const __nv_bfloat16*>(x), residual, weight, weight_f32, T, H, 0, eps, h,
                   static_cast<__nv_bfloat16*>(y), codes, scales};
  return stream_f32 ? launch_stream<float>(a, st) : launch_stream<__nv_bfloat16>(a, st);
}

}  // namespace kmoe
