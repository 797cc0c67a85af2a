// Block-scaled E4M3 products of many rows: rows times weights and rows times
// transposed weights, dense or by expert (fp8_gemm.cu has the definition, the
// operands' layouts and the kernel for few rows).
//
// Here the rows are the MMA's M: a tile is 128 rows x 256 features.  A TMEM
// lane is a row, so a thread's factor for a block of the sum is one product
// of two scales for 128 features, and the epilogue is one read of TMEM and
// one multiply-add a value; with the rows in the MMA's N it needs a factor a
// column, from shared memory that the tensor core is reading.
//
// Roles: warp 0 TMA, warp 1 MMA (both converged, one elected lane issues),
// warps 4 .. 15 the epilogue: three groups of four (one warp per TMEM lane
// quarter) that take the eight 32-column chunks in turn.  Every wait is
// bounded.
#include "fp8_dev.cuh"

namespace kmoe {

template <bool BACK_>
struct Fp8WideCfg {
  static constexpr bool BACK = BACK_;  // the weights transposed, read MN-major
  static constexpr int BM = 128, BN = 256;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = 4;
  static constexpr int NG = 3, NCH = 3;  // groups, and the most 32-column chunks of one
  static constexpr int EPI_WARPS = 4 * NG;
  static constexpr int CTRL_WARPS = 4;
  static constexpr int THREADS = 32 * (CTRL_WARPS + EPI_WARPS);
  // 96 accumulators a thread and 32 values being read
  static constexpr int CTRL_REGS = 32, EPI_REGS = 160;
  static constexpr int NACC = 2;
  static constexpr int BAR_OFF = STAGES * STAGE;
  static constexpr int TAB_OFF = BAR_OFF + 256;
  static constexpr int TAB_INTS = kMaxE + 1;
  static constexpr int SMEM = 1024 + TAB_OFF + (2 * TAB_INTS + 40) * 4;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(128 * CTRL_REGS + 32 * EPI_WARPS * EPI_REGS <= THREADS * 128, "register split");
};

template <class C>
__device__ __forceinline__ Fp8Item wide_item(const Fp8Args& a, const int32_t* first, const int32_t* unit, int w) {
  Fp8Item it;
  it.e = segment_of_unit(unit, a.E, w / a.FT);
  const int u0 = unit[it.e], nt = unit[it.e + 1] - u0;
  const int r = w - u0 * a.FT;
  it.f0 = r / nt * C::BN;
  const int at = r % nt * C::BM;
  it.c0 = first[it.e] + at;
  it.n = min(C::BM, first[it.e + 1] - it.c0);
  it.kb = 0;
  it.kn = a.KB;
  return it;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) fp8_gemm_wide_kernel(const __grid_constant__ Fp8Maps maps,
                                                                     const Fp8Args a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* acc_empty = acc_full + C::NACC;
  uint64_t* done = acc_empty + C::NACC;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* first = reinterpret_cast<int32_t*>(smem + C::TAB_OFF);
  int32_t* unit = first + C::TAB_INTS;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::NACC; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], C::EPI_WARPS);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.b);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::NACC * C::BN);
    tmem_relinquish();
  }
  chain_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;  // long before any wait can give up
  tc_fence_before();
  segment_prefix(a.seg, a.E, a.M, C::BM, first, unit, unit + C::TAB_INTS);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = a.FT * unit[a.E];
  const uint64_t budget = a.budget_ns;

  if (warp < C::CTRL_WARPS) {
    // (of the registers that the block was launched with)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::CTRL_REGS));
    if (warp == 0) {
      // ------------------------------------------------------------ loads
      const uint64_t pol_w = policy_evict_normal(), pol_x = policy_evict_last();
      uint32_t it = 0;
      bool ok = true;
      for (int w = blockIdx.x; ok && w < total; w += gridDim.x) {
        const Fp8Item wk = wide_item<C>(a, first, unit, w);
        const int boxes = a.F - wk.f0 > 128 ? 2 : 1;  // of 128 features
        const uint32_t tx = C::A_BYTES + boxes * 16384;
        for (int kb = 0; kb < wk.kn; ++kb, ++it) {
          const int s = it % C::STAGES;
          if (!wait_warp(&empty[s], ((it / C::STAGES) & 1u) ^ 1u, budget, a.err, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + s * C::STAGE;
          const int k0 = kb * kScaleBlock;
          mbar_arrive_expect_tx_el(&full[s], tx);
          tma_load_2d_el(sa, &maps.b, &full[s], k0, wk.c0, pol_x);
          for (int i = 0; i < boxes; ++i) {
            const int f = wk.f0 + i * 128;
            tma_load_3d_el(sa + C::A_BYTES + i * 16384, &maps.a, &full[s], C::BACK ? f : k0, C::BACK ? k0 : f, wk.e,
                           pol_w);
          }
        }
      }
      if (!ok) {
        // let the copies already issued land before the CTA can exit
        const uint32_t from = it > static_cast<uint32_t>(C::STAGES) ? it - C::STAGES : 0u;
        for (uint32_t i = from; i < it; ++i)
          mbar_wait_warp(&full[i % C::STAGES], (i / C::STAGES) & 1u, 20000000ull, nullptr, nullptr);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA
      constexpr uint32_t kStepB = C::BACK ? 256 : 2;  // 32 of the sum, as in fp8_gemm.cu
      const uint64_t adesc0 = sdesc_kmajor_sw128(smem_u32(smem));
      const uint64_t bdesc0 = C::BACK ? make_sdesc(smem_u32(smem + C::A_BYTES), 16384, 1024, 2)
                                      : sdesc_kmajor_sw128(smem_u32(smem + C::A_BYTES));
      uint32_t it = 0;
      bool ok = true;
      for (int w = blockIdx.x; ok && w < total; w += gridDim.x) {
        const Fp8Item wk = wide_item<C>(a, first, unit, w);
        const uint32_t idesc = idesc_f8(128, min(C::BN, a.F - wk.f0), false, C::BACK);  // F is a multiple of 16
        for (int kb = 0; kb < wk.kn; ++kb, ++it) {
          const int s = it % C::STAGES;
          const uint32_t b = it % C::NACC;
          if (!wait_warp(&acc_empty[b], ((it / C::NACC) & 1u) ^ 1u, budget, a.err, abort_flag) ||
              !wait_warp(&full[s], (it / C::STAGES) & 1u, budget, a.err, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t so = static_cast<uint64_t>(s) * (C::STAGE >> 4);
          const uint32_t d = tmem + b * C::BN;
#pragma unroll
          for (int i = 0; i < 4; ++i) mma_f8_el(d, adesc0 + so + i * 2, bdesc0 + so + i * kStepB, idesc, i > 0);
          tc_commit_el(&empty[s]);
          tc_commit_el(&acc_full[b]);
        }
      }
      tc_commit_el(done);
      mbar_wait_warp(done, 0, budget, a.err, nullptr);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::EPI_REGS));
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int grp = (warp - C::CTRL_WARPS) >> 2;
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    uint32_t it = 0;
    bool ok = true;
    for (int w = blockIdx.x; ok && w < total; w += gridDim.x) {
      const Fp8Item wk = wide_item<C>(a, first, unit, w);
      const int row = q * 32 + lane;
      const int nf = min(C::BN, a.F - wk.f0);
      // the group's chunk i holds features 32 (3 i + grp) ..
      const int nch = ((nf + 31) / 32 - grp + C::NG - 1) / C::NG;
      // scales of a block of the sum: this row's, and the tile's two blocks of
      // 128 features'; rows past the tile take its last one's
      const float* x_sf = a.b_sf + wk.c0 + min(row, wk.n - 1);
      const float* w_sf = a.a_sf + wk.e * a.a_se + static_cast<long long>(wk.f0 >> 7) * a.a_sm;
      const int second = nf > 128 ? a.a_sm : 0;
      float2 acc[C::NCH][16];
#pragma unroll
      for (int i = 0; i < C::NCH; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[i][j] = make_float2(0.f, 0.f);
      struct Scales {
        float x, w0, w1;
      };
      auto load = [&](int kb, Scales& s) {
        if (kb >= wk.kn) return;
        s.x = __ldg(x_sf);
        s.w0 = __ldg(w_sf);
        s.w1 = __ldg(w_sf + second);
        x_sf += a.ldb;
        w_sf += a.a_sk;
      };
      Scales s0{}, s1{};
      load(0, s0);
      load(1, s1);
      for (int kb = 0; kb < wk.kn; ++kb, ++it) {
        const uint32_t b = it % C::NACC;
        const float lo = s0.x * s0.w0, hi = s0.x * s0.w1;
        s0 = s1;
        load(kb + 2, s1);
        if (!wait_warp(&acc_full[b], (it / C::NACC) & 1u, budget, a.err, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t t = tmem + lanes + b * C::BN + grp * 32;
#pragma unroll
        for (int i = 0; i < C::NCH; ++i) {
          if (i < nch) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(t + i * C::NG * 32, r);
            tmem_ld_wait_for(r);
            if (i == nch - 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&acc_empty[b]);
            }
            const float f = i * C::NG + grp < 4 ? lo : hi;
            const float2 ff = make_float2(f, f);
#pragma unroll
            for (int j = 0; j < 16; ++j)
              acc[i][j] = __ffma2_rn(make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), ff,
                                     acc[i][j]);
          }
        }
        if (nch <= 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[b]);
        }
      }
      if (!ok) break;
      if (row < wk.n) {
#pragma unroll
        for (int i = 0; i < C::NCH; ++i) {
          if (i >= nch) continue;
          const int f = wk.f0 + (i * C::NG + grp) * 32;
          const long long at = static_cast<long long>(wk.c0 + row) * a.F + f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // eight features
            if (f + 8 * j >= a.F) continue;
            const float2* d = acc[i] + 4 * j;
            if (a.f32) {
              float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) + 2 * j;
              o[0] = make_float4(d[0].x, d[0].y, d[1].x, d[1].y);
              o[1] = make_float4(d[2].x, d[2].y, d[3].x, d[3].y);
            } else {
              uint32_t u[4];
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                const __nv_bfloat162 p = __floats2bfloat162_rn(d[v].x, d[v].y);
                u[v] = *reinterpret_cast<const uint32_t*>(&p);
              }
              reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at)[j] = make_uint4(u[0], u[1], u[2], u[3]);
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::NACC * C::BN);
  }
}

template <class C>
static cudaError_t launch_cfg(const Fp8Maps& maps, Fp8Args a, int sms, cudaStream_t st) {
  static bool set[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!set[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(fp8_gemm_wide_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  a.FT = (a.F + C::BN - 1) / C::BN;
  // no more CTAs than there can be items
  const long long items = (static_cast<long long>(a.M) / C::BM + (a.M < a.E ? a.M : a.E)) * a.FT;
  return launch_chained(fp8_gemm_wide_kernel<C>, dim3(static_cast<unsigned>(items < sms ? items : sms)),
                        dim3(C::THREADS), C::SMEM, st, true, maps, a);
}

cudaError_t launch_fp8_gemm_wide(bool back, const Fp8Maps& maps, const Fp8Args& a, int sms, cudaStream_t st) {
  return back ? launch_cfg<Fp8WideCfg<true>>(maps, a, sms, st) : launch_cfg<Fp8WideCfg<false>>(maps, a, sms, st);
}

}  // namespace kmoe
