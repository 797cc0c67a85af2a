// The weights' gradient of the block-scaled products, dense or by expert:
//
//   dw[e, n, k] = sum over e's blocks b of 128 rows:
//                   sy[b, n] sx[b, k] sum_{m in b} dy[m, n] x[m, k]
//
// Both scales are powers of two (kmoe_quantize_fp8_cols writes no others), so
// the tensor core applies them (tcgen05.mma kind::mxf8f6f4, one UE8M0 scale for
// 32 of the sum, the same four times) and eight blocks add up in one TMEM
// accumulator: no pass over the accumulator for each block.  The runs of eight
// are added in fp32 registers (see RUN).  A scale that is no power of two makes
// its row or column NaN.
//
// A cluster of two CTAs computes a tile of 256 features k (the MMA's M, 128 a
// CTA) x 224 features n with tcgen05.mma.cta_group::2: each CTA loads its
// features k and half of the features n, and holds the accumulator of its
// features k.  Both operands are read as they lie in memory, MN-major.  Two
// accumulators: a run's sums and stores overlap the next one's products.  An expert has
// few blocks (1024 rows are eight), so the fp32 stores weigh as much as the
// products.
//
// The scales of four blocks are one 32-bit word a feature; warps 2 and 3 gather
// them into the 32 x 16 byte order that tcgen05.cp copies into TMEM (each CTA its
// own features k and all n), and a block's MMAs select their byte.
//
// Roles in each CTA: warp 0 TMA, warp 1 MMA (the even CTA's, for both), warps 2
// and 3 the scales, warps 4 .. 11 the stores.  Loads complete on the even CTA's
// barriers, commits arrive at both CTAs'.  Every wait on an mbarrier is bounded; the
// cluster's barrier at the end is reached by every warp after its own waits.
//
// 16384 rows of 16 experts, 7168 x 3584: 460 us, 1830 TFLOP/s and 1.6 GB of
// stores; without the stores 360, without the loads 347, without both 283 (the
// products and the scales' copies).  One CTA a tile 569, the accumulators read
// and scaled for each block instead 1411.  One expert with all of them 312.
#include "fp8_dev.cuh"

namespace kmoe {

struct WgradCfg {
  static constexpr int BN = kWeightGradColumns;
  static constexpr int A_BYTES = 128 * 128, B_BYTES = 128 * 128;  // a block's 128 features k, and a box of n
  static constexpr int STAGE = A_BYTES + B_BYTES;                  // (two blocks a stage: 473 us where one takes 463)
  // blocks that the tensor core sums by itself: its additions truncate, which over
  // 32 blocks is off by 2e-7 of the sum and over 512 by 7e-6; in runs of eight,
  // added in fp32, by 7e-8 and 2e-7, in the same time
  static constexpr int RUN = 8;
  static constexpr int STAGES = 192 * 1024 / STAGE;
  static constexpr int CTRL_WARPS = 4, EPI_WARPS = 8;
  static constexpr int THREADS = 32 * (CTRL_WARPS + EPI_WARPS);
  static constexpr int CTRL_REGS = 120, EPI_REGS = 192;
  static constexpr int NACC = 2;
  static constexpr int SF_SLOTS = 4;        // of four blocks' scales in shared memory
  static constexpr int SF_BYTES = 3 * 512;  // 128 features k, 256 features n
  static constexpr int SF_COL = NACC * BN;  // in TMEM: two slots of 12 columns
  static constexpr int SF_OFF = STAGES * STAGE;
  static constexpr int BAR_OFF = SF_OFF + SF_SLOTS * SF_BYTES;
  static constexpr int TAB_OFF = BAR_OFF + 256;
  static constexpr int TAB_INTS = kMaxE + 1;
  static constexpr int SMEM = 1024 + TAB_OFF + (2 * TAB_INTS + 40) * 4;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(SF_COL + 24 <= 512, "TMEM columns");
  static_assert(32 * (CTRL_WARPS * CTRL_REGS + EPI_WARPS * EPI_REGS) <= THREADS * 168, "register split");
  static_assert(RUN % 4 == 0, "a group of four blocks' scales stays within a run");
  static_assert((2 * STAGES + 2 * NACC + 2 * SF_SLOTS + 1) * 8 + 8 <= 256, "barriers");
};

__device__ __forceinline__ Fp8Item wgrad_item(const Fp8Args& a, const int32_t* unit, int w) {
  Fp8Item it;
  const int per = a.FT * a.CT;
  it.e = w / per;
  const int r = w - it.e * per;
  it.f0 = r % a.FT * 256;
  it.c0 = r / a.FT * WgradCfg::BN;
  it.n = min(WgradCfg::BN, a.C - it.c0);
  it.kb = min(unit[it.e], a.KB);
  it.kn = min(unit[it.e + 1], a.KB) - it.kb;
  return it;
}

// Columns that each CTA of a pair loads and multiplies for a tile of n.
__device__ __forceinline__ int wgrad_half(int n) { return (n + 31) / 32 * 16; }

// The UE8M0 byte of a scale: its exponent, NaN for anything but a normal power of two.
__device__ __forceinline__ uint32_t ue8m0_of(float s) {
  const uint32_t u = __float_as_uint(s), e = u >> 23;
  return (u & 0x807FFFFFu) != 0u || e == 0u ? 0xFFu : e;
}

__global__ void __launch_bounds__(WgradCfg::THREADS, 1) fp8_wgrad_kernel(const __grid_constant__ Fp8Maps maps,
                                                                        const Fp8Args a) {
  using C = WgradCfg;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* acc_empty = acc_full + C::NACC;
  uint64_t* sf_full = acc_empty + C::NACC;
  uint64_t* sf_empty = sf_full + C::SF_SLOTS;
  uint64_t* done = sf_empty + C::SF_SLOTS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* first = reinterpret_cast<int32_t*>(smem + C::TAB_OFF);
  int32_t* unit = first + C::TAB_INTS;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool lead = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::NACC; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * C::EPI_WARPS);  // of both CTAs
    }
    for (int s = 0; s < C::SF_SLOTS; ++s) {
      mbar_init(&sf_full[s], 2);  // both CTAs' scales
      mbar_init(&sf_empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.b);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  chain_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;  // long before any wait can give up
  tc_fence_before();
  segment_prefix(a.seg, a.E, a.M, kScaleBlock, first, unit, unit + C::TAB_INTS);
  cluster_sync();  // both CTAs' barriers and TMEM are there
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = a.E * a.FT * a.CT;
  const int w0 = blockIdx.x >> 1, dw = gridDim.x >> 1;
  const uint64_t budget = a.budget_ns;

  if (warp < C::CTRL_WARPS) {
    // (of the registers that the block was launched with)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::CTRL_REGS));
    if (warp == 0) {
      // -------------------------------------------------------------- loads
      const uint64_t pol = policy_evict_last();
      const uint32_t lead_full = cluster_map(full, 0);
      uint32_t it = 0;
      bool ok = true;
      for (int w = w0; ok && w < total; w += dw) {
        const Fp8Item wk = wgrad_item(a, unit, w);
        // this CTA's half of the MMA's columns starts on a multiple of 16 bytes
        const int c0 = wk.c0 + rank * wgrad_half(wk.n), f0 = wk.f0 + rank * 128;
        for (int kb = 0; kb < wk.kn; ++kb, ++it) {
          const int s = it % C::STAGES;
          if (!wait_warp(&empty[s], ((it / C::STAGES) & 1u) ^ 1u, budget, a.err, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + s * C::STAGE;
          const int k0 = (wk.kb + kb) * kScaleBlock;
          if (lead) mbar_arrive_expect_tx_el(&full[s], 2u * C::STAGE);
          tma_load_2d_pair_el(st, &maps.a, lead_full + 8u * s, f0, k0, pol);
          tma_load_2d_pair_el(st + C::A_BYTES, &maps.b, lead_full + 8u * s, c0, k0, pol);
        }
      }
      if (!ok) {
        // let the copies already issued land before the CTA can exit
        if (lead) {
          const uint32_t from = it > static_cast<uint32_t>(C::STAGES) ? it - C::STAGES : 0u;
          for (uint32_t i = from; i < it; ++i)
            mbar_wait_warp(&full[i % C::STAGES], (i / C::STAGES) & 1u, 20000000ull, nullptr, nullptr);
        } else {
          spin_ns(100000ull);
        }
      }
    } else if (warp == 1) {
      // -------------------------------------------------------------- MMA
      if (lead) {
        // 32 of the sum are 32 rows of 128 bytes of an MN-major operand (8-row
        // groups 1024 bytes apart).
        const uint64_t adesc0 = make_sdesc(smem_u32(smem), 16384, 1024, 2);
        const uint64_t bdesc0 = make_sdesc(smem_u32(smem + C::A_BYTES), 16384, 1024, 2);
        const uint64_t sfdesc0 = sdesc_sf_32x16(smem_u32(smem + C::SF_OFF));
        uint32_t it = 0, li = 0, grp = 0;  // stages, runs, groups of four blocks
        bool ok = true;
        for (int w = w0; ok && w < total; w += dw) {
          const Fp8Item wk = wgrad_item(a, unit, w);
          if (wk.kn <= 0) continue;
          uint32_t b = 0;
          const int nmma = 2 * wgrad_half(wk.n);
          const uint32_t idesc = idesc_mxf8f6f4(256, nmma, MX_E4M3, MX_E4M3, 0, 0) | (1u << 15) | (1u << 16);
          for (int kb = 0; kb < wk.kn; ++kb, ++it) {
            if (kb % C::RUN == 0) {
              b = li % C::NACC;
              ok = mbar_wait_warp<true>(&acc_empty[b], ((li / C::NACC) & 1u) ^ 1u, budget, a.err, abort_flag);
              if (!ok) break;
              ++li;
            }
            const uint32_t d = tmem + b * C::BN;
            const int s = it % C::STAGES;
            if (!wait_warp(&full[s], (it / C::STAGES) & 1u, budget, a.err, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sf = tmem + C::SF_COL + (grp & 1u) * 12;
            if ((kb & 3) == 0) {
              const uint32_t sl = grp % C::SF_SLOTS;
              ok = mbar_wait_warp<true>(&sf_full[sl], (grp / C::SF_SLOTS) & 1u, budget, a.err, abort_flag);
              if (!ok) break;
              tc_fence_after();
              const uint64_t sd = sfdesc0 + sl * (C::SF_BYTES >> 4);
              tc_cp_32x128b_warpx4_pair_el(sf, sd);
              tc_cp_32x128b_warpx4_pair_el(sf + 4, sd + 32);
              if (nmma > 128) tc_cp_32x128b_warpx4_pair_el(sf + 8, sd + 64);
              tc_commit_pair_el(&sf_empty[sl]);
            }
            const uint64_t so = static_cast<uint64_t>(s) * (C::STAGE >> 4);
            const uint32_t id = idesc | (static_cast<uint32_t>(kb & 3) << 4) | (static_cast<uint32_t>(kb & 3) << 29);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_mxf8f6f4_pair_el(d, adesc0 + so + j * 256, bdesc0 + so + j * 256, id, sf, sf + 4,
                                   kb % C::RUN != 0 || j != 0);
            const bool last = kb == wk.kn - 1;
            if ((kb & 3) == 3 || last) ++grp;
            tc_commit_pair_el(&empty[s]);
            if (kb % C::RUN == C::RUN - 1 || last) tc_commit_pair_el(&acc_full[b]);
          }
        }
        tc_commit_pair_el(done);
        mbar_wait_warp(done, 0, budget, a.err, nullptr);
      }
    } else {
      // -------------------------------------------------------------- scales
      // (groups of four blocks by the two warps in turn)
      const uint32_t lead_sf_full = cluster_map(sf_full, 0);
      uint32_t grp = 0;
      bool ok = true;
      for (int w = w0; ok && w < total; w += dw) {
        const Fp8Item wk = wgrad_item(a, unit, w);
        for (int kb = 0; kb < wk.kn; kb += 4, ++grp) {
          if ((grp & 1u) != (warp & 1u)) continue;
          // features 32 j + lane: four of k, then eight of n; past an edge the last
          // one's (no product that is stored uses those), all loads in flight at once
          const int last = min(4, wk.kn - kb) - 1;
          const long long b0 = wk.kb + kb;
          float v[12][4];
#pragma unroll
          for (int j = 0; j < 12; ++j) {
            const int at = j < 4 ? min(wk.f0 + rank * 128 + 32 * j + lane, a.F - 1)
                                 : wk.c0 + min(32 * (j - 4) + lane, wk.n - 1);
            const float* src = j < 4 ? a.a_sf : a.b_sf;
            const int cols = j < 4 ? a.F : a.C;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j][i] = __ldg(src + (b0 + min(i, last)) * cols + at);
          }
          const uint32_t sl = grp % C::SF_SLOTS;
          if (!wait_warp(&sf_empty[sl], ((grp / C::SF_SLOTS) & 1u) ^ 1u, budget, a.err, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* dst = smem + C::SF_OFF + sl * C::SF_BYTES + lane * 16;
#pragma unroll
          for (int j = 0; j < 12; ++j)
            *reinterpret_cast<uint32_t*>(dst + (j >> 2) * 512 + (j & 3) * 4) =
                ue8m0_of(v[j][0]) | ue8m0_of(v[j][1]) << 8 | ue8m0_of(v[j][2]) << 16 | ue8m0_of(v[j][3]) << 24;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (lead)
              mbar_arrive(&sf_full[sl]);
            else
              mbar_arrive_remote(lead_sf_full + 8u * sl);
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::EPI_REGS));
    // -------------------------------------------------------------- stores
    const int q = warp & 3;
    const int half = (warp - C::CTRL_WARPS) >> 2;  // of the tile's 16-column chunks, in turn
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t lead_acc_empty = cluster_map(acc_empty, 0);
    uint32_t li = 0;
    for (int w = w0; w < total; w += dw) {
      const Fp8Item wk = wgrad_item(a, unit, w);
      const int f = wk.f0 + rank * 128 + q * 32 + lane;
      float* out = static_cast<float*>(a.out) + (static_cast<long long>(wk.e) * a.C + wk.c0) * a.F + f;
      if (wk.kn <= 0) {  // no rows: zeros
        if (f < a.F)
          for (int c = half; c < wk.n; c += 2) __stcs(out + static_cast<long long>(c) * a.F, 0.f);
        continue;
      }
      float sum[C::BN / 32][16];
      bool ok = true;
      for (int kb = 0; kb < wk.kn; kb += C::RUN, ++li) {
        const uint32_t b = li % C::NACC;
        ok = wait_warp(&acc_full[b], (li / C::NACC) & 1u, budget, a.err, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t t = tmem + lanes + b * C::BN;
        const bool begin = kb == 0, end = kb + C::RUN >= wk.kn;
#pragma unroll
        for (int i = 0; i < C::BN / 32; ++i) {
          const int c = 32 * i + 16 * half;
          if (c >= wk.n) break;  // (n is a multiple of 16)
          uint32_t r[16];
          tmem_ld_32x32b_x16(t + c, r);
          tmem_ld_wait_for(r);
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[i][j] = (begin ? 0.f : sum[i][j]) + __uint_as_float(r[j]);
          if (end && f < a.F) {  // 32 features of one n a store
#pragma unroll
            for (int j = 0; j < 16; ++j) __stcs(out + static_cast<long long>(c + j) * a.F, sum[i][j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (lead)
            mbar_arrive(&acc_empty[b]);
          else
            mbar_arrive_remote(lead_acc_empty + 8u * b);
        }
      }
      if (!ok) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no MMA of the pair and no remote arrive is outstanding past here
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

cudaError_t launch_fp8_wgrad(const Fp8Maps& maps, Fp8Args a, int sms, cudaStream_t st) {
  static int pairs_of[kMaxDevices] = {};  // co-resident clusters of two, per device
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see chain_wait
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(2 * (sms / 2));
  cfg.blockDim = dim3(WgradCfg::THREADS);
  cfg.dynamicSmemBytes = WgradCfg::SMEM;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int& pairs = pairs_of[dev];
  if (pairs == 0) {
    cudaError_t e =
        cudaFuncSetAttribute(fp8_wgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, WgradCfg::SMEM);
    if (e != cudaSuccess) return e;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, fp8_wgrad_kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (n <= 0) return cudaErrorInvalidConfiguration;
    pairs = n < sms / 2 ? n : sms / 2;
  }
  a.FT = (a.F + 255) / 256;
  const long long items = static_cast<long long>(a.E) * a.FT * a.CT;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (items < pairs ? items : pairs)));
  cfg.stream = st;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, fp8_wgrad_kernel, maps, a);
}

}  // namespace kmoe
