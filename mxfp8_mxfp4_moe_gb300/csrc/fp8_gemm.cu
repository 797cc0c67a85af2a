// Products of E4M3 operands with a scale for each block of 128 values of the
// sum: rows times weights and rows times transposed weights (the rows'
// gradient), dense or by expert.  This kernel takes the batches with few rows
// for each expert, fp8_gemm_wide.cu those with many; fp8_wgrad.cu has the
// weights' gradient.
//
//   out[r, f] = sum over blocks b of 128:  sx[b, r] sw(f, b) sum_{i in b} x[r, i] w[f, i]
//
// A block's inner sum is four tcgen05.mma (kind::f8f6f4, K = 32) into a fresh
// TMEM accumulator; the epilogue warps read it while the next block's runs in
// another accumulator, multiply by the product of the two scales and add in fp32
// registers.  That product may leave fp32's normal range, which the header says;
// finding such blocks in the epilogue and giving them their scales one after the
// other was measured at 2 to 28 % of fp8_gemm_wide.cu's time for every call (each
// read of shared memory, vote or register more lengthens the accumulators'
// hand-over) and 1 to 4 % here.
// The features f are the MMA's M, the rows its N (16 .. BN), so that a few
// rows cost few columns.  Operands that are contiguous along the sum are
// K-major; transposed weights are read as they lie in memory, MN-major
// (128-byte swizzle either way).
//
// Roles: warp 0 TMA, warp 1 MMA (both converged, one elected lane issues), warp
// 2 the scales (a ring in shared memory, some blocks ahead of their use: with
// few rows a block takes less time than a read of global memory), warps 3 .. 6
// the epilogue, one per TMEM lane quarter.  Every wait on an mbarrier is bounded;
// the cluster's barriers, which are not, are reached by every warp after its own.
//
// Where there are too few items for the SMs, a cluster of `split` CTAs takes
// one item: each sums a part of the blocks, and the parts are added in order
// through distributed shared memory, each CTA a share of the accumulators.
//
// Bound by HBM's reads of the weights where they are many (2048 rows of 64
// experts, 7168 x 3584: 256-264 us, 6.2-6.4 TB/s), by the chain of launch,
// first load, blocks and exchange where they are one matrix: one row 7168 x
// 7168 13.3 us with the 51 MB of weights from HBM (3.9 TB/s; eight matrices in
// turn), 10.7 with one matrix again and again, part of which stays in L2; 16 rows
// 2048 x 7168 7.4 us.  Transposed the same (13.2; 2048 rows of 64 experts 260-271).
#include <type_traits>

#include "fp8_dev.cuh"

namespace kmoe {

// 16 lanes x 32 columns: this thread reads, of each 8 columns g, columns 2q
// and 2q + 1 (q = lane % 4) of lane lane / 4 (r[4g], r[4g + 1]) and of the lane
// eight below (r[4g + 2], r[4g + 3]).
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// 8x8 matrices of 16-bit values, a row a quad of lanes, transposed.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <bool BACK_>
struct Fp8Cfg {
  static constexpr bool BACK = BACK_;  // the weights transposed, read MN-major
  static constexpr int BN = 32;        // rows of a tile
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int BOX = kFp8BoxRows;
  static constexpr int STAGE = A_BYTES + BN * 128;
  // two CTAs on an SM, so that one can start while another ends
  static constexpr int CTAS_PER_SM = 2;
  static constexpr int STAGES = 100 * 1024 / STAGE;
  static constexpr int EPI_WARPS = 4;
  static constexpr int CTRL_WARPS = 3;
  static constexpr int THREADS = 32 * (CTRL_WARPS + EPI_WARPS);
  static constexpr int NACC = 4;
  static constexpr int TMEM_COLS = NACC * BN;
  // ring of scales: a block's BN rows and its features'
  static constexpr int RING = 16, AHEAD = RING - NACC - 1;  // slots, and blocks loaded ahead
  static constexpr int SLOT = BN + 4;                       // floats
  static constexpr int SC_OFF = STAGES * STAGE;
  static constexpr int BAR_OFF = SC_OFF + RING * SLOT * 4;
  static constexpr int TAB_OFF = BAR_OFF + 256;
  static constexpr int TAB_INTS = kMaxE + 1;
  static constexpr int SMEM = 1024 + TAB_OFF + (2 * TAB_INTS + 40) * 4;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert((2 * STAGES + 2 * NACC + 1) * 8 + 8 <= 256, "barriers");
  static_assert(EPI_WARPS * 32 * BN * 4 <= STAGES * STAGE, "a cluster's parts go where the stages were");
};

template <class C>
__device__ __forceinline__ Fp8Item fp8_item(const Fp8Args& a, const int32_t* first, const int32_t* unit, int w,
                                            int rank) {
  Fp8Item it;
  it.e = segment_of_unit(unit, a.E, w / a.FT);
  const int u0 = unit[it.e], nt = unit[it.e + 1] - u0;
  const int r = w - u0 * a.FT;
  it.f0 = r / nt * 128;
  // an expert's rows in tiles of nearly the same size
  const int rows = first[it.e + 1] - first[it.e];
  const int per = ((rows + nt - 1) / nt + 15) / 16 * 16;
  const int at = r % nt * per;
  it.c0 = first[it.e] + at;
  it.n = min(per, rows - at);
  const int per_cta = (a.KB + a.split - 1) / a.split;
  it.kb = min(rank * per_cta, a.KB);
  it.kn = min(per_cta, a.KB - it.kb);
  return it;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::CTAS_PER_SM) fp8_gemm_kernel(const __grid_constant__ Fp8Maps maps,
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
  const int rank = static_cast<int>(cluster_ctarank());  // 0 without a cluster
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::NACC; ++b) {
      mbar_init(&acc_full[b], 2);  // the block's products, and its scales
      mbar_init(&acc_empty[b], C::EPI_WARPS);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.b);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  chain_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;  // long before any wait can give up
  tc_fence_before();
  segment_prefix(a.seg, a.E, a.M, C::BN, first, unit, unit + C::TAB_INTS);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint64_t budget = a.budget_ns;
  const int w0 = blockIdx.x / a.split, dw = gridDim.x / a.split;
  const int total = product_items(a.FT, unit[a.E], a.items);

  if (warp < C::CTRL_WARPS) {
    if (warp == 0) {
      // ------------------------------------------------------------ loads
      const uint64_t pol_a = policy_evict_normal(), pol_b = policy_evict_last();
      uint32_t it = 0;
      bool ok = true;
      for (int w = w0; ok && w < total; w += dw) {
        const Fp8Item wk = fp8_item<C>(a, first, unit, w, rank);
        const int boxes = (wk.n + C::BOX - 1) / C::BOX;
        const uint32_t tx = C::A_BYTES + boxes * C::BOX * 128;
        for (int kb = 0; kb < wk.kn; ++kb, ++it) {
          const int s = it % C::STAGES;
          if (!wait_warp(&empty[s], ((it / C::STAGES) & 1u) ^ 1u, budget, a.err, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + s * C::STAGE;
          uint8_t* sb = sa + C::A_BYTES;
          const int k0 = (wk.kb + kb) * kScaleBlock;
          mbar_arrive_expect_tx_el(&full[s], tx);
          tma_load_3d_el(sa, &maps.a, &full[s], C::BACK ? wk.f0 : k0, C::BACK ? k0 : wk.f0, wk.e, pol_a);
          for (int i = 0; i < boxes; ++i)
            tma_load_2d_el(sb + i * C::BOX * 128, &maps.b, &full[s], k0, wk.c0 + i * C::BOX, pol_b);
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
      // Steps of 32 along the sum: 32 bytes inside a K-major swizzle atom, 32
      // rows of 128 bytes of an MN-major one (8-row groups 1024 bytes apart).
      constexpr uint32_t kStepA = C::BACK ? 256 : 2;
      const uint64_t adesc0 =
          C::BACK ? make_sdesc(smem_u32(smem), 16384, 1024, 2) : sdesc_kmajor_sw128(smem_u32(smem));
      const uint64_t bdesc0 = sdesc_kmajor_sw128(smem_u32(smem + C::A_BYTES));
      uint32_t it = 0;
      bool ok = true;
      for (int w = w0; ok && w < total; w += dw) {
        const Fp8Item wk = fp8_item<C>(a, first, unit, w, rank);
        const uint32_t idesc = idesc_f8(128, (wk.n + 15) & ~15, C::BACK, false);
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
          for (int i = 0; i < 4; ++i)
            mma_f8_el(d, adesc0 + so + i * kStepA, bdesc0 + so + i * 2, idesc, i > 0);
          tc_commit_el(&empty[s]);
          tc_commit_el(&acc_full[b]);
        }
      }
      tc_commit_el(done);
      mbar_wait_warp(done, 0, budget, a.err, nullptr);
    }
    else {
      // ------------------------------------------------------------ scales
      // The rows' lie in the order in which the eight that a thread needs are two
      // 16-byte pieces: rows 8g + 2q + {0, 1}, g even and the g after it.
      const uint32_t ring = smem_u32(smem + C::SC_OFF) +
                            ((lane >> 4) * 16 + ((lane & 7) >> 1) * 4 + ((lane >> 3) & 1) * 2 + (lane & 1)) * 4;
      const uint32_t ring_w = smem_u32(smem + C::SC_OFF) + C::BN * 4;
      int w = w0 - dw, kb = 0, kn = 0, n = 0;  // the block that is loaded next
      const float *x_sf = nullptr, *w_sf = nullptr;
      bool more = true;
      uint32_t issued = 0;
      auto issue = [&] {
        while (more && kb >= kn) {  // the next item
          w += dw;
          more = w < total;
          if (more) {
            const Fp8Item wk = fp8_item<C>(a, first, unit, w, rank);
            kb = 0;
            kn = wk.kn;
            n = wk.n;
            x_sf = a.b_sf + static_cast<long long>(wk.kb) * a.ldb + wk.c0;
            w_sf = a.a_sf + wk.e * a.a_se + static_cast<long long>(wk.f0 >> 7) * a.a_sm + wk.kb * a.a_sk;
          }
        }
        if (more) {
          const uint32_t slot = (issued & (C::RING - 1)) * (C::SLOT * 4);
          cp_async4(ring + slot, x_sf + min(lane, n - 1));
          if (lane == 0) cp_async4(ring_w + slot, w_sf);
          x_sf += a.ldb;
          w_sf += a.a_sk;
          ++kb;
          ++issued;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
#pragma unroll 1
      for (int i = 0; i < C::AHEAD; ++i) issue();
#pragma unroll 1
      for (uint32_t it = 0;; ++it) {
        const uint32_t b = it % C::NACC;
        if (it < issued && !wait_warp(&acc_empty[b], ((it / C::NACC) & 1u) ^ 1u, budget, a.err, abort_flag)) break;
        issue();  // the slot's last block was read before the accumulator above was released
        if (it >= issued) break;
        asm volatile("cp.async.wait_group %0;" ::"n"(C::AHEAD) : "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_full[b]);
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    if (a.split > 1) {  // (the epilogue's exchange)
      cluster_sync();
      cluster_sync();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int ew = warp - C::CTRL_WARPS;
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    uint32_t it = 0;
    bool ok = true, exchanged = false;
    for (int w = w0; ok && w < total; w += dw) {
      const Fp8Item wk = fp8_item<C>(a, first, unit, w, rank);
      const int f0 = wk.f0 + q * 32;  // the warp's first feature
      float2 acc[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] = make_float2(0.f, 0.f);
      for (int kb = 0; kb < wk.kn; ++kb, ++it) {
        const uint32_t b = it % C::NACC;
        if (!wait_warp(&acc_full[b], (it / C::NACC) & 1u, budget, a.err, abort_flag)) {
          ok = false;
          break;
        }
        __syncwarp();
        tc_fence_after();
        const uint32_t t = tmem + lanes + b * C::BN;
        uint32_t r[32];
        tmem_ld_16x256b_x4(t, r);
        tmem_ld_16x256b_x4(t + (16u << 16), r + 16);
        const float* const scale = reinterpret_cast<const float*>(smem + C::SC_OFF) + (it & (C::RING - 1)) * C::SLOT;
        const float sw = scale[C::BN];
        float2 s[4];  // of rows 8 g + 2 q + {0, 1}
#pragma unroll
        for (int g = 0; g < 4; g += 2) {
          const float4 v = *reinterpret_cast<const float4*>(scale + 8 * g + (lane & 3) * 4);
          s[g] = make_float2(v.x * sw, v.y * sw);
          s[g + 1] = make_float2(v.z * sw, v.w * sw);
        }
        tmem_ld_wait_for(r);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[b]);
#pragma unroll
        for (int h = 0; h < 4; ++h)  // features lane / 4 + 8 h
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const uint32_t* v = r + (h >> 1) * 16 + 4 * g + (h & 1) * 2;
            acc[4 * h + g] =
                __ffma2_rn(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), s[g], acc[4 * h + g]);
          }
      }
      if (!ok) break;
      // accumulator j: rows c, c + 1 of features f0 + 8 h + lane / 4
      auto store = [&](int j, float2 d) {
        const int c = 8 * (j & 3), h = j >> 2;
        if (c >= wk.n) return;
        if (a.f32) {
          const int f = f0 + 8 * h + (lane >> 2), cc = c + 2 * (lane & 3);
          float* o = static_cast<float*>(a.out) + static_cast<long long>(wk.c0 + cc) * a.F + f;
          if (f < a.F && cc < wk.n) o[0] = d.x;
          if (f < a.F && cc + 1 < wk.n) o[a.F] = d.y;
        } else {
          // two features of one row a lane
          const __nv_bfloat162 p = __floats2bfloat162_rn(d.x, d.y);
          const uint32_t u = transpose_8x8(*reinterpret_cast<const uint32_t*>(&p));
          const int f = f0 + 8 * h + 2 * (lane & 3), cc = c + (lane >> 2);
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + static_cast<long long>(wk.c0 + cc) * a.F + f;
          if (f < a.F && cc < wk.n) *reinterpret_cast<uint32_t*>(o) = u;
        }
      };
      // the parts of S CTAs: each adds up every S-th accumulator, all its reads in flight at once
      auto exchange = [&](auto clusters) {
        constexpr int S = decltype(clusters)::value, NJ = 16 / S;
        // every load of this CTA has been used: its stages are free
        constexpr int kStride = C::EPI_WARPS * 32;
        float2* const part = reinterpret_cast<float2*>(smem) + ew * 32 + lane;
#pragma unroll
        for (int j = 0; j < 16; ++j) part[j * kStride] = acc[j];
        cluster_sync();
        exchanged = true;
        float2 v[NJ][S];
#pragma unroll
        for (int i = 0; i < NJ; ++i)
#pragma unroll
          for (int r = 0; r < S; ++r) v[i][r] = ld_shared_cluster_f2(cluster_map(part + (i * S + rank) * kStride, r));
#pragma unroll
        for (int i = 0; i < NJ; ++i) {
#pragma unroll
          for (int r = 1; r < S; ++r) {
            v[i][0].x += v[i][r].x;
            v[i][0].y += v[i][r].y;
          }
          store(i * S + rank, v[i][0]);
        }
      };
      switch (a.split) {
        case 1:
#pragma unroll
          for (int j = 0; j < 16; ++j) store(j, acc[j]);
          break;
        case 2: exchange(std::integral_constant<int, 2>{}); break;
        case 4: exchange(std::integral_constant<int, 4>{}); break;
        default: exchange(std::integral_constant<int, 8>{}); break;
      }
    }
    if (a.split > 1) {
      if (!exchanged) cluster_sync();
      cluster_sync();  // the other CTAs have read this one's part
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <class C>
static cudaError_t launch_cfg(const Fp8Maps& maps, Fp8Args a, int sms, cudaStream_t st) {
  static bool set[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!set[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(fp8_gemm_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  a.items = static_cast<int>(fp8_most_tiles(a.M, a.E, C::BN) * a.FT);
  a.split = product_split(a.items, C::CTAS_PER_SM * sms, a.KB, 4);
  return launch_product(fp8_gemm_kernel<C>, C::THREADS, C::SMEM, C::CTAS_PER_SM * sms, maps, a, st);
}

cudaError_t launch_fp8_gemm(bool back, const Fp8Maps& maps, const Fp8Args& a, int sms, cudaStream_t st) {
  return back ? launch_cfg<Fp8Cfg<true>>(maps, a, sms, st) : launch_cfg<Fp8Cfg<false>>(maps, a, sms, st);
}

}  // namespace kmoe
