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
// Where there are too few items for the SMs, a cluster of `split` CTAs takes
// one item, as in fp8_gemm.cu.
//
// Roles: warp 0 TMA, warp 1 MMA (both converged, one elected lane issues),
// warp 2 the scales (a ring in shared memory, some blocks ahead of their use),
// warps 4 .. 11 the epilogue: two groups of four (one warp per TMEM lane
// quarter), each with 128 features of the tile.  Every wait on an mbarrier is
// bounded; the clusters' barriers are reached by every warp after its own waits.
//
// A block of the sum takes 584 cycles of the tensor core, at least 520 of the
// epilogue (TMEM reads and multiply-adds of 128 x 256 values) and 880 of its
// 48 KB through TMA; with the two accumulators' handshake it comes to about
// 1030.  8192 rows, 7168 x 7168: 336 us, 2500 TFLOP/s (1.30 of the bf16 peak,
// 0.65 of twice it); 64 experts with 512 rows each 1394 us; 896 experts with 146
// rows each on average, 2048 x 2048, 1100-1140 (bytes: 683), whose second tiles are
// mostly empty.  Measured at 8192 rows: the rows in the MMA's N 708-1048, CTA pairs
// 1038 (a pair's accumulators handed over without any loads 775, one CTA's 304), 12
// or 16 epilogue warps 354-432, accumulators in halves 429.
#include <type_traits>

#include "fp8_dev.cuh"

namespace kmoe {

template <bool BACK_, bool SPLIT_>
struct Fp8WideCfg {
  static constexpr bool BACK = BACK_;    // the weights transposed, read MN-major
  static constexpr bool SPLIT = SPLIT_;  // a cluster shares an item (its exchange costs the others registers)
  static constexpr int BM = 128, BN = 256;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = 4;
  // a group's four warps hold 128 features of the tile, 16 of which they read
  // while the 16 before are added
  static constexpr int NG = 2, NCH = 8;
  static constexpr int EPI_WARPS = 4 * NG;
  static constexpr int CTRL_WARPS = 4;
  static constexpr int THREADS = 32 * (CTRL_WARPS + EPI_WARPS);
  static constexpr int CTRL_REGS = 104, EPI_REGS = 200;
  static constexpr int NACC = 2;
  // ring of scales: a block's 128 rows and its tile's two blocks of features
  static constexpr int RING = 8, AHEAD = 4;  // slots, and blocks loaded ahead
  static constexpr int SLOT = 128 + 4;       // floats
  static constexpr int SC_OFF = STAGES * STAGE;
  // rows on their way out: 32 of 64 bytes a warp
  static constexpr int OUT_OFF = SC_OFF + (RING * SLOT * 4 + 15) / 16 * 16;
  static constexpr int BAR_OFF = OUT_OFF + EPI_WARPS * 2048;
  static constexpr int TAB_OFF = BAR_OFF + 256;
  static constexpr int TAB_INTS = kMaxE + 1;
  static constexpr int SMEM = 1024 + TAB_OFF + (2 * TAB_INTS + 40) * 4;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(RING >= AHEAD + NACC + 1, "a slot is written again when its block has been read");
  static_assert(EPI_WARPS * 32 * NCH * 8 * 8 <= STAGES * STAGE, "a cluster's parts go where the stages were");
  static_assert(128 * CTRL_REGS + 32 * EPI_WARPS * EPI_REGS <= THREADS * 168, "register split");
};

template <class C>
__device__ __forceinline__ Fp8Item wide_item(const Fp8Args& a, const int32_t* first, const int32_t* unit, int w,
                                             int rank) {
  Fp8Item it;
  it.e = segment_of_unit(unit, a.E, w / a.FT);
  const int u0 = unit[it.e], nt = unit[it.e + 1] - u0;
  const int r = w - u0 * a.FT;
  it.f0 = r / nt * C::BN;
  const int at = r % nt * C::BM;
  it.c0 = first[it.e] + at;
  it.n = min(C::BM, first[it.e + 1] - it.c0);
  if constexpr (C::SPLIT) {
    const int per_cta = (a.KB + a.split - 1) / a.split;
    it.kb = min(rank * per_cta, a.KB);
    it.kn = min(per_cta, a.KB - it.kb);
  } else {
    it.kb = 0;
    it.kn = a.KB;
  }
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
  const int rank = C::SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
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
    tmem_alloc(tmem_slot, C::NACC * C::BN);
    tmem_relinquish();
  }
  chain_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;  // long before any wait can give up
  tc_fence_before();
  segment_prefix(a.seg, a.E, a.M, C::BM, first, unit, unit + C::TAB_INTS);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint64_t budget = a.budget_ns;
  const int ctas = C::SPLIT ? a.split : 1;
  const int w0 = blockIdx.x / ctas, dw = gridDim.x / ctas;
  const int total = product_items(a.FT, unit[a.E], a.items);

  if (warp < C::CTRL_WARPS) {
    // (of the registers that the block was launched with)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::CTRL_REGS));
    if (warp == 0) {
      // ------------------------------------------------------------ loads
      const uint64_t pol_w = policy_evict_normal(), pol_x = policy_evict_last();
      uint32_t it = 0;
      bool ok = true;
      for (int w = w0; ok && w < total; w += dw) {
        const Fp8Item wk = wide_item<C>(a, first, unit, w, rank);
        const int boxes = a.F - wk.f0 > 128 ? 2 : 1;  // of 128 features
        const uint32_t tx = C::A_BYTES + boxes * 16384;
        for (int kb = 0; kb < wk.kn; ++kb, ++it) {
          const int s = it % C::STAGES;
          if (!wait_warp(&empty[s], ((it / C::STAGES) & 1u) ^ 1u, budget, a.err, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + s * C::STAGE;
          const int k0 = (wk.kb + kb) * kScaleBlock;
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
      for (int w = w0; ok && w < total; w += dw) {
        const Fp8Item wk = wide_item<C>(a, first, unit, w, rank);
        const uint32_t idesc = idesc_f8(128, min(C::BN, a.F - wk.f0), false, C::BACK);  // F is a multiple of 16
        for (int kb = 0; kb < wk.kn; ++kb, ++it) {
          const int s = it % C::STAGES;
          const uint32_t b = it % C::NACC;
          if (!wait_warp(&full[s], (it / C::STAGES) & 1u, budget, a.err, abort_flag) ||
              !wait_warp(&acc_empty[b], ((it / C::NACC) & 1u) ^ 1u, budget, a.err, abort_flag)) {
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
    } else if (warp == 2) {
      // ------------------------------------------------------------ scales
      const uint32_t ring = smem_u32(smem + C::SC_OFF);
      // the block that is loaded next: the issued-th of this CTA's
      int w = w0 - dw, kb = 0, kn = 0;
      const float *x_sf = nullptr, *w_sf = nullptr;
      bool more = true;
      uint32_t issued = 0;
      int n = 0, second = 0;
      auto issue = [&] {
        while (more && kb >= kn) {  // the next item
          w += dw;
          more = w < total;
          if (more) {
            const Fp8Item wk = wide_item<C>(a, first, unit, w, rank);
            kb = 0;
            kn = wk.kn;
            n = wk.n;
            x_sf = a.b_sf + static_cast<long long>(wk.kb) * a.ldb + wk.c0;
            w_sf = a.a_sf + wk.e * a.a_se + static_cast<long long>(wk.f0 >> 7) * a.a_sm + wk.kb * a.a_sk;
            second = a.F - wk.f0 > 128 ? a.a_sm : 0;
          }
        }
        if (more) {
          const uint32_t at = ring + (issued & (C::RING - 1)) * (C::SLOT * 4);
#pragma unroll
          for (int j = 0; j < 4; ++j) cp_async4(at + (32 * j + lane) * 4, x_sf + min(32 * j + lane, n - 1));
          if (lane < 2) cp_async4(at + (128 + lane) * 4, w_sf + lane * second);
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
    if constexpr (C::SPLIT) {  // (the epilogue's exchange)
      cluster_sync();
      cluster_sync();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::EPI_REGS));
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int grp = (warp - C::CTRL_WARPS) >> 2;
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    uint8_t* const out_smem = smem + C::OUT_OFF + (warp - C::CTRL_WARPS) * 2048;
    auto release = [&](uint32_t b) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[b]);
    };
    uint32_t it = 0;
    bool ok = true, exchanged = false;
    for (int w = w0; ok && w < total; w += dw) {
      const Fp8Item wk = wide_item<C>(a, first, unit, w, rank);
      const int row = q * 32 + lane;
      const int g0 = wk.f0 + grp * 128;  // the group's first feature
      const int ng = a.F - g0;           // and how many there are from there (128 used)
      float2 acc[C::NCH][8];
#pragma unroll
      for (int i = 0; i < C::NCH; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = make_float2(0.f, 0.f);
      // The blocks of the sum, for whole groups and for ones with fewer features:
      // two loops, so that neither's registers follow the other's.
      auto blocks = [&](auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        for (int kb = 0; kb < wk.kn; ++kb, ++it) {
          const uint32_t b = it % C::NACC;
          if (!wait_warp(&acc_full[b], (it / C::NACC) & 1u, budget, a.err, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t t = tmem + lanes + b * C::BN + grp * 128;
          const float* slot = reinterpret_cast<const float*>(smem + C::SC_OFF) + (it & (C::RING - 1)) * C::SLOT;
          uint32_t r[2][16];
          tmem_ld_32x32b_x16(t, r[0]);
          const float f = slot[row] * slot[128 + grp];
#pragma unroll
          for (int i = 0; i < C::NCH; ++i) {
            if (!WHOLE && 16 * i >= ng) continue;
            if (!WHOLE && i > 0) tmem_ld_32x32b_x16(t + 16 * i, r[i & 1]);
            tmem_ld_wait_for(r[i & 1]);
            if (WHOLE && i + 1 < C::NCH) tmem_ld_32x32b_x16(t + 16 * (i + 1), r[(i + 1) & 1]);
            if (WHOLE && i + 1 == C::NCH) release(b);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              acc[i][j] = __ffma2_rn(make_float2(__uint_as_float(r[i & 1][2 * j]), __uint_as_float(r[i & 1][2 * j + 1])),
                                     make_float2(f, f), acc[i][j]);
          }
          if (!WHOLE) {
            tmem_ld_wait_for(r[0]);
            release(b);
          }
        }
      };
      if (ng >= 128)
        blocks(std::true_type{});
      else
        blocks(std::false_type{});
      if (!ok) break;
      // Rows go out by way of shared memory, 64 bytes of each at a time: a
      // store covers eight rows' pieces instead of 32 rows' 16 bytes.  The
      // 16-byte pieces of a row are stored at piece ^ (row / 2 & 3).
      uint8_t* const mine = out_smem + lane * 64;
      const int o_row = lane >> 2, o_piece = lane & 3;
      auto out_piece = [&](int j, const uint4& v) {
        *reinterpret_cast<uint4*>(mine + ((j ^ ((lane >> 1) & 3)) << 4)) = v;
      };
      // the staged 64 bytes of the rows, from byte `at` of a row of `bytes` on
      auto flush = [&](long long at, long long bytes, int pieces) {
        __syncwarp();
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int r = 8 * v + o_row;
          const uint4 u = *reinterpret_cast<const uint4*>(out_smem + r * 64 + ((o_piece ^ ((r >> 1) & 3)) << 4));
          if (q * 32 + r < wk.n && o_piece < pieces)
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + (wk.c0 + q * 32 + r) * bytes + at + o_piece * 16) =
                u;
        }
        __syncwarp();
      };
      // 16 features of a row as fp32
      auto pieces_f32 = [&](const float2* d) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          out_piece(j, make_uint4(__float_as_uint(d[2 * j].x), __float_as_uint(d[2 * j].y),
                                  __float_as_uint(d[2 * j + 1].x), __float_as_uint(d[2 * j + 1].y)));
      };
      // and as bf16, pieces p and p + 1
      auto pieces_bf16 = [&](const float2* d, int p) {
        uint32_t u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(d[j].x, d[j].y);
          u[j] = *reinterpret_cast<const uint32_t*>(&v);
        }
        out_piece(p, make_uint4(u[0], u[1], u[2], u[3]));
        out_piece(p + 1, make_uint4(u[4], u[5], u[6], u[7]));
      };
      // the parts of S CTAs: each adds up and stores an S-th of the chunks
      auto exchange = [&](auto clusters) {
        constexpr int S = decltype(clusters)::value, NJ = C::NCH / S;
        // every load of this CTA has been used: its stages are free
        constexpr int kStride = C::EPI_WARPS * 32;
        float2* const part = reinterpret_cast<float2*>(smem) + (warp - C::CTRL_WARPS) * 32 + lane;
#pragma unroll
        for (int i = 0; i < C::NCH; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) part[(8 * i + j) * kStride] = acc[i][j];
        cluster_sync();
        exchanged = true;
#pragma unroll
        for (int n = 0; n < NJ; ++n) {
          const int i = rank * NJ + n;
          float2 v[S][8];
#pragma unroll
          for (int r = 0; r < S; ++r)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[r][j] = ld_shared_cluster_f2(cluster_map(part + (8 * i + j) * kStride, r));
#pragma unroll
          for (int r = 1; r < S; ++r)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              v[0][j].x += v[r][j].x;
              v[0][j].y += v[r][j].y;
            }
          if (16 * i >= ng) continue;
          if (a.f32) {
            pieces_f32(v[0]);
            flush((g0 + 16 * i) * 4LL, a.F * 4LL, 4);
          } else {
            pieces_bf16(v[0], 0);
            flush((g0 + 16 * i) * 2LL, a.F * 2LL, 2);
          }
        }
      };
      if constexpr (C::SPLIT) {
        switch (a.split) {
          case 2: exchange(std::integral_constant<int, 2>{}); break;
          case 4: exchange(std::integral_constant<int, 4>{}); break;
          default: exchange(std::integral_constant<int, 8>{}); break;
        }
      } else {
#pragma unroll
        for (int i = 0; i < C::NCH; ++i) {
          if (a.f32) {
            if (16 * i >= ng) continue;
            pieces_f32(acc[i]);
            flush((g0 + 16 * i) * 4LL, a.F * 4LL, 4);
          } else {
            pieces_bf16(acc[i], (i & 1) * 2);
            if ((i & 1) && 16 * (i - 1) < ng) flush((g0 + 16 * (i - 1)) * 2LL, a.F * 2LL, 16 * i < ng ? 4 : 2);
          }
        }
      }
    }
    if constexpr (C::SPLIT) {
      if (!exchanged) cluster_sync();
      cluster_sync();  // the other CTAs have read this one's part
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
static cudaError_t launch_cfg(const Fp8Maps& maps, const Fp8Args& a, int sms, cudaStream_t st) {
  static bool set[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!set[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(fp8_gemm_wide_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  return launch_product(fp8_gemm_wide_kernel<C>, C::THREADS, C::SMEM, sms, maps, a, st);
}

cudaError_t launch_fp8_gemm_wide(bool back, const Fp8Maps& maps, Fp8Args a, int sms, cudaStream_t st) {
  using C = Fp8WideCfg<false, false>;
  a.FT = (a.F + C::BN - 1) / C::BN;
  a.items = static_cast<int>(fp8_most_tiles(a.M, a.E, C::BM) * a.FT);
  a.split = product_split(a.items, sms, a.KB, 8);
  if (a.split > 1)
    return back ? launch_cfg<Fp8WideCfg<true, true>>(maps, a, sms, st)
                : launch_cfg<Fp8WideCfg<false, true>>(maps, a, sms, st);
  return back ? launch_cfg<Fp8WideCfg<true, false>>(maps, a, sms, st)
              : launch_cfg<Fp8WideCfg<false, false>>(maps, a, sms, st);
}

}  // namespace kmoe
