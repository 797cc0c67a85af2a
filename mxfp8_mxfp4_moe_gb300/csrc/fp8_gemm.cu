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
// another accumulator, multiply by the two scales and add in fp32 registers.
// The features f are the MMA's M, the rows its N (16 .. BN), so that a few
// rows cost few columns.  Operands that are contiguous along the sum are
// K-major; transposed weights are read as they lie in memory, MN-major
// (128-byte swizzle either way).
//
// Roles: warp 0 TMA, warp 1 MMA (both converged, one elected lane issues),
// the others the epilogue: groups of four warps (one per TMEM lane quarter)
// that take the 32-column chunks in turn.  Every wait is bounded.
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

template <bool BACK_, int BN_>
struct Fp8Cfg {
  static constexpr bool BACK = BACK_;  // the weights transposed, read MN-major
  static constexpr int BN = BN_;       // columns of a tile
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int BOX = fp8_box_rows(BN);
  static constexpr int STAGE = A_BYTES + BN * 128;
  static constexpr int STAGES = 200 * 1024 / STAGE < 10 ? 200 * 1024 / STAGE : 10;
  // an epilogue warp holds up to 64 columns of 32 features (a TMEM quarter), and
  // in as many registers the block being read
  static constexpr int CW = BN < 64 ? BN : 64;
  static constexpr int NCH = CW / 32;  // 32-column chunks
  static constexpr int NG = BN / CW;   // groups of four warps
  static constexpr int EPI_WARPS = 4 * NG;
  static constexpr int CTRL_WARPS = 2;
  static constexpr int THREADS = 32 * (CTRL_WARPS + EPI_WARPS);
  static constexpr int NACC = 512 / BN < 4 ? 512 / BN : 4;
  static constexpr int TMEM_COLS = BN * NACC <= 128 ? 128 : 512;
  static constexpr int SC_OFF = STAGES * STAGE;
  static constexpr int SC_BYTES = EPI_WARPS * 2 * CW * 4;
  static constexpr int BAR_OFF = SC_OFF + SC_BYTES;
  static constexpr int TAB_OFF = BAR_OFF + 256;
  static constexpr int TAB_INTS = kMaxE + 1;
  static constexpr int SMEM = 1024 + TAB_OFF + (2 * TAB_INTS + 40) * 4;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert((2 * STAGES + 2 * NACC + 1) * 8 + 8 <= 256, "barriers");
  static_assert(BN * NACC <= TMEM_COLS, "TMEM columns");
};

template <class C>
__device__ __forceinline__ Fp8Item fp8_item(const Fp8Args& a, const int32_t* first, const int32_t* unit, int w) {
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
  it.kb = 0;
  it.kn = a.KB;
  return it;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) fp8_gemm_kernel(const __grid_constant__ Fp8Maps maps,
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
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  chain_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;  // long before any wait can give up
  tc_fence_before();
  segment_prefix(a.seg, a.E, a.M, C::BN, first, unit, unit + C::TAB_INTS);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = a.FT * unit[a.E];
  const uint64_t budget = a.budget_ns;

  if (warp < C::CTRL_WARPS) {
    if (warp == 0) {
      // ------------------------------------------------------------ loads
      const uint64_t pol_a = policy_evict_normal(), pol_b = policy_evict_last();
      uint32_t it = 0;
      bool ok = true;
      for (int w = blockIdx.x; ok && w < total; w += gridDim.x) {
        const Fp8Item wk = fp8_item<C>(a, first, unit, w);
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
          const int k0 = kb * kScaleBlock;
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
      for (int w = blockIdx.x; ok && w < total; w += gridDim.x) {
        const Fp8Item wk = fp8_item<C>(a, first, unit, w);
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
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int ew = warp - C::CTRL_WARPS;
    const int grp = ew >> 2;
    float* const ring = reinterpret_cast<float*>(smem + C::SC_OFF) + ew * 2 * C::CW;
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    // A chunk's scales lie in the order in which the eight that a thread needs
    // are two 16-byte pieces: columns 8g + 2q + {0, 1}, g even and the g after it.
    float* const my_scale = ring + (lane >> 4) * 16 + ((lane & 7) >> 1) * 4 + ((lane >> 3) & 1) * 2 + (lane & 1);
    uint32_t it = 0;
    bool ok = true;
    for (int w = blockIdx.x; ok && w < total; w += gridDim.x) {
      const Fp8Item wk = fp8_item<C>(a, first, unit, w);
      const int f0 = wk.f0 + q * 32;  // the warp's first feature
      // the group's 32-column chunks start at column(0), column(1)
      auto column = [&](int i) { return (i * C::NG + grp) * 32; };
      const int nch = (wk.n - grp * 32 + C::NG * 32 - 1) / (C::NG * 32);  // chunks with columns of the tile
      const float* b_sf = a.b_sf + wk.c0 + lane;
      const float* a_sf = a.a_sf + wk.e * a.a_se + static_cast<long long>(wk.f0 >> 7) * a.a_sm;
      // a block's scales: this lane's column of each chunk (0 past the tile), and the weights'
      struct Scales {
        float b[C::NCH], a;
      };
      auto load = [&](int kb, Scales& s) {
        if (kb >= wk.kn) return;
#pragma unroll
        for (int j = 0; j < C::NCH; ++j) {
          s.b[j] = 0.f;
          if (column(j) + lane < wk.n) s.b[j] = __ldg(b_sf + column(j));
        }
        s.a = __ldg(a_sf);
        b_sf += a.ldb;
        a_sf += a.a_sk;
      };
      float2 acc[C::CW / 2];
#pragma unroll
      for (int i = 0; i < C::CW / 2; ++i) acc[i] = make_float2(0.f, 0.f);
      Scales s0{}, s1{};
      load(0, s0);
      load(1, s1);
      for (int kb = 0; kb < wk.kn; ++kb, ++it) {
        const uint32_t b = it % C::NACC;
        float* const mine = my_scale + (kb & 1) * C::CW;
#pragma unroll
        for (int j = 0; j < C::NCH; ++j) mine[32 * j] = s0.b[j] * s0.a;
        s0 = s1;
        load(kb + 2, s1);
        if (!wait_warp(&acc_full[b], (it / C::NACC) & 1u, budget, a.err, abort_flag)) {
          ok = false;
          break;
        }
        __syncwarp();
        tc_fence_after();
        const uint32_t t = tmem + lanes + b * C::BN;
        uint32_t r[C::NCH][32];
#pragma unroll
        for (int i = 0; i < C::NCH; ++i)
          if (i < nch) {
            tmem_ld_16x256b_x4(t + column(i), r[i]);
            tmem_ld_16x256b_x4(t + (16u << 16) + column(i), r[i] + 16);
          }
#pragma unroll
        for (int i = 0; i < C::NCH; ++i) tmem_ld_wait_for(r[i]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[b]);
        const float* const scale = ring + (kb & 1) * C::CW + (lane & 3) * 4;
#pragma unroll
        for (int i = 0; i < C::NCH; ++i) {
          if (i >= nch) continue;
#pragma unroll
          for (int g = 0; g < 4; g += 2) {
            const float4 sv = *reinterpret_cast<const float4*>(scale + 32 * i + 8 * g);
#pragma unroll
            for (int h = 0; h < 4; ++h) {  // features lane / 4 + 8 h
              const uint32_t* v = r[i] + (h >> 1) * 16 + 4 * g + (h & 1) * 2;
              const float2 x0 = make_float2(__uint_as_float(v[0]), __uint_as_float(v[1]));
              const float2 x1 = make_float2(__uint_as_float(v[4]), __uint_as_float(v[5]));
              float2* d = acc + (4 * i + h) * 4 + g;
              d[0] = __ffma2_rn(x0, make_float2(sv.x, sv.y), d[0]);
              d[1] = __ffma2_rn(x1, make_float2(sv.z, sv.w), d[1]);
            }
          }
        }
      }
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < C::NCH; ++i) {
        if (i >= nch) continue;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int c = column(i) + 8 * g;
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const float2 d = acc[(4 * i + h) * 4 + g];
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
              if (f < a.F && cc < wk.n)
                *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + static_cast<long long>(wk.c0 + cc) * a.F + f) = u;
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
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <class C>
static cudaError_t launch_cfg(const Fp8Maps& maps, const Fp8Args& a, int sms, cudaStream_t st) {
  static bool set[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!set[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(fp8_gemm_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  // no more CTAs than there can be items
  const long long units = static_cast<long long>(a.M) / C::BN + (a.M < a.E ? a.M : a.E);
  const long long items = units * a.FT;
  return launch_chained(fp8_gemm_kernel<C>, dim3(static_cast<unsigned>(items < sms ? items : sms)), dim3(C::THREADS),
                        C::SMEM, st, true, maps, a);
}

cudaError_t launch_fp8_gemm(bool back, const Fp8Maps& maps, const Fp8Args& a, int sms, cudaStream_t st) {
  if (fp8_tile_columns(a.M, a.E) == 32)
    return back ? launch_cfg<Fp8Cfg<true, 32>>(maps, a, sms, st) : launch_cfg<Fp8Cfg<false, 32>>(maps, a, sms, st);
  return back ? launch_cfg<Fp8Cfg<true, 128>>(maps, a, sms, st) : launch_cfg<Fp8Cfg<false, 128>>(maps, a, sms, st);
}

}  // namespace kmoe
