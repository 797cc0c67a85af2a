// Products of E4M3 operands with a scale for each block of 128 values of the
// sum: rows times weights, rows times transposed weights (the rows' gradient)
// and columns times columns (the weights' gradient), dense or by expert.
//
//   D[f, c] = sum over blocks b of 128:  sa(f, b) sb(c, b) sum_{i in b} A[f, i] B[c, i]
//
// A block's inner sum is four tcgen05.mma (kind::f8f6f4, K = 32) into a fresh
// TMEM accumulator; the epilogue warps read it while the next block's runs in
// another accumulator, multiply by the two scales and add in fp32 registers.
// The features f are the MMA's M (128 lanes), the rows its N (16 .. BN), so
// that a few rows cost few columns; sa is one value a block for a weight tile
// (its scales are for 128 x 128) and one a lane for the weights' gradient.
//
// Operands that are contiguous along the sum are K-major; the transposed
// weights and both operands of the weights' gradient are read as they lie in
// memory, MN-major (128-byte swizzle either way).
//
// Roles: warp 0 TMA, warp 1 MMA (both converged, one elected lane issues),
// the others the epilogue: groups of four warps (one per TMEM lane quarter)
// that take the 16-column chunks in turn.  Every wait is bounded.
#include <cuda_bf16.h>

#include "fp8.cuh"

namespace kmoe {

// Instruction descriptor of kind::f8f6f4: fp32 D (bits 4-5), E4M3 operands,
// bit 15 / 16 A / B is MN-major, 17-22 N >> 3, 24-28 M >> 4.
__host__ __device__ constexpr uint32_t idesc_f8(uint32_t M, uint32_t N, bool a_mn, bool b_mn) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ void mma_f8_el(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred e, p;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <Fp8Kind KIND_, int BN_>
struct Fp8Cfg {
  static constexpr Fp8Kind KIND = KIND_;
  static constexpr int BN = BN_;  // columns of a tile
  static constexpr bool WGRAD = KIND == FP8_WEIGHT_GRAD;
  static constexpr bool A_MN = KIND != FP8_ROWS;
  static constexpr bool B_MN = WGRAD;
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = BN * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = 200 * 1024 / STAGE < 10 ? 200 * 1024 / STAGE : 10;
  static constexpr int NG = BN >= 128 ? 2 : 1;  // epilogue groups of four warps
  static constexpr int EPI_WARPS = 4 * NG;
  static constexpr int THREADS = 32 * (2 + EPI_WARPS);
  static constexpr int CW = BN / NG;      // columns of a group
  static constexpr int CPL = CW / 32;     // scales a lane loads for a block
  static constexpr int NACC = 512 / BN < 4 ? 512 / BN : 4;
  static constexpr int TMEM_COLS = NACC * BN < 32 ? 32 : NACC * BN;
  static constexpr int SC_OFF = STAGES * STAGE;
  static constexpr int SC_BYTES = EPI_WARPS * 2 * CW * 4;
  static constexpr int BAR_OFF = SC_OFF + SC_BYTES;
  static constexpr int TAB_OFF = BAR_OFF + 512;
  static constexpr int TAB_INTS = kMaxE + 1;
  static constexpr int SMEM = 1024 + TAB_OFF + (2 * TAB_INTS + 40) * 4;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert((2 * STAGES + 2 * NACC + 1) * 8 + 8 <= 512, "barriers");
  static_assert((TMEM_COLS & (TMEM_COLS - 1)) == 0 && TMEM_COLS <= 512, "TMEM columns");
};

struct Fp8Item {
  int e, f0;   // expert, first feature
  int c0, n;   // first column (a row of the batch, or of dW's n) and how many
  int kb, kn;  // first block of the sum and how many
};

template <class C>
__device__ __forceinline__ int fp8_items(const Fp8Args& a, const int32_t* unit) {
  return C::WGRAD ? a.E * a.FT * a.CT : a.FT * unit[a.E];
}

template <class C>
__device__ __forceinline__ Fp8Item fp8_item(const Fp8Args& a, const int32_t* first, const int32_t* unit, int w) {
  Fp8Item it;
  if constexpr (C::WGRAD) {
    const int per = a.FT * a.CT;
    it.e = w / per;
    const int r = w - it.e * per;
    it.f0 = r / a.CT * 128;
    it.c0 = r % a.CT * C::BN;
    it.n = min(C::BN, a.C - it.c0);
    it.kb = min(unit[it.e], a.KB);
    it.kn = min(unit[it.e + 1], a.KB) - it.kb;
  } else {
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
  }
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
  segment_prefix(a.seg, a.E, a.M, C::WGRAD ? kScaleBlock : C::BN, first, unit, unit + C::TAB_INTS);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = fp8_items<C>(a, unit);
  const uint64_t budget = a.budget_ns;

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    const uint64_t pol_a = policy_evict_normal(), pol_b = policy_evict_last();
    uint32_t it = 0;
    bool ok = true;
    for (int w = blockIdx.x; ok && w < total; w += gridDim.x) {
      const Fp8Item wk = fp8_item<C>(a, first, unit, w);
      constexpr int kBox = C::WGRAD ? 128 : kFp8BoxRows;
      const int boxes = (wk.n + kBox - 1) / kBox;
      const uint32_t tx = C::A_BYTES + boxes * kBox * 128;
      for (int kb = 0; kb < wk.kn; ++kb, ++it) {
        const int s = it % C::STAGES;
        if (!mbar_wait_warp(&empty[s], ((it / C::STAGES) & 1u) ^ 1u, budget, a.err, abort_flag)) {
          ok = false;
          break;
        }
        uint8_t* sa = smem + s * C::STAGE;
        uint8_t* sb = sa + C::A_BYTES;
        const int k0 = (wk.kb + kb) * kScaleBlock;
        mbar_arrive_expect_tx_el(&full[s], tx);
        if constexpr (C::WGRAD) {
          tma_load_2d_el(sa, &maps.a, &full[s], wk.f0, k0, pol_a);
          for (int i = 0; i < boxes; ++i)
            tma_load_2d_el(sb + i * kBox * 128, &maps.b, &full[s], wk.c0 + i * kBox, k0, pol_b);
        } else {
          if constexpr (C::A_MN)
            tma_load_3d_el(sa, &maps.a, &full[s], wk.f0, k0, wk.e, pol_a);
          else
            tma_load_3d_el(sa, &maps.a, &full[s], k0, wk.f0, wk.e, pol_a);
          for (int i = 0; i < boxes; ++i)
            tma_load_2d_el(sb + i * kBox * 128, &maps.b, &full[s], k0, wk.c0 + i * kBox, pol_b);
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
    // Steps of 32 along the sum: 32 bytes inside a K-major swizzle atom, 32
    // rows of 128 bytes of an MN-major one (8-row groups 1024 bytes apart, the
    // next 128 columns 16 KB on).
    constexpr uint32_t kStepA = C::A_MN ? 256 : 2, kStepB = C::B_MN ? 256 : 2;
    const uint64_t adesc0 = C::A_MN ? make_sdesc(smem_u32(smem), 16384, 1024, 2) : sdesc_kmajor_sw128(smem_u32(smem));
    const uint64_t bdesc0 = C::B_MN ? make_sdesc(smem_u32(smem + C::A_BYTES), 16384, 1024, 2)
                                    : sdesc_kmajor_sw128(smem_u32(smem + C::A_BYTES));
    uint32_t it = 0;
    bool ok = true;
    for (int w = blockIdx.x; ok && w < total; w += gridDim.x) {
      const Fp8Item wk = fp8_item<C>(a, first, unit, w);
      const uint32_t idesc = idesc_f8(128, (wk.n + 15) & ~15, C::A_MN, C::B_MN);
      for (int kb = 0; kb < wk.kn; ++kb, ++it) {
        const int s = it % C::STAGES;
        const uint32_t b = it % C::NACC;
        if (!mbar_wait_warp(&acc_empty[b], ((it / C::NACC) & 1u) ^ 1u, budget, a.err, abort_flag) ||
            !mbar_wait_warp(&full[s], (it / C::STAGES) & 1u, budget, a.err, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t so = static_cast<uint64_t>(s) * (C::STAGE >> 4);
        const uint32_t d = tmem + b * C::BN;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mma_f8_el(d, adesc0 + so + i * kStepA, bdesc0 + so + i * kStepB, idesc, i > 0);
        tc_commit_el(&empty[s]);
        tc_commit_el(&acc_full[b]);
      }
    }
    tc_commit_el(done);
    mbar_wait_warp(done, 0, budget, a.err, nullptr);
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int grp = (warp - 2) >> 2;
    float* sc = reinterpret_cast<float*>(smem + C::SC_OFF) + (warp - 2) * 2 * C::CW;
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    uint32_t it = 0;
    bool ok = true;
    for (int w = blockIdx.x; ok && w < total; w += gridDim.x) {
      const Fp8Item wk = fp8_item<C>(a, first, unit, w);
      const int f = wk.f0 + q * 32 + lane;
      // column of the group's value i (i-th of CW), 16-column chunks in turn
      auto column = [&](int i) { return ((i >> 4) * C::NG + grp) * 16 + (i & 15); };
      const float* a_sf;
      long long a_step;
      if constexpr (C::WGRAD) {
        a_sf = a.a_sf + static_cast<long long>(wk.kb) * a.F + min(f, a.F - 1);
        a_step = a.F;
      } else {
        a_sf = a.a_sf + wk.e * a.a_se + static_cast<long long>(wk.f0 >> 7) * a.a_sm;
        a_step = a.a_sk;
      }
      const float* b_sf = a.b_sf + static_cast<long long>(wk.kb) * a.ldb + wk.c0;
      // the scales of a block: this lane's columns (0 past the tile) and sa
      struct Scales {
        float b[C::CPL], a;
      };
      auto load = [&](int kb) {
        Scales s{};
        if (kb >= wk.kn) return s;
#pragma unroll
        for (int j = 0; j < C::CPL; ++j) {
          const int c = column(lane + 32 * j);
          s.b[j] = c < wk.n ? __ldg(b_sf + static_cast<long long>(kb) * a.ldb + c) : 0.f;
        }
        s.a = __ldg(a_sf + kb * a_step);
        return s;
      };
      float2 acc[C::CW / 2];
#pragma unroll
      for (int i = 0; i < C::CW / 2; ++i) acc[i] = make_float2(0.f, 0.f);
      Scales s0 = load(0), s1 = load(1);
      for (int kb = 0; kb < wk.kn; ++kb, ++it) {
        const Scales s = s0;
        s0 = s1;
        s1 = load(kb + 2);
        float* buf = sc + (kb & 1) * C::CW;
#pragma unroll
        for (int j = 0; j < C::CPL; ++j) buf[lane + 32 * j] = C::WGRAD ? s.b[j] : s.b[j] * s.a;
        __syncwarp();
        const uint32_t b = it % C::NACC;
        if (!mbar_wait_warp(&acc_full[b], (it / C::NACC) & 1u, budget, a.err, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t t = tmem + lanes + b * C::BN;
#pragma unroll
        for (int i = 0; i < C::CW / 16; ++i) {
          const int c = (i * C::NG + grp) * 16;
          if (c < wk.n) {
            uint32_t r[16];
            tmem_ld_32x32b_x16(t + c, r);
            tmem_ld_wait();
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const float4 sv = reinterpret_cast<const float4*>(buf + 16 * i)[v];
              float2 x0 = make_float2(__uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]));
              float2 x1 = make_float2(__uint_as_float(r[4 * v + 2]), __uint_as_float(r[4 * v + 3]));
              if constexpr (C::WGRAD) {
                x0 = __fmul2_rn(x0, make_float2(s.a, s.a));
                x1 = __fmul2_rn(x1, make_float2(s.a, s.a));
              }
              acc[8 * i + 2 * v] = __ffma2_rn(x0, make_float2(sv.x, sv.y), acc[8 * i + 2 * v]);
              acc[8 * i + 2 * v + 1] = __ffma2_rn(x1, make_float2(sv.z, sv.w), acc[8 * i + 2 * v + 1]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[b]);
      }
      if (!ok) break;
      if (f < a.F) {
        const long long row0 = C::WGRAD ? static_cast<long long>(wk.e) * a.C + wk.c0 : wk.c0;
        auto store = [&](int i, float v) {
          const int c = column(i);
          if (c >= wk.n) return;
          const long long at = (row0 + c) * a.F + f;
          if (C::WGRAD || a.f32)
            static_cast<float*>(a.out)[at] = v;
          else
            static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
        };
#pragma unroll
        for (int i = 0; i < C::CW / 2; ++i) {
          store(2 * i, acc[i].x);
          store(2 * i + 1, acc[i].y);
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

int fp8_tile_columns(int M, int E) {
  const int avg = (M + E - 1) / E;
  return avg <= 32 ? 32 : (avg <= 128 ? 128 : 256);
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
  const long long units = C::WGRAD ? static_cast<long long>(a.E) * a.CT
                                   : static_cast<long long>(a.M) / C::BN + (a.M < a.E ? a.M : a.E);
  const long long items = units * a.FT;
  return launch_chained(fp8_gemm_kernel<C>, dim3(static_cast<unsigned>(items < sms ? items : sms)), dim3(C::THREADS),
                        C::SMEM, st, true, maps, a);
}

cudaError_t launch_fp8_gemm(Fp8Kind kind, const Fp8Maps& maps, const Fp8Args& a, int sms, cudaStream_t st) {
  if (kind == FP8_WEIGHT_GRAD) return launch_cfg<Fp8Cfg<FP8_WEIGHT_GRAD, 256>>(maps, a, sms, st);
  const int bn = fp8_tile_columns(a.M, a.E);
  if (kind == FP8_ROWS) {
    if (bn == 32) return launch_cfg<Fp8Cfg<FP8_ROWS, 32>>(maps, a, sms, st);
    if (bn == 128) return launch_cfg<Fp8Cfg<FP8_ROWS, 128>>(maps, a, sms, st);
    return launch_cfg<Fp8Cfg<FP8_ROWS, 256>>(maps, a, sms, st);
  }
  if (bn == 32) return launch_cfg<Fp8Cfg<FP8_ROWS_GRAD, 32>>(maps, a, sms, st);
  if (bn == 128) return launch_cfg<Fp8Cfg<FP8_ROWS_GRAD, 128>>(maps, a, sms, st);
  return launch_cfg<Fp8Cfg<FP8_ROWS_GRAD, 256>>(maps, a, sms, st);
}

}  // namespace kmoe
