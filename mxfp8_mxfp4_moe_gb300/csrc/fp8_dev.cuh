// Device pieces shared by the kernels of the block-scaled E4M3 products.
#pragma once
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

// Waits for this warp's TMEM reads; the values of `r` are read after it.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// mbar_wait_warp for waits of a few hundred cycles, once or twice a block: the
// lanes poll without a vote and the clock that bounds the wait (reading it takes
// longer than most of these waits) is looked at from the 256th poll on.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint64_t budget_ns, uint32_t* err,
                                          volatile int* abort) {
  bool there = false;
  for (int i = 0; i < 256 && !there; ++i) there = mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, there)) return true;
  return mbar_wait_warp(bar, parity, budget_ns, err, abort);
}

// 4 bytes to shared memory, in the thread's cp.async group.
__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ float2 ld_shared_cluster_f2(uint32_t cluster_addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(cluster_addr) : "memory");
  return v;
}

// CTAs of a cluster that share an item where `items` (at most) are too few for
// the CTAs that can run at once: up to eight, with `least` blocks of the sum for
// each.  Such a cluster has one item, and its CTAs meet once.  One row, 7168 x
// 7168, the same weights again and again: clusters of 1, 2 and 4 take 21.5, 13.8
// and 10.6 us.  fp8_gemm.cu's tiles
// want four blocks for each CTA, fp8_gemm_wide.cu's eight: their exchange is
// eight times larger (128 rows, 4096 x 4096: four blocks each 25 us, eight 12.5).
__host__ inline int product_split(long long items, int resident, int KB, int least) {
  int split = 1;
  while (split < 8 && items * split * 2 <= resident && KB >= 2 * least * split) split *= 2;
  return split;
}

// Launches a product's kernel for at most a.items work items on up to
// `resident` CTAs; a.split is product_split's.
template <typename Kernel>
__host__ inline cudaError_t launch_product(Kernel kernel, int threads, int smem, int resident, const Fp8Maps& maps,
                                           const Fp8Args& a, cudaStream_t st) {
  const long long ctas = static_cast<long long>(a.items) * a.split;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see chain_wait
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = a.split;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(ctas < resident ? ctas : resident));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = a.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps, a);
}

// Work items of `units` tiles of rows and `ft` of features, of which the launch
// counted on at most `items`, which an ascending table keeps to.  One whose segments
// overlap can hold more, beyond an int too; those are left out (a cluster that
// shares an item takes one even then, as its CTAs meet once).
__host__ __device__ __forceinline__ int product_items(int ft, int units, int items) {
  const long long all = static_cast<long long>(ft) * units;
  return all < items ? static_cast<int>(all) : items;
}

// A work item: features f0 .. of expert e for the columns (rows of the batch)
// c0 .. c0 + n, over blocks kb .. kb + kn of the sum.
struct Fp8Item {
  int e, f0;
  int c0, n;
  int kb, kn;
};

}  // namespace kmoe
