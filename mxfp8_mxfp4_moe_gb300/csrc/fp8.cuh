// Arguments and launchers of the products of E4M3 operands with a scale for
// each block of 128 (fp8_gemm.cu) and of their quantisers (fp8_quant.cu).
#pragma once
#include "common.cuh"

namespace kmoe {

constexpr int kScaleBlock = 128;  // values a scale

struct Fp8Maps {
  CUtensorMap a;  // weights in boxes of 128 x 128 (weight gradient: x)
  CUtensorMap b;  // boxes of 128 x kFp8BoxRows rows (weight gradient: dy)
};

struct Fp8Args {
  const int32_t* seg;  // [E + 1] first row of each expert; null: one expert, all rows
  const float* a_sf;   // weights' scales [E][.][.] (strides below); weight gradient: x's, [blocks][F]
  const float* b_sf;   // rows' scales [KB][ldb]; weight gradient: dy's, [blocks][ldb]
  void* out;
  uint32_t* err;
  unsigned long long budget_ns;
  long long a_se;  // strides of a weight scale by expert, feature block and sum block
  int a_sm, a_sk;
  int E, M;        // experts, rows
  int F, FT;       // features and tiles of 128 of them
  int C, CT;       // weight gradient: columns and tiles of them
  int KB;          // blocks of the sum (weight gradient: blocks there are)
  int ldb;
  int f32;         // out is fp32, else bf16
  int split;       // CTAs of a cluster that share an item's blocks (products; set at the launch, as is
  int items;       // the most work items that an ascending table gives)
};

// Tiles of up to `per` rows that M rows of E experts can have, whatever the
// counts.
__host__ inline long long fp8_most_tiles(long long M, int E, int per) {
  const long long with = M < E ? M : E;  // experts that can have rows
  return (M + (per - 1) * with) / per;
}
// Whether M rows of E experts are few for each, fp8_gemm.cu's; else
// fp8_gemm_wide.cu's.  One matrix of 7168 x 7168, from HBM: 8 to 32 rows take
// 13.6 us there, 18.5 to 23 in tiles of 128.  8 experts of 7168 x 3584 with 4 to
// 32 rows each 38 to 39 us, in tiles of 128 41 to 52 (transposed 34 to 35 and
// 35 to 36).  64 experts: 246 to 265 us, in tiles of 128 245 to 253 (transposed
// 248 to 270 and 233 to 237): the rule looks at the average alone and errs by up
// to 12 % there, and by up to 16 % where half of the rows are one expert's (2048
// rows: 327 and 275 us).
__host__ inline bool fp8_few_rows(int M, int E) { return (M + E - 1) / E <= 32; }
// Rows of a TMA box of the rows: tiles of up to 32 are cut to multiples of 16
// (a copy takes the time of its rows), those of many are 128.
constexpr int kFp8BoxRows = 8, kFp8WideBoxRows = 128;

cudaError_t launch_fp8_gemm(bool back, const Fp8Maps& maps, const Fp8Args& a, int sms, cudaStream_t st);
cudaError_t launch_fp8_gemm_wide(bool back, const Fp8Maps& maps, Fp8Args a, int sms, cudaStream_t st);
constexpr int kWeightGradColumns = 224;  // n of a tile of the weights' gradient
cudaError_t launch_fp8_wgrad(const Fp8Maps& maps, Fp8Args a, int sms, cudaStream_t st);

cudaError_t launch_fp8_quant_rows(const void* x, int rows, int cols, uint8_t* codes, float* scales, cudaStream_t st);
// workspace: scales by token and a slot a row, or null.
cudaError_t launch_fp8_quant_scatter(const void* x, int T, int cols, int k, const int32_t* row_of_slot, uint8_t* codes,
                                     float* scales, void* workspace, cudaStream_t st);
cudaError_t launch_fp8_quant_weights(const void* w, int E, int N, int K, uint8_t* codes, float* scales,
                                     cudaStream_t st);
cudaError_t launch_fp8_quant_cols(const void* x, int rows, int cols, const int32_t* seg, int E, uint8_t* codes,
                                  float* scales, cudaStream_t st);

// Rows that hold `rows` rows of E experts with every expert's first on a
// multiple of 128: sum of ceil(c_e / 128) blocks over any counts c_e.
__host__ inline long long fp8_padded_rows(long long rows, int E) {
  const long long with = rows < E ? rows : E;  // experts that can have rows
  return (rows + 127 * with) / 128 * 128;
}

// The first row of expert e, held inside the rows there are whatever the
// table says.
__device__ __forceinline__ int segment_start(const int32_t* seg, int e, int M) {
  return seg == nullptr ? (e == 0 ? 0 : M) : min(max(__ldg(seg + e), 0), M);
}

// Units that are counted: more than an ascending table can have, and a sum of two
// fits an int.  Tables whose segments overlap can hold more, which are left out.
constexpr int kMaxUnits = (1 << 30) - 1;
__host__ __device__ __forceinline__ int add_units(int a, int b) { return a + b < kMaxUnits ? a + b : kMaxUnits; }

// Shared-memory prefixes over the experts, for all threads of a block:
// first[e] = expert e's first row (held in [0, M]), unit[e] = units before it (at
// most kMaxUnits), a unit being up to `per` rows, 32 at least; both with E + 1
// entries.  `tmp` holds 33 ints.
__device__ __forceinline__ void segment_prefix(const int32_t* seg, int E, int M, int per, int32_t* first,
                                               int32_t* unit, int32_t* tmp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  for (int e = threadIdx.x; e <= E; e += blockDim.x) first[e] = segment_start(seg, e, M);
  __syncthreads();
  // chunks of 32 experts: prefixes inside (of at most 2^30 / 32 units each), then
  // over the (at most 32) chunks
  const int chunks = (E + 31) / 32;
  for (int c = warp; c < chunks; c += nw) {
    const int e = c * 32 + lane;
    const int rows = e < E ? max(first[e + 1] - first[e], 0) : 0;
    int v = (rows + per - 1) / per;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v += u;
    }
    if (e < E) unit[e + 1] = v;
    if (lane == 31) tmp[c] = v;
  }
  __syncthreads();
  if (warp == 0) {
    int v = lane < chunks ? tmp[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v = add_units(v, u);
    }
    v = __shfl_up_sync(0xffffffffu, v, 1);
    if (lane < chunks) tmp[lane] = lane > 0 ? v : 0;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) unit[e + 1] = add_units(unit[e + 1], tmp[e >> 5]);
  if (threadIdx.x == 0) unit[0] = 0;
  __syncthreads();
}

// The expert whose units [unit[e], unit[e + 1]) hold u < unit[E].
__host__ __device__ __forceinline__ int segment_of_unit(const int32_t* unit, int E, int u) {
  int lo = 0, hi = E;  // the largest e with unit[e] <= u has units
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (unit[mid] <= u) lo = mid; else hi = mid;
  }
  return lo;
}

}  // namespace kmoe
