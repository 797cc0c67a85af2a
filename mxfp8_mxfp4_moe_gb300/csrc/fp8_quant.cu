// Quantisers of the block-scaled products: bf16 to E4M3 codes with one
// power-of-two fp32 scale for each 128 values, the rule of kmoe_quantize_mx
// over other groups:
//   s = 2^e, the smallest e >= -126 with amax <= 448 * 2^e;  code = e4m3(x / s)
// (round to nearest even, saturating; NaN is left out of amax and becomes 0).
// A power of two makes x / s exact, so codes and scales are the definition's
// bit for bit; e4m3 keeps its relative precision under any scale.
//
//   fp8_quant_rows_kernel     128 columns of one row: the sum of rows x weights
//   fp8_quant_scatter_kernel  the same, each token's row once, written to the
//                             expert-sorted rows of its k slots
//   fp8_sort_scales_kernel    the scales of those rows, where they are many
//   fp8_quant_cols_kernel     128 rows of one column (the sum of the weights'
//                             gradient; every expert's rows from a multiple of
//                             128 on, zeros behind them)
//   fp8_quant_weights_kernel  128 x 128 weights
//
// Bound by HBM where rows are many: 32768 x 7168 rows 104 us (6.8 TB/s), 8192
// tokens into 16 rows each 174 us (6.2 TB/s), 16384 x 7168 by columns 60 us
// (5.9 TB/s), weights 4 x 7168 x 7168 92 us (6.7 TB/s).
#include "fp8.cuh"
#include "mx_dev.cuh"

namespace kmoe {

// Scale byte (e + 127 of 2^e) for the largest magnitude of a group.
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t amax) { return max(e4m3_scale_byte(amax), 1u); }
__device__ __forceinline__ float fp8_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

__device__ __forceinline__ uint32_t bf16x2_amax(const uint4& q) {
  auto b2 = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
  const __nv_bfloat162 m =
      __hmax2(__hmax2(__habs2(b2(q.x)), __habs2(b2(q.y))), __hmax2(__habs2(b2(q.z)), __habs2(b2(q.w))));
  const uint32_t u = *reinterpret_cast<const uint32_t*>(&m);
  return max(u & 0x7FFFu, u >> 16);
}

// 16 values of one row, NaN dropped, and their largest magnitude.
struct Vals16 {
  uint4 a, b;
  uint32_t amax;
};
__device__ __forceinline__ Vals16 load16(const __nv_bfloat16* p) {
  Vals16 v;
  v.a = __ldg(reinterpret_cast<const uint4*>(p));
  v.b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  v.amax = max(bf16_amax_nan(v.a), bf16_amax_nan(v.b));
  if (v.amax > 0x7F80u) {
    v.a = bf16_drop_nan(v.a);
    v.b = bf16_drop_nan(v.b);
    v.amax = max(bf16x2_amax(v.a), bf16x2_amax(v.b));
  }
  return v;
}
// The largest of a group's eight lanes.
__device__ __forceinline__ uint32_t max8(uint32_t v) {
#pragma unroll
  for (int off = 1; off < 8; off <<= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// A warp takes 512 columns of one row (16 a lane), a block the same columns of
// eight rows, whose scales of one group are adjacent: whole sectors.
__global__ void __launch_bounds__(256) fp8_quant_rows_kernel(const __nv_bfloat16* __restrict__ x, int rows, int cols,
                                                             uint8_t* __restrict__ codes,
                                                             float* __restrict__ scales) {
  chain_wait();
  __shared__ float s_scale[4][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * 8 + warp;
  const int col = blockIdx.y * 512 + lane * 16;
  const bool in = row < rows && col < cols;
  const long long at = static_cast<long long>(row) * cols + col;
  Vals16 v{};
  if (in) v = load16(x + at);
  const uint32_t byte = fp8_scale_byte(max8(v.amax));
  if (in) {
    const uint2 lo = e4m3_chunk(v.a, byte), hi = e4m3_chunk(v.b, byte);
    *reinterpret_cast<uint4*>(codes + at) = make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
  if ((lane & 7) == 0) s_scale[lane >> 3][warp] = fp8_scale(byte);
  __syncthreads();
  if (threadIdx.x < 32) {
    const int g = threadIdx.x >> 3, r = blockIdx.x * 8 + (threadIdx.x & 7);
    const int grp = blockIdx.y * 4 + g;
    if (r < rows && grp * 128 < cols) scales[static_cast<long long>(grp) * rows + r] = s_scale[g][threadIdx.x & 7];
  }
}

// A row's scales are a line apart, so storing them here is a partial sector a
// value; LATER keeps them by token (`scales` [T][groups]) and notes each row's
// slot for fp8_sort_scales_kernel.
template <bool LATER>
__global__ void __launch_bounds__(512) fp8_quant_scatter_kernel(const __nv_bfloat16* __restrict__ x, int cols, int k,
                                                                long long R, const int32_t* __restrict__ row_of_slot,
                                                                uint8_t* __restrict__ codes, float* __restrict__ scales,
                                                                int32_t* __restrict__ slot_of_row) {
  chain_wait();
  __shared__ int s_row[kMaxK];
  const long long t = blockIdx.x;
  if (threadIdx.x < k) {
    const int r = row_of_slot[t * k + threadIdx.x];
    const bool in = r >= 0 && r < R;
    s_row[threadIdx.x] = in ? r : -1;
    if (LATER && in) slot_of_row[r] = static_cast<int>(t * k + threadIdx.x);
  }
  __syncthreads();
  const int step = blockDim.x * 16 * gridDim.y;
  // whole groups of eight lanes stay in the loop together
  for (int c0 = (blockIdx.y * blockDim.x + (threadIdx.x & ~31)) * 16; c0 < cols; c0 += step) {
    const int col = c0 + (threadIdx.x & 31) * 16;
    const bool in = col < cols;
    Vals16 v{};
    if (in) v = load16(x + t * cols + col);
    const uint32_t byte = fp8_scale_byte(max8(v.amax));
    if (!in) continue;
    const uint2 lo = e4m3_chunk(v.a, byte), hi = e4m3_chunk(v.b, byte);
    const uint4 out = make_uint4(lo.x, lo.y, hi.x, hi.y);
    const float scale = fp8_scale(byte);
    if (LATER && (threadIdx.x & 7) == 0) scales[t * ((cols + 127) / 128) + (col >> 7)] = scale;
    for (int j = 0; j < k; ++j) {
      const int r = s_row[j];
      if (r < 0) continue;
      *reinterpret_cast<uint4*>(codes + static_cast<long long>(r) * cols + col) = out;
      if (!LATER && (threadIdx.x & 7) == 0) scales[(col >> 7) * R + r] = scale;
    }
  }
}

// The scales by token [T][groups] into the sorted rows' lines [groups][R]: 32
// rows a block, 64 groups at a time, turned in shared memory.  slot_of_row may
// hold anything for rows without a slot, which are left out.
__global__ void __launch_bounds__(256) fp8_sort_scales_kernel(const float* __restrict__ by_token, int groups, int k,
                                                              long long R, const int32_t* __restrict__ row_of_slot,
                                                              const int32_t* __restrict__ slot_of_row,
                                                              float* __restrict__ scales) {
  chain_wait();
  __shared__ float s_tile[32][65];
  __shared__ int s_token[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long r0 = blockIdx.x * 32LL;
  if (warp == 0) {
    const long long r = r0 + lane;
    const int s = r < R ? slot_of_row[r] : -1;
    s_token[lane] = s >= 0 && s < R && row_of_slot[s] == r ? s / k : -1;
  }
  __syncthreads();
  for (int g0 = 0; g0 < groups; g0 += 64) {
    for (int i = warp; i < 32; i += 8) {
      const int t = s_token[i];
      if (t < 0) continue;
      for (int g = lane; g < min(64, groups - g0); g += 32)
        s_tile[i][g] = __ldg(by_token + static_cast<long long>(t) * groups + g0 + g);
    }
    __syncthreads();
    if (s_token[lane] >= 0)
      for (int g = warp; g < min(64, groups - g0); g += 8) scales[(g0 + g) * R + r0 + lane] = s_tile[lane][g];
    __syncthreads();
  }
}

// One tile of 128 rows x 128 columns of weights a step, with one scale: 16 lanes
// of 8 columns by 16 rows, eight rows a thread.  blockIdx.x = expert and row
// tile.
__global__ void __launch_bounds__(256) fp8_quant_weights_kernel(const __nv_bfloat16* __restrict__ w, int rows, int cols,
                                                                uint8_t* __restrict__ codes,
                                                                float* __restrict__ scales) {
  chain_wait();
  __shared__ uint32_t s_max[8];
  const int warp = threadIdx.x >> 5;
  const int cg = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  const int tiles = (rows + 127) / 128;
  const int e = blockIdx.x / tiles, i0 = blockIdx.x % tiles * 128;
  const long long src = static_cast<long long>(e) * rows + i0;
  const int n = min(128, rows - i0);
  for (int c0 = blockIdx.y * 128; c0 < cols; c0 += gridDim.y * 128) {
    const int col = c0 + cg * 8;
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + 16 * i;
      v[i] = make_uint4(0, 0, 0, 0);
      if (r < n && col < cols) v[i] = __ldg(reinterpret_cast<const uint4*>(w + (src + r) * cols + col));
    }
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t m = bf16_amax_nan(v[i]);
      if (m > 0x7F80u) {
        v[i] = bf16_drop_nan(v[i]);
        m = bf16x2_amax(v[i]);
      }
      a = max(a, m);
    }
    a = __reduce_max_sync(0xffffffffu, a);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_max[warp] = a;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 8; ++u) a = max(a, s_max[u]);
    const uint32_t byte = fp8_scale_byte(a);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + 16 * i;
      if (r < n && col < cols)
        *reinterpret_cast<uint2*>(codes + (src + r) * cols + col) = e4m3_chunk(v[i], byte);
    }
    if (threadIdx.x == 0)
      scales[static_cast<long long>(blockIdx.x) * ((cols + 127) / 128) + c0 / 128] = fp8_scale(byte);
  }
}

// A block takes 128 rows x 128 columns a step, a scale for each column: a lane
// four columns, a warp kColRows rows, all of them in registers and in flight at
// once; one exchange of the columns' largest stands between loads and stores.
// blockIdx.x = a block of 128 rows of the padded order.  Eight warps of 16 rows,
// four blocks an SM; 4095 x 7168: 13.7 us, 16384 x 7168: 60 (four warps of 32
// rows 14.4 and 69, sixteen of eight 19.6 and 73; 64 rows of 64 columns a half
// warp, without the barrier, 15.7 and 67).
constexpr int kColWarps = 8, kColRows = 128 / kColWarps;
__global__ void __launch_bounds__(32 * kColWarps, 4) fp8_quant_cols_kernel(
    const __nv_bfloat16* __restrict__ x, int rows, int cols, int E, const int32_t* __restrict__ seg,
    uint8_t* __restrict__ codes, float* __restrict__ scales) {
  chain_wait();
  __shared__ int32_t first[kMaxE + 1], unit[kMaxE + 1], tmp[33];
  __shared__ uint2 s_max[2][kColWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  segment_prefix(seg, E, rows, 128, first, unit, tmp);
  const int b = blockIdx.x;
  if (b >= unit[E]) return;
  const int e = segment_of_unit(unit, E, b);
  const int at = (b - unit[e]) * 128, r0 = kColRows * warp;
  const int n = min(128, first[e + 1] - first[e] - at) - r0;  // rows that are there from r0 on
  const long long src = first[e] + at + r0, dst = static_cast<long long>(b) * 128 + r0;
  int turn = 0;
  for (int c0 = blockIdx.y * 128; c0 < cols; c0 += gridDim.y * 128) {
    const int col = c0 + lane * 4;
    const bool in = col < cols;
    uint2 v[kColRows];
    const __nv_bfloat16* p = x + src * cols + col;
#pragma unroll
    for (int i = 0; i < kColRows; ++i) {
      v[i] = make_uint2(0, 0);
      if (in && i < n) v[i] = __ldg(reinterpret_cast<const uint2*>(p + static_cast<long long>(i) * cols));
    }
    // largest magnitudes of the four columns, two a word (as integers, so that NaN shows)
    auto largest = [&] {
      uint2 m = make_uint2(0, 0);
#pragma unroll
      for (int i = 0; i < kColRows; ++i) {
        m.x = __vmaxu2(m.x, v[i].x & 0x7FFF7FFFu);
        m.y = __vmaxu2(m.y, v[i].y & 0x7FFF7FFFu);
      }
      turn ^= 1;  // the other half of s_max was read before the last barrier
      s_max[turn][warp][lane] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kColWarps; ++w) {
        const uint2 o = s_max[turn][w][lane];
        m.x = __vmaxu2(m.x, o.x);
        m.y = __vmaxu2(m.y, o.y);
      }
      return m;
    };
    uint2 m = largest();
    const uint32_t top = __vmaxu2(m.x, m.y);
    if (__any_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16) > 0x7F80u)) {  // the same in every warp
      auto drop = [](uint32_t w) {
        return ((w & 0x7FFFu) > 0x7F80u ? 0u : w & 0xFFFFu) | ((w & 0x7FFF0000u) > 0x7F800000u ? 0u : w & 0xFFFF0000u);
      };
#pragma unroll
      for (int i = 0; i < kColRows; ++i) v[i] = make_uint2(drop(v[i].x), drop(v[i].y));
      m = largest();
    }
    if (!in) continue;
    const uint32_t amax[4] = {m.x & 0xFFFFu, m.x >> 16, m.y & 0xFFFFu, m.y >> 16};
    float inv[4];  // 1 / s: a power of two, so x / s is exact
    float* s = scales + static_cast<long long>(b) * cols + col;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t byte = fp8_scale_byte(amax[j]);
      inv[j] = exp2i(127 - static_cast<int>(byte));
      if (warp == 0) s[j] = fp8_scale(byte);
    }
    uint8_t* q = codes + dst * cols + col;
#pragma unroll
    for (int i = 0; i < kColRows; ++i) {
      auto two = [](uint32_t w, float lo, float hi) {
        return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
            make_float2(__uint_as_float(w << 16) * lo, __uint_as_float(w & 0xFFFF0000u) * hi), __NV_SATFINITE,
            __NV_E4M3));
      };
      *reinterpret_cast<uint32_t*>(q + static_cast<long long>(i) * cols) =
          two(v[i].x, inv[0], inv[1]) | two(v[i].y, inv[2], inv[3]) << 16;
    }
  }
}

cudaError_t launch_fp8_quant_rows(const void* x, int rows, int cols, uint8_t* codes, float* scales, cudaStream_t st) {
  return launch_chained(fp8_quant_rows_kernel, dim3((rows + 7) / 8, (cols + 511) / 512), dim3(256), 0, st, true,
                        static_cast<const __nv_bfloat16*>(x), rows, cols, codes, scales);
}

cudaError_t launch_fp8_quant_scatter(const void* x, int T, int cols, int k, const int32_t* row_of_slot, uint8_t* codes,
                                     float* scales, void* workspace, cudaStream_t st) {
  const int chunks = (cols / 16 + 31) / 32;  // warps a row takes
  // few tokens: a warp a block, so that their stores spread over the SMs (two blocks of warps an SM)
  const int threads = T < 304 ? 32 : 32 * (chunks < 16 ? chunks : 16);
  const dim3 grid(T, T < 304 ? chunks : 1);
  const long long R = static_cast<long long>(T) * k;
  const auto* rows = static_cast<const __nv_bfloat16*>(x);
  if (workspace == nullptr)
    return launch_chained(fp8_quant_scatter_kernel<false>, grid, dim3(threads), 0, st, true, rows, cols, k, R,
                          row_of_slot, codes, scales, static_cast<int32_t*>(nullptr));
  const int groups = (cols + 127) / 128;
  float* by_token = static_cast<float*>(workspace);
  int32_t* slot_of_row = static_cast<int32_t*>(workspace) + static_cast<long long>(T) * groups;
  const cudaError_t e = launch_chained(fp8_quant_scatter_kernel<true>, grid, dim3(threads), 0, st, true, rows, cols, k,
                                       R, row_of_slot, codes, by_token, slot_of_row);
  if (e != cudaSuccess) return e;
  return launch_chained(fp8_sort_scales_kernel, dim3(static_cast<unsigned>((R + 31) / 32)), dim3(256), 0, st, true,
                        static_cast<const float*>(by_token), groups, k, R, row_of_slot,
                        static_cast<const int32_t*>(slot_of_row), scales);
}

// Blocks along the columns for `tiles_down` tiles of rows: about eight an SM
// (weights 4 x 7168 x 7168: 92 us, with one for all of the columns 139; 16384 x
// 7168 by columns of 16 experts: 60 us, with four an SM 66, with sixteen 60).
static int column_split(int tiles_down, int cols) {
  const int tiles = (cols + 127) / 128, split = (1216 + tiles_down - 1) / tiles_down;
  return split < 1 ? 1 : (split < tiles ? split : tiles);
}

cudaError_t launch_fp8_quant_weights(const void* w, int E, int N, int K, uint8_t* codes, float* scales,
                                     cudaStream_t st) {
  const int down = E * ((N + 127) / 128);
  return launch_chained(fp8_quant_weights_kernel, dim3(down, column_split(down, K)), dim3(256), 0, st, true,
                        static_cast<const __nv_bfloat16*>(w), N, K, codes, scales);
}

cudaError_t launch_fp8_quant_cols(const void* x, int rows, int cols, const int32_t* seg, int E, uint8_t* codes,
                                  float* scales, cudaStream_t st) {
  const int down = static_cast<int>(fp8_padded_rows(rows, E) / 128);
  return launch_chained(fp8_quant_cols_kernel, dim3(down, column_split(down, cols)), dim3(32 * kColWarps), 0, st,
                        true, static_cast<const __nv_bfloat16*>(x), rows, cols, E, seg, codes, scales);
}

}  // namespace kmoe
