// Tokens sorted by expert and back, as calls of their own:
//
//   kmoe_sort_tokens        a stable counting sort of the T * k slots by expert
//   kmoe_permute            out[row of slot (t, j)] = x[t]
//   kmoe_unpermute          out[t] = sum_j w[t, j] * y[row of slot (t, j)]
//   kmoe_unpermute_backward d_y[row] = w[t, j] * d_out[t],
//                           d_w[t, j] = sum_h d_out[t, h] * y[row, h]
//
// The sort: slots in chunks of 1024, each ranked and counted by a block
// (sort_rank_kernel), the chunks' counts turned into prefixes by a warp an
// expert (sort_scan_kernel), the rows written (sort_place_kernel).  Up to one
// chunk of slots is one block's work (sort_small_kernel).
//
// The moves are bound by HBM: a token's row is read once and written k times,
// or k rows are read and summed, 16 bytes a lane.  8192 tokens, k = 16: the sort
// (896 experts) takes 9.7 us, and with 7168 bf16 columns the rows out 306 us and
// back 289 (6.5 and 6.9 TB/s), the gradient 568 (6.8 TB/s).
#include <cuda_bf16.h>

#include "common.cuh"
#include "sort.cuh"

namespace kmoe {

namespace {

// Rank of every thread's slot among the block's slots of the same expert that
// stand before it; cnt [E] (zeroed, synchronised) ends as the block's counts.
__device__ __forceinline__ int stable_rank(int id, int nwarps, int* cnt) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned peers = __match_any_sync(0xffffffffu, id);
  const unsigned lower = peers & ((1u << lane) - 1u);
  int my = -1;
  for (int w = 0; w < nwarps; ++w) {  // the same bound for every thread
    int base = 0;
    if (warp == w && id >= 0) base = cnt[id];
    __syncwarp();
    if (warp == w && id >= 0) {
      my = base + __popc(lower);
      if (lower == 0) cnt[id] = base + __popc(peers);
    }
    __syncthreads();
  }
  return my;
}

// seg[e] = sum of tot[0 .. e) for e in [0, E], by all of a block's 32 warps
// (E <= 1024, one expert a thread); tmp holds 32 ints.
__device__ __forceinline__ void prefix_1024(const int* tot, int E, int* seg, int* tmp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = threadIdx.x;
  const int c = e < E ? tot[e] : 0;
  int v = c;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += u;
  }
  if (lane == 31) tmp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int t = tmp[lane];
    const int own = t;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, t, off);
      if (lane >= off) t += u;
    }
    tmp[lane] = t - own;
  }
  __syncthreads();
  if (e < E) seg[e + 1] = tmp[warp] + v;
  if (e == 0) seg[0] = 0;
  __syncthreads();
}

__global__ void __launch_bounds__(kRankChunk) sort_small_kernel(const int32_t* __restrict__ ids, int R, int E,
                                                                int32_t* __restrict__ row_of_slot,
                                                                int32_t* __restrict__ slot_of_row,
                                                                int32_t* __restrict__ seg_start) {
  chain_wait();
  __shared__ int cnt[kMaxE], seg[kMaxE + 1], tmp[32];
  const int s = threadIdx.x;
  for (int e = s; e < E; e += kRankChunk) cnt[e] = 0;
  const int raw = s < R ? ids[s] : -1;
  const int id = raw >= 0 && raw < E ? raw : -1;
  __syncthreads();
  const int rank = stable_rank(id, (R + 31) >> 5, cnt);
  prefix_1024(cnt, E, seg, tmp);
  for (int e = s; e <= E; e += kRankChunk) seg_start[e] = seg[e];
  if (s < R) {
    const int row = id >= 0 ? seg[id] + rank : -1;
    row_of_slot[s] = row;
    if (row >= 0) slot_of_row[row] = s;
    if (s >= seg[E]) slot_of_row[s] = -1;
  }
}

// Ranks inside a chunk go to row_of_slot for the time being; counts [E][chunks].
__global__ void __launch_bounds__(kRankChunk) sort_rank_kernel(const int32_t* __restrict__ ids, int R, int E,
                                                               int32_t* __restrict__ rank, int32_t* __restrict__ counts) {
  chain_wait();
  __shared__ int cnt[kMaxE];
  for (int e = threadIdx.x; e < E; e += kRankChunk) cnt[e] = 0;
  const int s = blockIdx.x * kRankChunk + threadIdx.x;
  const int raw = s < R ? ids[s] : -1;
  const int id = raw >= 0 && raw < E ? raw : -1;
  __syncthreads();
  const int my = stable_rank(id, kRankChunk / 32, cnt);
  if (s < R) rank[s] = my;
  for (int e = threadIdx.x; e < E; e += kRankChunk) counts[static_cast<size_t>(e) * gridDim.x + blockIdx.x] = cnt[e];
}

// A warp an expert: the chunks' counts become what stands before them.
__global__ void __launch_bounds__(256) sort_scan_kernel(int32_t* __restrict__ counts, int chunks, int E,
                                                        int32_t* __restrict__ total) {
  chain_wait();
  const int lane = threadIdx.x & 31;
  const int e = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (e >= E) return;
  int32_t* c = counts + static_cast<size_t>(e) * chunks;
  int run = 0;
  for (int i = 0; i < chunks; i += 32) {
    const int own = i + lane < chunks ? c[i + lane] : 0;
    int v = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v += u;
    }
    if (i + lane < chunks) c[i + lane] = run + v - own;
    run += __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) total[e] = run;
}

__global__ void __launch_bounds__(kRankChunk) sort_place_kernel(const int32_t* __restrict__ ids, int R, int E,
                                                                const int32_t* __restrict__ counts,
                                                                const int32_t* __restrict__ total,
                                                                int32_t* __restrict__ row_of_slot,
                                                                int32_t* __restrict__ slot_of_row,
                                                                int32_t* __restrict__ seg_start) {
  chain_wait();
  __shared__ int seg[kMaxE + 1], tmp[32];
  prefix_1024(total, E, seg, tmp);
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= E; e += kRankChunk) seg_start[e] = seg[e];
  const int s = blockIdx.x * kRankChunk + threadIdx.x;
  if (s >= R) return;
  const int raw = ids[s];
  int row = -1;
  if (raw >= 0 && raw < E)
    row = seg[raw] + counts[static_cast<size_t>(raw) * gridDim.x + blockIdx.x] + row_of_slot[s];
  row_of_slot[s] = row;
  if (row >= 0) slot_of_row[row] = s;
  if (s >= seg[E]) slot_of_row[s] = -1;
}

// ---------------------------------------------------------------- moves

// chunks: 16-byte pieces of a row
__global__ void __launch_bounds__(512) permute_rows_kernel(const uint4* __restrict__ x, int chunks, int k, int R,
                                                           const int32_t* __restrict__ row_of_slot,
                                                           uint4* __restrict__ out) {
  chain_wait();
  __shared__ int s_row[kMaxK];
  const long long t = blockIdx.x;
  if (threadIdx.x < k) {
    const int r = row_of_slot[t * k + threadIdx.x];
    s_row[threadIdx.x] = r >= 0 && r < R ? r : -1;
  }
  __syncthreads();
  for (int i = blockIdx.y * blockDim.x + threadIdx.x; i < chunks; i += gridDim.y * blockDim.x) {
    const uint4 v = __ldg(x + t * chunks + i);
    for (int j = 0; j < k; ++j)
      if (s_row[j] >= 0) out[static_cast<long long>(s_row[j]) * chunks + i] = v;
  }
}

__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// One thread sums a 16-byte piece of the token's k rows, in slot order.
// y and out of either type: N values a piece (8 bf16 or 4 fp32).
template <bool Y32, bool O32>
__global__ void __launch_bounds__(256) unpermute_kernel(const uint4* __restrict__ y, int chunks, int k, int R,
                                                        const int32_t* __restrict__ row_of_slot,
                                                        const float* __restrict__ w, void* __restrict__ out) {
  constexpr int N = Y32 ? 4 : 8;
  chain_wait();
  __shared__ int s_row[kMaxK];
  __shared__ float s_w[kMaxK];
  __shared__ int s_n;
  const long long t = blockIdx.x;
  // the live slots, in order
  if (threadIdx.x < 32) {
    const int j = threadIdx.x;
    const int r = j < k ? row_of_slot[t * k + j] : -1;
    const bool live = r >= 0 && r < R;
    const unsigned mask = __ballot_sync(0xffffffffu, live);
    if (live) {
      const int at = __popc(mask & ((1u << j) - 1u));
      s_row[at] = r;
      s_w[at] = w ? w[t * k + j] : 1.f;
    }
    if (j == 0) s_n = __popc(mask);
  }
  __syncthreads();
  const int n = s_n;
  for (int i = blockIdx.y * blockDim.x + threadIdx.x; i < chunks; i += gridDim.y * blockDim.x) {
    float acc[N];
#pragma unroll
    for (int v = 0; v < N; ++v) acc[v] = 0.f;
    auto add = [&](const uint4& q, float wj) {
      const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if constexpr (Y32) {
          acc[v] = fmaf(wj, __uint_as_float(u[v]), acc[v]);
        } else {
          acc[2 * v] = fmaf(wj, lo_of(u[v]), acc[2 * v]);
          acc[2 * v + 1] = fmaf(wj, hi_of(u[v]), acc[2 * v + 1]);
        }
      }
    };
    int j = 0;
    for (; j + 4 <= n; j += 4) {
      uint4 q[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) q[v] = __ldcs(y + static_cast<long long>(s_row[j + v]) * chunks + i);
#pragma unroll
      for (int v = 0; v < 4; ++v) add(q[v], s_w[j + v]);
    }
    for (; j < n; ++j) add(__ldcs(y + static_cast<long long>(s_row[j]) * chunks + i), s_w[j]);
    const long long at = (t * chunks + i) * N;
    if constexpr (O32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
#pragma unroll
      for (int v = 0; v < N / 4; ++v) o[v] = make_float4(acc[4 * v], acc[4 * v + 1], acc[4 * v + 2], acc[4 * v + 3]);
    } else if constexpr (Y32) {
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) =
          make_uint2(pack2(acc[0], acc[1]), pack2(acc[2], acc[3]));
    } else {
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + at) =
          make_uint4(pack2(acc[0], acc[1]), pack2(acc[2], acc[3]), pack2(acc[4], acc[5]), pack2(acc[6], acc[7]));
    }
  }
}

// A slot is one warp's, or four warps' where slots are few (129 tokens, k = 8,
// 3584 columns: 7.4 us with the call); pieces of eight values.  y and d_y may be
// the same memory: a lane reads its pieces, four at a time, before it stores
// them.
template <bool G32, bool Y32, int WPS>
__global__ void __launch_bounds__(256) unpermute_backward_kernel(const void* __restrict__ d_out,
                                                                 const void* y,
                                                                 const int32_t* __restrict__ row_of_slot,
                                                                 const float* __restrict__ w, int R, int H, int k,
                                                                 void* d_y, float* __restrict__ d_w) {
  chain_wait();
  __shared__ float s_part[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = blockIdx.x * (8 / WPS) + warp / WPS;
  float acc = 0.f;
  if (s < R) {
    const int row = row_of_slot[s];
    if (row >= 0 && row < R) {
      const float wj = w[s];
      const long long g0 = static_cast<long long>(s / k) * (H / 8), y0 = static_cast<long long>(row) * (H / 8);
      constexpr int NY = Y32 ? 2 : 1, NG = G32 ? 2 : 1, STEP = 32 * WPS;  // 16-byte words of a piece
      auto eight = [](const uint4* q, auto f32, float(&v)[8]) {
        if constexpr (decltype(f32)::value) {
          const uint32_t u[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(u[j]);
        } else {
          const uint32_t u[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) v[2 * j] = lo_of(u[j]), v[2 * j + 1] = hi_of(u[j]);
        }
      };
      float part[4] = {0.f, 0.f, 0.f, 0.f};
      const int n = H / 8;
      for (int i0 = lane + 32 * (warp % WPS); i0 < n; i0 += 4 * STEP) {
        uint4 yv[4][NY], gv[4][NG];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int i = i0 + p * STEP;
          if (i >= n) continue;
#pragma unroll
          for (int j = 0; j < NY; ++j) yv[p][j] = __ldcs(static_cast<const uint4*>(y) + (y0 + i) * NY + j);
#pragma unroll
          for (int j = 0; j < NG; ++j) gv[p][j] = __ldg(static_cast<const uint4*>(d_out) + (g0 + i) * NG + j);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int i = i0 + p * STEP;
          if (i >= n) continue;
          float g[8], v[8];
          eight(yv[p], std::bool_constant<Y32>{}, v);
          eight(gv[p], std::bool_constant<G32>{}, g);
#pragma unroll
          for (int u = 0; u < 8; ++u) part[u & 3] = fmaf(g[u], v[u], part[u & 3]);
          uint4* o = static_cast<uint4*>(d_y) + (y0 + i) * NY;
          if constexpr (Y32) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              __stcs(o + j, make_uint4(__float_as_uint(wj * g[4 * j]), __float_as_uint(wj * g[4 * j + 1]),
                                       __float_as_uint(wj * g[4 * j + 2]), __float_as_uint(wj * g[4 * j + 3])));
          } else {
            __stcs(o, make_uint4(pack2(wj * g[0], wj * g[1]), pack2(wj * g[2], wj * g[3]), pack2(wj * g[4], wj * g[5]),
                                 pack2(wj * g[6], wj * g[7])));
          }
        }
      }
      acc = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    }
  }
  if constexpr (WPS > 1) {  // the slot's warps in order
    if (lane == 0) s_part[warp] = acc;
    __syncthreads();
    acc = 0.f;
#pragma unroll
    for (int v = 0; v < WPS; ++v) acc += s_part[warp / WPS * WPS + v];
  }
  if (s < R && lane == 0 && warp % WPS == 0) d_w[s] = acc;
}

// Blocks along a row for a token's k rows: few tokens spread over the SMs.
int row_split(int T, int chunks, int threads) {
  const int steps = (chunks + threads - 1) / threads;
  return T < 608 ? steps : 1;
}

}  // namespace

size_t sort_workspace_bytes(long long R, int E) {
  const size_t chunks = static_cast<size_t>((R + kRankChunk - 1) / kRankChunk);
  return chunks <= 1 ? 256 : align_up(chunks * E * 4, 256) + align_up(static_cast<size_t>(E) * 4, 256);
}

cudaError_t launch_sort_tokens(const int32_t* ids, int R, int E, int32_t* row_of_slot, int32_t* slot_of_row,
                               int32_t* seg_start, void* workspace, cudaStream_t st) {
  if (R <= kRankChunk)
    return launch_chained(sort_small_kernel, dim3(1), dim3(kRankChunk), 0, st, true, ids, R, E, row_of_slot,
                          slot_of_row, seg_start);
  const int chunks = (R + kRankChunk - 1) / kRankChunk;
  int32_t* counts = static_cast<int32_t*>(workspace);
  int32_t* total = counts + align_up(static_cast<size_t>(chunks) * E * 4, 256) / 4;
  cudaError_t e = launch_chained(sort_rank_kernel, dim3(chunks), dim3(kRankChunk), 0, st, true, ids, R, E, row_of_slot,
                                 counts);
  if (e != cudaSuccess) return e;
  e = launch_chained(sort_scan_kernel, dim3((E + 7) / 8), dim3(256), 0, st, true, counts, chunks, E, total);
  if (e != cudaSuccess) return e;
  return launch_chained(sort_place_kernel, dim3(chunks), dim3(kRankChunk), 0, st, true, ids, R, E,
                        static_cast<const int32_t*>(counts), static_cast<const int32_t*>(total), row_of_slot,
                        slot_of_row, seg_start);
}

cudaError_t launch_permute_rows(const void* x, const int32_t* row_of_slot, int T, int chunks, int k, void* out,
                                cudaStream_t st) {
  int threads = (chunks + 31) / 32 * 32;
  threads = threads < 128 ? 128 : (threads > 512 ? 512 : threads);
  if (T < 608) threads = 128;
  return launch_chained(permute_rows_kernel, dim3(T, row_split(T, chunks, threads)), dim3(threads), 0, st, true,
                        static_cast<const uint4*>(x), chunks, k, T * k, row_of_slot, static_cast<uint4*>(out));
}

cudaError_t launch_unpermute(const void* y, const int32_t* row_of_slot, const float* w, int T, int H, int k, bool y32,
                             bool o32, void* out, cudaStream_t st) {
  const int chunks = H / (y32 ? 4 : 8);
  const int threads = T < 608 ? 64 : 256;
  const dim3 grid(T, row_split(T, chunks, threads));
  auto* kernel = y32 ? (o32 ? unpermute_kernel<true, true> : unpermute_kernel<true, false>)
                     : (o32 ? unpermute_kernel<false, true> : unpermute_kernel<false, false>);
  return launch_chained(kernel, grid, dim3(threads), 0, st, true, static_cast<const uint4*>(y), chunks, k, T * k,
                        row_of_slot, w, out);
}

cudaError_t launch_unpermute_backward(const void* d_out, const void* y, const int32_t* row_of_slot, const float* w,
                                      int T, int H, int k, bool g32, bool y32, void* d_y, float* d_w,
                                      cudaStream_t st) {
  const int R = T * k;
  const bool few = R < 152 * 16;  // fewer slots than two warps a scheduler
  auto pick = [&](auto wps) {
    constexpr int W = decltype(wps)::value;
    return g32 ? (y32 ? unpermute_backward_kernel<true, true, W> : unpermute_backward_kernel<true, false, W>)
               : (y32 ? unpermute_backward_kernel<false, true, W> : unpermute_backward_kernel<false, false, W>);
  };
  auto* kernel = few ? pick(std::integral_constant<int, 4>{}) : pick(std::integral_constant<int, 1>{});
  const int per = few ? 2 : 8;
  return launch_chained(kernel, dim3((R + per - 1) / per), dim3(256), 0, st, true, d_out, y, row_of_slot, w, R, H, k,
                        d_y, d_w);
}

}  // namespace kmoe
