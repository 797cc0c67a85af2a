// Pieces shared by the norm (norm.cu) and its gradient (norm_backward.cu).
//
// Both move each element once and do little with it, so memory bounds them.
// Rows belong to teams: a block, or a warp where a row is short (at most 128
// chunks).  A team's threads hold fixed chunks of 8 elements (16 bytes of
// bf16) of the row, NC each, and walk rows team, team + teams, ...  A row's
// inputs come through a ring of stages in shared memory, filled with cp.async
// some rows ahead: the bytes in flight that keep HBM busy then cost no
// registers and no occupancy.  A thread reads only what it copied itself, so
// the ring needs no barrier; a block's row costs one (for the sum).
//
// Rows whose width is no multiple of 8 start inside a 16-byte word.  Chunks
// are cut at the words of the tensor, not of the row: a row is `lead` =
// (t * H) mod 8 elements into its first chunk, and its first and last chunks
// are shared with its neighbours (loaded whole, stored by element).  The
// number of teams is a multiple of 8 (or each has one row), so lead is the
// same for all rows of a team and the weights stay in registers.
#pragma once
#include <cuda_bf16.h>

#include "mx_dev.cuh"
#include "norm.cuh"

namespace kmoe {

// ---------------------------------------------------------------- chunks of 8 elements
// In fp32 a chunk is four float2: the additions and products below are the
// two-wide fp32 instructions, half the issue slots of scalar ones.
template <class T>
struct Vec8 {
  uint4 q[sizeof(T) / 2];
};
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ void unpack(const Vec8<__nv_bfloat16>& a, float2 (&v)[4]) {
  v[0] = unpack2(a.q[0].x);
  v[1] = unpack2(a.q[0].y);
  v[2] = unpack2(a.q[0].z);
  v[3] = unpack2(a.q[0].w);
}
__device__ __forceinline__ void unpack(const Vec8<float>& a, float2 (&v)[4]) {
  v[0] = make_float2(__uint_as_float(a.q[0].x), __uint_as_float(a.q[0].y));
  v[1] = make_float2(__uint_as_float(a.q[0].z), __uint_as_float(a.q[0].w));
  v[2] = make_float2(__uint_as_float(a.q[1].x), __uint_as_float(a.q[1].y));
  v[3] = make_float2(__uint_as_float(a.q[1].z), __uint_as_float(a.q[1].w));
}
__device__ __forceinline__ uint32_t pack2(float2 a) {
  const __nv_bfloat162 p = __float22bfloat162_rn(a);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ void pack(const float2 (&v)[4], Vec8<__nv_bfloat16>& a) {
  a.q[0] = make_uint4(pack2(v[0]), pack2(v[1]), pack2(v[2]), pack2(v[3]));
}
__device__ __forceinline__ void pack(const float2 (&v)[4], Vec8<float>& a) {
  a.q[0] = make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                      __float_as_uint(v[1].y));
  a.q[1] = make_uint4(__float_as_uint(v[2].x), __float_as_uint(v[2].y), __float_as_uint(v[3].x),
                      __float_as_uint(v[3].y));
}
__device__ __forceinline__ void zero(float2 (&v)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) v[p] = make_float2(0.f, 0.f);
}
// Zeroes what a chunk that starts at element j0 of a row holds of the row's neighbours.
__device__ __forceinline__ void mask_edge(float2 (&v)[4], int j0, int H) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    if (j0 + 2 * p < 0 || j0 + 2 * p >= H) v[p].x = 0.f;
    if (j0 + 2 * p + 1 < 0 || j0 + 2 * p + 1 >= H) v[p].y = 0.f;
  }
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most `left` of this thread's youngest groups are in flight.
__device__ __forceinline__ void cp_async_wait(int left) {
  if (left <= 0)
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (left == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (left == 2)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 3;" ::: "memory");
}

// One chunk of a tensor of `total` elements into its ring slot (the planes of
// a 4-byte type are `slots` apart, so that lanes touch consecutive words).
// The tensor's last chunk may be short: the rest is filled with zeros.
template <class T, bool RAGGED>
__device__ __forceinline__ void load_chunk(uint4* dst, int slots, const T* src, size_t at, size_t total) {
#pragma unroll
  for (int p = 0; p < static_cast<int>(sizeof(T)) / 2; ++p) {
    constexpr int per = 16 / sizeof(T);
    const size_t e = at + p * per;
    if (!RAGGED || e + per <= total) {
      cp_async16(dst + p * slots, src + e, 16);
    } else {
      const uint32_t n = e < total ? static_cast<uint32_t>(total - e) * sizeof(T) : 0u;
      cp_async16(dst + p * slots, n ? src + e : src, n);
    }
  }
}
template <class T>
__device__ __forceinline__ void read_chunk(const uint4* src, int slots, float2 (&v)[4]) {
  Vec8<T> a;
#pragma unroll
  for (int p = 0; p < static_cast<int>(sizeof(T)) / 2; ++p) a.q[p] = src[p * slots];
  unpack(a, v);
}
// Stores the chunk whose first element is element j0 (negative before the
// row's start) of the row at `row`.
template <class T, bool RAGGED>
__device__ __forceinline__ void store_chunk(T* row, int j0, int H, const Vec8<T>& a) {
  if (!RAGGED || (j0 >= 0 && j0 + 8 <= H)) {
#pragma unroll
    for (int p = 0; p < static_cast<int>(sizeof(T)) / 2; ++p) reinterpret_cast<uint4*>(row + j0)[p] = a.q[p];
  } else {
    const T* e = reinterpret_cast<const T*>(&a);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (j0 + i >= 0 && j0 + i < H) row[j0 + i] = e[i];
  }
}
// The weights of a chunk as fp32, 0 outside the row.
template <bool RAGGED>
__device__ __forceinline__ void load_weight(const void* weight, bool f32, int j0, int H, float2 (&w)[4]) {
  if constexpr (!RAGGED) {
    if (f32) {
      Vec8<float> a;
      a.q[0] = __ldg(reinterpret_cast<const uint4*>(static_cast<const float*>(weight) + j0));
      a.q[1] = __ldg(reinterpret_cast<const uint4*>(static_cast<const float*>(weight) + j0) + 1);
      unpack(a, w);
    } else {
      Vec8<__nv_bfloat16> a;
      a.q[0] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(weight) + j0));
      unpack(a, w);
    }
  } else {
    auto at = [&](int j) {
      if (j < 0 || j >= H) return 0.f;
      return f32 ? static_cast<const float*>(weight)[j] : __bfloat162float(static_cast<const __nv_bfloat16*>(weight)[j]);
    };
#pragma unroll
    for (int p = 0; p < 4; ++p) w[p] = make_float2(at(j0 + 2 * p), at(j0 + 2 * p + 1));
  }
}

// Sums of N values over a team, the same on every thread, in a fixed order.
// Blocks: `s_part` holds N x 2 x 32 floats, its halves used by alternate rows
// (`odd`), so one barrier a row suffices: a thread that writes a half again
// has passed the barrier of the row between, which every reader reached after
// it had read.
template <int N, bool WARP>
__device__ __forceinline__ void team_sum(float (&v)[N], float* s_part, int odd) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], off);
  if constexpr (!WARP) {
    float* part = s_part + odd * N * 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if (lane == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) part[n * 32 + warp] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float s = lane < nw ? part[n * 32 + lane] : 0.f;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      v[n] = s;
    }
  }
}

// ---------------------------------------------------------------- element-wise path
// Tensors that do not start on a 16-byte boundary, and rows wider than a
// block's registers hold (16384): one element a thread and step, the row
// parked in shared memory.
__device__ __forceinline__ float load_f(const float* p, size_t i) { return p[i]; }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p, size_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ void store_f(float* p, size_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store_f(__nv_bfloat16* p, size_t i, float v) { p[i] = __float2bfloat16_rn(v); }

// Sum over the block, the same value on every thread.  Warps in order.
__device__ __forceinline__ float block_sum(float v, float* s_part) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) s += s_part[w];
  return s;
}

// The shared-memory limit of a kernel, raised once per device.
template <class K>
__host__ inline cudaError_t allow_smem(K* kernel, int (&ready)[kMaxDevices]) {
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!ready[dev]) {  // benign race (idempotent)
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem);
    if (e != cudaSuccess) return e;
    ready[dev] = 1;
  }
  return cudaSuccess;
}

}  // namespace kmoe
