// Host interface of the norm kernels (norm.cu, norm_backward.cu).
#pragma once
#include "common.cuh"

namespace kmoe {

constexpr int kMaxNormH = 32768;       // columns of the element-wise path (a row of fp32 in shared memory)
constexpr int kNormSmem = 224 * 1024;  // shared memory that a block may ask for
constexpr int kNormSMs = 152;          // SMs the grids are laid out for
constexpr int kMaxStages = 4;          // of a row kernel's ring (cp_async_wait knows so many)

// Partial rows of the weight gradient: at most two blocks an SM.  Their number
// and so the summation order follow from the shape, the stream's type and
// whether the tensors take the row kernels, not from the GPU.
constexpr int kNormMaxParts = 2 * kNormSMs;
__host__ inline size_t norm_part_bytes(int T, int H) {
  return static_cast<size_t>(T < kNormMaxParts ? T : kNormMaxParts) * H * 4;
}

// Launch shape of a row kernel (norm_dev.cuh): chunks per thread, threads and
// blocks, ring stages.  nc = 0: the row does not fit, take the element-wise path.
struct NormPlan {
  int nc, threads, blocks, stages;
  bool warp;  // a warp, not a block, has a row
  size_t smem;
};

// chunk_bytes: ring bytes of one chunk of one row (all its tensors).
// Blocks an SM: rows in flight help until the streams of many rows hurt HBM.
// Measured per direction (1 / 2 blocks, us): the forward, 512 threads an SM:
// H = 7168 with codes 85.5 / 97.0, H = 4096 86 / 98, H = 2048 (2 / 4 blocks)
// 83 / 99; the gradient, 1024 chunks an SM: H = 7168 75.9 / 78.4, H = 3584
// 90 / 77.8.  Ragged rows do more for each byte and want twice as many: H =
// 7001, T = 4096, forward 45.5 / 42.7, gradient 59.6 / 51.6.  So do batches of
// a bf16 stream whose outputs mostly stay in L2, up to 2^24 elements: H = 7168,
// forward with codes, T = 256 8.2 / 7.8, 512 12.3 / 10.3, 1024 16.5 / 16.5, 2048
// 26.6 / 24.7, 4096 44.0 / 49.0; H = 4096, T = 2048 17.7 / 16.4 (an fp32 stream:
// H = 5000, T = 1024 16.8 / 18.7).
__host__ inline NormPlan plan_norm(int T, int H, int chunk_bytes, bool backward) {
  NormPlan p{};
  const bool ragged = H % 8 != 0;
  const int C = ragged ? (H + 14) / 8 : H / 8;  // chunks a row can touch
  int teams_per_block = 1, per_sm;
  if (C <= 128) {
    p.warp = true;
    p.nc = C <= 32 ? 1 : (C <= 64 ? 2 : 4);
    p.threads = 256;
    teams_per_block = 8;
    per_sm = 4;
  } else {
    p.nc = C <= 512 ? 1 : (C <= 1024 ? 2 : 4);
    p.threads = ((C + p.nc - 1) / p.nc + 31) / 32 * 32;
    if (p.threads > 512) return NormPlan{};
    per_sm = (backward ? 1024 / (p.threads * p.nc) : 512 / p.threads) * (ragged ? 2 : 1);
    if (per_sm < 1) per_sm = 1;
    const bool bf16_forward = !backward && chunk_bytes == 32;
    if (bf16_forward && !ragged && static_cast<long long>(T) * H <= (1 << 24)) per_sm *= 2;
  }
  if (backward && per_sm > 2) per_sm = 2;  // kNormMaxParts
  const size_t stage = static_cast<size_t>(p.threads) * p.nc * chunk_bytes;
  if (stage * per_sm > kNormSmem) per_sm = 1;
  if (stage > kNormSmem) return NormPlan{};
  // no more blocks than the rows of the longest need: the gradient's partial rows are fewer
  const int want = (T + teams_per_block - 1) / teams_per_block, most = kNormSMs * per_sm;
  const int rows = (want + most - 1) / most;
  p.blocks = (want + rows - 1) / rows;
  if (ragged && rows > 1) p.blocks = (p.blocks + 7) / 8 * 8;  // most is a multiple of 8
  p.stages = static_cast<int>(kNormSmem / per_sm / stage);
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  if (p.stages > rows) p.stages = rows;
  p.smem = stage * p.stages;
  return p;
}

cudaError_t launch_rmsnorm(const void* x, const void* residual, const void* weight, int T, int H, float eps,
                           bool stream_f32, bool weight_f32, void* h, void* y, uint8_t* codes, uint8_t* scales,
                           cudaStream_t st);
cudaError_t launch_rmsnorm_backward(const void* dy, const void* h, const void* weight, const void* dh_in, int T, int H,
                                    float eps, bool stream_f32, bool weight_f32, void* dh, float* dweight, float* part,
                                    cudaStream_t st);

}  // namespace kmoe
