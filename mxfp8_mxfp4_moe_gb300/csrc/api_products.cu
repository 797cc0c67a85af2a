// C-ABI entry points of the sort by expert and back and of the block-scaled
// E4M3 products (declared and documented in include/kmoe.h): argument checks,
// tensor maps and launches.
#include "api.cuh"
#include "fp8.cuh"
#include "sort.cuh"

using namespace kmoe;

namespace {

constexpr int kMaxCols = 1 << 20;  // columns of a product's operands and of the rows moved

int check_slots(int T, int k) {
  if (T < 0 || k <= 0 || k > kMaxK) return KMOE_ERR_ARG;
  return static_cast<long long>(T) * k > kMaxRows ? KMOE_ERR_SHAPE : KMOE_OK;
}

int check_rows(int T, int H, int k, uint32_t flags, uint32_t known) {
  const int st = check_slots(T, k);
  if (st != KMOE_OK) return st;
  if (H <= 0 || (flags & ~known) != 0u) return KMOE_ERR_ARG;
  return H % 8 != 0 || H > kMaxCols ? KMOE_ERR_SHAPE : KMOE_OK;
}

// Widths of a quantiser's or a product's operand: whole 16-byte pieces.
int check_cols(int cols) {
  if (cols <= 0) return KMOE_ERR_ARG;
  return cols % 16 != 0 || cols > kMaxCols ? KMOE_ERR_SHAPE : KMOE_OK;
}

int blocks_of(int n) { return (n + kScaleBlock - 1) / kScaleBlock; }

// Weights [E][N][K] in boxes of 128 x 128.
bool make_weights_map(CUtensorMap* m, const void* base, int E, int N, int K) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t gdim[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(E)};
  cuuint64_t gstr[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(K) * N};
  cuuint32_t box[3] = {128, 128, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), gdim, gstr, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_codes_map(CUtensorMap* m, const void* base, long long rows, int cols, uint32_t box_rows) {
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, static_cast<uint64_t>(cols), static_cast<uint64_t>(rows),
                  static_cast<uint64_t>(cols), 128, box_rows);
}

int check_workspace(const void* workspace, size_t ws_bytes) {
  if (!workspace || ws_bytes < KMOE_GEMM_FP8_WORKSPACE_BYTES) return KMOE_ERR_WORKSPACE;
  return aligned(workspace, 256) ? KMOE_OK : KMOE_ERR_ALIGN;
}

}  // namespace

extern "C" {

size_t kmoe_sort_workspace_size(int T, int E, int k) {
  if (check_slots(T, k) != KMOE_OK || E <= 0 || E > kMaxE) return 0;
  return sort_workspace_bytes(static_cast<long long>(T) * k, E);
}

int kmoe_sort_tokens(const int32_t* topk_ids, int T, int E, int k, int32_t* row_of_slot, int32_t* slot_of_row,
                     int32_t* seg_start, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  const int st = check_slots(T, k);
  if (st != KMOE_OK) return st;
  if (E <= 0 || E > kMaxE || !seg_start) return KMOE_ERR_ARG;
  if (!workspace || ws_bytes < kmoe_sort_workspace_size(T, E, k)) return KMOE_ERR_WORKSPACE;
  if (T > 0 && (!topk_ids || !row_of_slot || !slot_of_row)) return KMOE_ERR_ARG;
  if (!aligned(topk_ids, 4) || !aligned(row_of_slot, 4) || !aligned(slot_of_row, 4) || !aligned(seg_start, 4) ||
      !aligned(workspace, 256))
    return KMOE_ERR_ALIGN;
  if (T == 0) {
    KMOE_CK(cudaMemsetAsync(seg_start, 0, static_cast<size_t>(E + 1) * 4, stream));
    return KMOE_OK;
  }
  KMOE_CK(launch_sort_tokens(topk_ids, T * k, E, row_of_slot, slot_of_row, seg_start, workspace, stream));
  return KMOE_OK;
}

int kmoe_permute(const void* x, const int32_t* row_of_slot, int T, int H, int k, uint32_t flags, void* out,
                 cudaStream_t stream) {
  const int st = check_rows(T, H, k, flags, KMOE_ROWS_F32);
  if (st != KMOE_OK) return st;
  if (T == 0) return KMOE_OK;
  if (!x || !row_of_slot || !out) return KMOE_ERR_ARG;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(row_of_slot, 4)) return KMOE_ERR_ALIGN;
  KMOE_CK(launch_permute_rows(x, row_of_slot, T, H / ((flags & KMOE_ROWS_F32) ? 4 : 8), k, out, stream));
  return KMOE_OK;
}

int kmoe_unpermute(const void* y, const int32_t* row_of_slot, const float* topk_w, int T, int H, int k, uint32_t flags,
                   void* out, cudaStream_t stream) {
  const int st = check_rows(T, H, k, flags, KMOE_ROWS_F32 | KMOE_OUT_F32);
  if (st != KMOE_OK) return st;
  if (T == 0) return KMOE_OK;
  if (!y || !row_of_slot || !out) return KMOE_ERR_ARG;
  if (!aligned(y, 16) || !aligned(out, 16) || !aligned(row_of_slot, 4) || !aligned(topk_w, 4)) return KMOE_ERR_ALIGN;
  KMOE_CK(launch_unpermute(y, row_of_slot, topk_w, T, H, k, (flags & KMOE_ROWS_F32) != 0u,
                           (flags & KMOE_OUT_F32) != 0u, out, stream));
  return KMOE_OK;
}

int kmoe_unpermute_backward(const void* d_out, const void* y, const int32_t* row_of_slot, const float* topk_w, int T,
                            int H, int k, uint32_t flags, void* d_y, float* d_w, cudaStream_t stream) {
  const int st = check_rows(T, H, k, flags, KMOE_ROWS_F32 | KMOE_OUT_F32);
  if (st != KMOE_OK) return st;
  if (T == 0) return KMOE_OK;
  if (!d_out || !y || !row_of_slot || !topk_w || !d_y || !d_w) return KMOE_ERR_ARG;
  if (!aligned(d_out, 16) || !aligned(y, 16) || !aligned(d_y, 16) || !aligned(row_of_slot, 4) || !aligned(topk_w, 4) ||
      !aligned(d_w, 4))
    return KMOE_ERR_ALIGN;
  KMOE_CK(launch_unpermute_backward(d_out, y, row_of_slot, topk_w, T, H, k, (flags & KMOE_OUT_F32) != 0u,
                                    (flags & KMOE_ROWS_F32) != 0u, d_y, d_w, stream));
  return KMOE_OK;
}

size_t kmoe_quantize_fp8_workspace_size(int rows, int cols, int k) {
  if (check_slots(rows, k) != KMOE_OK || check_cols(cols) != KMOE_OK) return 0;
  // from where the sorted scales in a pass of their own are worth its launch (7168 columns, without / with it:
  // R = 131072 217 / 174 us, 65536 102 / 97, 32768 (k = 8, 16) 52 / 50 and 44 / 46, 16384 27 / 28, 8184 11.4 / 13.6)
  const long long R = static_cast<long long>(rows) * k;
  if (k == 1 || R < 65536) return 0;
  return align_up((static_cast<size_t>(rows) * blocks_of(cols) + static_cast<size_t>(R)) * 4, 256);
}

int kmoe_quantize_fp8(const void* x_bf16, int rows, int cols, const int32_t* row_of_slot, int k, uint8_t* codes,
                      float* scales, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  int st = check_slots(rows, k);
  if (st == KMOE_OK) st = check_cols(cols);
  if (st != KMOE_OK) return st;
  if (!row_of_slot && k != 1) return KMOE_ERR_ARG;
  const size_t need = row_of_slot ? kmoe_quantize_fp8_workspace_size(rows, cols, k) : 0;
  if (need && workspace && ws_bytes < need) return KMOE_ERR_WORKSPACE;
  if (rows == 0) return KMOE_OK;
  if (!x_bf16 || !codes || !scales) return KMOE_ERR_ARG;
  if (!aligned(x_bf16, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(row_of_slot, 4) ||
      !aligned(workspace, 4))
    return KMOE_ERR_ALIGN;
  KMOE_CK(row_of_slot ? launch_fp8_quant_scatter(x_bf16, rows, cols, k, row_of_slot, codes, scales,
                                                 need ? workspace : nullptr, stream)
                      : launch_fp8_quant_rows(x_bf16, rows, cols, codes, scales, stream));
  return KMOE_OK;
}

int kmoe_quantize_fp8_weights(const void* w_bf16, int E, int N, int K, uint8_t* codes, float* scales,
                              cudaStream_t stream) {
  if (E <= 0 || E > kMaxE) return KMOE_ERR_ARG;
  int st = check_cols(N);
  if (st == KMOE_OK) st = check_cols(K);
  if (st != KMOE_OK) return st;
  if (!w_bf16 || !codes || !scales) return KMOE_ERR_ARG;
  if (!aligned(w_bf16, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return KMOE_ERR_ALIGN;
  KMOE_CK(launch_fp8_quant_weights(w_bf16, E, N, K, codes, scales, stream));
  return KMOE_OK;
}

int kmoe_fp8_padded_rows(int rows, int E) {
  if (rows < 0 || rows > kMaxRows || E <= 0 || E > kMaxE) return -1;
  return static_cast<int>(fp8_padded_rows(rows, E));
}

int kmoe_quantize_fp8_cols(const void* x_bf16, int rows, int cols, const int32_t* seg_start, int E, uint8_t* codes,
                           float* scales, cudaStream_t stream) {
  if (rows < 0 || E <= 0 || E > kMaxE || (!seg_start && E != 1)) return KMOE_ERR_ARG;
  const int st = check_cols(cols);
  if (st != KMOE_OK) return st;
  if (rows > kMaxRows) return KMOE_ERR_SHAPE;
  if (rows == 0) return KMOE_OK;
  if (!x_bf16 || !codes || !scales) return KMOE_ERR_ARG;
  if (!aligned(x_bf16, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(seg_start, 4))
    return KMOE_ERR_ALIGN;
  KMOE_CK(launch_fp8_quant_cols(x_bf16, rows, cols, seg_start, E, codes, scales, stream));
  return KMOE_OK;
}

int kmoe_gemm_fp8(const uint8_t* x, const float* x_scales, const uint8_t* w, const float* w_scales,
                  const int32_t* seg_start, int M, int N, int K, int E, uint32_t flags, void* out, void* workspace,
                  size_t ws_bytes, cudaStream_t stream) {
  if (M < 0 || E <= 0 || E > kMaxE || (!seg_start && E != 1)) return KMOE_ERR_ARG;
  if ((flags & ~(KMOE_GEMM_TRANSPOSE | KMOE_GEMM_OUT_F32)) != 0u) return KMOE_ERR_ARG;
  int st = check_cols(N);
  if (st == KMOE_OK) st = check_cols(K);
  if (st != KMOE_OK) return st;
  const bool back = (flags & KMOE_GEMM_TRANSPOSE) != 0u, f32 = (flags & KMOE_GEMM_OUT_F32) != 0u;
  Fp8Args a{};
  a.F = back ? K : N;
  a.FT = blocks_of(a.F);
  // work items are counted in an int
  if (M > kMaxRows || (static_cast<long long>(M) / 16 + E) * a.FT > kMaxRows) return KMOE_ERR_SHAPE;
  st = check_workspace(workspace, ws_bytes);
  if (st != KMOE_OK) return st;
  if (M == 0) return KMOE_OK;
  if (!x || !x_scales || !w || !w_scales || !out) return KMOE_ERR_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4) || !aligned(seg_start, 4) ||
      !aligned(out, 16))
    return KMOE_ERR_ALIGN;
  a.seg = seg_start;
  a.a_sf = w_scales;
  a.b_sf = x_scales;
  a.out = out;
  a.err = static_cast<uint32_t*>(workspace);
  a.budget_ns = kWaitBudgetNs;
  const int nb = blocks_of(N), kb = blocks_of(K);
  a.a_se = static_cast<long long>(nb) * kb;
  a.a_sm = back ? 1 : kb;
  a.a_sk = back ? kb : 1;
  a.E = E;
  a.M = M;
  a.KB = back ? nb : kb;
  a.ldb = M;
  a.f32 = f32;
  const bool few = fp8_few_rows(M, E);
  Fp8Maps m;
  if (!make_weights_map(&m.a, w, E, N, K) ||
      !make_codes_map(&m.b, x, M, back ? N : K, few ? kFp8BoxRows : kFp8WideBoxRows))
    return KMOE_ERR_CUDA;
  const int sms = num_sms();
  if (sms <= 0) return KMOE_ERR_CUDA;
  KMOE_CK(few ? launch_fp8_gemm(back, m, a, sms, stream) : launch_fp8_gemm_wide(back, m, a, sms, stream));
  return KMOE_OK;
}

int kmoe_gemm_fp8_wgrad(const uint8_t* dy, const float* dy_scales, const uint8_t* x, const float* x_scales,
                        const int32_t* seg_start, int P, int N, int K, int E, float* dw, void* workspace,
                        size_t ws_bytes, cudaStream_t stream) {
  if (P < 0 || E <= 0 || E > kMaxE || (!seg_start && E != 1)) return KMOE_ERR_ARG;
  int st = check_cols(N);
  if (st == KMOE_OK) st = check_cols(K);
  if (st != KMOE_OK) return st;
  if (P > kMaxRows + 128LL * kMaxE || P % kScaleBlock != 0 ||
      static_cast<long long>(E) * blocks_of(N) * blocks_of(K) > kMaxRows)
    return KMOE_ERR_SHAPE;
  st = check_workspace(workspace, ws_bytes);
  if (st != KMOE_OK) return st;
  if (!dw || (P > 0 && (!dy || !dy_scales || !x || !x_scales))) return KMOE_ERR_ARG;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dy_scales, 4) || !aligned(x_scales, 4) ||
      !aligned(seg_start, 4) || !aligned(dw, 4))
    return KMOE_ERR_ALIGN;
  if (P == 0) {
    KMOE_CK(cudaMemsetAsync(workspace, 0, 4, stream));
    KMOE_CK(cudaMemsetAsync(dw, 0, static_cast<size_t>(E) * N * K * 4, stream));
    return KMOE_OK;
  }
  Fp8Args a{};
  a.seg = seg_start;
  a.a_sf = x_scales;
  a.b_sf = dy_scales;
  a.out = dw;
  a.err = static_cast<uint32_t*>(workspace);
  a.budget_ns = kWaitBudgetNs;
  a.E = E;
  a.M = P;  // no expert has more rows
  a.KB = P / kScaleBlock;
  a.F = K;
  a.FT = blocks_of(K);
  a.C = N;
  a.CT = (N + kWeightGradColumns - 1) / kWeightGradColumns;
  a.ldb = N;
  Fp8Maps m;
  if (!make_codes_map(&m.a, x, P, K, 128) || !make_codes_map(&m.b, dy, P, N, 128)) return KMOE_ERR_CUDA;
  const int sms = num_sms();
  if (sms <= 0) return KMOE_ERR_CUDA;
  KMOE_CK(launch_fp8_wgrad(m, a, sms, stream));
  return KMOE_OK;
}

}  // extern "C"
