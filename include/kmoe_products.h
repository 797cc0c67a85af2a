/*
 * kmoe -- expert products in 8 bits: part of kmoe.h, which includes it and has
 * the conventions (device pointers, streams, status codes, empty batches).
 */
#ifndef KMOE_PRODUCTS_H_
#define KMOE_PRODUCTS_H_

#include "kmoe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Expert products in 8 bits, for experts (or a dense projection) whose
 * weights are E4M3 with a scale for each block of 128 x 128, as FP8 checkpoints
 * hold them: the tokens' rows sorted by expert and summed back with their
 * weights, the quantisers and the products, and the gradients of each.  A step
 * of such experts is
 *   kmoe_sort_tokens, kmoe_quantize_fp8 (into sorted rows), kmoe_gemm_fp8, the
 *   activation, kmoe_quantize_fp8, kmoe_gemm_fp8, kmoe_unpermute
 * and back
 *   kmoe_unpermute_backward, kmoe_quantize_fp8, kmoe_gemm_fp8 with
 *   KMOE_GEMM_TRANSPOSE (the rows' gradient), kmoe_quantize_fp8_cols and
 *   kmoe_gemm_fp8_wgrad (the weights'), ..., kmoe_unpermute without weights.
 * At most 2^30 rows (tokens times k) and 2^20 columns.  These kernels are
 * launched with programmatic stream serialization and wait for what is queued
 * before them.  Calls that can overlap on the GPU take a workspace each. */

/* Tokens sorted by expert: a stable sort of the slots s = t * k + j by
 * topk_ids[s].
 *   row_of_slot [T, k]: the sorted row of a slot, -1 where its id is outside
 *   [0, E); slot_of_row [T * k]: its inverse, -1 for rows from seg_start[E] on;
 *   seg_start [E + 1]: each expert's first row, and the number of sorted rows
 * (all int32, out; seg_start is written for T = 0 too).  E <= 1024, k <= 32
 * (k > E is allowed: an expert may stand in several slots of a token).
 * workspace: kmoe_sort_workspace_size bytes (0 for invalid sizes), 256-byte
 * aligned. */
size_t kmoe_sort_workspace_size(int T, int E, int k);
int kmoe_sort_tokens(const int32_t* topk_ids, int T, int E, int k, int32_t* row_of_slot, int32_t* slot_of_row,
                     int32_t* seg_start, void* workspace, size_t ws_bytes, cudaStream_t stream);

/* Types of the moved rows: of the sorted rows (x and out of kmoe_permute, y,
 * d_y) and of the tokens' (out of kmoe_unpermute, d_out); bf16 without the flag. */
#define KMOE_ROWS_F32 1u
#define KMOE_OUT_F32 2u

/* out[row_of_slot[t, j]] = x[t] for the slots that have a row; the other rows
 * of out keep their contents.  x [T, H] and out [T * k, H] of one type
 * (KMOE_ROWS_F32), 16-byte aligned, H a multiple of 8.  Its gradient is
 * kmoe_unpermute without weights.  Entries of row_of_slot outside [0, T * k)
 * count as -1, here and below; no two may be the same row. */
int kmoe_permute(const void* x, const int32_t* row_of_slot, int T, int H, int k, uint32_t flags, void* out,
                 cudaStream_t stream);

/* out[t] = sum over slots j, in order, of topk_w[t, j] * y[row_of_slot[t, j]]
 * (topk_w null: the sum of the rows), in fp32, rounded once; slots without a
 * row add nothing and a token without any gets 0.
 *   y [T * k, H] (KMOE_ROWS_F32), topk_w [T, k] float or null, out [T, H]
 *   (KMOE_OUT_F32); y and out 16-byte aligned, H a multiple of 8. */
int kmoe_unpermute(const void* y, const int32_t* row_of_slot, const float* topk_w, int T, int H, int k, uint32_t flags,
                   void* out, cudaStream_t stream);

/* Gradient of kmoe_unpermute:
 *   d_y[row_of_slot[t, j]] = topk_w[t, j] * d_out[t]   (y's type, rounded once)
 *   d_w[t, j] = sum_h d_out[t, h] * y[row_of_slot[t, j], h]   (fp32)
 * and for slots without a row d_w = 0; rows of d_y without a slot keep their
 * contents.  d_out [T, H] (KMOE_OUT_F32), y and d_y [T * k, H] (KMOE_ROWS_F32;
 * d_y may be y), all 16-byte aligned, H a multiple of 8. */
int kmoe_unpermute_backward(const void* d_out, const void* y, const int32_t* row_of_slot, const float* topk_w, int T,
                            int H, int k, uint32_t flags, void* d_y, float* d_w, cudaStream_t stream);

/* Quantisation to E4M3 codes with one power-of-two fp32 scale for each 128
 * values, the rule of kmoe_quantize_mx over other groups: s = 2^e with the
 * smallest e >= -126 such that amax <= 448 * 2^e (2^127 beside an infinity),
 * NaN left out of amax; code = x / s rounded to nearest even, saturating; NaN
 * becomes +0.  Groups at an edge hold what there is.  Columns (N, K) are
 * multiples of 16; x and codes 16-byte aligned.
 *
 * Rows: groups of 128 columns of a row.  codes [rows, cols], scales
 * [ceil(cols/128), rows] float: one line of scales for each 128 columns, as
 * kmoe_gemm_fp8 reads them.  With row_of_slot [rows, k] (kmoe_sort_tokens')
 * row t goes to the sorted rows of its k slots instead: codes [rows * k, cols],
 * scales [ceil(cols/128), rows * k]; rows without a slot keep their contents.
 * Without it k is 1.
 *   workspace: kmoe_quantize_fp8_workspace_size bytes (0: none is used), 4-byte
 *   aligned, or null: many sorted rows' scales are then stored more slowly. */
size_t kmoe_quantize_fp8_workspace_size(int rows, int cols, int k);
int kmoe_quantize_fp8(const void* x_bf16, int rows, int cols, const int32_t* row_of_slot, int k, uint8_t* codes,
                      float* scales, void* workspace, size_t ws_bytes, cudaStream_t stream);

/* Weights [E, N, K]: blocks of 128 x 128 of an expert.  codes [E, N, K], scales
 * [E, ceil(N/128), ceil(K/128)] float.  E <= 1024. */
int kmoe_quantize_fp8_weights(const void* w_bf16, int E, int N, int K, uint8_t* codes, float* scales,
                              cudaStream_t stream);

/* Columns: groups of 128 rows of a column, for kmoe_gemm_fp8_wgrad, whose sum
 * runs over the rows.  Every expert's rows [seg_start[e], seg_start[e+1])
 * (int32 [E + 1] on the device, ascending; null: E = 1, all rows) start on a
 * multiple of 128 rows of the codes, in the experts' order, with zero codes
 * behind its last: codes [P, cols] and scales [P/128, cols] float for P =
 * kmoe_fp8_padded_rows(rows, E), enough for any counts (-1 for invalid sizes).
 * Blocks behind the last expert's keep their contents. */
int kmoe_fp8_padded_rows(int rows, int E);
int kmoe_quantize_fp8_cols(const void* x_bf16, int rows, int cols, const int32_t* seg_start, int E, uint8_t* codes,
                           float* scales, cudaStream_t stream);

/* kmoe_gemm_fp8's flags: multiply by the transposed weights (the rows'
 * gradient); out is fp32, else bf16. */
#define KMOE_GEMM_TRANSPOSE 1u
#define KMOE_GEMM_OUT_F32 2u
#define KMOE_GEMM_FP8_WORKSPACE_BYTES ((size_t)256)

/* Products of E4M3 rows with E4M3 weights, each expert's rows with its weights:
 *   out[m, n] = sum_b x_scales[b, m] * w_scales[e, n/128, b] *
 *               sum_{k in block b of 128} x[m, k] * w[e, n, k]
 * for m in [seg_start[e], seg_start[e+1]), or with KMOE_GEMM_TRANSPOSE
 *   out[m, k] = sum_b x_scales[b, m] * w_scales[e, b, k/128] *
 *               sum_{n in block b of 128} x[m, n] * w[e, n, k].
 * A block's products are summed by the tensor cores, the scaled blocks in fp32,
 * in the order of b; where there are few rows up to eight ranges of blocks are
 * summed so, each by itself, and then the ranges in their order.  How many depends
 * on the sizes of the call and the GPU's SMs: equal calls give equal bits, a row in
 * a call of another size may differ in its last ones.  out is rounded once.
 *   Scales are any fp32 values whose product, which is taken first, is a normal
 * fp32 number or 0.  Below 2^-126 it loses bits, by which a block is off by up to
 * 2^-125 (kmoe_quantize_fp8's smallest scale, 2^-126, is that of zeros, which stay
 * exact, and of values below 2^-117); from 2^128 on it is an infinity, and so is
 * the block, or NaN where its sum is 0.
 *   x [M, K] (transposed: [M, N]) codes, x_scales [ceil(cols/128), M] float
 *   (kmoe_quantize_fp8's); w [E, N, K] codes, w_scales [E, ceil(N/128),
 *   ceil(K/128)] float (kmoe_quantize_fp8_weights', or a checkpoint's);
 *   seg_start [E + 1] int32 on the device, ascending, from 0 (null: E = 1, all
 *   rows); out [M, N] (transposed: [M, K]).  Rows outside all segments keep
 *   their contents.  N and K multiples of 16; x, w and out 16-byte aligned.
 *   workspace: KMOE_GEMM_FP8_WORKSPACE_BYTES, 256-byte aligned: its first word
 *   is the device error word (kmoe_device_error), cleared by every call that
 *   has rows (one without leaves it as it is): what an earlier call in the same
 *   workspace left there is gone, so it is read before, or each call has a
 *   workspace of its own. */
int kmoe_gemm_fp8(const uint8_t* x, const float* x_scales, const uint8_t* w, const float* w_scales,
                  const int32_t* seg_start, int M, int N, int K, int E, uint32_t flags, void* out, void* workspace,
                  size_t ws_bytes, cudaStream_t stream);

/* The weights' gradient, each expert's from its rows:
 *   dw[e, n, k] = sum over e's blocks b of 128 rows of dy_scales[b, n] *
 *                 x_scales[b, k] * sum_{m in b} dy[m, n] * x[m, k]
 * dy [P, N], x [P, K] codes and scales [P/128, .] as kmoe_quantize_fp8_cols
 * writes them for the same rows and seg_start, P a multiple of 128 (a scale that
 * is no normal power of two makes its row or column of dw NaN); dw [E, N, K]
 * float (out, every element: an expert without rows gets zeros, P = 0 included).
 * The tensor cores sum up to 1024 rows, in fp32 whose additions may truncate;
 * those sums are added in fp32, in order.  Workspace as kmoe_gemm_fp8; the error
 * word is cleared by every call. */
int kmoe_gemm_fp8_wgrad(const uint8_t* dy, const float* dy_scales, const uint8_t* x, const float* x_scales,
                        const int32_t* seg_start, int P, int N, int K, int E, float* dw, void* workspace,
                        size_t ws_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* KMOE_PRODUCTS_H_ */
