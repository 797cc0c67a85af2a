// Launchers of the sort by expert and the moves of rows (sort.cu).
#pragma once
#include <type_traits>

#include "common.cuh"

namespace kmoe {

size_t sort_workspace_bytes(long long R, int E);
cudaError_t launch_sort_tokens(const int32_t* ids, int R, int E, int32_t* row_of_slot, int32_t* slot_of_row,
                               int32_t* seg_start, void* workspace, cudaStream_t st);
// `chunks`: 16-byte pieces of a row.
cudaError_t launch_permute_rows(const void* x, const int32_t* row_of_slot, int T, int chunks, int k, void* out,
                                cudaStream_t st);
cudaError_t launch_unpermute(const void* y, const int32_t* row_of_slot, const float* w, int T, int H, int k, bool y32,
                             bool o32, void* out, cudaStream_t st);
cudaError_t launch_unpermute_backward(const void* d_out, const void* y, const int32_t* row_of_slot, const float* w,
                                      int T, int H, int k, bool g32, bool y32, void* d_y, float* d_w, cudaStream_t st);

}  // namespace kmoe
