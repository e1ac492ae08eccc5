// moe_sort.cuh -- launchers of the operators that bring a routed layer's tokens into
// the order of their experts and back (moe_sort.cu).
#pragma once

#include "ffn_internal.cuh"

namespace ffn {

size_t moe_sort_workspace(int64_t pairs, int64_t experts);   // never falls as pairs grow
// x rows of row_bytes (a multiple of 16) and, x_scales given, nscales floats each
cudaError_t launch_moe_sort(const void *x, const float *x_scales, const int32_t *idx, void *xs, float *xs_scales,
                            int32_t *pos, int32_t *offsets, int64_t rows, int64_t row_bytes, int64_t nscales,
                            int experts, int k, void *workspace, cudaStream_t s);
// w null: 1; res null: none
cudaError_t launch_moe_unsort(const void *ys, const int32_t *pos, const float *w, const void *res, void *y,
                              int64_t rows, int64_t d, int k, int dt, cudaStream_t s);
cudaError_t launch_moe_unsort_backward(const void *dy, const void *ys, const int32_t *pos, const float *w, void *dys,
                                       float *dw, int64_t rows, int64_t d, int k, int dt, cudaStream_t s);

}  // namespace ffn
