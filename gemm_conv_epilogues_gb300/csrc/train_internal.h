// Internal declarations of the layer-norm (forward with statistics, backward)
// and grouped-product kernels: what their entry points pass to the launchers.
#pragma once

#include "tf_internal.h"

namespace tf {

// LayerNorm with saved statistics, and its backward pass (tf_layernorm_forward,
// tf_layernorm_backward); strides in elements, optional pointers may be null.
struct NormArgs {
    const void *x, *res;
    const float *gamma, *beta;
    void *y, *sum;
    float *mean, *rstd;
    int64_t x_stride, res_stride, y_stride, sum_stride, rows;
    int hidden, dtype;
    float eps;
};
struct NormGradArgs {
    const void *dy, *x, *dres;
    const float *gamma, *mean, *rstd;
    void *dx;
    float *dgamma, *dbeta, *ws;   // ws is null when neither weight gradient is wanted
    int64_t dy_stride, x_stride, dres_stride, dx_stride, rows;
    int hidden, dtype, accumulate;
};
cudaError_t launch_layernorm_forward(const NormArgs &a, cudaStream_t st);
int64_t layernorm_backward_workspace(int64_t rows, int64_t hidden, int dtype);
cudaError_t launch_layernorm_backward(const NormGradArgs &a, cudaStream_t st);

// Grouped products (tf_grouped_matmul and its two gradients).
enum { GROUPED_FORWARD = 0, GROUPED_DGRAD = 1, GROUPED_WGRAD = 2 };
struct GroupedArgs {
    const void *x, *dy, *w;       // FORWARD: x, w; DGRAD: dy, w; WGRAD: dy, x
    const float *bias;
    const int *offsets;
    void *y, *pre;                // outputs of FORWARD; DGRAD writes y (dx) and reads pre
    float *dw, *dbias, *ws;
    int64_t x_stride, dy_stride, y_stride, pre_stride, ws_bytes;
    int rows, groups, N, K, act, dtype, accumulate;
};
// 32-bit tile counts and row indices (rows + one tile stay below 2^31)
constexpr int64_t kGroupedMaxGroups = 1024, kGroupedMaxWidth = 65536, kGroupedMaxRows = (int64_t)1 << 22;
cudaError_t launch_grouped_unaligned(const GroupedArgs &a, int mode, cudaStream_t st);
cudaError_t launch_grouped_bias_grad(const GroupedArgs &a, cudaStream_t st);
cudaError_t launch_grouped(const GroupedArgs &a, int mode, cudaStream_t st);
int64_t grouped_wgrad_workspace(int64_t rows, int groups, int64_t N, int64_t K, int dtype);

}  // namespace tf
