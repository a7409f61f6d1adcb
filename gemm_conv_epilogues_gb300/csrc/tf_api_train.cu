// C entry points of the layer norm with saved statistics, its backward pass
// and the grouped products: argument checks and launch.  Every check runs on
// the host before anything is launched.
#include <cuda_runtime.h>

#include "train_internal.h"

using namespace tf;

namespace {

bool aligned_to(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool aligned16(const void *p) { return aligned_to(p, 16); }

int from_cuda(cudaError_t e)
{
    if (e == cudaSuccess) return TF_OK;
    if (e == cudaErrorNotSupported) {
        cudaGetLastError();
        return TF_ERR_UNSUPPORTED;
    }
    return TF_ERR_CUDA;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- layer norm, forward and backward

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30;   // 32-bit row counters, with room for a step past the end

size_t element_size(int dtype) { return dtype == TF_FP32 ? 4 : 2; }
bool bad_dtype(int dtype) { return dtype < TF_FP16 || dtype > TF_FP32; }

// A [rows][cols] operand that the call reads or writes: present, with rows
// that do not overlap.  With no rows nothing is touched and null is fine.
bool bad_matrix(const void *p, int64_t stride, int64_t rows, int64_t cols) { return rows > 0 && (!p || stride < cols); }
bool bad_optional(const void *p, int64_t stride, int64_t cols) { return p && stride < cols; }
// rows*stride stays far inside 64-bit offsets
bool long_stride(int64_t stride) { return stride > ((int64_t)1 << 31); }

}  // namespace

int tf_layernorm_forward(const void *x, int64_t x_stride, const void *res, int64_t res_stride, const float *gamma,
                         const float *beta, void *y, int64_t y_stride, void *sum, int64_t sum_stride, float *mean,
                         float *rstd, int64_t rows, int64_t hidden, float eps, int dtype, tf_stream_t stream)
{
    if (rows < 0 || hidden <= 0 || !(eps >= 0.0f) || bad_dtype(dtype)) return TF_ERR_INVALID_ARG;
    if (bad_matrix(x, x_stride, rows, hidden) || bad_matrix(y, y_stride, rows, hidden) ||
        bad_optional(res, res_stride, hidden) || bad_optional(sum, sum_stride, hidden))
        return TF_ERR_INVALID_ARG;
    if (hidden > kClusterMaxHidden || rows > kMaxRows || long_stride(x_stride) || long_stride(y_stride) ||
        (res && long_stride(res_stride)) || (sum && long_stride(sum_stride)))
        return TF_ERR_UNSUPPORTED;
    const size_t es = element_size(dtype);
    if (!aligned_to(x, es) || !aligned_to(res, es) || !aligned_to(y, es) || !aligned_to(sum, es) ||
        !aligned_to(gamma, 4) || !aligned_to(beta, 4) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return TF_ERR_UNSUPPORTED;
    if (rows == 0) return TF_OK;
    NormArgs a = {};
    a.x = x; a.res = res; a.gamma = gamma; a.beta = beta; a.y = y; a.sum = sum; a.mean = mean; a.rstd = rstd;
    a.x_stride = x_stride; a.res_stride = res_stride; a.y_stride = y_stride; a.sum_stride = sum_stride;
    a.rows = rows; a.hidden = (int)hidden; a.dtype = dtype; a.eps = eps;
    return from_cuda(launch_layernorm_forward(a, (cudaStream_t)stream));
}

int64_t tf_layernorm_backward_workspace_size(int64_t rows, int64_t hidden, int dtype)
{
    if (rows < 0 || rows > kMaxRows || hidden <= 0 || hidden > kClusterMaxHidden || bad_dtype(dtype)) return 0;
    return layernorm_backward_workspace(rows, hidden, dtype);
}

int tf_layernorm_backward(const void *dy, int64_t dy_stride, const void *x, int64_t x_stride, const float *gamma,
                          const float *mean, const float *rstd, const void *dres, int64_t dres_stride, void *dx,
                          int64_t dx_stride, float *dgamma, float *dbeta, int64_t rows, int64_t hidden, int accumulate,
                          int dtype, void *workspace, int64_t workspace_bytes, tf_stream_t stream)
{
    if (rows < 0 || hidden <= 0 || bad_dtype(dtype)) return TF_ERR_INVALID_ARG;
    if (bad_matrix(dy, dy_stride, rows, hidden) || bad_matrix(x, x_stride, rows, hidden) ||
        bad_matrix(dx, dx_stride, rows, hidden) || bad_optional(dres, dres_stride, hidden) ||
        (rows > 0 && (!mean || !rstd)))
        return TF_ERR_INVALID_ARG;
    if (hidden > kClusterMaxHidden || rows > kMaxRows || long_stride(dy_stride) || long_stride(x_stride) ||
        long_stride(dx_stride) || (dres && long_stride(dres_stride)))
        return TF_ERR_UNSUPPORTED;
    const size_t es = element_size(dtype);
    if (!aligned_to(dy, es) || !aligned_to(x, es) || !aligned_to(dx, es) || !aligned_to(dres, es) ||
        !aligned_to(gamma, 4) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(dgamma, 4) ||
        !aligned_to(dbeta, 4))
        return TF_ERR_UNSUPPORTED;
    const bool weights = dgamma || dbeta;
    const int64_t need = weights ? layernorm_backward_workspace(rows, hidden, dtype) : 0;
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return TF_ERR_INVALID_ARG;
        if (!aligned16(workspace)) return TF_ERR_UNSUPPORTED;
    }
    if (rows == 0 && (!weights || accumulate)) return TF_OK;
    NormGradArgs a = {};
    a.dy = dy; a.x = x; a.dres = dres; a.gamma = gamma; a.mean = mean; a.rstd = rstd; a.dx = dx;
    a.dgamma = dgamma; a.dbeta = dbeta; a.ws = weights ? static_cast<float *>(workspace) : nullptr;
    a.dy_stride = dy_stride; a.x_stride = x_stride; a.dres_stride = dres_stride; a.dx_stride = dx_stride;
    a.rows = rows; a.hidden = (int)hidden; a.dtype = dtype; a.accumulate = accumulate;
    return from_cuda(launch_layernorm_backward(a, (cudaStream_t)stream));
}

// ---------------------------------------------------------------- grouped products

namespace {

// Sizes shared by the three products.
int check_grouped(const int *offsets, int64_t rows, int64_t groups, int64_t N, int64_t K, int act, int dtype)
{
    if (rows < 0 || groups <= 0 || N <= 0 || K <= 0 || !offsets || bad_dtype(dtype) || act < TF_ACT_NONE ||
        act > TF_ACT_GELU)
        return TF_ERR_INVALID_ARG;
    if (dtype == TF_FP32 || groups > kGroupedMaxGroups || N > kGroupedMaxWidth || K > kGroupedMaxWidth ||
        rows > kGroupedMaxRows || !aligned_to(offsets, 4))
        return TF_ERR_UNSUPPORTED;
    return TF_OK;
}

}  // namespace

int tf_grouped_matmul(const void *x, int64_t x_stride, const void *w, const float *bias, const int32_t *offsets,
                      void *y, int64_t y_stride, void *pre, int64_t pre_stride, int64_t rows, int64_t groups, int64_t N,
                      int64_t K, int act, int dtype, tf_stream_t stream)
{
    const int rc = check_grouped(offsets, rows, groups, N, K, act, dtype);
    if (rc == TF_ERR_INVALID_ARG || !w || bad_matrix(x, x_stride, rows, K) || bad_matrix(y, y_stride, rows, N) ||
        bad_optional(pre, pre_stride, N))
        return TF_ERR_INVALID_ARG;
    if (rc != TF_OK || long_stride(x_stride) || long_stride(y_stride) || (pre && long_stride(pre_stride)) ||
        !aligned_to(x, 2) || !aligned_to(w, 2) || !aligned_to(y, 2) || !aligned_to(pre, 2) || !aligned_to(bias, 4))
        return TF_ERR_UNSUPPORTED;
    if (rows == 0) return TF_OK;
    GroupedArgs a = {};
    a.x = x; a.w = w; a.bias = bias; a.offsets = offsets; a.y = y; a.pre = pre;
    a.x_stride = x_stride; a.y_stride = y_stride; a.pre_stride = pre_stride;
    a.rows = (int)rows; a.groups = (int)groups; a.N = (int)N; a.K = (int)K; a.act = act; a.dtype = dtype;
    return from_cuda(launch_grouped(a, GROUPED_FORWARD, (cudaStream_t)stream));
}

int tf_grouped_matmul_dgrad(const void *dy, int64_t dy_stride, const void *w, const int32_t *offsets, const void *pre,
                            int64_t pre_stride, void *dx, int64_t dx_stride, int64_t rows, int64_t groups, int64_t N,
                            int64_t K, int act, int dtype, tf_stream_t stream)
{
    const int rc = check_grouped(offsets, rows, groups, N, K, act, dtype);
    if (rc == TF_ERR_INVALID_ARG || !w || bad_matrix(dy, dy_stride, rows, N) || bad_matrix(dx, dx_stride, rows, K) ||
        (act != TF_ACT_NONE && bad_matrix(pre, pre_stride, rows, K)))
        return TF_ERR_INVALID_ARG;
    if (rc != TF_OK || long_stride(dy_stride) || long_stride(dx_stride) ||
        (act != TF_ACT_NONE && long_stride(pre_stride)) || !aligned_to(dy, 2) || !aligned_to(w, 2) ||
        !aligned_to(dx, 2) || !aligned_to(pre, 2))
        return TF_ERR_UNSUPPORTED;
    if (rows == 0) return TF_OK;
    GroupedArgs a = {};
    a.dy = dy; a.w = w; a.offsets = offsets; a.y = dx; a.pre = act == TF_ACT_NONE ? nullptr : const_cast<void *>(pre);
    a.dy_stride = dy_stride; a.y_stride = dx_stride; a.pre_stride = pre_stride;
    a.rows = (int)rows; a.groups = (int)groups; a.N = (int)N; a.K = (int)K; a.act = act; a.dtype = dtype;
    return from_cuda(launch_grouped(a, GROUPED_DGRAD, (cudaStream_t)stream));
}

int64_t tf_grouped_matmul_wgrad_workspace_size(int64_t rows, int64_t groups, int64_t N, int64_t K, int dtype)
{
    int one = 0;
    if (check_grouped(&one, rows, groups, N, K, TF_ACT_NONE, dtype) != TF_OK) return 0;
    return grouped_wgrad_workspace(rows, (int)groups, N, K, dtype);
}

int tf_grouped_matmul_wgrad(const void *dy, int64_t dy_stride, const void *x, int64_t x_stride, const int32_t *offsets,
                            float *dw, float *dbias, int64_t rows, int64_t groups, int64_t N, int64_t K, int accumulate,
                            int dtype, void *workspace, int64_t workspace_bytes, tf_stream_t stream)
{
    const int rc = check_grouped(offsets, rows, groups, N, K, TF_ACT_NONE, dtype);
    if (rc == TF_ERR_INVALID_ARG || !dw || workspace_bytes < 0 || (workspace_bytes > 0 && !workspace) ||
        bad_matrix(dy, dy_stride, rows, N) || bad_matrix(x, x_stride, rows, K))
        return TF_ERR_INVALID_ARG;
    if (rc != TF_OK || long_stride(dy_stride) || long_stride(x_stride) || !aligned_to(dy, 2) || !aligned_to(x, 2) ||
        !aligned_to(dw, 4) || !aligned_to(dbias, 4) || !aligned16(workspace))
        return TF_ERR_UNSUPPORTED;
    GroupedArgs a = {};
    a.dy = dy; a.x = x; a.offsets = offsets; a.dw = dw; a.dbias = dbias;
    a.ws = static_cast<float *>(workspace); a.ws_bytes = workspace ? workspace_bytes : 0;
    a.dy_stride = dy_stride; a.x_stride = x_stride; a.accumulate = accumulate;
    a.rows = (int)rows; a.groups = (int)groups; a.N = (int)N; a.K = (int)K; a.dtype = dtype;
    return from_cuda(launch_grouped(a, GROUPED_WGRAD, (cudaStream_t)stream));
}

}  // extern "C"
