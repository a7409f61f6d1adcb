// C entry points of the embedding, its gradient, and the cross entropy over a
// vocabulary with its gradients: argument checks and launch.  Every check runs
// on the host before anything is launched.
#include <cuda_runtime.h>

#include "lm_internal.h"

using namespace tf;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30;           // 32-bit row numbers in the sorted keys
constexpr int64_t kMaxWords = ((int64_t)1 << 31) - 2;    // 32-bit words there, the last one for none

bool aligned_to(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
size_t element_size(int dtype) { return dtype == TF_FP32 ? 4 : 2; }
bool bad_dtype(int dtype) { return dtype < TF_FP16 || dtype > TF_FP32; }
bool bad_index(int index) { return index != TF_INT32 && index != TF_INT64; }
size_t index_size(int index) { return index == TF_INT64 ? 8 : 4; }
// A [rows][cols] operand: present, with rows that do not overlap; with no rows nothing is touched.
bool bad_matrix(const void *p, int64_t stride, int64_t rows, int64_t cols) { return rows > 0 && (!p || stride < cols); }
bool long_stride(int64_t stride) { return stride > ((int64_t)1 << 31); }

int from_cuda(cudaError_t e)
{
    if (e == cudaSuccess) return TF_OK;
    if (e == cudaErrorNotSupported) {
        cudaGetLastError();
        return TF_ERR_UNSUPPORTED;
    }
    return TF_ERR_CUDA;
}

bool finite(float f) { return f - f == 0.0f; }

}  // namespace

extern "C" {

int tf_embedding_forward(const void *tokens, int index, const void *table, void *y, int64_t y_stride, int64_t rows,
                         int64_t vocab, int64_t hidden, float scale, int64_t padding, int dtype, tf_stream_t stream)
{
    if (rows < 0 || vocab <= 0 || hidden <= 0 || bad_dtype(dtype) || bad_index(index) || !finite(scale) ||
        (rows > 0 && (!tokens || !table)) || bad_matrix(y, y_stride, rows, hidden))
        return TF_ERR_INVALID_ARG;
    const size_t es = element_size(dtype);
    if (rows > kMaxRows || vocab > kMaxWords || hidden > kClusterMaxHidden || long_stride(y_stride) ||
        !aligned_to(tokens, index_size(index)) || !aligned_to(table, es) || !aligned_to(y, es))
        return TF_ERR_UNSUPPORTED;
    if (rows == 0) return TF_OK;
    EmbedArgs a = {};
    a.tokens = {tokens, index == TF_INT64}; a.table = table; a.y = y; a.y_stride = y_stride;
    a.rows = rows; a.vocab = vocab; a.hidden = (int)hidden; a.scale = scale; a.padding = padding; a.dtype = dtype;
    a.err = device_error_word();
    return a.err ? from_cuda(launch_embedding_forward(a, (cudaStream_t)stream)) : TF_ERR_CUDA;
}

int64_t tf_embedding_backward_workspace_size(int64_t rows, int64_t vocab, int64_t hidden)
{
    if (rows < 0 || rows > kMaxRows || vocab <= 0 || vocab > kMaxWords || hidden <= 0 || hidden > kClusterMaxHidden) return 0;
    return embedding_backward_workspace(rows, vocab, hidden);
}

int tf_embedding_backward(const void *dy, int64_t dy_stride, const void *tokens, int index, float *dtable, int64_t rows,
                          int64_t vocab, int64_t hidden, float scale, int64_t padding, int accumulate, int dtype,
                          void *workspace, int64_t workspace_bytes, tf_stream_t stream)
{
    if (rows < 0 || vocab <= 0 || hidden <= 0 || bad_dtype(dtype) || bad_index(index) || !finite(scale) || !dtable ||
        (rows > 0 && !tokens) || bad_matrix(dy, dy_stride, rows, hidden))
        return TF_ERR_INVALID_ARG;
    const size_t es = element_size(dtype);
    if (rows > kMaxRows || vocab > kMaxWords || hidden > kClusterMaxHidden || long_stride(dy_stride) ||
        !aligned_to(tokens, index_size(index)) || !aligned_to(dy, es) || !aligned_to(dtable, 4))
        return TF_ERR_UNSUPPORTED;
    if (rows == 0 && accumulate) return TF_OK;
    const int64_t need = embedding_backward_workspace(rows, vocab, hidden);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return TF_ERR_INVALID_ARG;
        if (!aligned_to(workspace, 16)) return TF_ERR_UNSUPPORTED;
    }
    EmbedArgs a = {};
    a.tokens = {tokens, index == TF_INT64}; a.dy = dy; a.dy_stride = dy_stride; a.dtable = dtable; a.ws = workspace;
    a.rows = rows; a.vocab = vocab; a.hidden = (int)hidden; a.scale = scale; a.padding = padding;
    a.accumulate = accumulate; a.dtype = dtype;
    a.err = device_error_word();
    return a.err ? from_cuda(launch_embedding_backward(a, (cudaStream_t)stream)) : TF_ERR_CUDA;
}

// ---------------------------------------------------------------- linear cross entropy

namespace {

// Sizes shared by the two passes.
int check_lce(const void *w, const void *targets, int index, int64_t rows, int64_t vocab, int64_t hidden, float scale,
              int dtype)
{
    if (rows < 0 || vocab <= 0 || hidden <= 0 || !w || (rows > 0 && !targets) || bad_dtype(dtype) || bad_index(index) ||
        !finite(scale * kLog2e) || !(scale > 0.0f))
        return TF_ERR_INVALID_ARG;
    if (dtype == TF_FP32 || rows > kLceMaxRows || vocab > kLceMaxVocab || hidden > kLceMaxHidden ||
        !aligned_to(w, hidden % 8 == 0 ? 16 : 2) || !aligned_to(targets, index_size(index)))
        return TF_ERR_UNSUPPORTED;
    return TF_OK;
}

int64_t lce_size(bool backward, int64_t rows, int64_t vocab, int64_t hidden, int dtype)
{
    const uint64_t one = 0;
    alignas(16) static const char word[16] = {};
    if (check_lce(word, &one, TF_INT64, rows, vocab, hidden, 1.0f, dtype) != TF_OK) return 0;
    return lce_workspace(backward, rows, vocab, hidden);
}

int check_workspace(const void *ws, int64_t bytes, int64_t need)
{
    if (!ws || bytes < need) return TF_ERR_INVALID_ARG;
    return aligned_to(ws, 16) ? TF_OK : TF_ERR_UNSUPPORTED;
}

}  // namespace

int64_t tf_linear_cross_entropy_forward_workspace_size(int64_t rows, int64_t vocab, int64_t hidden, int dtype)
{
    return lce_size(false, rows, vocab, hidden, dtype);
}

int tf_linear_cross_entropy_forward(const void *x, int64_t x_stride, const void *w, const void *targets, int index,
                                    float *loss, float *lse, int64_t rows, int64_t vocab, int64_t hidden, float scale,
                                    int64_t ignore, int dtype, void *workspace, int64_t workspace_bytes,
                                    tf_stream_t stream)
{
    const int rc = check_lce(w, targets, index, rows, vocab, hidden, scale, dtype);
    if (rc == TF_ERR_INVALID_ARG || bad_matrix(x, x_stride, rows, hidden) || (rows > 0 && (!loss || !lse)))
        return TF_ERR_INVALID_ARG;
    if (rc != TF_OK || long_stride(x_stride) || !aligned_to(x, 2) || !aligned_to(loss, 4) || !aligned_to(lse, 4))
        return TF_ERR_UNSUPPORTED;
    if (rows == 0) return TF_OK;
    if (const int ws = check_workspace(workspace, workspace_bytes, lce_workspace(false, rows, vocab, hidden))) return ws;
    LceArgs a = {};
    a.targets = {targets, index == TF_INT64}; a.x = x; a.w = w; a.loss = loss; a.lse = lse; a.ws = workspace;
    a.x_stride = x_stride; a.rows = rows; a.vocab = vocab; a.ignore = ignore; a.hidden = (int)hidden;
    a.dtype = dtype; a.scale = scale;
    a.err = device_error_word();
    return a.err ? from_cuda(launch_lce_forward(a, (cudaStream_t)stream)) : TF_ERR_CUDA;
}

int64_t tf_linear_cross_entropy_backward_workspace_size(int64_t rows, int64_t vocab, int64_t hidden, int dtype)
{
    return lce_size(true, rows, vocab, hidden, dtype);
}

int tf_linear_cross_entropy_backward(const void *x, int64_t x_stride, const void *w, const void *targets, int index,
                                     const float *lse, const float *dloss, const float *dlse, void *dx,
                                     int64_t dx_stride, void *dw, int64_t rows, int64_t vocab, int64_t hidden,
                                     float scale, int64_t ignore, int accumulate, int dw_dtype, int dtype,
                                     void *workspace, int64_t workspace_bytes, tf_stream_t stream)
{
    const int rc = check_lce(w, targets, index, rows, vocab, hidden, scale, dtype);
    if (rc == TF_ERR_INVALID_ARG || bad_matrix(x, x_stride, rows, hidden) || (rows > 0 && !lse) ||
        (dx && dx_stride < hidden) || (!dx && !dw) || bad_dtype(dw_dtype))
        return TF_ERR_INVALID_ARG;
    const bool f32 = dw_dtype == TF_FP32;
    if (rc != TF_OK || long_stride(x_stride) || (dx && long_stride(dx_stride)) || !aligned_to(x, 2) || !aligned_to(lse, 4) ||
        !aligned_to(dloss, 4) || !aligned_to(dlse, 4) || !aligned_to(dx, 2) || !aligned_to(dw, f32 ? 4 : 2) ||
        (dw && ((!f32 && dw_dtype != dtype) || (accumulate && !f32))))
        return TF_ERR_UNSUPPORTED;
    if (rows == 0 && (!dw || accumulate)) return TF_OK;
    if (const int ws = check_workspace(workspace, workspace_bytes, lce_workspace(true, rows, vocab, hidden))) return ws;
    LceArgs a = {};
    a.targets = {targets, index == TF_INT64}; a.x = x; a.w = w; a.lse = const_cast<float *>(lse);
    a.dloss = dloss; a.dlse = dlse; a.dx = rows > 0 ? dx : nullptr; a.dw = dw; a.ws = workspace;
    a.x_stride = x_stride; a.dx_stride = dx_stride; a.rows = rows; a.vocab = vocab; a.ignore = ignore;
    a.hidden = (int)hidden; a.dtype = dtype; a.dw_dtype = dw_dtype; a.accumulate = accumulate; a.scale = scale;
    a.err = device_error_word();
    return a.err ? from_cuda(launch_lce_backward(a, (cudaStream_t)stream)) : TF_ERR_CUDA;
}

}  // extern "C"
