// LayerNorm for training and serving in fp16, bf16 and fp32, any width up to
// 131072 and any row stride: the forward pass with the residual sum and the
// row statistics saved, and the backward pass with the weights' gradients.
//
//   s = x + res;  mean, var over the row (biased);  rstd = 1/sqrt(var + eps)
//   y = (s - mean)*rstd*gamma + beta
// With xh = (s - mean)*rstd and w = dy*gamma:
//   dx = rstd*(w - mean(w) - xh*mean(w*xh)) + dres
//   dgamma = sum over rows of dy*xh,  dbeta = sum over rows of dy
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "train_internal.h"

namespace tf {
namespace {

__device__ __forceinline__ float widen(float a) { return a; }
__device__ __forceinline__ float widen(__half a) { return __half2float(a); }
__device__ __forceinline__ float widen(__nv_bfloat16 a) { return __bfloat162float(a); }
__device__ __forceinline__ void put(float *p, float a) { *p = a; }
__device__ __forceinline__ void put(__half *p, float a) { *p = __float2half_rn(a); }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float a) { *p = __float2bfloat16_rn(a); }

constexpr int kThreads = 256;

// Sum over the CTA, returned to every thread.
__device__ __forceinline__ float cta_sum(float v, float *red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    cta_sync();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    cta_sync();
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) t += red[i];
    return t;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_forward_kernel(const NormArgs a)
{
    pdl_begin();
    __shared__ float red[kThreads / 32];
    const T *x0 = reinterpret_cast<const T *>(a.x), *r0 = reinterpret_cast<const T *>(a.res);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = x0 + row * a.x_stride;
        const T *r = r0 ? r0 + row * a.res_stride : nullptr;
        auto value = [&](int c) { return r ? widen(x[c]) + widen(r[c]) : widen(x[c]); };
        float sum = 0.0f;
        for (int c = threadIdx.x; c < a.hidden; c += kThreads) sum += value(c);
        const float mean = cta_sum(sum, red) / (float)a.hidden;
        float sq = 0.0f;
        for (int c = threadIdx.x; c < a.hidden; c += kThreads) {
            const float d = value(c) - mean;
            sq = fmaf(d, d, sq);
        }
        const float rstd = 1.0f / sqrtf(cta_sum(sq, red) / (float)a.hidden + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        for (int c = threadIdx.x; c < a.hidden; c += kThreads) {
            const float s = value(c), n = (s - mean) * rstd;
            put(reinterpret_cast<T *>(a.y) + row * a.y_stride + c,
                fmaf(n, a.gamma ? a.gamma[c] : 1.0f, a.beta ? a.beta[c] : 0.0f));
            if (a.sum) put(reinterpret_cast<T *>(a.sum) + row * a.sum_stride + c, s);
        }
    }
}

// CTA p takes rows p, p + gridDim.x, ...; its column sums of dy*xh and dy go
// to row p of the workspace's two [gridDim.x][hidden] arrays.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_backward_kernel(const NormGradArgs a)
{
    pdl_begin();
    __shared__ float red[kThreads / 32];
    float *pg = a.ws ? a.ws + (int64_t)blockIdx.x * a.hidden : nullptr;
    float *pb = a.ws ? pg + (int64_t)gridDim.x * a.hidden : nullptr;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = reinterpret_cast<const T *>(a.x) + row * a.x_stride;
        const T *dy = reinterpret_cast<const T *>(a.dy) + row * a.dy_stride;
        const T *dr = a.dres ? reinterpret_cast<const T *>(a.dres) + row * a.dres_stride : nullptr;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float c1 = 0.0f, c2 = 0.0f;
        for (int c = threadIdx.x; c < a.hidden; c += kThreads) {
            const float xh = (widen(x[c]) - mean) * rstd, g = widen(dy[c]), w = a.gamma ? g * a.gamma[c] : g;
            c1 += w;
            c2 = fmaf(w, xh, c2);
            if (pg) {
                pg[c] = row == blockIdx.x ? g * xh : fmaf(g, xh, pg[c]);
                pb[c] = row == blockIdx.x ? g : pb[c] + g;
            }
        }
        c1 = cta_sum(c1, red) / (float)a.hidden;
        c2 = cta_sum(c2, red) / (float)a.hidden;
        for (int c = threadIdx.x; c < a.hidden; c += kThreads) {
            const float xh = (widen(x[c]) - mean) * rstd, g = widen(dy[c]), w = a.gamma ? g * a.gamma[c] : g;
            float d = rstd * (w - c1 - xh * c2);
            if (dr) d += widen(dr[c]);
            put(reinterpret_cast<T *>(a.dx) + row * a.dx_stride + c, d);
        }
    }
}

// dgamma and dbeta: the partial sums of a column, added in order.
__global__ void __launch_bounds__(kThreads) norm_weight_grad_kernel(const NormGradArgs a, int parts)
{
    pdl_begin();
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= a.hidden) return;
    float g = 0.0f, b = 0.0f;
    for (int p = 0; p < parts; ++p) {
        g += a.ws[(int64_t)p * a.hidden + c];
        b += a.ws[(int64_t)(parts + p) * a.hidden + c];
    }
    if (a.dgamma) a.dgamma[c] = a.accumulate ? a.dgamma[c] + g : g;
    if (a.dbeta) a.dbeta[c] = a.accumulate ? a.dbeta[c] + b : b;
}

int parts_for(int64_t rows)
{
    const int64_t most = 2 * (int64_t)sm_count();
    return (int)(rows < most ? rows : most);
}

}  // namespace

cudaError_t launch_layernorm_forward(const NormArgs &a, cudaStream_t st)
{
    const int64_t most = 8 * (int64_t)sm_count();
    const dim3 grid((unsigned)(a.rows < most ? a.rows : most));
    if (a.dtype == TF_FP32) return launch_pdl(norm_forward_kernel<float>, grid, dim3(kThreads), 0, st, a);
    if (a.dtype == TF_BF16) return launch_pdl(norm_forward_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, a);
    return launch_pdl(norm_forward_kernel<__half>, grid, dim3(kThreads), 0, st, a);
}

int64_t layernorm_backward_workspace(int64_t rows, int64_t hidden, int dtype)
{
    return (int64_t)parts_for(rows) * hidden * 2 * 4;
}

cudaError_t launch_layernorm_backward(const NormGradArgs &a, cudaStream_t st)
{
    const int parts = parts_for(a.rows);
    cudaError_t e = cudaSuccess;
    if (a.rows > 0) {
        const dim3 grid((unsigned)parts);
        if (a.dtype == TF_FP32)
            e = launch_pdl(norm_backward_kernel<float>, grid, dim3(kThreads), 0, st, a);
        else if (a.dtype == TF_BF16)
            e = launch_pdl(norm_backward_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, a);
        else
            e = launch_pdl(norm_backward_kernel<__half>, grid, dim3(kThreads), 0, st, a);
    }
    if (e != cudaSuccess || (!a.dgamma && !a.dbeta)) return e;
    return launch_pdl(norm_weight_grad_kernel, dim3((unsigned)((a.hidden + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                      st, a, parts);
}

}  // namespace tf
