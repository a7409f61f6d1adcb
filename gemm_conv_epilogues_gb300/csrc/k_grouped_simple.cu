// Grouped products on the CUDA cores, for operands that no tensor map can
// address (rows that are not multiples of 16 bytes, or unaligned bases):
//   FORWARD  y[m][n]    = act(sum_k x[m][k] w[e][n][k] + bias[e][n])   for m in group e
//   DGRAD    dx[m][k]   = (sum_n dy[m][n] w[e][n][k]) * act'(pre[m][k])
//   WGRAD    dw[e][n][k] = sum_{m in e} dy[m][n] x[m][k]
// One kernel: a 64 x 64 output tile per CTA, 16 steps of the reduction staged
// in shared memory as fp32 at a time, 4 x 4 fp32 sums per thread.  Loads go
// along whichever index is contiguous.  Bound by the FMA pipe.
#include "grouped.cuh"

namespace tf {
namespace {

using namespace grouped;

constexpr int TM = 64, TN = 64, TK = 16, kThreads = 256;

template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads) grouped_simple_kernel(const GroupedArgs a, uint32_t *err)
{
    pdl_begin();
    __shared__ Schedule sch;
    __shared__ float As[TK][TM + 4], Bs[TK][TN + 4];
    const T *A = reinterpret_cast<const T *>(MODE == GROUPED_FORWARD ? a.x : a.dy);
    const T *B = reinterpret_cast<const T *>(MODE == GROUPED_WGRAD ? a.x : a.w);
    const int64_t lda = MODE == GROUPED_FORWARD ? a.x_stride : a.dy_stride;
    const int outM = MODE == GROUPED_WGRAD ? a.N : 0;
    const int outN = MODE == GROUPED_FORWARD ? a.N : a.K;
    const int ntn = (outN + TN - 1) / TN, ntm = (outM + TM - 1) / TM;
    make_schedule(sch, a.offsets, a.groups, a.rows, MODE == GROUPED_WGRAD ? 1 << 30 : TM, ntn, err);
    if (sch.bad) return;
    const int64_t tiles = MODE == GROUPED_WGRAD ? (int64_t)a.groups * ntm * ntn : sch.tile[a.groups];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;

    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        int e, m0, n0, red;
        if (MODE == GROUPED_WGRAD) {
            e = (int)(t / ((int64_t)ntm * ntn));
            const int r = (int)(t - (int64_t)e * ntm * ntn);
            m0 = r / ntn * TM;
            n0 = r % ntn * TN;
            red = sch.row[e + 1] - sch.row[e];
        } else {
            e = group_of_tile(sch, a.groups, (int)t);
            const int r = (int)t - sch.tile[e];
            m0 = sch.row[e] + r / ntn * TM;
            n0 = r % ntn * TN;
            red = MODE == GROUPED_FORWARD ? a.K : a.N;
        }
        const int mend = MODE == GROUPED_WGRAD ? a.N : sch.row[e + 1];
        const int64_t row0 = sch.row[e];
        const T *We = MODE == GROUPED_WGRAD ? nullptr : B + (int64_t)e * a.N * a.K;
        float acc[4][4] = {};
        for (int k0 = 0; k0 < red; k0 += TK) {
#pragma unroll
            for (int i = 0; i < TM * TK / kThreads; ++i) {
                const int idx = threadIdx.x + i * kThreads;
                // the index that is contiguous in memory runs fastest over the threads
                const int m = MODE == GROUPED_WGRAD ? idx % TM : idx / TK;
                const int k = MODE == GROUPED_WGRAD ? idx / TM : idx % TK;
                float v = 0.0f;
                if (m0 + m < mend && k0 + k < red)
                    v = Half2Of<T>::widen(MODE == GROUPED_WGRAD ? A[(row0 + k0 + k) * lda + m0 + m]
                                                                : A[(int64_t)(m0 + m) * lda + k0 + k]);
                As[k][m] = v;
                const int n = MODE == GROUPED_FORWARD ? idx / TK : idx % TN;
                const int kb = MODE == GROUPED_FORWARD ? idx % TK : idx / TN;
                v = 0.0f;
                if (n0 + n < outN && k0 + kb < red)
                    v = Half2Of<T>::widen(MODE == GROUPED_FORWARD ? We[(int64_t)(n0 + n) * a.K + k0 + kb]
                                          : MODE == GROUPED_DGRAD ? We[(int64_t)(k0 + kb) * a.K + n0 + n]
                                                                  : B[(row0 + k0 + kb) * a.x_stride + n0 + n]);
                Bs[kb][n] = v;
            }
            cta_sync();
#pragma unroll
            for (int k = 0; k < TK; ++k) {
                float av[4], bv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    av[i] = As[k][ty * 4 + i];
                    bv[i] = Bs[k][tx + 16 * i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
            }
            cta_sync();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = m0 + ty * 4 + i;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx + 16 * j;
                if (m >= mend || n >= outN) continue;
                float v = acc[i][j];
                if (MODE == GROUPED_FORWARD) {
                    if (a.bias) v += a.bias[(int64_t)e * a.N + n];
                    if (a.pre) reinterpret_cast<T *>(a.pre)[m * a.pre_stride + n] = Half2Of<T>::round(v);
                    reinterpret_cast<T *>(a.y)[m * a.y_stride + n] = Half2Of<T>::round(act_value(a.act, v));
                } else if (MODE == GROUPED_DGRAD) {
                    if (a.act != TF_ACT_NONE)
                        v *= act_slope(a.act, Half2Of<T>::widen(reinterpret_cast<const T *>(a.pre)[m * a.pre_stride + n]));
                    reinterpret_cast<T *>(a.y)[m * a.y_stride + n] = Half2Of<T>::round(v);
                } else {
                    float *dst = a.dw + ((int64_t)e * a.N + m) * a.K + n;
                    *dst = a.accumulate ? *dst + v : v;
                }
            }
        }
    }
}

// dbias[e][n] = sum of dy[m][n] over group e's rows.  A CTA takes 64 columns of
// one group: VEC columns per thread (8: 16-byte loads), 64/VEC threads side by
// side, the others on rows of their own, four loads each in flight; the CTA's
// partial sums are added in order.  Bound by HBM: dy once.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) grouped_bias_grad_kernel(const GroupedArgs a, uint32_t *err)
{
    pdl_begin();
    constexpr int ACROSS = 64 / VEC, DOWN = 256 / ACROSS;
    __shared__ float red[DOWN][65];
    __shared__ int bad;
    if (threadIdx.x == 0) bad = 0;
    cta_sync();
    for (int i = threadIdx.x; i <= a.groups; i += blockDim.x) {
        const int v = a.offsets[i];
        if (v < 0 || v > a.rows || (i > 0 && a.offsets[i - 1] > v)) bad = 1;
    }
    cta_sync();
    if (bad) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(err, TF_DEVERR_OFFSETS);
        return;
    }
    const int e = blockIdx.y, q = threadIdx.x / ACROSS, c = (int)threadIdx.x % ACROSS * VEC, n = blockIdx.x * 64 + c;
    const int lo = a.offsets[e], hi = a.offsets[e + 1];
    const T *dy = reinterpret_cast<const T *>(a.dy) + n;
    float sum[VEC] = {};
    if (n < a.N)   // (N is a multiple of VEC)
        for (int m = lo + q; m < hi; m += 4 * DOWN) {
            if constexpr (VEC == 8) {
                uint4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = m + i * DOWN < hi ? __ldg(reinterpret_cast<const uint4 *>(dy + (int64_t)(m + i * DOWN) * a.dy_stride))
                                             : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = Half2Of<T>::unpack(w[j]);
                        sum[2 * j] += f.x;
                        sum[2 * j + 1] += f.y;
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (m + i * DOWN < hi) sum[0] += Half2Of<T>::widen(dy[(int64_t)(m + i * DOWN) * a.dy_stride]);
            }
        }
#pragma unroll
    for (int j = 0; j < VEC; ++j) red[q][c + j] = sum[j];
    cta_sync();
    if (threadIdx.x < 64 && blockIdx.x * 64 + threadIdx.x < (unsigned)a.N) {
        float t = 0.0f;
        for (int i = 0; i < DOWN; ++i) t += red[i][threadIdx.x];
        float *dst = a.dbias + (int64_t)e * a.N + blockIdx.x * 64 + threadIdx.x;
        *dst = a.accumulate ? *dst + t : t;
    }
}

template <typename T>
cudaError_t launch_typed(const GroupedArgs &a, int mode, uint32_t *err, cudaStream_t st)
{
    const int outN = mode == GROUPED_FORWARD ? a.N : a.K;
    const int64_t ntn = (outN + TN - 1) / TN;
    const int64_t most = mode == GROUPED_WGRAD ? (int64_t)a.groups * ((a.N + TM - 1) / TM) * ntn
                                               : ((int64_t)a.rows / TM + a.groups) * ntn;
    const unsigned grid = (unsigned)(most < (int64_t)sm_count() * 4 ? most : (int64_t)sm_count() * 4);
    if (mode == GROUPED_FORWARD)
        return launch_pdl(grouped_simple_kernel<T, GROUPED_FORWARD>, dim3(grid), dim3(kThreads), 0, st, a, err);
    if (mode == GROUPED_DGRAD)
        return launch_pdl(grouped_simple_kernel<T, GROUPED_DGRAD>, dim3(grid), dim3(kThreads), 0, st, a, err);
    return launch_pdl(grouped_simple_kernel<T, GROUPED_WGRAD>, dim3(grid), dim3(kThreads), 0, st, a, err);
}

}  // namespace

cudaError_t launch_grouped_simple(const GroupedArgs &a, int mode, cudaStream_t st)
{
    uint32_t *err = device_error_word();
    if (!err) return cudaErrorInitializationError;
    return a.dtype == TF_BF16 ? launch_typed<__nv_bfloat16>(a, mode, err, st) : launch_typed<__half>(a, mode, err, st);
}

cudaError_t launch_grouped_bias_grad(const GroupedArgs &a, cudaStream_t st)
{
    uint32_t *err = device_error_word();
    if (!err) return cudaErrorInitializationError;
    const dim3 grid((unsigned)((a.N + 63) / 64), (unsigned)a.groups);
    const bool vec = a.N % 8 == 0 && a.dy_stride % 8 == 0 && (reinterpret_cast<uintptr_t>(a.dy) & 15u) == 0;
    auto launch = [&](auto kern) { return launch_pdl(kern, grid, dim3(256), 0, st, a, err); };
    if (a.dtype == TF_BF16)
        return vec ? launch(grouped_bias_grad_kernel<__nv_bfloat16, 8>) : launch(grouped_bias_grad_kernel<__nv_bfloat16, 1>);
    return vec ? launch(grouped_bias_grad_kernel<__half, 8>) : launch(grouped_bias_grad_kernel<__half, 1>);
}

}  // namespace tf
