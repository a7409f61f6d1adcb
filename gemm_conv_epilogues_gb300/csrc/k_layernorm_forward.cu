// LayerNorm's forward pass for training and serving, fp16, bf16 and fp32, any
// width up to 131072 and any row stride, one pass over HBM:
//   s = x + res;  mean, biased var of the row;  rstd = 1/sqrt(var + eps)
//   y = (s - mean)*rstd*gamma + beta;  s, mean and rstd saved on request
// Bound by HBM: x, res, y and s once each.  The statistics come from the fp32
// values in registers, the deviations in a second pass over them, so a mean
// far from zero costs no digits of the variance.
#include "norm_rows.cuh"

namespace tf {
namespace {

using namespace norm;

template <typename T, bool ALIGNED, bool CLUSTER, int NT>
__global__ void __launch_bounds__(kMaxThreads)
    norm_forward_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ Sources src,
                        const __grid_constant__ Geometry g, uint32_t *err, uint64_t wait_ns)
{
    pdl_begin();
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float2 red[2][kMaxThreads / 32];
    __shared__ __align__(8) float2 slot[2][kMaxRanks];
    __shared__ __align__(8) uint64_t xbar[2];
    const uint32_t rank = CLUSTER ? ptx::cluster_ctarank() : 0u;
    const int gt = threadIdx.x % g.group, c0 = (int)rank * g.slice;
    auto ring = start_ring<T, ALIGNED, CLUSTER, NT>(g, smem, src, a.hidden, a.rows, blockIdx.x / g.csize,
                                                    gridDim.x / g.csize, c0, err, wait_ns, xbar);
    Exchange xch = {slot, xbar, rank, (uint32_t)g.csize, wait_ns, err, false};
    const int width = ring.width;

    float ga[kCols], be[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
        const int c = col_of<T, ALIGNED>(j, gt, g.group);
        ga[j] = a.gamma && c < width ? __ldg(a.gamma + c0 + c) : 1.0f;
        be[j] = a.beta && c < width ? __ldg(a.beta + c0 + c) : 0.0f;
    }
    const float inv_h = 1.0f / (float)a.hidden, inv_w = 1.0f / (float)width;
    const int lane = threadIdx.x & 31;
    const float n_l = CLUSTER && lane < g.csize ? (float)min(a.hidden - lane * g.slice, g.slice) : 0.0f;
    const float inv_n_l = CLUSTER && lane < g.csize ? 1.0f / n_l : 0.0f;

    Edge ex = load_edge(ring, 0, ring.first, gt, g.group), er = {0.0f, 0.0f};
    if (NT > 1) er = load_edge(ring, 1, ring.first, gt, g.group);
    int it = 0;
    for (int64_t row = ring.first; row < a.rows; row += ring.step, ++it) {
        float s[kCols];
        ring.wait(it);
        load_cols(ring, 0, it, gt, g.group, ex, s);
        if (NT > 1) {
            float r[kCols];
            load_cols(ring, 1, it, gt, g.group, er, r);
#pragma unroll
            for (int j = 0; j < kCols; ++j) s[j] += r[j];
        }
        ex = load_edge(ring, 0, row + ring.step, gt, g.group);
        if (NT > 1) er = load_edge(ring, 1, row + ring.step, gt, g.group);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < kCols; ++j) sum += s[j];
        const float total = group_sum(sum, 0.0f, g.group, red[0]).x;
        if (gt == 0) {   // every thread of the group holds its columns: the stage takes a later row
            ptx::fence_proxy_async_smem();
            ring.issue(it + g.stages);
        }
        const float centre = total * (CLUSTER ? inv_w : inv_h);   // of the slice, in a cluster
        float sq = 0.0f;
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            const float d = s[j] - centre;
            if (col_of<T, ALIGNED>(j, gt, g.group) < width) sq = fmaf(d, d, sq);
        }
        float m2 = group_sum(sq, 0.0f, g.group, red[1]).x, mean = centre;
        if constexpr (CLUSTER) {
            // the slices' (sum, M2) pairs merged pairwise (Chan et al.): M2 = sum M2_r + sum n_r (mean_r - mean)^2,
            // lane r of every warp taking rank r's terms
            const float2 *pairs = xch.swap(make_float2(total, m2), it);
            const float2 pr = lane < g.csize ? pairs[lane] : make_float2(0.0f, 0.0f);
            float t = pr.x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            mean = t * inv_h;
            const float d = pr.x * inv_n_l - mean;
            m2 = lane < g.csize ? fmaf(n_l * d, d, pr.y) : 0.0f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m2 += __shfl_xor_sync(0xffffffffu, m2, o);
        }
        const float rstd = rsqrtf(m2 * inv_h + a.eps);
        if (gt == 0 && rank == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        if (a.sum) store_cols<T, ALIGNED>(reinterpret_cast<T *>(a.sum) + row * a.sum_stride + c0, width, gt, g.group, s);
#pragma unroll
        for (int j = 0; j < kCols; ++j) s[j] = fmaf((s[j] - mean) * rstd, ga[j], be[j]);
        store_cols<T, ALIGNED>(reinterpret_cast<T *>(a.y) + row * a.y_stride + c0, width, gt, g.group, s);
    }
    if (gt == 0) ring.drain();
    if constexpr (CLUSTER) ptx::cluster_sync();   // no CTA leaves while a peer's push to it may be in flight
}

template <typename T>
cudaError_t launch_typed(const NormArgs &a, cudaStream_t st)
{
    constexpr int size = (int)sizeof(T);
    uint32_t *err = device_error_word();
    if (!err) return cudaErrorInitializationError;
    const bool aligned = a.hidden * size % 16 == 0 && aligned_rows(a.x, a.x_stride, size) &&
                         aligned_rows(a.res, a.res_stride, size) && aligned_rows(a.y, a.y_stride, size) &&
                         aligned_rows(a.sum, a.sum_stride, size);
    const Sources src = {{a.x, a.res}, {a.x_stride, a.res_stride}};
    const Geometry g = geometry(a.hidden, size, aligned, a.res ? 2 : 1);
    auto pick = [&](auto nt) {
        constexpr int NT = decltype(nt)::value;
        return g.csize > 1
                   ? (aligned ? norm_forward_kernel<T, true, true, NT> : norm_forward_kernel<T, false, true, NT>)
                   : (aligned ? norm_forward_kernel<T, true, false, NT> : norm_forward_kernel<T, false, false, NT>);
    };
    return launch_rows(a.res ? pick(std::integral_constant<int, 2>()) : pick(std::integral_constant<int, 1>()), g,
                       launch_units(g, a.rows), st, a, src, g, err, wait_limit_ns());
}

}  // namespace

cudaError_t launch_layernorm_forward(const NormArgs &a, cudaStream_t st)
{
    if (a.dtype == TF_FP32) return launch_typed<float>(a, st);
    return a.dtype == TF_BF16 ? launch_typed<__nv_bfloat16>(a, st) : launch_typed<__half>(a, st);
}

}  // namespace tf
