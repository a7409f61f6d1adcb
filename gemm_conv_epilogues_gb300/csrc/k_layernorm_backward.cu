// LayerNorm's backward pass, fp16, bf16 and fp32, any width up to 131072 and
// any row stride.  With xh = (x - mean)*rstd and w = dy*gamma:
//   dx = rstd*(w - mean_row(w) - xh*mean_row(w*xh)) + dres
//   dgamma = sum over rows of dy*xh,  dbeta = sum over rows of dy
// One pass over HBM: dy, x (and dres) read once, dx written once.  A thread
// keeps its columns' dgamma and dbeta in fp32 registers over all the rows its
// CTA takes; a CTA's sums go to the workspace and a second, small kernel adds
// them in order, so that equal calls give equal bits (no atomics).
#include "norm_rows.cuh"

namespace tf {
namespace {

using namespace norm;

template <typename T, bool ALIGNED, bool CLUSTER, int NT>
__global__ void __launch_bounds__(kMaxThreads)
    norm_backward_kernel(const __grid_constant__ NormGradArgs a, const __grid_constant__ Sources src,
                         const __grid_constant__ Geometry g, uint32_t *err, uint64_t wait_ns)
{
    pdl_begin();
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float2 red[2][kMaxThreads / 32];
    __shared__ __align__(8) float2 slot[2][kMaxRanks];
    __shared__ __align__(8) uint64_t xbar[2];
    const uint32_t rank = CLUSTER ? ptx::cluster_ctarank() : 0u;
    const int gt = threadIdx.x % g.group, c0 = (int)rank * g.slice;
    const int64_t unit = blockIdx.x / g.csize;
    auto ring = start_ring<T, ALIGNED, CLUSTER, NT>(g, smem, src, a.hidden, a.rows, unit, gridDim.x / g.csize, c0, err,
                                                    wait_ns, xbar);
    Exchange xch = {slot, xbar, rank, (uint32_t)g.csize, wait_ns, err, false};
    const int width = ring.width;

    float ga[kCols], dg[kCols], db[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
        const int c = col_of<T, ALIGNED>(j, gt, g.group);
        ga[j] = a.gamma && c < width ? __ldg(a.gamma + c0 + c) : 1.0f;
        dg[j] = db[j] = 0.0f;
    }
    const float inv_h = 1.0f / (float)a.hidden;
    Edge ed = load_edge(ring, 0, ring.first, gt, g.group), ex = load_edge(ring, 1, ring.first, gt, g.group);
    Edge er = {0.0f, 0.0f};
    if (NT > 2) er = load_edge(ring, 2, ring.first, gt, g.group);
    // the row statistics, one row ahead
    float mean = 0.0f, rstd = 0.0f;
    if (ring.first < a.rows) {
        mean = __ldg(a.mean + ring.first);
        rstd = __ldg(a.rstd + ring.first);
    }
    int it = 0;
    for (int64_t row = ring.first; row < a.rows; row += ring.step, ++it) {
        float d[kCols], xh[kCols];
        Held<T, ALIGNED> dr;
        ring.wait(it);
        load_cols(ring, 0, it, gt, g.group, ed, d);
        load_cols(ring, 1, it, gt, g.group, ex, xh);
        if (NT > 2) hold_cols(ring, 2, it, gt, g.group, er, dr);
        const int64_t next = row + ring.step;
        ed = load_edge(ring, 0, next, gt, g.group);
        ex = load_edge(ring, 1, next, gt, g.group);
        if (NT > 2) er = load_edge(ring, 2, next, gt, g.group);
        const float shift = -mean * rstd, scale = rstd;
        if (next < a.rows) {
            mean = __ldg(a.mean + next);
            rstd = __ldg(a.rstd + next);
        }
        float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
        for (int j = 0; j < kCols; ++j) {   // past the slice dy is zero and adds nothing
            xh[j] = fmaf(xh[j], scale, shift);
            dg[j] = fmaf(d[j], xh[j], dg[j]);
            db[j] += d[j];
            d[j] *= ga[j];
            c1 += d[j];
            c2 = fmaf(d[j], xh[j], c2);
        }
        float2 c = group_sum(c1, c2, g.group, red[it & 1]);
        if (gt == 0) {   // every thread of the group holds its columns: the stage takes a later row
            ptx::fence_proxy_async_smem();
            ring.issue(it + g.stages);
        }
        if constexpr (CLUSTER) {
            const float2 *pairs = xch.swap(c, it);
            c = make_float2(0.0f, 0.0f);
            for (int r = 0; r < g.csize; ++r) {
                c.x += pairs[r].x;
                c.y += pairs[r].y;
            }
        }
        const float k1 = -c.x * inv_h * scale, k2 = -c.y * inv_h * scale;
#pragma unroll
        for (int j = 0; j < kCols; ++j) d[j] = fmaf(d[j], scale, fmaf(xh[j], k2, k1));
        if (NT > 2) add_held(dr, d);
        store_cols<T, ALIGNED>(reinterpret_cast<T *>(a.dx) + row * a.dx_stride + c0, width, gt, g.group, d);
    }
    if (gt == 0) ring.drain();

    if (a.ws) {
        // this CTA's sums: row `unit` of dgamma's and of dbeta's [units][hidden] array
        float *wg = a.ws + unit * a.hidden + c0, *wb = wg + (int64_t)(gridDim.x / g.csize) * a.hidden;
        if (g.group < g.threads) {   // eight warps with rows of their own: added in order in shared memory
            float *acc = reinterpret_cast<float *>(smem);
            for (int w = 0; w < g.threads / g.group; ++w) {
                cta_sync();   // every warp is done with its ring, and with the previous warp's turn
                if ((int)threadIdx.x / g.group != w) continue;
#pragma unroll
                for (int j = 0; j < kCols; ++j) {
                    const int c = col_of<T, ALIGNED>(j, gt, g.group);
                    if (c < width) {
                        acc[c] = w ? acc[c] + dg[j] : dg[j];
                        acc[kWarpCols + c] = w ? acc[kWarpCols + c] + db[j] : db[j];
                    }
                }
            }
            cta_sync();
            for (int c = threadIdx.x; c < width; c += g.threads) {
                wg[c] = acc[c];
                wb[c] = acc[kWarpCols + c];
            }
        } else {
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
                const int c = col_of<T, ALIGNED>(j, gt, g.group);
                if (c < width) {
                    wg[c] = dg[j];
                    wb[c] = db[j];
                }
            }
        }
    }
    if constexpr (CLUSTER) ptx::cluster_sync();
}

// dgamma and dbeta: a column's partial sums, added in an order that depends on
// their number alone: warp w takes parts w, w + 16, ..., then the 16 sums in order.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(kSumWarps * 32) norm_weight_grad_kernel(const NormGradArgs a, int parts)
{
    pdl_begin();
    __shared__ float red[kSumWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const float *src = a.ws + (blockIdx.y ? (int64_t)parts * a.hidden : 0) + c;
    float t = 0.0f;
    if (c < a.hidden) {
        int p = warp;
        for (; p + 3 * kSumWarps < parts; p += 4 * kSumWarps) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = src[(int64_t)(p + i * kSumWarps) * a.hidden];
            t += (v[0] + v[1]) + (v[2] + v[3]);
        }
        for (; p < parts; p += kSumWarps) t += src[(int64_t)p * a.hidden];
    }
    red[warp][lane] = t;
    cta_sync();
    float *out = blockIdx.y ? a.dbeta : a.dgamma;
    if (warp == 0 && c < a.hidden && out) {
        t = 0.0f;
#pragma unroll
        for (int w = 0; w < kSumWarps; ++w) t += red[w][lane];
        out[c] = a.accumulate ? out[c] + t : t;
    }
}

// The widest set of partial sums any alignment of the operands gives.
int64_t most_units(int64_t rows, int64_t hidden, int dtype)
{
    const int size = dtype == TF_FP32 ? 4 : 2;
    int64_t most = 0;
    for (bool aligned : {false, true}) {
        const int64_t u = launch_units(geometry(hidden, size, aligned, 3), rows);
        if (u > most) most = u;
    }
    return most;
}

template <typename T>
cudaError_t launch_typed(const NormGradArgs &a, int64_t *units, cudaStream_t st)
{
    constexpr int size = (int)sizeof(T);
    uint32_t *err = device_error_word();
    if (!err) return cudaErrorInitializationError;
    const bool aligned = a.hidden * size % 16 == 0 && aligned_rows(a.dy, a.dy_stride, size) &&
                         aligned_rows(a.x, a.x_stride, size) && aligned_rows(a.dres, a.dres_stride, size) &&
                         aligned_rows(a.dx, a.dx_stride, size);
    const Sources src = {{a.dy, a.x, a.dres}, {a.dy_stride, a.x_stride, a.dres_stride}};
    const Geometry g = geometry(a.hidden, size, aligned, a.dres ? 3 : 2);
    *units = launch_units(g, a.rows);
    auto pick = [&](auto nt) {
        constexpr int NT = decltype(nt)::value;
        return g.csize > 1
                   ? (aligned ? norm_backward_kernel<T, true, true, NT> : norm_backward_kernel<T, false, true, NT>)
                   : (aligned ? norm_backward_kernel<T, true, false, NT> : norm_backward_kernel<T, false, false, NT>);
    };
    return launch_rows(a.dres ? pick(std::integral_constant<int, 3>()) : pick(std::integral_constant<int, 2>()), g,
                       *units, st, a, src, g, err, wait_limit_ns());
}

}  // namespace

int64_t layernorm_backward_workspace(int64_t rows, int64_t hidden, int dtype)
{
    return rows > 0 ? most_units(rows, hidden, dtype) * hidden * 2 * 4 : 0;
}

cudaError_t launch_layernorm_backward(const NormGradArgs &a, cudaStream_t st)
{
    int64_t units = 0;   // with no rows there are no partial sums, and the gradients become zero
    cudaError_t e = cudaSuccess;
    if (a.rows > 0)
        e = a.dtype == TF_FP32   ? launch_typed<float>(a, &units, st)
            : a.dtype == TF_BF16 ? launch_typed<__nv_bfloat16>(a, &units, st)
                                 : launch_typed<__half>(a, &units, st);
    if (e != cudaSuccess || (!a.dgamma && !a.dbeta)) return e;
    return launch_pdl(norm_weight_grad_kernel, dim3((unsigned)((a.hidden + 31) / 32), 2), dim3(kSumWarps * 32), 0, st, a,
                      (int)units);
}

}  // namespace tf
