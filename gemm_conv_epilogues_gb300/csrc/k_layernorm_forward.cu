// LayerNorm's forward pass for training and serving, fp16, bf16 and fp32, any
// width up to 131072 and any row stride, one pass over HBM:
//   s = x + res;  mean, biased var of the row;  rstd = 1/sqrt(var + eps)
//   y = (s - mean)*rstd*gamma + beta;  s, mean and rstd saved on request
// Bound by HBM: x, res, y and s once each (16384 x 4096 bf16: 85 us, 6.3 TB/s;
// 50001 x 640 fp16 without residual: 29 us).  The statistics come from the fp32
// values in registers, the deviations in a second pass over them, so a mean
// far from zero costs no digits of the variance.
#include "norm_rows.cuh"

namespace tf {
namespace {

using namespace norm;

// Columns per thread: 16 at 128 registers; 8 at 64 for narrow rows and where they
// are element-wise; 24 for 16-bit rows that then take one warp, with gamma and
// beta in shared memory.  Fewer registers would spill, which costs far more than
// more threads gain: with most of the SM's memory in the rings, the little L1
// left does not hold them.  (Element-wise rows of several CTAs take 16, too, in
// CTAs of 512.)
int cols_of(bool aligned, int size, int64_t hidden)
{
    if (!aligned) return hidden > kSlice ? 16 : 8;
    if (hidden <= 256) return 8;
    return size == 2 && hidden > 512 && hidden <= 768 ? 24 : 16;
}
constexpr int sm_threads(int cols) { return cols == 8 ? 1024 : 512; }

// GROUP: threads per row where the columns are element-wise or pairs (a constant
// makes them immediate offsets), 0 for 16-byte vectors.  SPAN: 0 for at most 256
// threads per row, 1 for up to 512, 2 for a cluster of such CTAs.
template <typename T, int GROUP, int SPAN, int NT, int COLS, int VEC = 16 / (int)sizeof(T)>
__global__ void __launch_bounds__(GROUP > 512 ? 1024 : GROUP > 256 || SPAN > 0 ? 512 : 256,
                                  GROUP > 512   ? 1
                                  : GROUP > 256 ? (COLS == 8 ? 2 : 1)
                                  : GROUP > 0   ? 4
                                  : SPAN > 0    ? 1
                                  : COLS == 8   ? 4
                                                : 2)
    norm_forward_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ Sources src,
                        const __grid_constant__ Geometry g, uint32_t *err, uint64_t wait_ns)
{
    constexpr bool ALIGNED = GROUP == 0, CLUSTER = SPAN == 2;
    static_assert(ALIGNED == kAligned<T, VEC>, "GROUP and VEC");
    using C = Cols<T, VEC, COLS>;
    constexpr int PAIRS = C::PAIRS;
    constexpr bool HELD = COLS <= 16;   // gamma and beta in registers
    pdl_begin();
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float2 red[2][kMaxGroup / 32];
    __shared__ __align__(8) float2 slot[2][kMaxRanks];
    __shared__ __align__(8) uint64_t xbar[2];
    const int rank = CLUSTER ? (int)ptx::cluster_ctarank() : 0;
    const int gsize = ALIGNED ? g.group : GROUP, gt = threadIdx.x % gsize, c0 = rank * g.slice;
    auto ring = start_ring<T, VEC, CLUSTER, NT>(g, smem, src, a.hidden, (int)a.rows, (int)blockIdx.x / g.csize,
                                                    (int)gridDim.x / g.csize, c0, err, wait_ns, xbar);
    Exchange xch = {slot, xbar, (uint32_t)rank, (uint32_t)g.csize, wait_ns, err, false};
    const int width = ring.width;

    float2 ga[HELD ? PAIRS : 1], be[HELD ? PAIRS : 1];
    // [PAIRS][gsize] pairs: the lanes' reads of one lie side by side
    float2 *gs = reinterpret_cast<float2 *>(smem + g.gamma_off), *bs = gs + PAIRS * gsize;
    auto pair_of = [&](const float *v, int p, int l, float none) {
        const int c = C::col(2 * p, l, gsize), d = C::col(2 * p + 1, l, gsize);
        return make_float2(v && c < width ? __ldg(v + c0 + c) : none, v && d < width ? __ldg(v + c0 + d) : none);
    };
    if (HELD) {
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) {
            ga[HELD ? p : 0] = pair_of(a.gamma, p, gt, 1.0f);
            be[HELD ? p : 0] = pair_of(a.beta, p, gt, 0.0f);
        }
    } else {
        for (int i = threadIdx.x; i < PAIRS * gsize; i += (int)blockDim.x) {
            gs[i] = pair_of(a.gamma, i / gsize, i % gsize, 1.0f);
            bs[i] = pair_of(a.beta, i / gsize, i % gsize, 0.0f);
        }
        cta_sync();
    }
    const float inv_h = 1.0f / (float)a.hidden, inv_n = 1.0f / (float)width;

    Edge<T, VEC> ex, er;
    load_edge(ring, 0, ring.first, gt, gsize, ex);
    if (NT > 1) load_edge(ring, 1, ring.first, gt, gsize, er);
    for (int row = ring.first, it = 0; row < ring.rows; row += ring.step, ++it, ring.advance()) {
        float2 s[PAIRS];
        ring.wait();
        put_edge(ring, 0, row, ex);
        if (NT > 1) put_edge(ring, 1, row, er);
        {
            C x, r;
            x.load(ring, 0, row, gt, gsize);
            if (NT > 1) r.load(ring, 1, row, gt, gsize);
#pragma unroll
            for (int p = 0; p < PAIRS; ++p) s[p] = NT > 1 ? fadd2(x.get(p), r.get(p)) : x.get(p);
        }
        load_edge(ring, 0, (int64_t)row + ring.step, gt, gsize, ex);
        if (NT > 1) load_edge(ring, 1, (int64_t)row + ring.step, gt, gsize, er);
        float2 sum = s[0];
#pragma unroll
        for (int p = 1; p < PAIRS; ++p) sum = fadd2(sum, s[p]);
        const float total = group_sum<false>(sum.x + sum.y, gsize, red[0]);
        if (gt == 0) ring.refill(row);   // every thread of the group holds its columns
        float mean = total * (CLUSTER ? inv_n : inv_h);   // of the slice, in a cluster
        float2 sq = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) {
            float2 d = fsub2(s[p], make_float2(mean, mean));
            if (!C::inside(2 * p, gt, gsize, width)) d.x = 0.0f;
            if (!C::inside(2 * p + 1, gt, gsize, width)) d.y = 0.0f;
            sq = ffma2(d, d, sq);
        }
        float m2 = group_sum<false>(sq.x + sq.y, gsize, red[1]);
        if constexpr (CLUSTER) {
            // the slices' (sum, M2) pairs merged pairwise (Chan et al.): M2 = sum M2_r + sum n_r (mean_r - mean)^2,
            // lane r of every warp taking rank r's terms
            const int lane = threadIdx.x & 31;
            const float n_l = lane < g.csize ? (float)min(a.hidden - lane * g.slice, g.slice) : 0.0f;
            const float2 *pairs = xch.swap(make_float2(total, m2), it);
            const float2 pr = lane < g.csize ? pairs[lane] : make_float2(0.0f, 0.0f);
            mean = warp_sum(pr.x) * inv_h;
            const float d = lane < g.csize ? pr.x / n_l - mean : 0.0f;
            m2 = warp_sum(fmaf(n_l * d, d, pr.y));
        }
        const float rstd = rsqrtf(m2 * inv_h + a.eps);
        if (gt == 0 && rank == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        if (a.sum) C::store(reinterpret_cast<T *>(a.sum) + (row * a.sum_stride + c0), width, gt, gsize, s);
#pragma unroll
        for (int p = 0; p < PAIRS; ++p)
            s[p] = ffma2(fmul2(fsub2(s[p], make_float2(mean, mean)), make_float2(rstd, rstd)), HELD ? ga[HELD ? p : 0] : gs[p * gsize + gt],
                         HELD ? be[HELD ? p : 0] : bs[p * gsize + gt]);
        C::store(reinterpret_cast<T *>(a.y) + (row * a.y_stride + c0), width, gt, gsize, s);
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
    auto whole = [&](int bytes) {   // every row starts and ends on a multiple of `bytes`
        return a.hidden * size % bytes == 0 && aligned_rows(a.x, a.x_stride, size, bytes) &&
               aligned_rows(a.res, a.res_stride, size, bytes) && aligned_rows(a.y, a.y_stride, size, bytes) &&
               aligned_rows(a.sum, a.sum_stride, size, bytes);
    };
    const bool aligned = whole(16);
    const int vec = aligned ? 16 / size : size == 2 && whole(4) ? 2 : 1;
    const Sources src = {{a.x, a.res}, {a.x_stride, a.res_stride}};
    const int cols = cols_of(aligned, size, a.hidden);
    const Geometry g = geometry(a.hidden, size, vec, cols, a.res ? 2 : 1, sm_threads(cols), false, a.rows,
                                cols > 16 ? 2 : 0);
    auto pick = [&](auto nt) {
        constexpr int NT = decltype(nt)::value;
        if (aligned) {
            if (g.csize > 1) return norm_forward_kernel<T, 0, 2, NT, 16>;
            if (cols == 8) return norm_forward_kernel<T, 0, 0, NT, 8>;
            if (cols == 24) return norm_forward_kernel<T, 0, 0, NT, size == 2 ? 24 : 16>;
            return g.group > 256 ? norm_forward_kernel<T, 0, 1, NT, 16> : norm_forward_kernel<T, 0, 0, NT, 16>;
        }
        auto unaligned = [&](auto v) {
            constexpr int VEC = decltype(v)::value;
            decltype(&norm_forward_kernel<T, 32, 0, NT, 8, VEC>) none = nullptr;   // refused by launch_rows()
            if (g.csize > 1) return g.group == 512 ? norm_forward_kernel<T, 512, 2, NT, 16, VEC> : none;
            switch (g.group) {
            case 32: return norm_forward_kernel<T, 32, 0, NT, 8, VEC>;
            case 64: return norm_forward_kernel<T, 64, 0, NT, 8, VEC>;
            case 128: return norm_forward_kernel<T, 128, 0, NT, 8, VEC>;
            case 192: return norm_forward_kernel<T, 192, 0, NT, 8, VEC>;
            case 256: return norm_forward_kernel<T, 256, 0, NT, 8, VEC>;
            case 320: return norm_forward_kernel<T, 320, 0, NT, 8, VEC>;
            case 384: return norm_forward_kernel<T, 384, 0, NT, 8, VEC>;
            case 448: return norm_forward_kernel<T, 448, 0, NT, 8, VEC>;
            case 512: return norm_forward_kernel<T, 512, 0, NT, 8, VEC>;
            case 640: return norm_forward_kernel<T, 640, 0, NT, 8, VEC>;
            case 768: return norm_forward_kernel<T, 768, 0, NT, 8, VEC>;
            case 896: return norm_forward_kernel<T, 896, 0, NT, 8, VEC>;
            case 1024: return norm_forward_kernel<T, 1024, 0, NT, 8, VEC>;
            default: return none;
            }
        };
        return vec == 2 ? unaligned(std::integral_constant<int, size == 2 ? 2 : 1>()) : unaligned(std::integral_constant<int, 1>());
    };
    int64_t units = launch_units(g, a.rows);
    return launch_rows(a.res ? pick(std::integral_constant<int, 2>()) : pick(std::integral_constant<int, 1>()), g,
                       units, st, a, src, g, err, wait_limit_ns());
}

}  // namespace

cudaError_t launch_layernorm_forward(const NormArgs &a, cudaStream_t st)
{
    if (a.dtype == TF_FP32) return launch_typed<float>(a, st);
    return a.dtype == TF_BF16 ? launch_typed<__nv_bfloat16>(a, st) : launch_typed<__half>(a, st);
}

}  // namespace tf
