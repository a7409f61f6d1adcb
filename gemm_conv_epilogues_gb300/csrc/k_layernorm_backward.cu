// LayerNorm's backward pass, fp16, bf16 and fp32, any width up to 131072 and
// any row stride.  With xh = (x - mean)*rstd and w = dy*gamma:
//   dx = rstd*(w - mean_row(w) - xh*mean_row(w*xh)) + dres
//   dgamma = sum over rows of dy*xh,  dbeta = sum over rows of dy
// One pass over HBM: dy, x (and dres) read once, dx written once.  A thread
// keeps its columns' dgamma and dbeta in fp32 registers over all the rows its
// group takes; the row groups of an SM form one CTA and add their sums in
// shared memory, one set per SM goes to the workspace, and a second, small
// kernel adds those in order, so that equal calls give equal bits (no atomics).
// Very many rows take several such launches.
// Bound by HBM: 16384 x 4096 bf16 with dres in 89 us, 80 of them this pass at
// 6.7 TB/s, the rest the second kernel; narrow rows by the chain of wait,
// shuffles and store of the one row that each of an SM's sixteen warps has in
// flight (50001 x 640 fp16: 45 us, 4.2 TB/s, 0.55 instructions per cycle and
// scheduler), odd widths by their element-wise columns (1999 x 5003 fp32: 32 us).
#include "norm_rows.cuh"

namespace tf {
namespace {

using namespace norm;

// Threads per SM, from the registers the columns take (two fp32 sums, gamma,
// and the row in its storage type): 128 registers for 16 columns and 24 (gamma
// in shared memory), 80 for 8; where those are element-wise 96, with dres 128,
// but for the widest groups.  Spilled registers cost far more than a few warps
// fewer, since with most of the SM's memory in the rings the little L1 that is
// left does not hold them (8000 x 3501 fp32 with dres: 86 us, spilled 152).
constexpr int sm_threads(int cols, bool aligned, int group, int tensors)
{
    if (cols > 8) return 512;
    if (aligned || group > 640) return 768;
    return tensors < 3 || group > 512 ? 640 : 512;
}

// ... and of a CTA with element-wise columns, which has whole groups only.
constexpr int cta_threads(int cols, int group, int tensors)
{
    const int n = sm_threads(cols, group == 0, group, tensors);
    return group == 0 || group > n ? n : n / group * group;
}

// Columns per thread: 16, or 8 for narrow rows and for element-wise columns (16
// above 6144 of them); 24 for 16-bit rows that then take one warp, whose sums
// need no barrier (50001 x 640 fp16: 45 us, 65 with two warps of 16; 32 columns
// for rows of 1024 were slower, 48 against 30).  With dres 24 do not fit the
// registers (122 us, with 16 columns 70).
int cols_for(int64_t hidden, int size, bool aligned, int tensors)
{
    if (!aligned) return hidden > 6144 ? 16 : 8;
    if (hidden <= 256) return 8;
    if (size == 2 && hidden > 512 && hidden <= 768 && tensors < 3) return 24;
    return 16;
}

// GROUP: threads per row where the columns are element-wise or pairs (a constant
// makes them immediate offsets), 0 for 16-byte vectors.
template <typename T, int GROUP, bool CLUSTER, int NT, int COLS, int VEC = 16 / (int)sizeof(T)>
__global__ void __launch_bounds__(CLUSTER ? 512 : cta_threads(COLS, GROUP, NT), 1)
    norm_backward_kernel(const __grid_constant__ NormGradArgs a, const __grid_constant__ Sources src,
                         const __grid_constant__ Geometry g, uint32_t *err, uint64_t wait_ns)
{
    constexpr bool ALIGNED = GROUP == 0;
    static_assert(ALIGNED == kAligned<T, VEC>, "GROUP and VEC");
    using C = Cols<T, VEC, COLS>;
    constexpr int PAIRS = C::PAIRS;
    constexpr bool HELD = COLS <= 16;   // gamma in registers
    pdl_begin();
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float2 red[2][768 / 32];
    __shared__ __align__(8) float2 slot[2][kMaxRanks];
    __shared__ __align__(8) uint64_t xbar[2];
    const int rank = CLUSTER ? (int)ptx::cluster_ctarank() : 0;
    const int gsize = ALIGNED ? g.group : GROUP, gt = threadIdx.x % gsize, c0 = rank * g.slice;
    const int unit = (int)blockIdx.x / g.csize, units = (int)gridDim.x / g.csize;
    auto ring = start_ring<T, VEC, CLUSTER, NT>(g, smem, src, a.hidden, (int)a.rows, unit, units, c0, err, wait_ns,
                                                    xbar);
    Exchange xch = {slot, xbar, (uint32_t)rank, (uint32_t)g.csize, wait_ns, err, false};
    const int width = ring.width;

    float2 ga[HELD ? PAIRS : 1], dg[PAIRS], db[PAIRS];
    // [PAIRS][gsize] pairs: the lanes' reads of one lie side by side
    float2 *gs = reinterpret_cast<float2 *>(smem + g.gamma_off);
    auto gamma_of = [&](int c) { return a.gamma && c < width ? __ldg(a.gamma + c0 + c) : 1.0f; };
    if (!HELD) {
        for (int i = threadIdx.x; i < PAIRS * gsize; i += (int)blockDim.x) {
            const int p = i / gsize, l = i % gsize;
            gs[i] = make_float2(gamma_of(C::col(2 * p, l, gsize)), gamma_of(C::col(2 * p + 1, l, gsize)));
        }
        cta_sync();
    }
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) {
        if (HELD) ga[HELD ? p : 0] = make_float2(gamma_of(C::col(2 * p, gt, gsize)), gamma_of(C::col(2 * p + 1, gt, gsize)));
        dg[p] = db[p] = make_float2(0.0f, 0.0f);
    }
    // (read anew for either use: held, the compiler would keep it in registers)
    auto gamma2 = [&](int p) {
        if (HELD) return ga[HELD ? p : 0];
        float2 v;
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(ptx::smem_u32(gs + p * gsize + gt)));
        return v;
    };
    const float inv_h = 1.0f / (float)a.hidden;
    Edge<T, VEC> ed, ex, er;
    load_edge(ring, 0, ring.first, gt, gsize, ed);
    load_edge(ring, 1, ring.first, gt, gsize, ex);
    if (NT > 2) load_edge(ring, 2, ring.first, gt, gsize, er);
    // the row statistics, one row ahead
    float mean = 0.0f, rstd = 0.0f;
    if (ring.first < ring.rows) {
        mean = __ldg(a.mean + ring.first);
        rstd = __ldg(a.rstd + ring.first);
    }
    for (int row = ring.first, it = 0; row < ring.rows; row += ring.step, ++it, ring.advance()) {
        C d, x, r;
        ring.wait();
        put_edge(ring, 0, row, ed);
        put_edge(ring, 1, row, ex);
        if (NT > 2) put_edge(ring, 2, row, er);
        d.load(ring, 0, row, gt, gsize);
        x.load(ring, 1, row, gt, gsize);
        if (NT > 2) r.load(ring, 2, row, gt, gsize);
        const int64_t next = (int64_t)row + ring.step;
        load_edge(ring, 0, next, gt, gsize, ed);
        load_edge(ring, 1, next, gt, gsize, ex);
        if (NT > 2) load_edge(ring, 2, next, gt, gsize, er);
        const float2 scale = make_float2(rstd, rstd), centre = make_float2(mean, mean);
        // (the difference first: x*rstd - mean*rstd would lose the digits of a row far from zero)
        auto normalised = [&](int p) { return fmul2(fsub2(x.get(p), centre), scale); };
        if (next < ring.rows) {
            mean = __ldg(a.mean + next);
            rstd = __ldg(a.rstd + next);
        }
        float2 c1 = make_float2(0.0f, 0.0f), c2 = c1;
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) {   // past the slice dy is zero and adds nothing
            const float2 fd = d.get(p), xh = normalised(p), w = fmul2(fd, gamma2(p));
            dg[p] = ffma2(fd, xh, dg[p]);
            db[p] = fadd2(db[p], fd);
            c1 = fadd2(c1, w);
            c2 = ffma2(w, xh, c2);
        }
        float2 c = group_sum2<!CLUSTER>(c1.x + c1.y, c2.x + c2.y, gsize, red[it & 1]);
        if (gt == 0) ring.refill(row);   // every thread of the group holds its columns
        if constexpr (CLUSTER) {
            const float2 *pairs = xch.swap(c, it);
            c = make_float2(0.0f, 0.0f);
            for (int i = 0; i < g.csize; ++i) {
                c.x += pairs[i].x;
                c.y += pairs[i].y;
            }
        }
        const float2 k1 = make_float2(-c.x * inv_h * scale.x, -c.x * inv_h * scale.x);
        const float2 k2 = make_float2(-c.y * inv_h * scale.x, -c.y * inv_h * scale.x);
        float2 out[PAIRS];
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) {
            const float2 xh = normalised(p);
            out[p] = ffma2(fmul2(d.get(p), gamma2(p)), scale, ffma2(xh, k2, k1));
            if (NT > 2) out[p] = fadd2(out[p], r.get(p));
        }
        C::store(reinterpret_cast<T *>(a.dx) + (row * a.dx_stride + c0), width, gt, gsize, out);
    }
    if (gt == 0) ring.drain();

    if (a.ws) {
        // this CTA's sums: row `unit` of dgamma's and of dbeta's [units][hidden] array
        float *wg = a.ws + (int64_t)unit * a.hidden + c0, *wb = wg + (int64_t)units * a.hidden;
        // the groups' sums, added as a tree in shared memory (16 groups one after the other took 5 us): thread
        // gt of every group has the same columns, [2*COLS][gsize] per group
        const int gid = (int)threadIdx.x / gsize;
        cta_sync();   // every group is done with its ring
        for (int n = g.threads / gsize; n > 1;) {
            const int half = (n + 1) / 2;
            float *at = reinterpret_cast<float *>(smem) + (gid < half ? gid : gid - half) * (2 * COLS * gsize) + gt;
            if (gid >= half && gid < n) {
#pragma unroll
                for (int p = 0; p < PAIRS; ++p) {
                    at[4 * p * gsize] = dg[p].x;
                    at[(4 * p + 1) * gsize] = dg[p].y;
                    at[(4 * p + 2) * gsize] = db[p].x;
                    at[(4 * p + 3) * gsize] = db[p].y;
                }
            }
            cta_sync();
            if (gid < n - half) {
#pragma unroll
                for (int p = 0; p < PAIRS; ++p) {
                    dg[p] = fadd2(dg[p], make_float2(at[4 * p * gsize], at[(4 * p + 1) * gsize]));
                    db[p] = fadd2(db[p], make_float2(at[(4 * p + 2) * gsize], at[(4 * p + 3) * gsize]));
                }
            }
            cta_sync();
            n = half;
        }
        if (gid == 0) {
#pragma unroll
            for (int p = 0; p < PAIRS; ++p) {
                const int c = C::col(2 * p, gt, gsize), d = C::col(2 * p + 1, gt, gsize);
                if (c < width) {
                    wg[c] = dg[p].x;
                    wb[c] = db[p].x;
                }
                if (d < width) {
                    wg[d] = dg[p].y;
                    wb[d] = db[p].y;
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
        for (int p = warp; p < parts; p += 8 * kSumWarps) {   // eight loads in flight
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int q = p + i * kSumWarps;
                v[i] = q < parts ? src[(int64_t)q * a.hidden] : 0.0f;
            }
            t += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        }
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

cudaError_t launch_weight_grad(const NormGradArgs &a, int64_t units, cudaStream_t st)
{
    return launch_pdl(norm_weight_grad_kernel, dim3((unsigned)((a.hidden + 31) / 32), 2), dim3(kSumWarps * 32), 0, st, a,
                      (int)units);
}

Geometry geometry_for(int64_t rows, int64_t hidden, int size, int vec, int tensors)
{
    const bool aligned = vec * size == 16;
    const int cols = cols_for(hidden, size, aligned, tensors);
    const int group = (int)(hidden + cols - 1) / cols;   // (rounded up by geometry())
    return geometry(hidden, size, vec, cols, tensors, sm_threads(cols, aligned, group, tensors), true, rows, cols > 16 ? 1 : 0);
}

// The most partial sums that any alignment, number of operands and number of
// rows up to `rows` gives.  One row per CTA gives the most, as long as there are
// SMs: with more rows a CTA takes several, and 153 rows may have half the partial
// sums of 152.
int64_t most_units(int64_t rows, int64_t hidden, int dtype)
{
    const int size = dtype == TF_FP32 ? 4 : 2;
    const int64_t sms = sm_count();
    if (rows > sms) rows = sms;
    int64_t most = 0;
    for (int tensors : {2, 3})
        for (int vec : {1, 2, 16 / size}) {
            const int64_t u = launch_units(geometry_for(rows, hidden, size, vec, tensors), rows);
            if (u > most) most = u;
        }
    return most;
}

// Rows that one launch takes where column sums are wanted: up to 1024 for each
// of its row groups.  A thread adds its rows one after the other, and equal
// terms of a much longer sum lose digits: 3e-4 over 37000 rows each, below 1e-5
// over 1024.  (Of 4096 16-bit columns a launch takes 311,000 rows, over 1 ms.)
int64_t rows_per_launch(const Geometry &g, const NormGradArgs &a)
{
    return a.ws ? 1024 * launch_units(g, a.rows) * (g.threads / g.group) : a.rows;
}

template <typename T>
cudaError_t launch_typed(const NormGradArgs &a, cudaStream_t st)
{
    constexpr int size = (int)sizeof(T);
    uint32_t *err = device_error_word();
    if (!err) return cudaErrorInitializationError;
    auto whole = [&](int bytes) {   // every row starts and ends on a multiple of `bytes`
        return a.hidden * size % bytes == 0 && aligned_rows(a.dy, a.dy_stride, size, bytes) &&
               aligned_rows(a.x, a.x_stride, size, bytes) && aligned_rows(a.dres, a.dres_stride, size, bytes) &&
               aligned_rows(a.dx, a.dx_stride, size, bytes);
    };
    const bool aligned = whole(16);
    const int vec = aligned ? 16 / size : size == 2 && whole(4) ? 2 : 1;
    const Geometry g = geometry_for(a.rows, a.hidden, size, vec, a.dres ? 3 : 2);
    auto pick = [&](auto nt) {
        constexpr int NT = decltype(nt)::value;
        if (aligned) {
            if (g.csize > 1) return norm_backward_kernel<T, 0, true, NT, 16>;
            switch (cols_for(a.hidden, size, true, NT)) {
            case 8: return norm_backward_kernel<T, 0, false, NT, 8>;
            case 24: return norm_backward_kernel<T, 0, false, NT, size == 2 && NT < 3 ? 24 : 16>;
            default: return norm_backward_kernel<T, 0, false, NT, 16>;
            }
        }
        auto unaligned = [&](auto v) {
            constexpr int VEC = decltype(v)::value;
            decltype(&norm_backward_kernel<T, 32, false, NT, 8, VEC>) none = nullptr;   // refused by launch_rows()
            if (cols_for(a.hidden, size, false, NT) == 16) {
                if (g.group != 512) return none;
                return g.csize > 1 ? norm_backward_kernel<T, 512, true, NT, 16, VEC>
                                   : norm_backward_kernel<T, 512, false, NT, 16, VEC>;
            }
            switch (g.group) {
            case 32: return norm_backward_kernel<T, 32, false, NT, 8, VEC>;
            case 64: return norm_backward_kernel<T, 64, false, NT, 8, VEC>;
            case 128: return norm_backward_kernel<T, 128, false, NT, 8, VEC>;
            case 192: return norm_backward_kernel<T, 192, false, NT, 8, VEC>;
            case 256: return norm_backward_kernel<T, 256, false, NT, 8, VEC>;
            case 320: return norm_backward_kernel<T, 320, false, NT, 8, VEC>;
            case 384: return norm_backward_kernel<T, 384, false, NT, 8, VEC>;
            case 448: return norm_backward_kernel<T, 448, false, NT, 8, VEC>;
            case 512: return norm_backward_kernel<T, 512, false, NT, 8, VEC>;
            case 640: return norm_backward_kernel<T, 640, false, NT, 8, VEC>;
            case 768: return norm_backward_kernel<T, 768, false, NT, 8, VEC>;
            default: return none;
            }
        };
        return vec == 2 ? unaligned(std::integral_constant<int, size == 2 ? 2 : 1>()) : unaligned(std::integral_constant<int, 1>());
    };
    auto kern = a.dres ? pick(std::integral_constant<int, 3>()) : pick(std::integral_constant<int, 2>());
    const int64_t run = rows_per_launch(g, a);
    NormGradArgs p = a;
    for (int64_t left = a.rows;;) {
        p.rows = left < run ? left : run;
        const Sources src = {{p.dy, p.x, p.dres}, {a.dy_stride, a.x_stride, a.dres_stride}};
        int64_t units = launch_units(g, p.rows);
        cudaError_t e = launch_rows(kern, g, units, st, p, src, g, err, wait_limit_ns());
        if (e == cudaSuccess && a.ws) e = launch_weight_grad(p, units, st);
        if (e != cudaSuccess || (left -= p.rows) == 0) return e;
        auto skip = [&](const void *&q, int64_t stride) {
            if (q) q = static_cast<const T *>(q) + p.rows * stride;
        };
        skip(p.dy, a.dy_stride);
        skip(p.x, a.x_stride);
        skip(p.dres, a.dres_stride);
        p.dx = static_cast<T *>(p.dx) + p.rows * a.dx_stride;
        p.mean += p.rows;
        p.rstd += p.rows;
        p.accumulate = 1;
    }
}

}  // namespace

int64_t layernorm_backward_workspace(int64_t rows, int64_t hidden, int dtype)
{
    return rows > 0 ? most_units(rows, hidden, dtype) * hidden * 2 * 4 : 0;
}

cudaError_t launch_layernorm_backward(const NormGradArgs &a, cudaStream_t st)
{
    // with no rows there are no partial sums, and the gradients become zero
    if (a.rows == 0) return launch_weight_grad(a, 0, st);
    return a.dtype == TF_FP32   ? launch_typed<float>(a, st)
           : a.dtype == TF_BF16 ? launch_typed<__nv_bfloat16>(a, st)
                                : launch_typed<__half>(a, st);
}

}  // namespace tf
