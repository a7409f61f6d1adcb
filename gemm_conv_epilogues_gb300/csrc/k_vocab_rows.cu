// Cross entropy of logits = scale * x w^T over a vocabulary, and its gradients:
//   lse[i] = log(sum over v of exp(l[i][v]));  loss[i] = lse[i] - l[i][target]
//   dl[i][v] = exp(l[i][v] - lse[i]) (dloss[i] + dlse[i]) - [v = target] dloss[i]
//   dx = scale * dl w;  dw = scale * dl^T x
// Here are the plan of a call and its kernels over rows; the products are in
// k_vocab_umma.cu.
//
//   gather   the rows that count (whose target is a word) are brought together in
//            the workspace, so that the others cost no products, and what they hold,
//            NaN included, reaches nothing; their outputs become zero
//   STATS    forward: maxima and sums of exponentials; `loss` joins them
//   DLOGITS, GRADS   backward, one piece of the vocabulary after the other: the
//            piece's gradients of the logits are the only ones in memory (256 MB at most)
//   dx       the splits' sums of dx are added and put in the rows' places
//
// Weights whose rows are not multiples of 16 bytes, which no tensor map can address,
// are copied piece by piece to rows that are.
#include <climits>

#include "grouped.cuh"
#include "lm_internal.h"

namespace tf {
namespace {

using grouped::Half2Of;

constexpr int kThreads = 256;
constexpr int64_t kDlBytes = (int64_t)256 << 20;     // a piece's gradients of the logits
constexpr int64_t kPackBytes = (int64_t)256 << 20;   // a piece's copied weights
constexpr int64_t kSplitBytes = (int64_t)128 << 20;  // dx's sums, where there are several

// ---------------------------------------------------------------- gather

enum { UNIT_FIRST_ROW = 0, UNIT_ALL_ROWS = 1, UNIT_GIVEN = 2 };   // (the last: unit[0] by unit_kernel)
struct GatherArgs {
    LceArgs a;
    int *count, *index, *target;
    float *z, *ca, *cb;        // backward
    float *unit;               // backward: the gradients of the logits are held times unit[0]; unit[1] is its inverse
    int unit_from;
    uint16_t *x;
    int64_t x_pitch;
    int per_block;             // rows
};

// 1: counts, 0: ignored (or outside the vocabulary, which the error word tells)
__device__ __forceinline__ bool counts(const LceArgs &a, int64_t i, int64_t *target, bool tell)
{
    const int64_t t = a.targets.at(i);
    *target = t;
    if (t == a.ignore) return false;
    if (t >= 0 && t < a.vocab) return true;
    if (tell) atomicOr(a.err, TF_DEVERR_INDEX);
    return false;
}

// `lanes` threads copy a row of 16-bit values, by the widest words that fit it.
__device__ __forceinline__ void copy_row(uint16_t *dst, const uint16_t *src, int n, int lane, int lanes)
{
    if ((reinterpret_cast<uintptr_t>(src) & 15u) == 0 && n % 8 == 0) {
        for (int c = lane; c < n / 8; c += 4 * lanes) {
            uint4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (c + u * lanes < n / 8) v[u] = reinterpret_cast<const uint4 *>(src)[c + u * lanes];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (c + u * lanes < n / 8) reinterpret_cast<uint4 *>(dst)[c + u * lanes] = v[u];
        }
    } else {
        for (int c = lane; c < n; c += 8 * lanes) {
            uint16_t v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (c + u * lanes < n) v[u] = src[c + u * lanes];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (c + u * lanes < n) dst[c + u * lanes] = v[u];
        }
    }
}

__device__ __forceinline__ void zero_row(uint16_t *dst, int n, int lane, int lanes)
{
    if ((reinterpret_cast<uintptr_t>(dst) & 15u) == 0 && n % 8 == 0)
        for (int c = lane; c < n / 8; c += lanes) reinterpret_cast<uint4 *>(dst)[c] = make_uint4(0, 0, 0, 0);
    else
        for (int c = lane; c < n; c += lanes) dst[c] = 0;
}

// The gradients of the logits are held in units of a typical |dloss|, which is often
// that of all rows: a target's (p - 1) dloss is then rounded near one, where it is
// off by no more than p, and not by dloss's own rounding, the same in every row (dx of 3300 rows
// with a mean's weights: relative error 2.9e-3 without, 1.8e-3 with units).  bf16 takes the first
// row's.  fp16, whose exponents are few, takes the largest, times 2^14:
// a word's share of 1e-5 would otherwise lie far below its smallest.
__device__ __forceinline__ float unit_of(float typical)
{
    return typical > 0x1p-40f && typical < 0x1p40f ? 1.0f / typical : 1.0f;
}

// fp16's, from all rows, by a CTA of THREADS threads.
template <int THREADS>
__device__ __forceinline__ float unit_of_all(const LceArgs &a)
{
    __shared__ float2 warps[THREADS / 32];
    float most = 0.0f, both = 0.0f;   // the largest |dloss|, and |dloss| + |dlse|, which bounds the gradients
    for (int64_t i = threadIdx.x; i < a.rows; i += THREADS) {
        int64_t target;
        if (!counts(a, i, &target, false)) continue;
        const float d = a.dloss ? fabsf(a.dloss[i]) : 1.0f;
        most = fmaxf(most, d);
        both = fmaxf(both, d + (a.dlse ? fabsf(a.dlse[i]) : 0.0f));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        both = fmaxf(both, __shfl_xor_sync(0xffffffffu, both, o));
    }
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = make_float2(most, both);
    __syncthreads();
    for (int w = 0; w < THREADS / 32; ++w) {
        most = fmaxf(most, warps[w].x);
        both = fmaxf(both, warps[w].y);
    }
    const float size = both <= 2.0f * most ? most : both;   // (the gradients stay below 2^15, or 2^14)
    return size > 0x1p-100f && size < 0x1p100f ? 0x1p14f / size : 1.0f;   // (a normal number, and its inverse too)
}

__global__ void __launch_bounds__(1024) unit_kernel(const __grid_constant__ LceArgs a, float *unit)
{
    pdl_begin();
    const float u = unit_of_all<1024>(a);
    if (threadIdx.x == 0) *unit = u;
}

// A CTA takes per_block rows; it counts those that count before them itself,
// which reads the targets once per CTA, but needs no CTA to wait for another.
template <bool BACKWARD>
__global__ void __launch_bounds__(kThreads, 4) gather_kernel(const __grid_constant__ GatherArgs g)
{
    pdl_begin();
    __shared__ int warps[kThreads / 32], least[kThreads / 32];
    __shared__ int place[kThreads];
    __shared__ float typical;   // |dloss| of the first row that counts
    const LceArgs &a = g.a;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int64_t first = (int64_t)blockIdx.x * g.per_block, end = min(first + g.per_block, a.rows);
    int before = 0, earliest = INT_MAX;
    for (int64_t i = t; i < first; i += 4 * kThreads) {   // four loads under way at a time
        int64_t target[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) target[u] = i + u * kThreads < first ? a.targets.at(i + u * kThreads) : -1;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i + u * kThreads < first && target[u] >= 0 && target[u] < a.vocab && target[u] != a.ignore) {
                ++before;
                earliest = min(earliest, (int)(i + u * kThreads));
            }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        earliest = min(earliest, __shfl_xor_sync(0xffffffffu, earliest, o));
    }
    if (lane == 0) {
        warps[warp] = before;
        least[warp] = earliest;
    }
    __syncthreads();
    before = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        before += warps[w];
        earliest = min(earliest, least[w]);
    }
    float unit = 1.0f;
    if (BACKWARD) {
        if (g.unit_from == UNIT_ALL_ROWS) unit = unit_of_all<kThreads>(a);
        else if (g.unit_from == UNIT_GIVEN) unit = g.unit[0];
        else if (t == 0) typical = before > 0 && a.dloss ? fabsf(a.dloss[earliest]) : 1.0f;
    }
    for (int64_t base = first; base < end; base += kThreads) {
        const int64_t i = base + t;
        int64_t target = 0;
        const bool live = i < end, used = live && counts(a, i, &target, true);
        const unsigned mask = __ballot_sync(0xffffffffu, used);
        __syncthreads();   // (warps and place have been read)
        if (lane == 0) warps[warp] = __popc(mask);
        __syncthreads();
        int at = before + __popc(mask & ((1u << lane) - 1u));
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) at += warps[w];
            before += warps[w];
        }
        place[t] = used ? at : -1;
        if (BACKWARD && used && at == 0 && a.dloss) typical = fabsf(a.dloss[i]);   // (the first of all)
        __syncthreads();
        if (used) {
            g.index[at] = (int)i;
            g.target[at] = (int)target;
            if (BACKWARD) {
                const float d = a.dloss ? a.dloss[i] : 1.0f;
                if (g.unit_from == UNIT_FIRST_ROW) unit = unit_of(typical);
                g.z[at] = a.lse[i];
                g.ca[at] = (a.dlse ? d + a.dlse[i] : d) * unit;
                g.cb[at] = d * unit;
            }
        } else if (live && !BACKWARD) {
            a.loss[i] = 0.0f;
            a.lse[i] = 0.0f;
        }
        const int lanes = g.per_block == 1 ? kThreads : 32, member = t % lanes;   // a row to a warp, or to the CTA
        for (int r = t / lanes; r < (int)min((int64_t)kThreads, end - base); r += kThreads / lanes) {
            const int64_t row = base + r;
            if (place[r] >= 0)
                copy_row(g.x + place[r] * g.x_pitch, static_cast<const uint16_t *>(a.x) + row * a.x_stride, a.hidden, member,
                         lanes);
            else if (a.dx)
                zero_row(static_cast<uint16_t *>(a.dx) + row * a.dx_stride, a.hidden, member, lanes);
        }
    }
    if (end == a.rows) {   // the last CTA
        if (t == 0) {
            *g.count = before;
            if (BACKWARD) g.unit[1] = 1.0f / (g.unit_from == UNIT_FIRST_ROW ? unit_of(typical) : unit);
        }
        // the K steps of dw read whole sixty-fours of rows
        for (int64_t r = before + warp; r < min((int64_t)(before + 63) / 64 * 64, a.rows); r += kThreads / 32)
            zero_row(g.x + r * g.x_pitch, (int)g.x_pitch, lane, 32);
    }
}

// ---------------------------------------------------------------- loss

struct LossArgs {
    const int *count, *index;
    const float2 *part;
    const float *at_target;
    float *loss, *lse;
    int rows, slots, per_block;
    float scale;
};

// `per_block` rows per CTA (one, or four, whose neighbouring slots fill a sector), a
// row's slots over the CTA's threads.
// The loss is taken from the maximum, so that a sure target's, whose sum of exponentials
// is one, is exactly zero.
__global__ void __launch_bounds__(kThreads) loss_kernel(const __grid_constant__ LossArgs p)
{
    pdl_begin();
    constexpr int WARPS = kThreads / 32;
    __shared__ float2 red[WARPS][4];
    const int count = *p.count, per = p.per_block, row0 = (int)blockIdx.x * per;
    if (row0 >= count) return;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, row = row0 + t % per, lanes = kThreads / per;
    const float c = p.scale * kLog2e;
    auto join = [&](float2 s, float2 v) {
        const float m = fmaxf(s.x, v.x), base = m == -INFINITY ? 0.0f : m;
        return make_float2(m, s.y * ex2_approx((s.x - base) * c) + v.y * ex2_approx((v.x - base) * c));
    };
    float2 s = make_float2(-INFINITY, 0.0f);
    if (row < count)
        for (int k = t / per; k < p.slots; k += 4 * lanes) {
            float2 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                v[u] = k + u * lanes < p.slots ? p.part[(int64_t)(k + u * lanes) * p.rows + row]
                                               : make_float2(-INFINITY, 0.0f);
            s = join(s, join(join(v[0], v[1]), join(v[2], v[3])));
        }
    for (int o = 16; o >= per; o >>= 1)
        s = join(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, s.y, o)));
    if (lane < per) red[warp][lane] = s;
    __syncthreads();
    if (t >= per || row >= count) return;
    for (int w = 1; w < WARPS; ++w) s = join(s, red[w][t]);
    const float over = logf(s.y);
    const int64_t i = p.index[row];
    p.loss[i] = fmaf(p.scale, s.x - p.at_target[row], over);
    p.lse[i] = fmaf(p.scale, s.x, over);
}

// ---------------------------------------------------------------- dx

struct DxArgs {
    const int *count, *index;
    const float *sums;   // [splits][rows][pitch]
    void *dx;
    int64_t pitch, stride, rows;
    int hidden, splits, bf16;
};

// A CTA per row, 4 columns per thread.
__global__ void __launch_bounds__(kThreads) dx_kernel(const __grid_constant__ DxArgs p)
{
    pdl_begin();
    const int row = (int)blockIdx.x;
    if (row >= *p.count) return;
    uint16_t *out = static_cast<uint16_t *>(p.dx) + (int64_t)p.index[row] * p.stride;
    const bool words = (reinterpret_cast<uintptr_t>(out) & 7u) == 0;
    for (int c = threadIdx.x * 4; c < p.hidden; c += kThreads * 4) {
        const float *src = p.sums + (int64_t)row * p.pitch + c;
        float4 t = *reinterpret_cast<const float4 *>(src);
#pragma unroll 4
        for (int s = 1; s < p.splits; ++s) {
            const float4 v = *reinterpret_cast<const float4 *>(src + (int64_t)s * p.rows * p.pitch);
            t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
        }
        uint2 v;
        if (p.bf16) v = make_uint2(Half2Of<__nv_bfloat16>::pack(t.x, t.y), Half2Of<__nv_bfloat16>::pack(t.z, t.w));
        else v = make_uint2(Half2Of<__half>::pack(t.x, t.y), Half2Of<__half>::pack(t.z, t.w));
        if (words && c + 4 <= p.hidden) {
            *reinterpret_cast<uint2 *>(out + c) = v;
        } else {
            const uint16_t e[4] = {(uint16_t)v.x, (uint16_t)(v.x >> 16), (uint16_t)v.y, (uint16_t)(v.y >> 16)};
            for (int k = 0; k < min(4, p.hidden - c); ++k) out[c + k] = e[k];
        }
    }
}

// ---------------------------------------------------------------- weights of odd widths

// A warp per row.  Eight values at any even address come as five aligned 32-bit words,
// shifted into place; what might lie before the weights or behind them is not read
// (a row's last one to eight values, and the first eight of all where they begin inside a word).
__global__ void __launch_bounds__(kThreads) pack_rows_kernel(const uint16_t *w, uint16_t *out, int64_t rows, int hidden,
                                                             int64_t pitch)
{
    pdl_begin();
    constexpr int UNROLL = 4;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
    const int lane = threadIdx.x & 31, whole = (hidden - 1) / 8;
    for (int64_t r = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); r < rows; r += step) {
        const uint16_t *src = w + r * hidden;
        uint16_t *dst = out + r * pitch;
        const bool inside = (reinterpret_cast<uintptr_t>(src) & 2u) != 0;
        const uint32_t *words = reinterpret_cast<const uint32_t *>(src - (inside ? 1 : 0));
        const int first = r == 0 && inside ? 1 : 0;
        for (int c = first + lane; c < whole; c += UNROLL * 32) {
            uint32_t v[UNROLL][5];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u)
                if (c + u * 32 < whole)
#pragma unroll
                    for (int k = 0; k < 5; ++k) v[u][k] = k < 4 || inside ? words[(c + u * 32) * 4 + k] : 0;
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                if (c + u * 32 >= whole) break;
                const int shift = inside ? 16 : 0;
                reinterpret_cast<uint4 *>(dst)[c + u * 32] =
                    make_uint4(__funnelshift_r(v[u][0], v[u][1], shift), __funnelshift_r(v[u][1], v[u][2], shift),
                               __funnelshift_r(v[u][2], v[u][3], shift), __funnelshift_r(v[u][3], v[u][4], shift));
            }
        }
        if (lane < 8 && first && lane < whole * 8) dst[lane] = src[lane];
        if (whole * 8 + lane < hidden && lane < 8) dst[whole * 8 + lane] = src[whole * 8 + lane];
    }
}

cudaError_t launch_pack(const LceArgs &a, int64_t v0, int64_t words, int64_t pitch, void *out, cudaStream_t st)
{
    const int64_t blocks = (words + kThreads / 32 - 1) / (kThreads / 32), most = 8 * (int64_t)sm_count();
    return launch_pdl(pack_rows_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(kThreads), 0, st,
                      static_cast<const uint16_t *>(a.w) + v0 * a.hidden, static_cast<uint16_t *>(out), words, a.hidden,
                      pitch);
}

// ---------------------------------------------------------------- plan

int64_t up(int64_t v, int64_t step) { return (v + step - 1) / step * step; }

// What a call keeps where in its workspace.  Where a choice depends on the rows,
// its bytes are those of the larger choice, so that they do not fall as rows grow.
struct Plan {
    int64_t x_pitch, w_pitch, dl_pitch, dx_pitch;
    int64_t piece;          // words
    int splits;             // of dx
    int64_t count, unit, index, target, z, ca, cb, at_target, part, x, dl, dx, pack, bytes;
};

// Words per piece where `most` bytes hold `per_word` each: as few pieces as fit, of
// equal size but for the last, in whole tiles.
int64_t piece_of(int64_t vocab, int64_t per_word, int64_t most)
{
    int64_t fit = most / per_word / 512 * 512;
    if (fit < 512) fit = 512;
    if (vocab <= fit) return vocab;
    const int64_t n = (vocab + fit - 1) / fit;
    return up((vocab + n - 1) / n, 512);
}

Plan plan_of(bool backward, int64_t rows, int64_t vocab, int64_t hidden)
{
    if (rows < 1) rows = 1;   // (dw alone, which becomes zero)
    Plan p = {};
    p.x_pitch = up(hidden, 8);
    p.w_pitch = p.x_pitch;
    p.dx_pitch = up(hidden, 4);
    const bool pack = hidden % 8 != 0;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t from = at;
        at += up(bytes, 256);
        return from;
    };
    p.count = take(4);
    p.unit = take(8);
    p.index = take(4 * rows);
    p.target = take(4 * rows);
    p.x = take(rows * p.x_pitch * 2);
    p.piece = vocab;
    if (pack) p.piece = piece_of(vocab, p.w_pitch * 2, kPackBytes);
    if (!backward) {
        p.at_target = take(4 * rows);
        // Two slots per tile of words.  lce_word_tile makes at most units*waves/down tiles of a piece
        // (down: row tiles), which is no more than words/256 + 1 + units/down, and rows/down is no more
        // than a row tile: 256 rows on half of the SMs, or 128 on all.
        const int64_t pieces = (vocab + p.piece - 1) / p.piece;
        p.part = take(8 * 2 * ((vocab / 256 + pieces) * rows + pieces * 128 * sm_count()));
    } else {
        p.z = take(4 * rows);
        p.ca = take(4 * rows);
        p.cb = take(4 * rows);
        const int64_t fits = piece_of(vocab, 2 * rows, kDlBytes);
        if (fits < p.piece) p.piece = fits;
        p.dl_pitch = up(p.piece, 64);
        const int64_t all = 2 * rows * up(vocab, 64), least = 2 * rows * 512, cap = kDlBytes > least ? kDlBytes : least;
        p.dl = take(all < cap ? all : cap);
        const int64_t row_bytes = p.dx_pitch * 4 * rows, by_bytes = kSplitBytes / row_bytes;
        const int64_t splits = lce_splits(rows, p.piece, hidden);
        p.splits = (int)(splits < by_bytes ? splits : by_bytes < 1 ? 1 : by_bytes);
        const int64_t most = 16 * row_bytes < kSplitBytes ? 16 * row_bytes : kSplitBytes;
        p.dx = take(row_bytes > most ? row_bytes : most);
    }
    if (pack) {
        const int64_t row_bytes = p.w_pitch * 2, fit = kPackBytes / row_bytes;
        p.pack = take(up(vocab < fit ? vocab : fit, 512) * row_bytes);
    }
    p.bytes = at;
    return p;
}

template <typename T>
T *at(void *ws, int64_t offset)
{
    return reinterpret_cast<T *>(static_cast<char *>(ws) + offset);
}

cudaError_t launch_gather(const LceArgs &a, const Plan &p, bool backward, cudaStream_t st)
{
    GatherArgs g = {};
    g.a = a;
    g.count = at<int>(a.ws, p.count);
    g.index = at<int>(a.ws, p.index);
    g.target = at<int>(a.ws, p.target);
    g.x = at<uint16_t>(a.ws, p.x);
    g.x_pitch = p.x_pitch;
    // a row per CTA while they all run at once (4 rows of 4096: 4.3 us, 8.9 with a row per warp), a row per
    // warp, or more where counting what lies before would take longer than that
    g.per_block = a.rows <= 4 * sm_count() ? 1 : a.rows <= 16384 ? 8 : (int)up((a.rows + 2047) / 2048, 8);
    const dim3 grid((unsigned)(a.rows ? (a.rows + g.per_block - 1) / g.per_block : 1));
    if (!backward) return launch_pdl(gather_kernel<false>, grid, dim3(kThreads), 0, st, g);
    g.z = at<float>(a.ws, p.z);
    g.ca = at<float>(a.ws, p.ca);
    g.cb = at<float>(a.ws, p.cb);
    g.unit = at<float>(a.ws, p.unit);
    // each CTA looks through a few rows itself, one kernel through many
    g.unit_from = a.dtype == TF_BF16 ? UNIT_FIRST_ROW : g.per_block == 1 ? UNIT_ALL_ROWS : UNIT_GIVEN;
    const cudaError_t e = g.unit_from == UNIT_GIVEN ? launch_pdl(unit_kernel, dim3(1), dim3(1024), 0, st, a, g.unit) : cudaSuccess;
    return e != cudaSuccess ? e : launch_pdl(gather_kernel<true>, grid, dim3(kThreads), 0, st, g);
}

LceProduct product_of(const LceArgs &a, const Plan &p)
{
    LceProduct m = {};
    m.count = at<int>(a.ws, p.count);
    m.target = at<int>(a.ws, p.target);
    m.x = at<void>(a.ws, p.x);
    m.x_pitch = p.x_pitch;
    m.w_pitch = a.hidden;
    m.rows = (int)a.rows;
    m.hidden = a.hidden;
    m.dtype = a.dtype;
    return m;
}

// The piece of the weights from word v0 on, where the products can address it.
cudaError_t piece_weights(const LceArgs &a, const Plan &p, int64_t v0, int64_t words, LceProduct *m, cudaStream_t st)
{
    m->v0 = (int)v0;
    m->words = (int)words;
    if (a.hidden % 8 == 0) {
        m->w = static_cast<const uint16_t *>(a.w) + v0 * a.hidden;
        return cudaSuccess;
    }
    m->w = at<void>(a.ws, p.pack);
    m->w_pitch = p.w_pitch;
    return launch_pack(a, v0, words, p.w_pitch, at<void>(a.ws, p.pack), st);
}

}  // namespace

int64_t lce_workspace(bool backward, int64_t rows, int64_t vocab, int64_t hidden)
{
    return plan_of(backward, rows, vocab, hidden).bytes;
}

cudaError_t launch_lce_forward(const LceArgs &a, cudaStream_t st)
{
    const Plan p = plan_of(false, a.rows, a.vocab, a.hidden);
    cudaError_t e = launch_gather(a, p, false, st);
    LceProduct m = product_of(a, p);
    m.part = at<float2>(a.ws, p.part);
    m.at_target = at<float>(a.ws, p.at_target);
    m.factor = a.scale * kLog2e;
    for (int64_t v0 = 0; e == cudaSuccess && v0 < a.vocab; v0 += p.piece) {
        const int64_t words = a.vocab - v0 < p.piece ? a.vocab - v0 : p.piece;
        e = piece_weights(a, p, v0, words, &m, st);
        if (e != cudaSuccess) return e;
        e = launch_lce_product(LCE_STATS, m, st);
        const int bn = lce_word_tile(a.rows, words);
        m.slot0 += 2 * (int)((words + bn - 1) / bn);
    }
    if (e != cudaSuccess) return e;
    LossArgs l = {};
    l.count = m.count; l.index = at<int>(a.ws, p.index); l.part = m.part; l.at_target = m.at_target;
    l.loss = a.loss; l.lse = a.lse; l.rows = (int)a.rows; l.slots = m.slot0;
    l.per_block = a.rows < 512 ? 1 : 4; l.scale = a.scale;
    return launch_pdl(loss_kernel, dim3((unsigned)((a.rows + l.per_block - 1) / l.per_block)), dim3(kThreads), 0, st, l);
}

cudaError_t launch_lce_backward(const LceArgs &a, cudaStream_t st)
{
    const Plan p = plan_of(true, a.rows, a.vocab, a.hidden);
    cudaError_t e = launch_gather(a, p, true, st);
    LceProduct m = product_of(a, p);
    m.z = at<float>(a.ws, p.z);
    m.ca = at<float>(a.ws, p.ca);
    m.cb = at<float>(a.ws, p.cb);
    m.unit = at<float>(a.ws, p.unit);
    m.dl = at<void>(a.ws, p.dl);
    m.dl_pitch = p.dl_pitch;
    m.dx = a.dx ? at<float>(a.ws, p.dx) : nullptr;
    m.dx_pitch = p.dx_pitch;
    m.splits = p.splits;
    m.dw_f32 = a.dw_dtype == TF_FP32;
    m.accumulate = a.accumulate;
    m.first = 1;
    m.factor = a.scale;
    for (int64_t v0 = 0; e == cudaSuccess && v0 < a.vocab; v0 += p.piece) {
        const int64_t words = a.vocab - v0 < p.piece ? a.vocab - v0 : p.piece;
        e = piece_weights(a, p, v0, words, &m, st);
        if (e != cudaSuccess) return e;
        if (a.rows > 0) e = launch_lce_product(LCE_DLOGITS, m, st);
        if (e != cudaSuccess) return e;
        m.dw = a.dw ? static_cast<char *>(a.dw) + v0 * a.hidden * (m.dw_f32 ? 4 : 2) : nullptr;
        e = launch_lce_product(LCE_GRADS, m, st);
        m.first = 0;
    }
    if (e != cudaSuccess || !a.dx || a.rows == 0) return e;
    DxArgs d = {m.count, at<int>(a.ws, p.index), m.dx, a.dx, p.dx_pitch, a.dx_stride, a.rows, a.hidden, p.splits,
                a.dtype == TF_BF16};
    return launch_pdl(dx_kernel, dim3((unsigned)a.rows), dim3(kThreads), 0, st, d);
}

}  // namespace tf
