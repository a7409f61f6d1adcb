// Row streaming shared by the layer-norm kernels (forward with statistics,
// backward): the rows of up to three tensors pass through a ring of
// shared-memory stages filled by bulk copies, so several rows per SM are on
// their way while one is reduced, and every element is read from HBM once.
//
// A row group of one or more warps works on one row at a time, each thread on
// COLS columns of it; a CTA holds one or several groups, which meet at named
// barriers of their own.  Rows wider than 8192 columns are cut into slices
// over the CTAs of a cluster, one group per CTA.  (Slices of 4096, with more
// CTAs per SM, were slower: 161 against 110 us for 8192 x 8192 bf16, forward
// with residual; the exchange lengthens every row.)
//
// Alignment.  With every row start and length a multiple of 16 bytes a row is
// one bulk copy and a thread's columns are 16-byte vectors.  Otherwise the
// copy takes the 16-byte pieces that lie inside the row, at the same offset
// from a 16-byte boundary in shared memory as in global memory; the up to 15
// bytes before and behind them are loaded one row ahead by the threads whose
// columns they are (copying them too would read past the tensor's ends).  A
// thread's columns are then single ones, or pairs where 16-bit rows consist of
// whole words (6000 x 5002 bf16 with residual, forward: 76 us, 100 one by one).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "ptx_sm100.cuh"
#include "train_internal.h"

namespace tf {
namespace norm {

constexpr int kSlice = 8192;              // columns of one CTA
constexpr int kMaxGroup = 1024;
constexpr int kClusterGroup = 512;
constexpr int kMaxStages = 8;
constexpr int kMaxTensors = 3;
constexpr int kMaxRanks = 16;

__device__ __forceinline__ float widen(float a) { return a; }
__device__ __forceinline__ float widen(__half a) { return __half2float(a); }
__device__ __forceinline__ float widen(__nv_bfloat16 a) { return __bfloat162float(a); }
__device__ __forceinline__ void narrow(float &p, float a) { p = a; }
__device__ __forceinline__ void narrow(__half &p, float a) { p = __float2half_rn(a); }
__device__ __forceinline__ void narrow(__nv_bfloat16 &p, float a) { p = __float2bfloat16_rn(a); }

template <typename T>
__device__ __forceinline__ void unpack(const uint4 &u, float *f)
{
    const T *h = reinterpret_cast<const T *>(&u);
#pragma unroll
    for (int i = 0; i < 16 / (int)sizeof(T); ++i) f[i] = widen(h[i]);
}

template <typename T>
__device__ __forceinline__ uint4 repack(const float *f)
{
    uint4 u;
    if constexpr (sizeof(T) == 4) {
        u = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same<T, __half>::value) {
                const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        u = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return u;
}

__device__ __forceinline__ void st_stream(void *p, uint4 v)
{
    asm volatile("st.global.cs.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Launch geometry, from the host.
struct Geometry {
    int group;          // threads per row (and CTA of the cluster)
    int threads;        // threads per CTA
    int per_sm;         // CTAs per SM
    int csize, slice;   // CTAs per row and columns per CTA
    int stages, tensor_bytes;   // ring of one row group: stages x tensors x tensor_bytes
    int bar_off;        // mbarriers behind the rings
    int gamma_off;      // parameter tables behind those, where the kernel keeps them there
    int smem;
};

// The tensors whose rows stream in (a kernel parameter).
struct Sources {
    const void *base[kMaxTensors];
    int64_t stride[kMaxTensors];
};

// VEC: neighbouring columns that a thread moves at once.  16 bytes of them for
// aligned rows; else one, or two of 16 bits (a word).
template <typename T, int VEC>
constexpr bool kAligned = VEC * (int)sizeof(T) == 16;
template <typename T, int VEC>
using Unit = typename std::conditional<VEC == 2, uint32_t, T>::type;   // of unaligned rows

// What one thread knows of its row group's ring of NT tensors.
template <typename T, int VEC, int NT>
struct Ring {
    static constexpr bool ALIGNED = kAligned<T, VEC>;
    const Sources &src;
    unsigned char *mem;
    uint64_t *full;
    int stages, tensor_bytes, c0, width;        // width: columns of this CTA's slice, from c0 on
    int first, step, rows;                      // this group's rows: first, first + step, ...
    uint64_t wait_ns;
    uint32_t *err;
    bool failed;
    int stage;                                  // of the current row; counted up, not divided out: rows are short
    uint32_t phase, pending;                    // pending: stages with a copy under way (the issuing thread's)

    __device__ __forceinline__ const T *at(int i, int64_t row) const
    {
        return reinterpret_cast<const T *>(src.base[i]) + (row * src.stride[i] + c0);
    }

    // Copies `row` into stage s (one thread of the group).
    __device__ __forceinline__ void issue(int s, int64_t row)
    {
        if (row >= rows || failed) return;
        unsigned char *dst = mem + s * NT * tensor_bytes;
        uint64_t *bar = &full[s];
        const uint32_t bytes = (uint32_t)width * (uint32_t)sizeof(T);
        if constexpr (ALIGNED) {
            ptx::mbar_arrive_expect_tx(bar, bytes * (uint32_t)NT);
#pragma unroll
            for (int i = 0; i < NT; ++i) ptx::bulk_load(dst + i * tensor_bytes, at(i, row), bytes, bar);
        } else {
            uint32_t total = 0;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const uint64_t a = reinterpret_cast<uint64_t>(at(i, row)), lo = (a + 15) & ~15ull, hi = (a + bytes) & ~15ull;
                if (hi > lo) total += (uint32_t)(hi - lo);
            }
            ptx::mbar_arrive_expect_tx(bar, total);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const uint64_t a = reinterpret_cast<uint64_t>(at(i, row)), lo = (a + 15) & ~15ull, hi = (a + bytes) & ~15ull;
                if (hi > lo)
                    ptx::bulk_load(dst + i * tensor_bytes + (lo - (a & ~15ull)), reinterpret_cast<const void *>(lo),
                                   (uint32_t)(hi - lo), bar);
            }
        }
        pending |= 1u << s;
    }

    // Waits for the current row.
    __device__ __forceinline__ void wait()
    {
        if (!failed && !ptx::mbar_wait(&full[stage], phase, wait_ns)) {
            failed = true;
            atomicOr(err, TF_DEVERR_PRODUCER_WAIT);
        }
        if (!failed) pending &= ~(1u << stage);
    }

    // The row `stages` after `row` takes the current stage, which every thread of the group has read (one thread).
    __device__ __forceinline__ void refill(int row)
    {
        ptx::fence_proxy_async_smem();
        issue(stage, (int64_t)row + (int64_t)stages * step);
    }

    __device__ __forceinline__ void advance()
    {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
        }
    }

    // Copies never waited for (after a time-out only) land before the CTA exits.
    __device__ __forceinline__ void drain()
    {
        for (int s = 0; s < stages; ++s)
            if ((pending >> s) & 1u)
                if (!ptx::mbar_wait(&full[s], s >= stage ? phase : phase ^ 1u, wait_ns))
                    atomicOr(err, TF_DEVERR_DRAIN_WAIT);
    }

    // Units of row `it` of tensor i that lie before and behind the copied pieces.
    __device__ __forceinline__ void edges(int i, int64_t row, int &head, int &tail) const
    {
        constexpr int size = (int)sizeof(Unit<T, VEC>);
        const uint64_t a = reinterpret_cast<uint64_t>(at(i, row)), bytes = (uint64_t)width * sizeof(T);
        const uint64_t lo = (a + 15) & ~15ull, hi = (a + bytes) & ~15ull;
        head = min(width / VEC, (int)((lo - a) / size));
        tail = hi > lo ? (int)((a + bytes - hi) / size) : width / VEC - head;
    }
};

// The edge units of one tensor's row that are this thread's columns (at most
// one of either edge), loaded a row ahead and put into the row's stage before
// the thread reads it: a thread reads its own columns only, so no barrier lies
// between.
template <typename T, int VEC>
struct Edge {
    Unit<T, VEC> head, tail;
    int head_at, tail_at;   // units, or -1
};

template <typename T, int VEC, int NT>
__device__ __forceinline__ void load_edge(const Ring<T, VEC, NT> &ring, int i, int64_t row, int gt, int gsize,
                                          Edge<T, VEC> &e)
{
    if constexpr (!kAligned<T, VEC>) {
        e.head_at = e.tail_at = -1;
        if (row < ring.rows) {
            int head, tail;
            ring.edges(i, row, head, tail);
            const Unit<T, VEC> *p = reinterpret_cast<const Unit<T, VEC> *>(ring.at(i, row));
            if (gt < head) {
                e.head_at = gt;
                e.head = p[gt];
            }
            // the last units, at most 15: those congruent to gt modulo the group's size
            const int n = ring.width / VEC, t0 = n - tail, d = (gt - t0) % gsize, c = t0 + (d < 0 ? d + gsize : d);
            if (c < n) {
                e.tail_at = c;
                e.tail = p[c];
            }
        }
    }
}

// Tensor i of the current row `row` in its stage.
template <typename T, int VEC, int NT>
__device__ __forceinline__ T *stage_row(const Ring<T, VEC, NT> &ring, int i, int row)
{
    unsigned char *s = ring.mem + (ring.stage * NT + i) * ring.tensor_bytes;
    if constexpr (!kAligned<T, VEC>) s += reinterpret_cast<uint64_t>(ring.at(i, row)) & 15u;
    return reinterpret_cast<T *>(s);
}

template <typename T, int VEC, int NT>
__device__ __forceinline__ void put_edge(const Ring<T, VEC, NT> &ring, int i, int row, const Edge<T, VEC> &edge)
{
    if constexpr (!kAligned<T, VEC>) {
        auto *p = reinterpret_cast<Unit<T, VEC> *>(stage_row(ring, i, row));
        if (edge.head_at >= 0) p[edge.head_at] = edge.head;
        if (edge.tail_at >= 0) p[edge.tail_at] = edge.tail;
    }
}

__device__ __forceinline__ float2 widen2(uint32_t u, __half)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}
__device__ __forceinline__ float2 widen2(uint32_t u, __nv_bfloat16)
{
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

__device__ __forceinline__ uint32_t narrow2(float2 f, __half)
{
    const __half2 h = __floats2half2_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t narrow2(float2 f, __nv_bfloat16)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A thread's COLS columns of one row, in the storage type; zero past the slice:
// the vectors (units) gt, gt + gsize, ... of VEC columns.  The arithmetic goes
// over pairs (packed fp32), which halves its instructions.
template <typename T, int VEC, int COLS>
struct Cols {
    static constexpr bool ALIGNED = kAligned<T, VEC>;
    static constexpr int NVEC = COLS / VEC;
    static constexpr int PAIRS = COLS / 2;
    uint4 v[ALIGNED ? NVEC : 1];
    Unit<T, VEC> e[ALIGNED ? 1 : NVEC];

    template <int NT>
    __device__ __forceinline__ void load(const Ring<T, VEC, NT> &ring, int i, int row, int gt, int gsize)
    {
        const T *p = stage_row(ring, i, row);
        const int n = ring.width / VEC;
#pragma unroll
        for (int k = 0; k < NVEC; ++k) {
            const int c = gt + k * gsize;
            if constexpr (ALIGNED) v[k] = c < n ? reinterpret_cast<const uint4 *>(p)[c] : make_uint4(0, 0, 0, 0);
            else if constexpr (VEC == 2) e[k] = c < n ? reinterpret_cast<const uint32_t *>(p)[c] : 0u;
            else if (c < n) e[k] = p[c];
            else narrow(e[k], 0.0f);
        }
    }
    // values 2p and 2p + 1
    __device__ __forceinline__ float2 get(int p) const
    {
        if constexpr (VEC == 2) {
            return widen2(e[p], T());
        } else if constexpr (VEC == 1) {
            return make_float2(widen(e[2 * p]), widen(e[2 * p + 1]));
        } else {
            constexpr int PER = VEC / 2;   // pairs per vector
            const uint4 &u = v[p / PER];
            if constexpr (sizeof(T) == 4)
                return p % PER ? make_float2(__uint_as_float(u.z), __uint_as_float(u.w))
                               : make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
            else
                return widen2(p % PER == 0 ? u.x : p % PER == 1 ? u.y : p % PER == 2 ? u.z : u.w, T());
        }
    }
    // column of value j within the slice
    __device__ __forceinline__ static int col(int j, int gt, int gsize) { return (gt + j / VEC * gsize) * VEC + j % VEC; }

    // whether value j lies in the slice (a vector does as a whole or not at all)
    __device__ __forceinline__ static bool inside(int j, int gt, int gsize, int width)
    {
        return gt + j / VEC * gsize < width / VEC;
    }

    __device__ __forceinline__ static void store(T *dst, int width, int gt, int gsize, const float2 (&f)[PAIRS])
    {
        if constexpr (ALIGNED) {
            const int n = width / VEC;
#pragma unroll
            for (int k = 0; k < NVEC; ++k) {
                const int c = gt + k * gsize;
                float w[VEC];
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    w[2 * j] = f[k * (VEC / 2) + j].x;
                    w[2 * j + 1] = f[k * (VEC / 2) + j].y;
                }
                if (c < n) st_stream(dst + c * VEC, repack<T>(w));
            }
        } else if constexpr (VEC == 2) {
#pragma unroll
            for (int p = 0; p < PAIRS; ++p)
                if (gt + p * gsize < width / 2) reinterpret_cast<uint32_t *>(dst)[gt + p * gsize] = narrow2(f[p], T());
        } else {
#pragma unroll
            for (int p = 0; p < PAIRS; ++p) {
                const int c = gt + 2 * p * gsize;
                if (c < width) narrow(dst[c], f[p].x);
                if (c + gsize < width) narrow(dst[c + gsize], f[p].y);
            }
        }
    }
};

// Barrier of one row group (a warp needs none).  NAMED: several groups of more
// than a warp share the CTA.  A kernel with named barriers takes all 16 of
// them, which limits the CTAs of an SM (1024-column rows in CTAs of one group:
// 59 us instead of 34), so one-group CTAs use the CTA's own.
template <bool NAMED>
__device__ __forceinline__ void group_sync(int gsize)
{
    if constexpr (NAMED) {
        __syncwarp();
        asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / gsize), "r"(gsize) : "memory");
    } else {
        cta_sync();
    }
}

__device__ __forceinline__ float warp_sum(float a)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    return a;
}

// Sums over the row group, in every thread of it.  `red` (one entry per warp of
// the CTA) is a buffer no thread of the group may still be reading: callers
// alternate two of them, and between a read and the next write of one lies the
// other one's barrier.
template <bool NAMED>
__device__ __forceinline__ float2 group_sum2(float a, float b, int gsize, float2 *red)
{
    a = warp_sum(a);
    b = warp_sum(b);
    if (gsize == 32) {
        __syncwarp();   // the lanes' reads of the stage come before its refill
        return make_float2(a, b);
    }
    const int warp = threadIdx.x >> 5, nw = gsize >> 5, w0 = warp / nw * nw;
    if ((threadIdx.x & 31) == 0) red[warp] = make_float2(a, b);
    group_sync<NAMED>(gsize);
    // the warps' pairs, all of them added in every lane (up to 16 by each half-warp)
    const int lane = nw > 16 ? threadIdx.x & 31 : threadIdx.x & 15;
    float2 t = lane < nw ? red[w0 + lane] : make_float2(0.0f, 0.0f);
    if (nw > 16) {
        t.x += __shfl_xor_sync(0xffffffffu, t.x, 16);
        t.y += __shfl_xor_sync(0xffffffffu, t.y, 16);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
        t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
    }
    return t;
}

template <bool NAMED>
__device__ __forceinline__ float group_sum(float a, int gsize, float2 *red)
{
    a = warp_sum(a);
    if (gsize == 32) {
        __syncwarp();
        return a;
    }
    const int warp = threadIdx.x >> 5, nw = gsize >> 5, w0 = warp / nw * nw;
    if ((threadIdx.x & 31) == 0) red[warp].x = a;
    group_sync<NAMED>(gsize);
    const int lane = nw > 16 ? threadIdx.x & 31 : threadIdx.x & 15;
    float t = lane < nw ? red[w0 + lane].x : 0.0f;
    if (nw > 16) t += __shfl_xor_sync(0xffffffffu, t, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return t;
}

// Exchange of one pair per CTA and row over a cluster: every CTA pushes its
// pair into slot[parity][its rank] of every CTA (st.async, completing on that
// CTA's barrier) and waits for all of them.  Double-buffered by row parity: a
// peer is at most one row ahead, since it cannot finish row i+1 without this
// CTA's pair of row i+1, sent after this CTA has read its slots of row i.
struct Exchange {
    float2 (*slot)[kMaxRanks];
    uint64_t *bar;
    uint32_t rank, nranks;
    uint64_t wait_ns;
    uint32_t *err;
    bool failed;

    // `pair` is held by every thread; returns the slots of this row.
    __device__ __forceinline__ const float2 *swap(float2 pair, int it)
    {
        const int p = it & 1;
        if (threadIdx.x == 0 && !failed) ptx::mbar_arrive_expect_tx(&bar[p], nranks * 8u);
        if (threadIdx.x < nranks)
            ptx::st_async_f32x2(ptx::mapa_shared(&slot[p][rank], threadIdx.x), pair.x, pair.y,
                                ptx::mapa_shared(&bar[p], threadIdx.x));
        if (!failed && !ptx::mbar_wait<true>(&bar[p], (uint32_t)(it >> 1) & 1u, wait_ns)) {
            failed = true;
            atomicOr(err, TF_DEVERR_EXCHANGE_WAIT);
        }
        return slot[p];
    }
};

// Shared set-up of both kernels: this thread's ring, with its barriers
// initialised and the first rows on their way.
template <typename T, int VEC, bool CLUSTER, int NT>
__device__ __forceinline__ Ring<T, VEC, NT> start_ring(const Geometry &g, unsigned char *smem, const Sources &src,
                                                           int hidden, int rows, int unit, int units, int c0,
                                                           uint32_t *err, uint64_t wait_ns, uint64_t *xbar)
{
    const int gid = threadIdx.x / g.group, ngroups = g.threads / g.group;
    Ring<T, VEC, NT> r{src,
                           smem + (size_t)gid * g.stages * NT * g.tensor_bytes,
                           reinterpret_cast<uint64_t *>(smem + g.bar_off) + gid * g.stages,
                           g.stages,
                           g.tensor_bytes,
                           c0,
                           min(hidden - c0, g.slice),
                           unit + gid * units,
                           units * ngroups,
                           rows,
                           wait_ns,
                           err,
                           false,
                           0,
                           0u,
                           0u};
    const bool issuer = threadIdx.x % g.group == 0;
    if (issuer) {
        for (int s = 0; s < g.stages; ++s) ptx::mbar_init(&r.full[s], 1);
        if (CLUSTER)
            for (int p = 0; p < 2; ++p) ptx::mbar_init(&xbar[p], 1);
        ptx::mbar_init_fence();
        for (int s = 0; s < g.stages; ++s) r.issue(s, r.first + (int64_t)s * r.step);
    }
    if constexpr (CLUSTER) ptx::cluster_sync();   // every CTA's exchange barriers exist before the first push
    else cta_sync();
    return r;
}

// ---------------------------------------------------------------- host side

// Rows of `hidden` columns, `tensors` of them streaming in, in a kernel whose
// threads take `cols` columns, `vec` at once, and of which an SM holds
// `sm_threads` threads.  MERGED: all the row groups of an SM in one CTA (whose column sums then leave
// the SM once).
inline Geometry geometry(int64_t hidden, int size, int vec, int cols, int tensors, int sm_threads, bool merged,
                         int64_t rows, int tables = 0)
{
    Geometry g;
    const bool aligned = vec * size == 16;
    const int csize = (int)((hidden + kSlice - 1) / kSlice);
    const int64_t slice = ((hidden + csize - 1) / csize + vec - 1) / vec * vec;
    g.csize = (int)((hidden + slice - 1) / slice);   // no CTA without columns
    g.slice = (int)slice;
    // element-wise groups are constants of the kernels: 32, multiples of 64, above 512 of 128
    const int step = aligned || slice <= 32 * cols ? 32 : slice <= 512 * cols ? 64 : 128;
    g.group = (int)(((slice + cols - 1) / cols + step - 1) / step * step);
    if (!aligned && cols > 8) g.group = kClusterGroup;
    g.tensor_bytes = (int)((slice * size + 15) / 16 * 16) + (aligned ? 0 : 32);
    const int ring = tensors * g.tensor_bytes + 8;
    // row groups per SM: as many as the registers hold, fewer where shared
    // memory has no room for two stages of each
    const bool one_cta = merged && g.csize == 1;
    // `tables` of the kernel's parameters (gamma, beta) per CTA
    const int sm_bytes = 226 * 1024, table_bytes = tables * cols * g.group * 4;
    auto room = [&](int n) {   // of one of n groups, past a CTA's own 2 KB (static memory, and what the system keeps)
        return one_cta ? (sm_bytes - 2048 - table_bytes) / n : sm_bytes / n - 2048 - table_bytes;
    };
    int groups = sm_threads / g.group;
    if (groups < 1) groups = 1;
    if (g.group > 32 && merged && groups > 15) groups = 15;   // named barriers
    while (groups > 1 && room(groups) < 2 * ring) --groups;
    const int64_t sms = sm_count();
    if (one_cta) {
        const int64_t need = (rows + sms - 1) / sms;
        if (groups > need) groups = need < 1 ? 1 : (int)need;
    }
    int stages = room(groups) / ring;
    if (stages > kMaxStages) stages = kMaxStages;
    if (stages < 1) stages = 1;
    g.stages = stages;
    const int in_cta = g.group == 32 && !merged ? (groups < 8 ? groups : 8) : one_cta ? groups : 1;
    g.threads = in_cta * g.group;
    g.per_sm = groups / in_cta;
    g.bar_off = in_cta * stages * tensors * g.tensor_bytes;
    g.gamma_off = (g.bar_off + in_cta * stages * 8 + 15) / 16 * 16;
    g.smem = g.gamma_off + table_bytes;
    // half the groups' column sums at a time lie there to be added
    if (merged && g.smem < in_cta / 2 * 8 * cols * g.group) g.smem = in_cta / 2 * 8 * cols * g.group;
    return g;
}

// CTAs (clusters) to launch for `rows` rows: as many as share the GPU at once,
// at most one row group per row.
inline int64_t launch_units(const Geometry &g, int64_t rows)
{
    const int in_cta = g.threads / g.group;
    int64_t units = (int64_t)sm_count() * g.per_sm / g.csize;
    const int64_t need = (rows + in_cta - 1) / in_cta;
    if (units > need) units = need;
    return units < 1 ? 1 : units;
}

// Clusters of this many CTAs, one CTA per SM, that the GPU holds at once: fewer
// than its SMs would make, since a cluster lies in one GPC.  (Too many run as a
// second wave: 2048 x 32768 bf16 forward took 190 us instead of 105.)
template <typename... KArgs>
cudaError_t resident_clusters(int *clusters, cudaLaunchConfig_t cfg, void (*kern)(KArgs...), int csize)
{
    const void *key = reinterpret_cast<const void *>(kern);
    if (recall(key, FACT_CLUSTERS + csize, clusters)) return cudaSuccess;
    cfg.blockDim = dim3(kClusterGroup);   // whose registers fill an SM, whatever the rows' width
    if (cudaOccupancyMaxActiveClusters(clusters, kern, &cfg) != cudaSuccess || *clusters < 1) {
        cudaGetLastError();
        return cudaErrorNotSupported;
    }
    remember(key, FACT_CLUSTERS + csize, *clusters);
    return cudaSuccess;
}

// `units` CTAs or clusters, at most as many as run at once.  No kernel (null)
// where none is built for the geometry's row groups: one built for others would
// wait at its barriers for threads that are not there.
template <typename... KArgs, typename... Args>
cudaError_t launch_rows(void (*kern)(KArgs...), const Geometry &g, int64_t &units, cudaStream_t st, Args... args)
{
    if (!kern) return cudaErrorNotSupported;
    const void *key = reinterpret_cast<const void *>(kern);
    cudaError_t e = raise_smem_limit(key);
    int allowed = 0;
    if (e == cudaSuccess && g.csize > 8 && !recall(key, FACT_WIDE_CLUSTERS, &allowed)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess) remember(key, FACT_WIDE_CLUSTERS, 1);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();   // a refused attribute is not an error of the caller's stream
        return cudaErrorNotSupported;
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see pdl_begin()
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)g.csize;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * g.csize));
    cfg.blockDim = dim3((unsigned)g.threads);
    cfg.dynamicSmemBytes = (size_t)g.smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = g.csize > 1 ? 2 : 1;
    // Clusters of 3, 5, 6 or 7 CTAs wait for the previous kernel's end: placed while its CTAs leave one by one,
    // fewer of them find room (3300 x 20480 bf16, backward: 200 us instead of 148).
    if (g.csize & (g.csize - 1)) {
        cfg.attrs = attr + 1;
        cfg.numAttrs = 1;
    }
    if (g.csize > 1) {
        int most = 0;
        e = resident_clusters(&most, cfg, kern, g.csize);
        if (e != cudaSuccess) return e;
        if (units > most) units = most;
        cfg.gridDim = dim3((unsigned)(units * g.csize));
    }
    return counted(cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...));
}

inline bool aligned_rows(const void *p, int64_t stride, int size, int bytes)
{
    return !p || (reinterpret_cast<uintptr_t>(p) % (unsigned)bytes == 0 && stride * size % bytes == 0);
}

}  // namespace norm
}  // namespace tf
