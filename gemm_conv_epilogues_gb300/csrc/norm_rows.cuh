// Row streaming shared by the layer-norm kernels (forward with statistics,
// backward): the rows of up to three tensors pass through a ring of
// shared-memory stages filled by bulk copies, so several rows per SM are on
// their way while one is reduced, and every element is read from HBM once.
//
// A row group (one warp for rows of at most 512 columns, else the whole CTA)
// works on one row at a time, each thread on kCols columns of it, held in fp32
// registers.  Rows wider than kSlice columns are cut into slices over the
// CTAs of a cluster.
//
// Alignment.  With every row start a multiple of 16 bytes (ALIGNED) a row is
// one bulk copy and a thread's columns are 16-byte vectors.  Otherwise the
// copy takes the 16-byte pieces that lie inside the row, at the same offset
// from a 16-byte boundary in shared memory as in global memory; the up to 15
// bytes before and behind them are loaded one row ahead by the threads whose
// columns they are (copying them too would read past the tensor's ends).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "ptx_sm100.cuh"
#include "train_internal.h"

namespace tf {
namespace norm {

constexpr int kCols = 16;                 // columns per thread
constexpr int kWarpCols = 32 * kCols;     // rows up to this width take one warp
constexpr int kMaxThreads = 512;
constexpr int kSlice = kMaxThreads * kCols;   // widest slice of one CTA
constexpr int kWarpRowThreads = 256;      // CTA of warp rows: eight rows at a time
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
    int group;          // threads per row: 32, or the CTA
    int threads;        // threads per CTA
    int csize, slice;   // CTAs per row and columns per CTA
    int tensors, stages, tensor_bytes;   // ring of one row group: stages x tensors x tensor_bytes
    int bar_off;        // mbarriers behind the rings
    int smem;
};

// The tensors whose rows stream in (a kernel parameter).
struct Sources {
    const void *base[kMaxTensors];
    int64_t stride[kMaxTensors];
};

// What one thread knows of its row group's ring of NT tensors.
template <typename T, bool ALIGNED, int NT>
struct Ring {
    const Sources &src;
    unsigned char *mem;
    uint64_t *full;
    int stages, tensor_bytes, c0, width;        // width: columns of this CTA's slice, from c0 on
    int64_t first, step, rows;                  // this group's rows: first, first + step, ...
    uint64_t wait_ns;
    uint32_t *err;
    bool failed;
    int issued, used;

    __device__ __forceinline__ const T *at(int i, int64_t row) const {
        return reinterpret_cast<const T *>(src.base[i]) + (row * src.stride[i] + c0);
    }

    // Copies the group's it-th row into its stage (one thread of the group).
    __device__ __forceinline__ void issue(int it)
    {
        const int64_t row = first + it * step;
        if (row >= rows || failed) return;
        unsigned char *dst = mem + (it % stages) * NT * tensor_bytes;
        uint64_t *bar = &full[it % stages];
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
        issued = it + 1;
    }

    __device__ __forceinline__ void wait(int it)
    {
        if (!failed && !ptx::mbar_wait(&full[it % stages], (uint32_t)(it / stages) & 1u, wait_ns)) {
            failed = true;
            atomicOr(err, TF_DEVERR_PRODUCER_WAIT);
        }
        used = it + 1;
    }

    // Copies issued but never waited for (after a time-out only) land before the CTA exits.
    __device__ __forceinline__ void drain()
    {
        for (int k = used; k < issued; ++k)
            if (!ptx::mbar_wait(&full[k % stages], (uint32_t)(k / stages) & 1u, wait_ns))
                atomicOr(err, TF_DEVERR_DRAIN_WAIT);
    }

    // Columns of row `it` of tensor i that lie before and behind the copied pieces.
    __device__ __forceinline__ void edges(int i, int64_t row, int &head, int &tail) const
    {
        const uint64_t a = reinterpret_cast<uint64_t>(at(i, row)), bytes = (uint64_t)width * sizeof(T);
        const uint64_t lo = (a + 15) & ~15ull, hi = (a + bytes) & ~15ull;
        head = min(width, (int)((lo - a) / sizeof(T)));
        tail = hi > lo ? (int)((a + bytes - hi) / sizeof(T)) : width - head;
    }
};

// A thread's (at most one) column of either edge of one tensor, loaded ahead.
struct Edge {
    float head, tail;
};

template <typename T, bool ALIGNED, int NT>
__device__ __forceinline__ Edge load_edge(const Ring<T, ALIGNED, NT> &ring, int i, int64_t row, int gt, int gsize)
{
    Edge e = {0.0f, 0.0f};
    if constexpr (!ALIGNED) {
        if (row < ring.rows) {
            int head, tail;
            ring.edges(i, row, head, tail);
            const T *p = ring.at(i, row);
            if (gt < head) e.head = widen(p[gt]);
            // the tail column of this thread: the one congruent to gt modulo the group's size
            const int t0 = ring.width - tail;
            int c = t0 + ((gt - t0) % gsize + gsize) % gsize;
            if (c < ring.width) e.tail = widen(p[c]);
        }
    }
    return e;
}

// The thread's kCols columns of tensor i of the group's it-th row, fp32; zero past the slice.
template <typename T, bool ALIGNED, int NT>
__device__ __forceinline__ void load_cols(const Ring<T, ALIGNED, NT> &ring, int i, int it, int gt, int gsize,
                                          const Edge &edge, float (&f)[kCols])
{
    constexpr int VEC = 16 / (int)sizeof(T);
    const unsigned char *src = ring.mem + ((it % ring.stages) * NT + i) * ring.tensor_bytes;
    if constexpr (ALIGNED) {
        const int nvec = ring.width / VEC;
#pragma unroll
        for (int k = 0; k < kCols / VEC; ++k) {
            const int v = gt + k * gsize;
            uint4 u = make_uint4(0, 0, 0, 0);
            if (v < nvec) u = reinterpret_cast<const uint4 *>(src)[v];
            unpack<T>(u, f + k * VEC);
        }
    } else {
        const int64_t row = ring.first + it * ring.step;
        int head, tail;
        ring.edges(i, row, head, tail);
        const T *p = reinterpret_cast<const T *>(src + (reinterpret_cast<uint64_t>(ring.at(i, row)) & 15u));
#pragma unroll
        for (int k = 0; k < kCols; ++k) {
            const int c = gt + k * gsize;
            f[k] = c >= ring.width ? 0.0f : c < head ? edge.head : c >= ring.width - tail ? edge.tail : widen(p[c]);
        }
    }
}

// The same columns, left in the storage type until they are needed (half the registers for 16-bit types).
template <typename T, bool ALIGNED>
struct Held {
    uint4 raw[ALIGNED ? kCols * (int)sizeof(T) / 16 : 1];
    T one[ALIGNED ? 1 : kCols];
};

template <typename T, bool ALIGNED, int NT>
__device__ __forceinline__ void hold_cols(const Ring<T, ALIGNED, NT> &ring, int i, int it, int gt, int gsize,
                                          const Edge &edge, Held<T, ALIGNED> &h)
{
    if constexpr (ALIGNED) {
        constexpr int VEC = 16 / (int)sizeof(T);
        const unsigned char *src = ring.mem + ((it % ring.stages) * NT + i) * ring.tensor_bytes;
#pragma unroll
        for (int k = 0; k < kCols / VEC; ++k) {
            const int v = gt + k * gsize;
            h.raw[k] = v < ring.width / VEC ? reinterpret_cast<const uint4 *>(src)[v] : make_uint4(0, 0, 0, 0);
        }
    } else {
        float f[kCols];
        load_cols(ring, i, it, gt, gsize, edge, f);
#pragma unroll
        for (int k = 0; k < kCols; ++k) narrow(h.one[k], f[k]);   // exact: the value came from T
    }
}

// f += the held columns.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void add_held(const Held<T, ALIGNED> &h, float (&f)[kCols])
{
    if constexpr (ALIGNED) {
        constexpr int VEC = 16 / (int)sizeof(T);
#pragma unroll
        for (int k = 0; k < kCols / VEC; ++k) {
            float v[VEC];
            unpack<T>(h.raw[k], v);
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[k * VEC + j] += v[j];
        }
    } else {
#pragma unroll
        for (int k = 0; k < kCols; ++k) f[k] += widen(h.one[k]);
    }
}

// Column of the thread's j-th value within its slice.
template <typename T, bool ALIGNED>
__device__ __forceinline__ int col_of(int j, int gt, int gsize)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    return ALIGNED ? (gt + j / VEC * gsize) * VEC + j % VEC : gt + j * gsize;
}

template <typename T, bool ALIGNED>
__device__ __forceinline__ void store_cols(T *dst, int width, int gt, int gsize, const float (&f)[kCols])
{
    constexpr int VEC = 16 / (int)sizeof(T);
    if constexpr (ALIGNED) {
#pragma unroll
        for (int k = 0; k < kCols / VEC; ++k) {
            const int v = gt + k * gsize;
            if (v * VEC < width) st_stream(dst + v * VEC, repack<T>(f + k * VEC));
        }
    } else {
#pragma unroll
        for (int k = 0; k < kCols; ++k) {
            const int c = gt + k * gsize;
            if (c < width) narrow(dst[c], f[k]);
        }
    }
}

// Sums of two values over the row group, in every thread of it.  `red` is a
// buffer no thread may still be reading: callers alternate two of them, and
// between a read and the next write of one lies the other one's barrier.
__device__ __forceinline__ float2 group_sum(float a, float b, int gsize, float2 *red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (gsize == 32) return make_float2(a, b);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
    cta_sync();
    const int lane = threadIdx.x & 31;
    float2 t = lane < (gsize >> 5) ? red[lane] : make_float2(0.0f, 0.0f);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
        t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
    }
    return make_float2(__shfl_sync(0xffffffffu, t.x, 0), __shfl_sync(0xffffffffu, t.y, 0));
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

__device__ __forceinline__ uint32_t cluster_nctarank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// Shared set-up of both kernels: this thread's ring, with its barriers
// initialised and the first rows on their way.
template <typename T, bool ALIGNED, bool CLUSTER, int NT>
__device__ __forceinline__ Ring<T, ALIGNED, NT> start_ring(const Geometry &g, unsigned char *smem, const Sources &src,
                                                           int hidden, int64_t rows, int64_t unit, int64_t units, int c0,
                                                           uint32_t *err, uint64_t wait_ns, uint64_t *xbar)
{
    const int gid = threadIdx.x / g.group, ngroups = g.threads / g.group;
    Ring<T, ALIGNED, NT> r{src,
                           smem + (size_t)gid * g.stages * NT * g.tensor_bytes,
                           reinterpret_cast<uint64_t *>(smem + g.bar_off) + gid * g.stages,
                           g.stages,
                           g.tensor_bytes,
                           c0,
                           min(hidden - c0, g.slice),
                           unit * ngroups + gid,
                           units * ngroups,
                           rows,
                           wait_ns,
                           err,
                           false,
                           0,
                           0};
    const bool issuer = threadIdx.x % g.group == 0;
    if (issuer) {
        for (int s = 0; s < g.stages; ++s) ptx::mbar_init(&r.full[s], 1);
        if (CLUSTER)
            for (int p = 0; p < 2; ++p) ptx::mbar_init(&xbar[p], 1);
        ptx::mbar_init_fence();
        for (int s = 0; s < g.stages; ++s) r.issue(s);
    }
    if constexpr (CLUSTER) ptx::cluster_sync();   // every CTA's exchange barriers exist before the first push
    else cta_sync();
    return r;
}

// ---------------------------------------------------------------- host side

// `ctas` of `threads` threads and 128 registers each share an SM's registers
// and its 227 KB of shared memory.
inline Geometry geometry(int64_t hidden, int size, bool aligned, int tensors)
{
    Geometry g;
    const int vec = aligned ? 16 / size : 1;
    int csize = (int)((hidden + kSlice - 1) / kSlice);
    int64_t slice = ((hidden + csize - 1) / csize + vec - 1) / vec * vec;
    csize = (int)((hidden + slice - 1) / slice);   // no CTA without columns
    g.csize = csize;
    g.slice = (int)slice;
    if (hidden <= kWarpCols) {
        g.group = 32;
        g.threads = kWarpRowThreads;
    } else {
        const int64_t per = (slice + kCols - 1) / kCols;
        int t = 64;
        while (t < per) t *= 2;
        g.group = g.threads = t;
    }
    g.tensors = tensors;
    g.tensor_bytes = (int)((slice * size + 15) / 16 * 16) + (aligned ? 0 : 32);
    const int groups = g.threads / g.group;
    const int per_sm = kMaxThreads / g.threads;
    const int budget = 224 * 1024 / per_sm - 2048;
    int stages = budget / (groups * tensors * g.tensor_bytes + groups * 8);
    if (stages > kMaxStages) stages = kMaxStages;
    if (stages < 1) stages = 1;
    g.stages = stages;
    g.bar_off = groups * stages * tensors * g.tensor_bytes;
    g.smem = g.bar_off + groups * stages * 8;
    if (g.group == 32 && g.smem < 2 * kWarpCols * 4) g.smem = 2 * kWarpCols * 4;   // the backward pass adds its warps' sums there
    return g;
}

// CTAs (clusters) to launch for `rows` rows: as many as share the GPU at once,
// at most one row group per row.
inline int64_t launch_units(const Geometry &g, int64_t rows)
{
    const int groups = g.threads / g.group;
    int64_t units = (int64_t)sm_count() * (kMaxThreads / g.threads) / g.csize;
    const int64_t need = (rows + groups - 1) / groups;
    if (units > need) units = need;
    return units < 1 ? 1 : units;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_rows(void (*kern)(KArgs...), const Geometry &g, int64_t units, cudaStream_t st, Args... args)
{
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, g.smem);
    if (e == cudaSuccess && g.csize > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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
    return counted(cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...));
}

inline bool aligned_rows(const void *p, int64_t stride, int size)
{
    return !p || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && stride * size % 16 == 0);
}

}  // namespace norm
}  // namespace tf
