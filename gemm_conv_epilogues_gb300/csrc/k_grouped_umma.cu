// Grouped products on the 5th-generation tensor cores.
//
// The weights' side is the MMA's M side and the rows (tokens) are its N side:
//   FORWARD  D[n][m] = sum_k w[e][n][k] x[m][k]     A = w (K-major),   B = x (K-major)
//   DGRAD    D[k][m] = sum_n w[e][n][k] dy[m][n]    A = w (M-major),   B = dy (K-major)
//   WGRAD    D[n][k] = sum_m dy[m][n] x[m][k]       A = dy (M-major),  B = x (N-major)
// A group has any number of rows while the weights' extents are whole tiles:
// with the rows on the N side, whose size an MMA takes in steps of 16, a
// ragged group costs the tensor cores its rows rounded up to 16 (32 on CTA
// pairs) where tiles of 128 or 256 rows would be half empty on average, and a
// group of one to sixteen rows streams its weights past the smallest MMA.  A
// group's rows are cut into tiles of equal width.
//
// Persistent kernel, one CTA (CG = 1) or CTA pair (CG = 2, cta_group::2) per SM
// (pair), work items (group, weights tile, row tile) from a schedule that every
// CTA computes from the offsets.  Warps:
//   0     TMA producer of a ring of K steps (64 deep, 128-byte swizzle)
//   1     TMEM allocator and MMA issuer; two 256-column fp32 accumulators, so
//         the epilogue of one tile overlaps the main loop of the next
//   2     WGRAD: zeroes what the last K step of a group holds of other rows
//   3     lists the CTA's coming items, 32 at a time, so that the issuing warps
//         do not stop for their searches and divisions
//   4-11  epilogue: TMEM -> registers -> bias, activation -> y
//   12-15 WGRAD: the bias gradient, from dy itself, beside the products (188 us
//         without it, 195 with it, 228 in a kernel of its own, which reads dy
//         once more)
//
// What bounds it, at 16384 rows in 16 uneven groups, bf16, weights 4096 x 2048
// (275 GFLOP; 142.7 us at the tensor cores' burst rate, 157.5 at the sustained one):
//   FORWARD with bias, GELU and the pre-activation saved: 174-178 us (207 in a
//     loop, under the power cap), 1.55-1.58
//     PFLOP/s, tensor pipe 75% busy; 159 without the epilogue's stores, and the
//     operands' loads alone take 146 (64 bytes per clock and SM from L2)
//   DGRAD with GELU's slope: 174-178 us (206 in a loop)
//   WGRAD with dbias: 251-256 us; the fp32 dw, 128 KB per tile, leaves the SM at
//     about 13 bytes per clock whichever way it is stored (fragments, 128-byte
//     rows or TMA), and the writes keep the loads waiting.  For a group of more
//     than 1024 rows (half of the rows here) the epilogue holds both accumulators
//     until its last store, so that the next item's MMAs do not run under it
//   16 rows in 16 groups of 2048 x 4096 (decoding): 39.5 us, 6.0 TB/s of weights
// Every wait is bounded (ptx::mbar_wait); a role that times out sets the
// device error word and winds down.
#include <cuda.h>

#include <mutex>
#include <type_traits>

#include "grouped.cuh"
#include "ptx_sm100.cuh"
#include "tensor_maps.h"

namespace tf {
namespace {

using namespace grouped;

constexpr int BM = 128;                 // weights rows per CTA (UMMA M, or half of the pair's 256)
constexpr int kMaxBN = 256;             // widest row tile: one accumulator is 256 TMEM columns
constexpr int kMaxStages = 24;
constexpr int kEpiWarps = 8, kFirstEpiWarp = 4;
constexpr int kBiasWarps = 4;           // WGRAD: warps that sum dy's columns for the bias gradient
constexpr int threads_of(int mode) { return 32 * (kFirstEpiWarp + kEpiWarps + (mode == GROUPED_WGRAD ? kBiasWarps : 0)); }
constexpr int kSmemLimit = 227 * 1024;
constexpr int kABytes = BM * BK * 2;
constexpr int kNumBars = 3 * kMaxStages + 9;      // full, empty, land; accumulators full x2, empty x2; drain;
                                                  // item lists ready x2, free x2
constexpr int kItemBytes = 64 * 32;               // two lists of 32 items
// An epilogue warp's box, 32 tokens x 32 weights rows of 16 bits: it turns the
// accumulator's columns into rows for 16-byte stores by the threads (TMA stores
// of the same boxes measured the same).
constexpr int kBoxBytes = 32 * 32 * 2;
// WGRAD: rows per accumulation.  The tensor cores truncate where fp32 additions
// round, so an accumulator's error grows with the number of MMAs it takes
// (relative error 1.4e-6 for groups of up to 2459 rows, against 2.9e-7 for fp32
// products).  A longer group is accumulated in parts: the first in one of the
// two accumulators, the second in the other, and the epilogue's threads add
// them; for a third part they leave the sum in the first.  (Adding the parts in
// memory took 316 us for groups of 1025 rows, 208 for 1023.)
constexpr int kMaxPartRows = 1024;
constexpr uint32_t kTmemCols = 512;

struct UmmaArgs {
    const int *offsets;
    const float *bias;
    void *y, *pre;     // WGRAD: y is dw
    uint32_t *err;
    uint64_t wait_ns;
    int64_t y_stride, pre_stride;
    int groups, rows;  // groups: with WGRAD's splits, real groups x splits
    int splits;
    int M;             // extent of the weights' side (N, or K for DGRAD)
    int red;           // reduction length of FORWARD and DGRAD
    int cols;          // WGRAD: K, the N side
    int bn;            // widest row tile the shared memory holds
    int box_rows;      // rows per token box
    int off_epi, off_bar, off_items, off_sched;   // the operand ring comes first
    int act, bf16, accumulate;
    const void *dy;    // WGRAD: for the bias gradient
    float *dbias;
    int64_t dy_stride;
};

__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 TMEM lanes x 32 columns as 8 x 8 blocks: lane l of the warp receives, for
// column block b, row l/4 (registers 4b, 4b+1) and row l/4 + 8 (4b+2, 4b+3),
// columns 8b + 2(l%4) and the next.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Four 8 x 8 blocks between registers and shared memory, transposed on the way:
// a lane's two values of a block are neighbours along a column of the block in
// memory.  Lane l gives the address of row l%8 of block l/8.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// One work item.  FORWARD, DGRAD: weights rows [m0, +128*CG), tokens [t0, +tv), MMA
// N = w.  WGRAD: dw rows [m0, +128*CG), columns [t0, +w) of group e from its rows
// [first, +tv), in `parts` parts of `len` rows (the last one shorter).
struct alignas(16) Item {
    int e, m0, t0, w, tv, first, len, parts;
};
static_assert(sizeof(Item) == 32, "two 16-byte loads");

// The schedule in shared memory: the rows of every group and the running count
// of their tiles.
struct Plan {
    const int *row, *tile;
    int mt;   // weights tiles
};

template <int MODE, int CG>
__device__ __forceinline__ Item item_of(const UmmaArgs &p, const Plan &s, int t)
{
    constexpr int STEP = 16 * CG;
    Item it;
    if (MODE == GROUPED_WGRAD) {
        const int ct = (p.cols + kMaxBN - 1) / kMaxBN, pos = t / (s.mt * ct), r = t - pos * (s.mt * ct);
        it.e = pos;
        it.m0 = r / ct * (BM * CG);
        it.t0 = r % ct * kMaxBN;
        const int left = min(kMaxBN, p.cols - it.t0);
        it.w = (left + 64 * CG - 1) / (64 * CG) * (64 * CG);
        it.first = s.row[it.e];
        it.tv = s.row[it.e + 1] - it.first;
        it.parts = max(1, (it.tv + kMaxPartRows - 1) / kMaxPartRows);
        it.len = ((it.tv + it.parts - 1) / it.parts + BK - 1) / BK * BK;
    } else {
        int lo = 0, hi = p.groups - 1;   // the last group that starts at or before tile t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s.tile[mid] <= t) lo = mid; else hi = mid - 1;
        }
        it.e = lo;
        const int r = t - s.tile[lo], T = s.row[lo + 1] - s.row[lo];
        const int ntt = (T + p.bn - 1) / p.bn;
        const int wt = ((T + ntt - 1) / ntt + STEP - 1) / STEP * STEP;   // equal widths, at most bn
        const int tt = r % ntt;
        it.m0 = r / ntt * (BM * CG);
        it.first = s.row[lo];
        it.t0 = it.first + tt * wt;
        it.tv = min(wt, T - tt * wt);
        it.w = (it.tv + STEP - 1) / STEP * STEP;
        it.parts = 1;
        it.len = 0;
    }
    return it;
}

// The item lists: list i of 32 lies in half i % 2 of the table.
struct Items {
    Item *table;
    uint64_t *ready, *free;
    uint64_t wait_ns;
    int cid, ncl, num_work;
};

// Calls f(item, part, first row, rows, K steps) for every part of every item of
// this CTA or pair, in order, until it returns false; false where a list never
// came.  All lanes of a warp call together.
template <int MODE, int KSUB, typename F>
__device__ __forceinline__ bool each_item(const UmmaArgs &p, const Items &s, F f)
{
    int i = 0;
    for (int t = s.cid; t < s.num_work; t += s.ncl, ++i) {
        const int half = (i >> 5) & 1;
        if ((i & 31) == 0) {
            const bool ok = ptx::mbar_wait(&s.ready[half], (uint32_t)(i >> 6) & 1u, s.wait_ns);
            if (!__all_sync(0xffffffffu, ok)) return false;
        }
        const int4 *src = reinterpret_cast<const int4 *>(&s.table[i & 63]);
        const int4 a = src[0], b = src[1];
        const Item it = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        if constexpr (MODE == GROUPED_WGRAD) {
            // parts are whole K steps but for the last
            for (int part = 0, done = 0; part < it.parts; ++part, done += it.len) {
                const int rows = min(it.len, it.tv - done);
                if (!f(it, part, it.first + done, rows, (rows + BK - 1) / BK)) return true;
            }
        } else {
            if (!f(it, 0, it.first, it.tv, (p.red + BK * KSUB - 1) / (BK * KSUB))) return true;
        }
        if ((i & 31) == 31) {
            __syncwarp();
            if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&s.free[half]);
        }
    }
    return true;
}

// The box [32 tokens][32 weights rows] (64-byte rows, the 16-byte pieces swizzled
// over pairs of rows, so that neither side meets a bank twice) to `count` rows of
// y or pre: four lanes per row.
__device__ __forceinline__ void store_box(void *dst, int64_t stride, const uint8_t *box, int n0, int M, int token, int count)
{
    const int lane = threadIdx.x & 31, piece = lane & 3, n = n0 + 8 * piece;
    uint16_t *out = reinterpret_cast<uint16_t *>(dst) + token * stride + n;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = (lane >> 2) + 8 * i;
        if (r < count && n < M)
            *reinterpret_cast<uint4 *>(out + r * stride) =
                *reinterpret_cast<const uint4 *>(box + r * 64 + ((piece ^ ((r >> 1) & 3)) * 16));
    }
}

// The rows of pre under a chunk, in the registers of the lanes that put them into the box.
__device__ __forceinline__ void load_pre(uint4 (&v)[4], const void *src, int64_t stride, int n0, int M, int token, int count)
{
    const int lane = threadIdx.x & 31, n = n0 + 8 * (lane & 3);
    const uint16_t *in = reinterpret_cast<const uint16_t *>(src) + token * stride + n;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = (lane >> 2) + 8 * i;
        v[i] = r < count && n < M ? __ldg(reinterpret_cast<const uint4 *>(in + r * stride)) : make_uint4(0, 0, 0, 0);
    }
}

// One 32 x 32 chunk of the accumulator, from the fragments of tmem_ld_16x256b_x4
// (r[0..15] weights rows 0..15, r[16..31] rows 16..31): bias and activation
// (FORWARD), or the slope at pre (DGRAD; its rows are in `pre`).
template <typename T, int MODE, int ACT>
__device__ __forceinline__ void finish_chunk(const UmmaArgs &p, const uint32_t (&r)[32], const float (&bias)[4],
                                             const uint4 (&pre)[4], uint8_t *box, int n0, int token, int count)
{
    const int lane = threadIdx.x & 31;
    // this lane's row of each of four blocks that lie side by side along n, tokens 8b + lane%8
    const uint32_t at = ptx::smem_u32(box) + (uint32_t)((lane & 7) * 64 + ((lane >> 3) ^ ((lane >> 1) & 3)) * 16);
    // block b's fragments: weights rows 8j + lane/4, j = 0..3
    auto pair = [&](int b, int j) {
        const int k = (j >> 1) * 16 + 4 * b + 2 * (j & 1);
        return make_float2(__uint_as_float(r[k]), __uint_as_float(r[k + 1]));
    };
    if constexpr (MODE == GROUPED_FORWARD) {
        auto emit = [&](auto value, void *dst, int64_t stride) {
            __syncwarp();   // the box has been read
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = value(fadd2(pair(b, j), dup2(bias[j])));
                    w[j] = Half2Of<T>::pack(v.x, v.y);
                }
                stmatrix_x4_trans(at + b * 512, w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
            store_box(dst, stride, box, n0, p.M, token, count);
        };
        if (p.pre) emit([](float2 z) { return z; }, p.pre, p.pre_stride);
        bool far = false;
        if (ACT != TF_ACT_NONE) {
            float least[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                least[j] = INFINITY;
#pragma unroll
                for (int b = 0; b < 4; ++b) least[j] = fminf(least[j], fminf(pair(b, j).x, pair(b, j).y));
                least[j] += bias[j];   // (adding keeps the order)
            }
            const float all = fminf(fminf(least[0], least[1]), fminf(least[2], least[3]));
            far = __any_sync(0xffffffffu, all < far_from(ACT));
        }
        if (far) emit([](float2 z) { return act_value2<ACT, true>(z); }, p.y, p.y_stride);
        else emit([](float2 z) { return act_value2<ACT, false>(z); }, p.y, p.y_stride);
    } else {
        __syncwarp();
        if (ACT != TF_ACT_NONE) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int q = (lane >> 2) + 8 * i;
                *reinterpret_cast<uint4 *>(box + q * 64 + (((lane & 3) ^ ((q >> 1) & 3)) * 16)) = pre[i];
            }
            __syncwarp();
        }
        auto emit = [&](auto far) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                uint32_t z[4], w[4];
                if (ACT != TF_ACT_NONE) ldmatrix_x4_trans(at + b * 512, z);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float2 v = pair(b, j);
                    if (ACT != TF_ACT_NONE) v = fmul2(v, act_slope2<ACT, decltype(far)::value>(Half2Of<T>::unpack(z[j])));
                    w[j] = Half2Of<T>::pack(v.x, v.y);
                }
                __syncwarp();   // (a block's four rows are read before they are replaced)
                stmatrix_x4_trans(at + b * 512, w[0], w[1], w[2], w[3]);
            }
        };
        bool far = false;
        if (ACT != TF_ACT_NONE) {
            uint32_t least = Half2Of<T>::min2(pre[0].x, pre[0].y);
            least = Half2Of<T>::min2(least, Half2Of<T>::min2(pre[0].z, pre[0].w));
#pragma unroll
            for (int i = 1; i < 4; ++i)
                least = Half2Of<T>::min2(least, Half2Of<T>::min2(Half2Of<T>::min2(pre[i].x, pre[i].y), Half2Of<T>::min2(pre[i].z, pre[i].w)));
            const float2 f = Half2Of<T>::unpack(least);
            far = __any_sync(0xffffffffu, fminf(f.x, f.y) < far_from(ACT));
        }
        if (far) emit(std::true_type());
        else emit(std::false_type());
        __syncwarp();
        store_box(p.y, p.y_stride, box, n0, p.M, token, count);
    }
}

// dbias[e][n] = sum of dy[m][n] over group e's rows, without the pipeline: a warp
// takes 64 columns of a group (16 where that leaves warps without work), 16
// bytes per lane, eight loads in flight, fp32 sums in levels, the lanes' rows
// added in a fixed order.
template <typename T>
__device__ __forceinline__ void bias_grad(const UmmaArgs &p, const Plan &s, int warp)
{
    const int lane = threadIdx.x & 31, warps = (int)gridDim.x * kBiasWarps;
    const int across = p.groups * ((p.M + 63) / 64) >= warps ? 8 : 2, down = 32 / across;
    const int piece = lane % across, r0 = lane / across, chunks = (p.M + 8 * across - 1) / (8 * across);
    for (int u = (int)blockIdx.x * kBiasWarps + warp; u < p.groups * chunks; u += warps) {
        const int e = u / chunks, n = (u % chunks * across + piece) * 8;
        const int lo = s.row[e], hi = s.row[e + 1];
        const uint16_t *src = reinterpret_cast<const uint16_t *>(p.dy) + n;
        float2 sum[4] = {};
        sum_rows(sum, lo + r0, n < p.M ? hi : lo, 8 * down, [&](int m, float2 (&rows)[4]) {
            uint4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = m + i * down < hi ? __ldg(reinterpret_cast<const uint4 *>(src + (int64_t)(m + i * down) * p.dy_stride))
                                         : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    rows[j] = i == 0 ? Half2Of<T>::unpack(w[j]) : fadd2(rows[j], Half2Of<T>::unpack(w[j]));
            }
        });
        __syncwarp();
        for (int o = across; o < 32; o <<= 1)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sum[j].x += __shfl_xor_sync(0xffffffffu, sum[j].x, o);
                sum[j].y += __shfl_xor_sync(0xffffffffu, sum[j].y, o);
            }
        if (r0 == 0 && n < p.M) {
            float *out = p.dbias + (int64_t)e * p.M + n;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                out[2 * j] = p.accumulate ? out[2 * j] + sum[j].x : sum[j].x;
                out[2 * j + 1] = p.accumulate ? out[2 * j + 1] + sum[j].y : sum[j].y;
            }
        }
    }
}

// KSUB: K blocks of 64 per stage.  Handing a stage over takes its issuers ~300
// cycles, so FORWARD and DGRAD take two (pairs, 16384 rows: 185 us against 189
// with one, DGRAD 186 against 195; single CTAs, 16 rows: 39.5 against 43.0, and
// 41.3 with four).  WGRAD, whose last block may be ragged, takes one.
template <int MODE, int CG, int KSUB>
__global__ void __launch_bounds__(threads_of(MODE), 1)
    grouped_umma_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                        const __grid_constant__ UmmaArgs p)
{
    constexpr bool PAIR = CG == 2;
    constexpr bool WG = MODE == GROUPED_WGRAD;
    constexpr bool A_MMAJOR = MODE != GROUPED_FORWARD;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + p.off_bar);
    uint64_t *empty = full + kMaxStages;
    uint64_t *land = empty + kMaxStages;    // WGRAD: this CTA's copies of a group's ragged last K step
    uint64_t *tfull = land + kMaxStages;
    uint64_t *tempty = tfull + 2;
    uint64_t *drain = tempty + 2;
    uint64_t *ready = drain + 1, *freed = ready + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(freed + 2);
    int *row = reinterpret_cast<int *>(smem + p.off_sched);      // [groups + 1]
    int *tile = row + p.groups + 1;                              // [groups + 1]
    int *bad = tile + p.groups + 1;                              // the offsets are invalid
    volatile int *dead = bad + 1;                                // a role has given up

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int crank = PAIR ? (int)ptx::cluster_ctarank() : 0;
    const int cid = (int)blockIdx.x / CG, ncl = (int)gridDim.x / CG;
    const bool leader = crank == 0;

    if (threadIdx.x < kMaxStages) {
        // WGRAD: one arrival per CTA, from the producers' side (which arrives CG times for a whole
        // K step) or from the CTAs' zeroing warps (a ragged one)
        ptx::mbar_init(&full[threadIdx.x], WG ? CG : 1);
        ptx::mbar_init(&empty[threadIdx.x], 1);
        ptx::mbar_init(&land[threadIdx.x], 1);
        ptx::mbar_init_fence();
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&tfull[i], 1);
            ptx::mbar_init(&tempty[i], CG * kEpiWarps);   // one lane per epilogue warp of either CTA
        }
        ptx::mbar_init(drain, 1);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&ready[i], 1);
            // the producer, the MMA issuer (of the first CTA), WGRAD's zeroing warp, the epilogue warps
            ptx::mbar_init(&freed[i], 1 + (leader ? 1 : 0) + (WG ? 1 : 0) + kEpiWarps);
        }
        ptx::mbar_init_fence();
        ptx::prefetch_tensormap(&tmap_a);
        ptx::prefetch_tensormap(&tmap_b);
        *bad = 0;
        *dead = 0;
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            ptx::tmem_alloc_pair(tmem_slot, kTmemCols);
            ptx::tmem_relinquish_pair();
        } else {
            ptx::tmem_alloc(tmem_slot, kTmemCols);
            ptx::tmem_relinquish();
        }
    }
    ptx::griddep_wait();   // the offsets may come from the stream's previous kernel
    ptx::griddep_launch_dependents();
    ptx::tc_fence_before();
    cta_sync();
    ptx::tc_fence_after();

    // ---- the schedule
    const Plan plan = {row, tile, (p.M + BM * CG - 1) / (BM * CG)};
    {
        int wrong = 0;
        const int real = WG ? p.groups / p.splits : p.groups;
        for (int i = threadIdx.x; i <= real; i += (int)blockDim.x) {
            const int v = p.offsets[i];
            wrong |= v < 0 || v > p.rows || (i > 0 && p.offsets[i - 1] > v);
            if (WG && p.splits > 1 && i < real) {   // a group's rows in `splits` runs of whole K steps, the last ones maybe empty
                const int T = max(0, p.offsets[i + 1] - v), len = ((T + p.splits - 1) / p.splits + BK - 1) / BK * BK;
                for (int s = 0; s < p.splits; ++s) row[i * p.splits + s] = v + min(T, s * len);
            } else {
                row[WG ? i * p.splits : i] = v;
            }
        }
        if (wrong) *bad = 1;
        cta_sync();
        if (warp == 0 && !WG) {
            int before = 0;
            for (int base = 0; base < p.groups; base += 32) {
                const int e = base + lane;
                int sum = 0, n = 0;
                if (e < p.groups && !*bad) n = (row[e + 1] - row[e] + p.bn - 1) / p.bn * plan.mt;
                sum = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int up = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += up;
                }
                if (e < p.groups) tile[e] = before + sum - n;
                before += __shfl_sync(0xffffffffu, sum, 31);
            }
            if (lane == 0) tile[p.groups] = before;
        }
        cta_sync();
    }
    int num_work = WG ? p.groups * plan.mt * ((p.cols + kMaxBN - 1) / kMaxBN) : tile[p.groups];
    if (*bad) {
        num_work = 0;
        if (threadIdx.x == 0) atomicOr(p.err, TF_DEVERR_OFFSETS);
    }
    if constexpr (PAIR) ptx::cluster_sync();   // the peer's barriers exist
    const uint32_t tmem_base = *tmem_slot;
    if ((ptx::smem_u32(smem) & 1023u) != 0) {
        num_work = 0;
        if (threadIdx.x == 0) atomicOr(p.err, TF_DEVERR_SMEM_ALIGN);
    }
    if constexpr (PAIR) {
        if (ptx::ld_shared_cluster_u32(ptx::mapa_shared(tmem_slot, (uint32_t)crank ^ 1u)) != tmem_base) {
            num_work = 0;
            if (threadIdx.x == 0) atomicOr(p.err, TF_DEVERR_PAIR_TMEM);
        }
    }

    // the ring: stages of KSUB K blocks, each A's tile and then B's
    const int sub_bytes = kABytes + (WG ? kMaxBN : p.bn) / CG * BK * 2, stage_bytes = sub_bytes * KSUB;
    const int stages = min(kMaxStages, p.off_epi / stage_bytes);
    auto give_up = [&](uint32_t why) {
        *dead = 1;
        atomicOr(p.err, why);
    };
    const Items items = {reinterpret_cast<Item *>(smem + p.off_items), ready, freed, p.wait_ns, cid, ncl, num_work};
    if (warp == 0) {
        // ------------------------------------------------------------ producer
        int stage = 0;
        uint32_t phase = 0, issued = 0, last_phase = 0;
        bool ok = true;
        const bool issuer = elect_one();
        ok &= each_item<MODE, KSUB>(p, items, [&](const Item &it, int, int first, int rows, int nkb) {
            const int mrow = it.m0 + crank * BM;
            // boxes of the N side this CTA loads: its half of the tile's rows (or columns)
            const int half = it.w / CG;
            const int nbox = WG ? half / 64 : (half + p.box_rows - 1) / p.box_rows;
            const uint32_t own = kABytes + (uint32_t)(nbox * (WG ? kChunkBytes : p.box_rows * BK * 2));
            for (int kb = 0; kb < nkb; ++kb) {
                const bool got = ptx::mbar_wait(&empty[stage], phase ^ 1u, p.wait_ns);
                if (!__all_sync(0xffffffffu, got)) return ok = false;
                if (issuer) {
                    const bool ragged = WG && kb == nkb - 1 && (rows & 15) != 0;
                    uint64_t *bar = ragged ? &land[stage] : &full[stage];
                    // K blocks of this stage (no box starts past the end of K)
                    const int subs = KSUB == 1 ? 1 : min(KSUB, (p.red + BK - 1) / BK - kb * KSUB);
                    if (ragged) {
                        ptx::mbar_arrive_expect_tx(bar, own);
                    } else if (leader) {
                        ptx::mbar_arrive_expect_tx(bar, CG * own * (uint32_t)subs);
                        if (WG && PAIR) ptx::mbar_arrive(bar);
                    }
                    const uint32_t bar_cl = PAIR ? ptx::mapa_shared(bar, ragged ? (uint32_t)crank : 0u) : 0u;
                    for (int sub = 0; sub < subs; ++sub) {
                        uint8_t *a_dst = smem + stage * stage_bytes + sub * sub_bytes, *b_dst = a_dst + kABytes;
                        const int k0 = (kb * KSUB + sub) * BK;
                        if constexpr (MODE == GROUPED_FORWARD) {
                            // a box that would start past the last weights row starts on it: its rows are never stored
                            const int n = min(mrow, p.M - 1);
                            if constexpr (PAIR) ptx::tma_load_3d_pair(a_dst, &tmap_a, bar_cl, k0, n, it.e);
                            else ptx::tma_load_3d(a_dst, &tmap_a, bar, k0, n, it.e);
                        } else {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                uint8_t *dst = a_dst + i * kChunkBytes;
                                const int c = min(mrow + 64 * i, (p.M - 1) & ~7);   // 16-byte aligned, inside the tensor
                                if constexpr (MODE == GROUPED_DGRAD) {
                                    if constexpr (PAIR) ptx::tma_load_3d_pair(dst, &tmap_a, bar_cl, c, k0, it.e);
                                    else ptx::tma_load_3d(dst, &tmap_a, bar, c, k0, it.e);
                                } else {
                                    if constexpr (PAIR) ptx::tma_load_2d_pair(dst, &tmap_a, bar_cl, c, first + k0);
                                    else ptx::tma_load_2d(dst, &tmap_a, bar, c, first + k0);
                                }
                            }
                        }
                        for (int i = 0; i < nbox; ++i) {
                            if constexpr (WG) {
                                const int c = min(it.t0 + crank * half + 64 * i, (p.cols - 1) & ~7);
                                if constexpr (PAIR) ptx::tma_load_2d_pair(b_dst + i * kChunkBytes, &tmap_b, bar_cl, c, first + k0);
                                else ptx::tma_load_2d(b_dst + i * kChunkBytes, &tmap_b, bar, c, first + k0);
                            } else {
                                // rows past the group are other groups' (or zero): their columns of D are never stored
                                const int m = min(it.t0 + crank * half + i * p.box_rows, p.rows - 1);
                                uint8_t *dst = b_dst + i * p.box_rows * (BK * 2);
                                if constexpr (PAIR) ptx::tma_load_2d_pair(dst, &tmap_b, bar_cl, k0, m);
                                else ptx::tma_load_2d(dst, &tmap_b, bar, k0, m);
                            }
                        }
                    }
                }
                __syncwarp();
                issued |= 1u << stage;
                last_phase = (last_phase & ~(1u << stage)) | (phase << stage);
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            return true;
        });
        if (!ok && lane == 0) give_up(TF_DEVERR_PRODUCER_WAIT);
        // every copy has landed before the CTA exits (a pair's complete on the first CTA's barriers)
        for (int s = 0; s < stages; ++s)
            if (leader && ((issued >> s) & 1u))
                if (!ptx::mbar_wait<PAIR>(&full[s], (last_phase >> s) & 1u, p.wait_ns) && lane == 0)
                    atomicOr(p.err, TF_DEVERR_DRAIN_WAIT);
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (leader) {
            int stage = 0, b = 0;
            uint32_t phase = 0, taken = 0;   // taken: parity of the uses of either accumulator
            bool ok = true;
            const bool issuer = elect_one();
            constexpr uint32_t a_step = desc_step(!A_MMAJOR), b_step = desc_step(!WG);
            const uint32_t a_low = desc_low(ptx::smem_u32(smem), !A_MMAJOR);
            const uint32_t b_low = desc_low(ptx::smem_u32(smem) + kABytes, !WG);
            auto mma = [](uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
                if constexpr (PAIR) ptx::umma_bf16_pair(d, desc_of(a), desc_of(b), id, acc);
                else ptx::umma_bf16(d, desc_of(a), desc_of(b), id, acc);
            };
            ok &= each_item<MODE, KSUB>(p, items, [&](const Item &it, int part, int, int rows, int nkb) {
                if (nkb == 0) return true;
                const uint32_t id = idesc(BM * CG, it.w, p.bf16 != 0, A_MMAJOR, WG);
                const int c = WG && part > 0 ? b ^ 1 : b;   // the accumulator
                bool got = ptx::mbar_wait<PAIR>(&tempty[c], ((taken >> c) & 1u) ^ 1u, p.wait_ns);
                if (!__all_sync(0xffffffffu, got)) return ok = false;
                ptx::tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)(c * kMaxBN);
                uint32_t acc = 0;   // the first K step begins its sums
                for (int kb = 0; kb < nkb; ++kb) {
                    got = ptx::mbar_wait<PAIR && WG>(&full[stage], phase, p.wait_ns);
                    if (!__all_sync(0xffffffffu, got)) return ok = false;
                    ptx::tc_fence_after();
                    const uint32_t a = a_low + (uint32_t)stage * (uint32_t)(stage_bytes >> 4);
                    const uint32_t bb = b_low + (uint32_t)stage * (uint32_t)(stage_bytes >> 4);
                    // WGRAD: sixteens of rows past the group's end are left out
                    const int steps = WG ? min(BK / UMMA_K, (rows - kb * BK + UMMA_K - 1) / UMMA_K) : BK / UMMA_K;
                    const int subs = KSUB == 1 ? 1 : min(KSUB, (p.red + BK - 1) / BK - kb * KSUB);
                    if (issuer) {
                        mma(d_tmem, a, bb, id, acc);
                        if (!WG || steps > 1) mma(d_tmem, a + a_step, bb + b_step, id, 1u);
                        if (!WG || steps > 2) mma(d_tmem, a + 2 * a_step, bb + 2 * b_step, id, 1u);
                        if (!WG || steps > 3) mma(d_tmem, a + 3 * a_step, bb + 3 * b_step, id, 1u);
#pragma unroll
                        for (int sub = 1; sub < KSUB; ++sub) {
                            if (sub >= subs) break;
                            const uint32_t as = a + (uint32_t)sub * (uint32_t)(sub_bytes >> 4), bs = bb + (uint32_t)sub * (uint32_t)(sub_bytes >> 4);
#pragma unroll
                            for (int k = 0; k < BK / UMMA_K; ++k) mma(d_tmem, as + k * a_step, bs + k * b_step, id, 1u);
                        }
                        if constexpr (PAIR) ptx::umma_commit_both(&empty[stage]);
                        else ptx::umma_commit(&empty[stage]);
                        if (kb == nkb - 1) {
                            if constexpr (PAIR) ptx::umma_commit_both(&tfull[c]);
                            else ptx::umma_commit(&tfull[c]);
                        }
                    }
                    __syncwarp();
                    acc = 1u;
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                taken ^= 1u << c;
                if (part == it.parts - 1) b ^= 1;
                return true;
            });
            if (!ok && lane == 0) give_up(TF_DEVERR_MMA_WAIT);
            if (issuer) {   // (the lane that issued the MMAs)
                if constexpr (PAIR) ptx::umma_commit_pair(ptx::smem_u32(drain));
                else ptx::umma_commit(drain);
            }
            __syncwarp();
            if (!ptx::mbar_wait(drain, 0, p.wait_ns) && lane == 0) atomicOr(p.err, TF_DEVERR_DRAIN_WAIT);
        }
    } else if (WG && warp == 2) {
        // ------------------------------------------------------------ zeroing warp
        // The last K step of a group holds rows of the next group (or what lies
        // behind the last): those of the sixteen that the last MMA reads become
        // zero in both operands, so that not even a NaN there reaches this group.
        uint32_t land_phase = 0;
        int blocks = 0;    // K steps before this item
        bool ok = true;
        ok &= each_item<MODE, KSUB>(p, items, [&](const Item &it, int, int, int rows, int nkb) {
            blocks += nkb;
            if ((rows & 15) == 0) return true;
            const int stage = (blocks - 1) % stages;
            ok = ptx::mbar_wait(&land[stage], (land_phase >> stage) & 1u, p.wait_ns);
            land_phase ^= 1u << stage;
            if (!__all_sync(0xffffffffu, ok)) return ok = false;
            const int r0 = rows - (nkb - 1) * BK, r1 = (r0 + 15) & ~15;
            uint8_t *base = smem + stage * stage_bytes;
            const int nbox = 2 + it.w / CG / 64;   // A's two boxes, then B's
            for (int i = lane; i < nbox * (r1 - r0) * 8; i += 32) {
                const int box = i / ((r1 - r0) * 8), j = i - box * ((r1 - r0) * 8);
                *reinterpret_cast<uint4 *>(base + box * kChunkBytes + r0 * 128 + j * 16) = make_uint4(0, 0, 0, 0);
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR) ptx::mbar_arrive_cluster(ptx::mapa_shared(&full[stage], 0));
                else ptx::mbar_arrive(&full[stage]);
            }
            __syncwarp();
            return true;
        });
        if (!ok && lane == 0) give_up(TF_DEVERR_MMA_WAIT);
    } else if (warp == 3) {
        // ------------------------------------------------------------ item lists
        bool ok = true;
        for (int k = 0; ok && cid + k * 32 * ncl < num_work; ++k) {
            const int half = k & 1, t = cid + (k * 32 + lane) * ncl;
            // the list before the last is used up after up to 64 items, each of which may take a while
            if (k >= 2)
                for (int tries = 0; !(ok = ptx::mbar_wait(&freed[half], (uint32_t)((k >> 1) - 1) & 1u, p.wait_ns)); ++tries)
                    if (tries == 64 || *dead) break;
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            if (t < num_work) items.table[half * 32 + lane] = item_of<MODE, CG>(p, plan, t);
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&ready[half]);
        }
        if (!ok && lane == 0) atomicOr(p.err, TF_DEVERR_PRODUCER_WAIT);
    } else if (warp >= kFirstEpiWarp && warp < kFirstEpiWarp + kEpiWarps) {
        // ------------------------------------------------------------ epilogue
        // Warp w reads TMEM lanes 32*(w%4) .. +31 (one weights row per lane) and
        // every second 32-column chunk.
        const int q = warp & 3, h = (warp - kFirstEpiWarp) >> 2;
        uint8_t *box = smem + p.off_epi + (warp - kFirstEpiWarp) * kBoxBytes;
        const bool slope = MODE == GROUPED_DGRAD && p.act != TF_ACT_NONE;
        int b = 0;
        uint32_t seen = 0;   // parity of the results of either accumulator
        bool ok = true;
        ok &= each_item<MODE, KSUB>(p, items, [&](const Item &it, int part, int, int, int nkb) {
            const int n0 = it.m0 + crank * BM + q * 32;
            const int width = WG ? min(kMaxBN, p.cols - it.t0) : it.tv;
            const bool mine = n0 < p.M;
            float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (MODE == GROUPED_FORWARD && p.bias) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = n0 + 8 * j + (lane >> 2);
                    if (n < p.M) bias[j] = __ldg(p.bias + (int64_t)it.e * p.M + n);
                }
            }
            uint4 pre[4] = {};
            if (slope && mine && h * 32 < width)
                load_pre(pre, p.pre, p.pre_stride, n0, p.M, it.t0 + h * 32, min(32, width - h * 32));
            const bool last = part == it.parts - 1;
            if (WG && part == 0 && !last) {   // a part to come completes after this one: wait for that
                seen ^= 1u << b;
                return true;
            }
            const int acc = WG && part > 0 ? b ^ 1 : b;   // the accumulator of this part
            if (nkb > 0) {
                const bool got = ptx::mbar_wait(&tfull[acc], (seen >> acc) & 1u, p.wait_ns);
                if (!__all_sync(0xffffffffu, got)) return ok = false;
                ptx::tc_fence_after();
            } else if (!WG || p.accumulate) {
                return true;   // a group without rows adds nothing
            }
            const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kMaxBN);
#pragma unroll 1
            for (int c = h; c * 32 < width && mine; c += kEpiWarps / 4) {
                uint32_t r[32];
                if constexpr (WG) {
                    if (nkb > 0) {
                        tmem_ld_16x256b_x4(taddr + (uint32_t)(c * 32), r);
                        tmem_ld_16x256b_x4(taddr + (16u << 16) + (uint32_t)(c * 32), r + 16);
                        ptx::tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) r[j] = 0u;
                    }
                    const uint32_t saddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * kMaxBN + c * 32);
                    if (part > 0) {   // plus the parts before
                        uint32_t u[32];
                        tmem_ld_16x256b_x4(saddr, u);
                        tmem_ld_16x256b_x4(saddr + (16u << 16), u + 16);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(u[j]));
                    }
                    if (!last) {
                        tmem_st_16x256b_x4(saddr, r);
                        tmem_st_16x256b_x4(saddr + (16u << 16), r + 16);
                        tmem_st_wait();
                        continue;
                    }
                    // rows l/4 + 8j of the 32, columns 8k + 2(l%4) and the next: 32-byte pieces of eight rows at a time
                    const int col = it.t0 + c * 32 + 2 * (lane & 3);
                    float *out = reinterpret_cast<float *>(p.y) + ((int64_t)it.e * p.M + n0 + (lane >> 2)) * p.cols + col;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (n0 + 8 * j + (lane >> 2) >= p.M) continue;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int i = (j >> 1) * 16 + 4 * k + 2 * (j & 1);
                            float2 *dst = reinterpret_cast<float2 *>(out + (int64_t)(8 * j) * p.cols + 8 * k);
                            if (col + 8 * k >= p.cols) continue;
                            float2 v = make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]));
                            if (p.accumulate) v = fadd2(v, *dst);
                            *dst = v;
                        }
                    }
                } else {
                    tmem_ld_16x256b_x4(taddr + (uint32_t)(c * 32), r);
                    tmem_ld_16x256b_x4(taddr + (16u << 16) + (uint32_t)(c * 32), r + 16);
                    const int count = min(32, width - c * 32), token = it.t0 + c * 32, next = c + kEpiWarps / 4;
                    ptx::tmem_ld_wait();
                    uint4 cur[4] = {pre[0], pre[1], pre[2], pre[3]};
                    if (slope && next * 32 < width)
                        load_pre(pre, p.pre, p.pre_stride, n0, p.M, it.t0 + next * 32, min(32, width - next * 32));
                    auto finish = [&](auto act) {
                        constexpr int ACT = decltype(act)::value;
                        if (p.bf16) finish_chunk<__nv_bfloat16, MODE, ACT>(p, r, bias, cur, box, n0, token, count);
                        else finish_chunk<__half, MODE, ACT>(p, r, bias, cur, box, n0, token, count);
                    };
                    if (p.act == TF_ACT_GELU) finish(std::integral_constant<int, TF_ACT_GELU>());
                    else if (p.act == TF_ACT_SILU) finish(std::integral_constant<int, TF_ACT_SILU>());
                    else finish(std::integral_constant<int, TF_ACT_NONE>());
                }
            }
            if (nkb > 0) {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    auto release = [&](int i) {
                        if constexpr (PAIR) ptx::mbar_arrive_cluster(ptx::mapa_shared(&tempty[i], 0));
                        else ptx::mbar_arrive(&tempty[i]);
                    };
                    release(acc);
                    if (last && part > 0) release(b);
                }
                seen ^= 1u << acc;
                if (last) b ^= 1;
            }
            return true;
        });
        if (!ok && lane == 0) give_up(TF_DEVERR_EPILOGUE_WAIT);
    } else if (WG && warp >= kFirstEpiWarp + kEpiWarps && p.dbias && num_work > 0) {
        // ------------------------------------------------------------ bias gradient
        if (p.bf16) bias_grad<__nv_bfloat16>(p, plan, warp - kFirstEpiWarp - kEpiWarps);
        else bias_grad<__half>(p, plan, warp - kFirstEpiWarp - kEpiWarps);
    }

    ptx::tc_fence_before();
    cta_sync();
    if constexpr (PAIR) ptx::cluster_sync();
    if (warp == 1) {
        ptx::tc_fence_after();
        if constexpr (PAIR) ptx::tmem_dealloc_pair(tmem_base, kTmemCols);
        else ptx::tmem_dealloc(tmem_base, kTmemCols);
    }
}

// ---------------------------------------------------------------- host side

// [groups][N][K] weights.
bool encode_groups(CUtensorMap *m, CUtensorMapDataType type, const void *base, int64_t groups, int64_t N, int64_t K,
                   int box_cols, int box_rows)
{
    const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)N, (cuuint64_t)groups};
    const cuuint64_t strides[2] = {(cuuint64_t)K * 2, (cuuint64_t)N * K * 2};
    const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
    return encode(m, type, 3, base, dims, strides, box);
}

// CTAs (or pairs) that can be resident at once, by device; the kernel's
// shared-memory limit is raised on the way.
template <int MODE, int CG, int KSUB>
cudaError_t resident(int *units)
{
    static std::mutex mu;
    static int known[64];
    int d = 0;
    cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess || d < 0 || d >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!known[d]) {
        auto kern = grouped_umma_kernel<MODE, CG, KSUB>;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
        if (e != cudaSuccess) return e;
        int n = sm_count();
        if (CG == 2) {
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)(n / 2 * 2));
            cfg.blockDim = dim3(threads_of(MODE));
            cfg.dynamicSmemBytes = kSmemLimit;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
            if (e != cudaSuccess) return e;
            if (n < 1) return cudaErrorNotSupported;
        }
        known[d] = n;
    }
    *units = known[d];
    return cudaSuccess;
}

template <int MODE, int CG, int KSUB>
cudaError_t launch_mode(const GroupedArgs &a, int bn, cudaStream_t st, int splits = 1)
{
    constexpr bool WG = MODE == GROUPED_WGRAD;
    UmmaArgs p = {};
    p.offsets = a.offsets;
    p.bias = a.bias;
    p.y = WG ? (splits > 1 ? a.ws : a.dw) : a.y;   // with splits, partial sums
    p.pre = a.pre;
    p.err = device_error_word();
    p.wait_ns = wait_limit_ns();
    if (!p.err) return cudaErrorInitializationError;
    p.y_stride = a.y_stride;
    p.pre_stride = a.pre_stride;
    p.groups = a.groups * splits;
    p.splits = splits;
    p.rows = a.rows;
    p.M = MODE == GROUPED_DGRAD ? a.K : a.N;
    p.red = MODE == GROUPED_DGRAD ? a.N : a.K;
    p.cols = a.K;
    p.bn = bn;
    p.box_rows = bn / CG < 64 ? bn / CG : 64;
    p.act = a.act;
    p.bf16 = a.dtype == TF_BF16;
    p.accumulate = splits > 1 ? 0 : a.accumulate;
    p.dy = a.dy;
    p.dy_stride = a.dy_stride;
    p.dbias = splits > 1 && a.dbias ? a.ws + (int64_t)p.groups * a.N * a.K : a.dbias;
    const int sched = (2 * (p.groups + 1) + 2) * 4;
    const int fixed = (WG ? 0 : kEpiWarps * kBoxBytes) + kItemBytes + kNumBars * 8 + 16 + sched;
    const int ring = (kSmemLimit - fixed) / 1024 * 1024;
    if (ring < 2 * KSUB * (kABytes + (WG ? kMaxBN : bn) / CG * BK * 2)) return cudaErrorNotSupported;
    p.off_epi = ring;
    p.off_items = p.off_epi + (WG ? 0 : kEpiWarps * kBoxBytes);
    p.off_bar = p.off_items + kItemBytes;
    p.off_sched = p.off_bar + kNumBars * 8 + 16;
    const int smem = p.off_sched + sched;

    cudaError_t e = bind_context();
    if (e != cudaSuccess) return e;
    const CUtensorMapDataType type = p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    CUtensorMap ta, tb;
    bool ok;
    if (MODE == GROUPED_FORWARD)
        ok = encode_groups(&ta, type, a.w, a.groups, a.N, a.K, BK, BM) &&
             encode_rows(&tb, type, a.x, a.rows, a.K, a.x_stride, BK, p.box_rows);
    else if (MODE == GROUPED_DGRAD)
        ok = encode_groups(&ta, type, a.w, a.groups, a.N, a.K, 64, BK) &&
             encode_rows(&tb, type, a.dy, a.rows, a.N, a.dy_stride, BK, p.box_rows);
    else
        ok = encode_rows(&ta, type, a.dy, a.rows, a.N, a.dy_stride, 64, BK) &&
             encode_rows(&tb, type, a.x, a.rows, a.K, a.x_stride, 64, BK);
    if (!ok) return cudaErrorInvalidValue;

    int units = 0;
    e = resident<MODE, CG, KSUB>(&units);
    if (e != cudaSuccess) return e;
    const int64_t mt = (p.M + BM * CG - 1) / (BM * CG);
    const int64_t most = WG ? (int64_t)p.groups * mt * ((a.K + kMaxBN - 1) / kMaxBN)
                            : ((int64_t)a.rows / bn + a.groups) * mt;
    if (most >= (int64_t)1 << 31) return cudaErrorNotSupported;
    if (units > most) units = (int)most;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * CG));
    cfg.blockDim = dim3(threads_of(MODE));
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 2 ? 2 : 1;
    return counted(cudaLaunchKernelEx(&cfg, grouped_umma_kernel<MODE, CG, KSUB>, ta, tb, p));
}

// WGRAD with fewer tiles than CTAs and long groups: every group's rows in
// `splits` runs, whose products a second kernel adds.  At least 512 rows per run
// on average, as far as the host knows (2 groups of 8000 rows, 256 x 320: 13.2
// us, 15.5 with 256 rows, 56 without splits; no difference at 4000 rows in 8 groups).
int wgrad_splits(int64_t rows, int groups, int64_t N, int64_t K)
{
    const int64_t tiles = (int64_t)groups * ((N + BM - 1) / BM) * ((K + kMaxBN - 1) / kMaxBN);
    int64_t s = sm_count() / tiles;
    if (s > rows / groups / 512) s = rows / groups / 512;
    if (s > kGroupedMaxGroups / groups) s = kGroupedMaxGroups / groups;
    return s < 2 ? 1 : (int)s;
}

// dw's partial sums [groups*splits][N][K], then dbias's [groups*splits][N].
int64_t split_bytes(int splits, int groups, int64_t N, int64_t K)
{
    return splits < 2 ? 0 : (int64_t)splits * groups * N * (K + 1) * 4;
}

// dst[e][i] (+)= the sum over s of src[e*splits + s][i], in order; 4 values per
// thread.  Nothing with invalid offsets, for which there are no partial sums.
__global__ void __launch_bounds__(256) split_sum_kernel(float *dw, float *dbias, const float *ws, const int *offsets,
                                                        int rows, int splits, int groups, int64_t NK, int64_t N,
                                                        int accumulate)
{
    pdl_begin();
    bool wrong = false;
    for (int i = threadIdx.x; i <= groups; i += 256) {
        const int v = offsets[i];
        wrong |= v < 0 || v > rows || (i > 0 && offsets[i - 1] > v);
    }
    if (__syncthreads_or(wrong)) return;
    const int64_t step = (int64_t)gridDim.x * 256, first = (int64_t)blockIdx.x * 256 + threadIdx.x;
    auto add = [&](float *dst, const float *src, int64_t n) {   // n values per group, a multiple of 4
        for (int64_t i = first; i < groups * n / 4; i += step) {
            const int64_t e = 4 * i / n, at = 4 * i - e * n;
            float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int s = 0; s < splits; ++s) {
                const float4 v = *reinterpret_cast<const float4 *>(src + (e * splits + s) * n + at);
                t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
            }
            float *out = dst + 4 * i;   // (dbias need not be 16-byte aligned)
            out[0] = accumulate ? out[0] + t.x : t.x;
            out[1] = accumulate ? out[1] + t.y : t.y;
            out[2] = accumulate ? out[2] + t.z : t.z;
            out[3] = accumulate ? out[3] + t.w : t.w;
        }
    };
    add(dw, ws, NK);
    if (dbias) add(dbias, ws + (int64_t)groups * splits * NK, N);
}

cudaError_t launch_sum(const GroupedArgs &a, int splits, cudaStream_t st)
{
    const int64_t NK = (int64_t)a.N * a.K, blocks = (a.groups * NK / 4 + 255) / 256, most = 8 * (int64_t)sm_count();
    return launch_pdl(split_sum_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, st, a.dw, a.dbias,
                      static_cast<const float *>(a.ws), a.offsets, a.rows, splits, a.groups, NK, (int64_t)a.N, a.accumulate);
}

template <int MODE>
cudaError_t launch_auto(const GroupedArgs &a, cudaStream_t st)
{
    const int64_t M = MODE == GROUPED_DGRAD ? a.K : a.N;
    const int64_t avg = a.rows / a.groups;   // rows per group, as far as the host knows
    if constexpr (MODE == GROUPED_WGRAD) {
        int splits = wgrad_splits(a.rows, a.groups, a.N, a.K);
        // Pairs for long groups only (16 groups of 2048 x 2048: of 2048 rows 219 us, single CTAs 226; of 512
        // rows 85 and 79; of 256 rows 70 and 59; 4096 x 2048 of 1024 rows 257 and 262): two CTAs' epilogues have
        // to end before either goes on.
        const bool pair = M > BM && a.K > 128 && avg >= 1024 && splits == 1;
        if (a.ws_bytes < split_bytes(splits, a.groups, a.N, a.K)) splits = 1;
        const cudaError_t e = pair ? launch_mode<MODE, 2, 1>(a, kMaxBN, st, splits) : launch_mode<MODE, 1, 1>(a, kMaxBN, st, splits);
        return e != cudaSuccess || splits == 1 ? e : launch_sum(a, splits, st);
    } else {
        // Pairs move the fewest operand bytes per product, which is what bounds large calls (16 groups of
        // 512 rows, 2048 x 2048: 57 us; single CTAs with tiles of 128 rows 65, of 256 rows 62).  Smaller tiles
        // win while they fill no more than one wave of SMs (8 groups of 128 rows, 1024 x 4096: 18.0 us, pairs
        // 24.3; 256 rows: 34 and 25), and where a group's rows would leave the wide one mostly empty (16 groups
        // of 32 rows, 2048 x 2048: 25.6 us with 64, 26.6 with 128, 28.0 on pairs; of 96 rows: 32.6, 28.2, 31.3;
        // 4 groups of one row, 4096 x 4096: 23.9 with 16 and 29.9 with 64, whose stages are larger and fewer).
        // A group's tiles of `bn` rows each, half a tile more on average for the ragged end:
        auto one_wave = [&](int bn) { return (M + BM - 1) / BM * (a.rows / bn + (a.groups + 1) / 2) <= sm_count(); };
        if (M > BM && avg > 96 && !one_wave(128)) return launch_mode<MODE, 2, 2>(a, kMaxBN, st);
        return launch_mode<MODE, 1, 2>(a, avg <= 8 ? 16 : avg <= 48 || one_wave(64) ? 64 : 128, st);
    }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

int64_t grouped_wgrad_workspace(int64_t rows, int groups, int64_t N, int64_t K, int)
{
    if (N % 8 != 0 || K % 8 != 0) return 0;
    return split_bytes(wgrad_splits(rows, groups, N, K), groups, N, K);
}

cudaError_t launch_grouped(const GroupedArgs &a, int mode, cudaStream_t st)
{
    // what a tensor map can address: 16-byte rows and bases
    auto rows_ok = [](const void *p, int64_t stride) { return !p || (aligned16(p) && stride % 8 == 0); };
    const bool dims = a.N % 8 == 0 && a.K % 8 == 0 && a.rows > 0;
    if (mode == GROUPED_FORWARD) {
        const bool tma = dims && rows_ok(a.x, a.x_stride) && rows_ok(a.y, a.y_stride) && rows_ok(a.pre, a.pre_stride) &&
                         aligned16(a.w);
        return tma ? launch_auto<GROUPED_FORWARD>(a, st) : launch_grouped_unaligned(a, mode, st);
    }
    if (mode == GROUPED_DGRAD) {
        const bool tma = dims && rows_ok(a.dy, a.dy_stride) && rows_ok(a.y, a.y_stride) && rows_ok(a.pre, a.pre_stride) &&
                         aligned16(a.w);
        return tma ? launch_auto<GROUPED_DGRAD>(a, st) : launch_grouped_unaligned(a, mode, st);
    }
    const bool tma = dims && rows_ok(a.dy, a.dy_stride) && rows_ok(a.x, a.x_stride) && aligned16(a.dw);
    if (tma) return launch_auto<GROUPED_WGRAD>(a, st);
    const cudaError_t e = launch_grouped_unaligned(a, mode, st);
    return e != cudaSuccess || !a.dbias ? e : launch_grouped_bias_grad(a, st);
}

}  // namespace tf
