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
//   4-11  epilogue: TMEM -> registers -> bias, activation -> y
// Every wait is bounded (ptx::mbar_wait); a role that times out sets the
// device error word and winds down.
#include <cuda.h>
#include <string.h>

#include <mutex>

#include "grouped.cuh"
#include "ptx_sm100.cuh"

namespace tf {
namespace {

using namespace grouped;

constexpr int BM = 128;                 // weights rows per CTA (UMMA M, or half of the pair's 256)
constexpr int BK = 64;                  // K step: one 128-byte swizzle row of 16-bit values
constexpr int UMMA_K = 16;
constexpr int kMaxBN = 256;             // widest row tile: one accumulator is 256 TMEM columns
constexpr int kMaxStages = 12;
constexpr int kEpiWarps = 8, kFirstEpiWarp = 4;
constexpr int kThreads = 32 * (kFirstEpiWarp + kEpiWarps);
constexpr int kSmemLimit = 227 * 1024;
constexpr int kABytes = BM * BK * 2;
constexpr int kChunkBytes = 64 * BK * 2;          // one 64 x 64 box of an M- or N-major operand
constexpr int kDwBoxBytes = 32 * 32 * 4;          // WGRAD epilogue box per warp
constexpr int kNumBars = 3 * kMaxStages + 5;      // full, empty, land; accumulators full x2, empty x2; drain
constexpr uint32_t kTmemCols = 512;

struct UmmaArgs {
    const int *offsets;
    const float *bias;
    void *y;
    const void *pre_in;
    void *pre_out;
    uint32_t *err;
    uint64_t wait_ns;
    int64_t y_stride, pre_stride;
    int groups, rows;
    int M;             // extent of the weights' side (N, or K for DGRAD)
    int red;           // reduction length of FORWARD and DGRAD
    int cols;          // WGRAD: K, the N side
    int bn;            // widest row tile
    int box_rows;      // rows per token box
    int stages, stage_bytes, off_dw, off_bar, off_sched;
    int act, bf16, accumulate;
};

// Shared-memory matrix descriptor of an M- or N-major tile written by TMA with
// 128-byte swizzling: boxes of 64 (M or N) x 64 (K) values, each a K row of 128
// bytes.  Eight K rows are one 1024-byte swizzle atom (stride byte offset); the
// next 64 M or N values are a box further on (leading byte offset).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr)
{
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(kChunkBytes >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

__device__ __forceinline__ uint32_t idesc(int m, int n, bool bf16, bool a_mmajor, bool b_nmajor)
{
    const uint32_t fmt = bf16 ? 1u : 0u;
    return (1u << 4) | (fmt << 7) | (fmt << 10) | ((a_mmajor ? 1u : 0u) << 15) | ((b_nmajor ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void tma_store_3d(const void *map, const void *src, int c0, int c1, int c2)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(c0),
                 "r"(c1), "r"(c2), "r"(ptx::smem_u32(src))
                 : "memory");
}

__device__ __forceinline__ void tma_add_3d(const void *map, const void *src, int c0, int c1, int c2)
{
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
                 "r"(c0), "r"(c1), "r"(c2), "r"(ptx::smem_u32(src))
                 : "memory");
}

// One work item.  FORWARD, DGRAD: weights rows [m0, +128*CG), tokens [t0, +tv),
// MMA N = w.  WGRAD: dw rows [m0, +128*CG), columns [t0, +w) of group e, rows
// `first` on; tv is the group's number of rows.
struct Item {
    int e, m0, t0, w, tv, first, nkb;
};

template <int MODE, int CG>
__device__ __forceinline__ Item item_of(const UmmaArgs &p, const int *row, const int *tile, int t)
{
    constexpr int STEP = 16 * CG;
    Item it;
    const int mt = (p.M + BM * CG - 1) / (BM * CG);
    if (MODE == GROUPED_WGRAD) {
        const int ct = (p.cols + kMaxBN - 1) / kMaxBN;
        it.e = t / (mt * ct);
        const int r = t - it.e * (mt * ct);
        it.m0 = r / ct * (BM * CG);
        it.t0 = r % ct * kMaxBN;
        const int left = min(kMaxBN, p.cols - it.t0);
        it.w = (left + 64 * CG - 1) / (64 * CG) * (64 * CG);
        it.first = row[it.e];
        it.tv = row[it.e + 1] - it.first;
        it.nkb = (it.tv + BK - 1) / BK;
    } else {
        int lo = 0, hi = p.groups - 1;   // the last group that starts at or before tile t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (tile[mid] <= t) lo = mid; else hi = mid - 1;
        }
        it.e = lo;
        const int r = t - tile[lo], T = row[lo + 1] - row[lo];
        const int ntt = (T + p.bn - 1) / p.bn;
        const int wt = ((T + ntt - 1) / ntt + STEP - 1) / STEP * STEP;   // equal widths, at most bn
        const int tt = r % ntt;
        it.m0 = r / ntt * (BM * CG);
        it.first = row[lo];
        it.t0 = it.first + tt * wt;
        it.tv = min(wt, T - tt * wt);
        it.w = (it.tv + STEP - 1) / STEP * STEP;
        it.nkb = (p.red + BK - 1) / BK;
    }
    return it;
}

// y (and pre) of one 32 x 32 chunk: lane = weights row n, r[j] = token j of `count`.
template <typename T, int MODE>
__device__ __forceinline__ void store_chunk(const UmmaArgs &p, const uint32_t (&r)[32], int count, int64_t token, int n,
                                            bool in, float bias)
{
    if (!in) return;
    T *y = reinterpret_cast<T *>(p.y) + token * p.y_stride + n;
    if (MODE == GROUPED_FORWARD) {
        T *z = p.pre_out ? reinterpret_cast<T *>(p.pre_out) + token * p.pre_stride + n : nullptr;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (j >= count) break;
            const float v = __uint_as_float(r[j]) + bias;
            if (z) z[j * p.pre_stride] = Half2Of<T>::round(v);
            y[j * p.y_stride] = Half2Of<T>::round(act_value(p.act, v));
        }
    } else {
        const T *z = reinterpret_cast<const T *>(p.pre_in) + token * p.pre_stride + n;
        T zv[32];
        if (p.act != TF_ACT_NONE) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (j < count) zv[j] = z[j * p.pre_stride];
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (j >= count) break;
            float v = __uint_as_float(r[j]);
            if (p.act != TF_ACT_NONE) v *= act_slope(p.act, Half2Of<T>::widen(zv[j]));
            y[j * p.y_stride] = Half2Of<T>::round(v);
        }
    }
}

template <int MODE, int CG>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_umma_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                        const __grid_constant__ CUtensorMap tmap_dw, const UmmaArgs p)
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
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    int *row = reinterpret_cast<int *>(smem + p.off_sched);      // [groups + 1]
    int *tile = row + p.groups + 1;                              // [groups + 1]
    int *bad = tile + p.groups + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int crank = PAIR ? (int)ptx::cluster_ctarank() : 0;
    const int cid = (int)blockIdx.x / CG, ncl = (int)gridDim.x / CG;
    const bool leader = crank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            // WGRAD: one arrival per CTA, from the producers' side (which arrives CG times for a whole
            // K step) or from the CTAs' zeroing warps (a ragged one)
            ptx::mbar_init(&full[s], WG ? CG : 1);
            ptx::mbar_init(&empty[s], 1);
            ptx::mbar_init(&land[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&tfull[i], 1);
            ptx::mbar_init(&tempty[i], CG * kEpiWarps);   // one lane per epilogue warp of either CTA
        }
        ptx::mbar_init(drain, 1);
        ptx::mbar_init_fence();
        ptx::prefetch_tensormap(&tmap_a);
        ptx::prefetch_tensormap(&tmap_b);
        if (WG) ptx::prefetch_tensormap(&tmap_dw);
        *bad = 0;
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

    // ---- the schedule: rows of every group and the running count of tiles
    {
        int wrong = 0;
        for (int i = threadIdx.x; i <= p.groups; i += kThreads) {
            const int v = p.offsets[i];
            row[i] = v;
            wrong |= v < 0 || v > p.rows || (i > 0 && p.offsets[i - 1] > v);
        }
        if (wrong) *bad = 1;
        cta_sync();
        if (warp == 0 && !WG) {
            const int mt = (p.M + BM * CG - 1) / (BM * CG);
            int before = 0;
            for (int base = 0; base < p.groups; base += 32) {
                const int e = base + lane;
                int sum = 0, n = 0;
                if (e < p.groups && !*bad) n = (row[e + 1] - row[e] + p.bn - 1) / p.bn * mt;
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
    int num_work = WG ? p.groups * ((p.M + BM * CG - 1) / (BM * CG)) * ((p.cols + kMaxBN - 1) / kMaxBN)
                      : tile[p.groups];
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

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, issued = 0, last_phase = 0;
            bool ok = true;
            for (int t = cid; ok && t < num_work; t += ncl) {
                const Item it = item_of<MODE, CG>(p, row, tile, t);
                const int mrow = it.m0 + crank * BM;
                for (int kb = 0; kb < it.nkb; ++kb) {
                    if (!ptx::mbar_wait(&empty[stage], phase ^ 1u, p.wait_ns)) {
                        ok = false;
                        break;
                    }
                    uint8_t *a_dst = smem + stage * p.stage_bytes, *b_dst = a_dst + kABytes;
                    const int k0 = kb * BK;
                    // boxes of the N side this CTA loads: its half of the tile's rows (or columns)
                    const int half = it.w / CG;
                    const int nbox = WG ? half / 64 : (half + p.box_rows - 1) / p.box_rows;
                    const uint32_t own = kABytes + (uint32_t)(nbox * (WG ? kChunkBytes : p.box_rows * BK * 2));
                    const bool ragged = WG && kb == it.nkb - 1 && (it.tv & 15) != 0;
                    uint64_t *bar = ragged ? &land[stage] : &full[stage];
                    if (ragged) {
                        ptx::mbar_arrive_expect_tx(bar, own);
                    } else if (leader) {
                        ptx::mbar_arrive_expect_tx(bar, CG * own);
                        if (WG && PAIR) ptx::mbar_arrive(bar);
                    }
                    const uint32_t bar_cl = PAIR ? ptx::mapa_shared(bar, ragged ? (uint32_t)crank : 0u) : 0u;
                    if constexpr (MODE == GROUPED_FORWARD) {
                        // a box that would start past the last weights row starts on it: its rows are never stored
                        const int n = min(mrow, p.M - 1);
                        if constexpr (PAIR) ptx::tma_load_3d_pair(a_dst, &tmap_a, bar_cl, k0, n, it.e);
                        else ptx::tma_load_3d(a_dst, &tmap_a, bar, k0, n, it.e);
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int c = min(mrow + 64 * i, (p.M - 1) & ~7);   // 16-byte aligned, inside the tensor
                            if constexpr (MODE == GROUPED_DGRAD) {
                                if constexpr (PAIR) ptx::tma_load_3d_pair(a_dst + i * kChunkBytes, &tmap_a, bar_cl, c, k0, it.e);
                                else ptx::tma_load_3d(a_dst + i * kChunkBytes, &tmap_a, bar, c, k0, it.e);
                            } else {
                                if constexpr (PAIR) ptx::tma_load_2d_pair(a_dst + i * kChunkBytes, &tmap_a, bar_cl, c, it.first + k0);
                                else ptx::tma_load_2d(a_dst + i * kChunkBytes, &tmap_a, bar, c, it.first + k0);
                            }
                        }
                    }
                    for (int i = 0; i < nbox; ++i) {
                        if constexpr (WG) {
                            const int c = min(it.t0 + crank * half + 64 * i, (p.cols - 1) & ~7);
                            if constexpr (PAIR) ptx::tma_load_2d_pair(b_dst + i * kChunkBytes, &tmap_b, bar_cl, c, it.first + k0);
                            else ptx::tma_load_2d(b_dst + i * kChunkBytes, &tmap_b, bar, c, it.first + k0);
                        } else {
                            // rows past the group are other groups' (or zero): their columns of D are never stored
                            const int m = min(it.t0 + crank * half + i * p.box_rows, p.rows - 1);
                            uint8_t *dst = b_dst + i * p.box_rows * (BK * 2);
                            if constexpr (PAIR) ptx::tma_load_2d_pair(dst, &tmap_b, bar_cl, k0, m);
                            else ptx::tma_load_2d(dst, &tmap_b, bar, k0, m);
                        }
                    }
                    issued |= 1u << stage;
                    last_phase = (last_phase & ~(1u << stage)) | (phase << stage);
                    if (++stage == p.stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) atomicOr(p.err, TF_DEVERR_PRODUCER_WAIT);
            // every copy has landed before the CTA exits (a pair's complete on the first CTA's barriers)
            for (int s = 0; s < p.stages; ++s)
                if (leader && ((issued >> s) & 1u))
                    if (!ptx::mbar_wait<PAIR>(&full[s], (last_phase >> s) & 1u, p.wait_ns))
                        atomicOr(p.err, TF_DEVERR_DRAIN_WAIT);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0 && leader) {
            int stage = 0, local = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = cid; ok && t < num_work; t += ncl) {
                const Item it = item_of<MODE, CG>(p, row, tile, t);
                if (it.nkb == 0) continue;
                const uint32_t id = idesc(BM * CG, it.w, p.bf16 != 0, A_MMAJOR, WG);
                const int b = local & 1;
                if (!ptx::mbar_wait<PAIR>(&tempty[b], (uint32_t)((local >> 1) & 1) ^ 1u, p.wait_ns)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)(b * kMaxBN);
                for (int kb = 0; kb < it.nkb; ++kb) {
                    if (!ptx::mbar_wait<PAIR && WG>(&full[stage], phase, p.wait_ns)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t a = ptx::smem_u32(smem + stage * p.stage_bytes), bb = a + kABytes;
                    // WGRAD: sixteens of rows past the group's end are left out
                    const int steps = WG ? min(BK / UMMA_K, (it.tv - kb * BK + UMMA_K - 1) / UMMA_K) : BK / UMMA_K;
                    for (int k = 0; k < steps; ++k) {
                        const uint64_t ad = A_MMAJOR ? sw128_mnmajor_desc(a + k * UMMA_K * 128)
                                                     : ptx::sw128_kmajor_desc(a + k * UMMA_K * 2);
                        const uint64_t bd = WG ? sw128_mnmajor_desc(bb + k * UMMA_K * 128)
                                               : ptx::sw128_kmajor_desc(bb + k * UMMA_K * 2);
                        const uint32_t acc = (kb > 0 || k > 0) ? 1u : 0u;
                        if constexpr (PAIR) ptx::umma_bf16_pair(d_tmem, ad, bd, id, acc);
                        else ptx::umma_bf16(d_tmem, ad, bd, id, acc);
                    }
                    if constexpr (PAIR) {
                        ptx::umma_commit_pair(ptx::mapa_shared(&empty[stage], 0));
                        ptx::umma_commit_pair(ptx::mapa_shared(&empty[stage], 1));
                    } else {
                        ptx::umma_commit(&empty[stage]);
                    }
                    if (++stage == p.stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                if constexpr (PAIR) {
                    ptx::umma_commit_pair(ptx::mapa_shared(&tfull[b], 0));
                    ptx::umma_commit_pair(ptx::mapa_shared(&tfull[b], 1));
                } else {
                    ptx::umma_commit(&tfull[b]);
                }
                ++local;
            }
            if (!ok) atomicOr(p.err, TF_DEVERR_MMA_WAIT);
            if constexpr (PAIR) ptx::umma_commit_pair(ptx::smem_u32(drain));
            else ptx::umma_commit(drain);
            if (!ptx::mbar_wait(drain, 0, p.wait_ns)) atomicOr(p.err, TF_DEVERR_DRAIN_WAIT);
        }
    } else if (WG && warp == 2) {
        // ------------------------------------------------------------ zeroing warp
        // The last K step of a group holds rows of the next group (or what lies
        // behind the last): those of the sixteen that the last MMA reads become
        // zero in both operands, so that not even a NaN there reaches this group.
        uint32_t land_phase = 0;
        int blocks = 0;    // K steps before this item
        bool ok = true;
        for (int t = cid; t < num_work; t += ncl) {
            const Item it = item_of<MODE, CG>(p, row, tile, t);
            blocks += it.nkb;
            if ((it.tv & 15) == 0) continue;
            const int stage = (blocks - 1) % p.stages;
            ok = ptx::mbar_wait(&land[stage], (land_phase >> stage) & 1u, p.wait_ns);
            land_phase ^= 1u << stage;
            if (!__all_sync(0xffffffffu, ok)) break;
            const int r0 = it.tv - (it.nkb - 1) * BK, r1 = (r0 + 15) & ~15;
            uint8_t *base = smem + stage * p.stage_bytes;
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
        }
        if (!ok && lane == 0) atomicOr(p.err, TF_DEVERR_MMA_WAIT);
    } else if (warp >= kFirstEpiWarp) {
        // ------------------------------------------------------------ epilogue
        // Warp w reads TMEM lanes 32*(w%4) .. +31 (one weights row per lane) and
        // every second 32-column chunk.
        const int q = warp & 3, h = (warp - kFirstEpiWarp) >> 2;
        uint8_t *box = smem + p.off_dw + (warp - kFirstEpiWarp) * kDwBoxBytes;
        int local = 0;
        bool ok = true;
        for (int t = cid; t < num_work; t += ncl) {
            const Item it = item_of<MODE, CG>(p, row, tile, t);
            const int n0 = it.m0 + crank * BM + q * 32, n = n0 + lane;
            const bool in = n < p.M;
            const int b = local & 1;
            float bias = 0.0f;
            if (MODE == GROUPED_FORWARD && p.bias && in) bias = __ldg(p.bias + (int64_t)it.e * p.M + n);
            if (it.nkb > 0) {
                const bool got = ptx::mbar_wait(&tfull[b], (uint32_t)(local >> 1) & 1u, p.wait_ns);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
            } else if (!WG || p.accumulate) {
                continue;   // a group without rows adds nothing
            }
            const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * kMaxBN);
            const int width = WG ? min(kMaxBN, p.cols - it.t0) : it.tv;
#pragma unroll 1
            for (int c = h; c * 32 < width; c += kEpiWarps / 4) {
                uint32_t r[32];
                if (!WG || it.nkb > 0) {
                    ptx::tmem_ld_32x32b_x32(taddr + (uint32_t)(c * 32), r);
                    ptx::tmem_ld_wait();
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[j] = 0u;
                }
                if constexpr (WG) {
                    if (lane == 0) ptx::bulk_wait_group_read<0>();
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; ++j)   // 128-byte swizzle: 16-byte piece j of row l lies at j ^ (l % 8)
                        *reinterpret_cast<uint4 *>(box + lane * 128 + ((j ^ (lane & 7)) * 16)) =
                            make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && n0 < p.M) {
                        // clipped at the group's N rows and K columns
                        if (p.accumulate) tma_add_3d(&tmap_dw, box, it.t0 + c * 32, n0, it.e);
                        else tma_store_3d(&tmap_dw, box, it.t0 + c * 32, n0, it.e);
                        ptx::bulk_commit_group();
                    }
                } else {
                    const int count = min(32, width - c * 32);
                    const int64_t token = it.t0 + c * 32;
                    if (p.bf16) store_chunk<__nv_bfloat16, MODE>(p, r, count, token, n, in, bias);
                    else store_chunk<__half, MODE>(p, r, count, token, n, in, bias);
                }
            }
            if (it.nkb > 0) {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR) ptx::mbar_arrive_cluster(ptx::mapa_shared(&tempty[b], 0));
                    else ptx::mbar_arrive(&tempty[b]);
                }
                ++local;
            }
        }
        if (WG && lane == 0) ptx::bulk_wait_group_all();
        if (!ok && lane == 0) atomicOr(p.err, TF_DEVERR_EPILOGUE_WAIT);
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

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled()
{
    static EncodeTiledFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return (EncodeTiledFn) nullptr;
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

bool encode(CUtensorMap *m, CUtensorMapDataType type, int rank, const void *base, const cuuint64_t *dims,
            const cuuint64_t *strides, const cuuint32_t *box)
{
    const cuuint32_t ones[3] = {1, 1, 1};
    EncodeTiledFn fn = encode_tiled();
    return fn && fn(m, type, (cuuint32_t)rank, const_cast<void *>(base), dims, strides, box, ones,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [rows][cols] matrix of 16-bit values, rows `stride` elements apart.
bool encode_rows(CUtensorMap *m, CUtensorMapDataType type, const void *base, int64_t rows, int64_t cols, int64_t stride,
                 int box_cols, int box_rows)
{
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    return encode(m, type, 2, base, dims, strides, box);
}

// [groups][N][K] weights or weights' gradients.
bool encode_groups(CUtensorMap *m, CUtensorMapDataType type, const void *base, int64_t groups, int64_t N, int64_t K,
                   int size, int box_cols, int box_rows)
{
    const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)N, (cuuint64_t)groups};
    const cuuint64_t strides[2] = {(cuuint64_t)K * size, (cuuint64_t)N * K * size};
    const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
    return encode(m, type, 3, base, dims, strides, box);
}

// CTAs (or pairs) that can be resident at once, by device; the kernel's
// shared-memory limit is raised on the way.
template <int MODE, int CG>
cudaError_t resident(int *units)
{
    static std::mutex mu;
    static int known[64];
    int d = 0;
    cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess || d < 0 || d >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!known[d]) {
        auto kern = grouped_umma_kernel<MODE, CG>;
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
            cfg.blockDim = dim3(kThreads);
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

template <int MODE, int CG>
cudaError_t launch_mode(const GroupedArgs &a, int bn, cudaStream_t st)
{
    constexpr bool WG = MODE == GROUPED_WGRAD;
    UmmaArgs p = {};
    p.offsets = a.offsets;
    p.bias = a.bias;
    p.y = a.y;
    p.pre_in = a.pre;
    p.pre_out = a.pre;
    p.err = device_error_word();
    p.wait_ns = wait_limit_ns();
    if (!p.err) return cudaErrorInitializationError;
    p.y_stride = a.y_stride;
    p.pre_stride = a.pre_stride;
    p.groups = a.groups;
    p.rows = a.rows;
    p.M = MODE == GROUPED_DGRAD ? a.K : a.N;
    p.red = MODE == GROUPED_DGRAD ? a.N : a.K;
    p.cols = a.K;
    p.bn = bn;
    p.box_rows = bn / CG < 64 ? bn / CG : 64;
    p.act = a.act;
    p.bf16 = a.dtype == TF_BF16;
    p.accumulate = a.accumulate;
    p.stage_bytes = kABytes + (WG ? kMaxBN : bn) / CG * BK * 2;
    const int fixed = (WG ? kEpiWarps * kDwBoxBytes : 0) + kNumBars * 8 + 16 + (2 * (a.groups + 1) + 1) * 4;
    p.stages = (kSmemLimit - fixed) / p.stage_bytes;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    if (p.stages < 2) return cudaErrorNotSupported;
    p.off_dw = p.stages * p.stage_bytes;
    p.off_bar = p.off_dw + (WG ? kEpiWarps * kDwBoxBytes : 0);
    p.off_sched = p.off_bar + kNumBars * 8 + 16;
    const int smem = p.off_sched + (2 * (a.groups + 1) + 1) * 4;

    const CUtensorMapDataType type = p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    CUtensorMap ta, tb, td;
    memset(&td, 0, sizeof td);
    bool ok;
    if (MODE == GROUPED_FORWARD)
        ok = encode_groups(&ta, type, a.w, a.groups, a.N, a.K, 2, BK, BM) &&
             encode_rows(&tb, type, a.x, a.rows, a.K, a.x_stride, BK, p.box_rows);
    else if (MODE == GROUPED_DGRAD)
        ok = encode_groups(&ta, type, a.w, a.groups, a.N, a.K, 2, 64, BK) &&
             encode_rows(&tb, type, a.dy, a.rows, a.N, a.dy_stride, BK, p.box_rows);
    else
        ok = encode_rows(&ta, type, a.dy, a.rows, a.N, a.dy_stride, 64, BK) &&
             encode_rows(&tb, type, a.x, a.rows, a.K, a.x_stride, 64, BK) &&
             encode_groups(&td, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.dw, a.groups, a.N, a.K, 4, 32, 32);
    if (!ok) return cudaErrorInvalidValue;

    int units = 0;
    cudaError_t e = resident<MODE, CG>(&units);
    if (e != cudaSuccess) return e;
    const int64_t mt = (p.M + BM * CG - 1) / (BM * CG);
    const int64_t most = WG ? (int64_t)a.groups * mt * ((a.K + kMaxBN - 1) / kMaxBN)
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
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 2 ? 2 : 1;
    return counted(cudaLaunchKernelEx(&cfg, grouped_umma_kernel<MODE, CG>, ta, tb, td, p));
}

template <int MODE>
cudaError_t launch_auto(const GroupedArgs &a, cudaStream_t st)
{
    const int64_t M = MODE == GROUPED_DGRAD ? a.K : a.N;
    const int64_t avg = a.rows / a.groups;   // rows per group, as far as the host knows
    if (MODE == GROUPED_WGRAD) return M > BM && a.K > 128 ? launch_mode<MODE, 2>(a, kMaxBN, st) : launch_mode<MODE, 1>(a, kMaxBN, st);
    if (M > BM && avg > 128) return launch_mode<MODE, 2>(a, kMaxBN, st);
    return launch_mode<MODE, 1>(a, avg <= 32 ? 32 : avg <= 64 ? 64 : avg <= 128 ? 128 : 256, st);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

int64_t grouped_wgrad_workspace(int64_t, int, int64_t, int64_t, int) { return 0; }

cudaError_t launch_grouped(const GroupedArgs &a, int mode, cudaStream_t st)
{
    // what a tensor map can address: 16-byte rows and bases
    const bool dims = a.N % 8 == 0 && a.K % 8 == 0 && a.rows > 0;
    cudaError_t e;
    if (mode == GROUPED_FORWARD) {
        const bool tma = dims && a.x_stride % 8 == 0 && aligned16(a.x) && aligned16(a.w);
        return tma ? launch_auto<GROUPED_FORWARD>(a, st) : launch_grouped_simple(a, mode, st);
    }
    if (mode == GROUPED_DGRAD) {
        const bool tma = dims && a.dy_stride % 8 == 0 && aligned16(a.dy) && aligned16(a.w);
        return tma ? launch_auto<GROUPED_DGRAD>(a, st) : launch_grouped_simple(a, mode, st);
    }
    const bool tma = dims && a.dy_stride % 8 == 0 && a.x_stride % 8 == 0 && aligned16(a.dy) && aligned16(a.x) &&
                     aligned16(a.dw);
    e = tma ? launch_auto<GROUPED_WGRAD>(a, st) : launch_grouped_simple(a, mode, st);
    if (e != cudaSuccess || !a.dbias) return e;
    return launch_grouped_bias_grad(a, st);
}

}  // namespace tf
