// The products of the cross entropy over a vocabulary on the 5th-generation
// tensor cores.  Logits never reach memory:
//   STATS    D[t][v] = sum_h x[t][h] w[v][h]; the epilogue keeps, per row and
//            stretch of the tile's words, the largest sum and the sum of exponentials
//   DLOGITS  the same sums again; the epilogue turns them into the gradients of
//            the logits, dl = e^(l - lse) ca - [v = target] cb, in the operands' type,
//            for one piece of the vocabulary
//   GRADS    of that piece, in one launch:
//              DX[t][h] = sum_v dl[t][v] w[v][h]   A = dl (K-major), B = w (N-major)
//              DW[v][h] = sum_t dl[t][v] x[t][h]   A = dl (M-major), B = x (N-major)
//
// Rows (DW: words) are the MMA's M side, so that a thread of the epilogue has a row
// of the tile to itself and reduces over the vocabulary in its registers.
//
// Persistent kernel, one CTA (CG = 1, tiles of 128 rows, for few rows) or CTA pair
// (CG = 2, cta_group::2, tiles of 256 rows) per SM (pair), with two 256-column fp32
// accumulators, so that the epilogue of one tile overlaps the main loop of the
// next.  (Pairs with tiles of 512 x 256, which load a quarter less per product but
// fill the TMEM with one tile: 1152 us instead of 1064 for a step of 8192 rows, 3300 of
// which count, over 32000 words of 2048; 5047 instead of 5005 for 4096 rows, 64000 words of 4096.)  Warps:
//   0     TMA producer of a ring of K steps (64 deep, 128-byte swizzle)
//   1     TMEM allocator and MMA issuer
//   4-11  epilogue
// The tensor cores truncate where fp32 additions round, so an accumulator's error grows with
// the number of MMAs it takes.  A logit's sum is cut into parts of 1024 terms, dw's into parts of
// 4096, whose accumulators alternate; the epilogue's threads add them in registers while
// the next part's MMAs run.  (In one accumulator the gradients of weights by a million rows of one sign
// came out 6e-3 low, now 2e-6.)  dx's sums, of which 16 bits are kept, are cut into parts of 16384 terms, which are
// tiles of their own that add to the fp32 sums in memory.
// What bounds it, 4096 rows, 64000 words of 4096, bf16 (2.15 TFLOP each): STATS 1.02-1.05 ms
// alone (2.05-2.1 PFLOP/s), DLOGITS in two pieces 1.08-1.10, GRADS 2.23-2.26.  In a loop the power cap holds the
// clock down: 1.7 PFLOP/s.  With 4096 rows and 16384 words of 2048 the tensor pipe is busy for 95, 92 and 96% of the
// active cycles, with 1024 rows and 128000 words of 2048 for 97, 94 and 92%.
// Four rows over 128000 words: 157 us, 6.7 TB/s of weights.
// Every wait is bounded (ptx::mbar_wait); a role that times out sets the device
// error word and winds down.
#include <cuda.h>

#include <mutex>

#include "grouped.cuh"
#include "lm_internal.h"
#include "ptx_sm100.cuh"
#include "tensor_maps.h"

namespace tf {
namespace {

using grouped::BK;
using grouped::desc_low;
using grouped::desc_of;
using grouped::desc_step;
using grouped::elect_one;
using grouped::Half2Of;
using grouped::idesc;
using grouped::kChunkBytes;
using grouped::UMMA_K;

constexpr int kMaxStages = 6, kRingBytes = 192 * 1024;
constexpr int kEpiWarps = 8, kFirstEpiWarp = 4;
constexpr int kThreads = 32 * (kFirstEpiWarp + kEpiWarps);
constexpr int kTileN = 256;
constexpr int kABytes = 128 * BK * 2;               // 128 rows of a K step
constexpr int stage_bytes(int cg) { return kABytes + 256 / cg * BK * 2; }
// Gradients whose dw sums have more than one part.  (The registers that parts take cost short
// sums time: gradients of 7 rows over 88000 words of 2560 318 us in this kernel, 270 in the other; of 300 rows over 32000
// words of 2048 158 and 140.)
constexpr int LCE_LONG_GRADS = 3;
constexpr bool of_grads(int mode) { return mode == LCE_GRADS || mode == LCE_LONG_GRADS; }
// K steps per part of a sum in registers: 1024 terms of a logit's, 4096 of dw's.
constexpr int kGradSteps = 64;
// K steps per part of dx's in memory: 16384 terms of one sign come out 8e-5 low, a sixth of fp16's half step.
// (Step of 1024 rows over 128000 words of 2048: 1.46 ms, uncut 1.45, with parts of 4096 terms 1.48; of 4096 rows, 64000
// words of 4096: 5.00, uncut 4.96, with parts of 4096 terms 5.06.)
constexpr int kDxSteps = 256;
constexpr int part_steps(int mode) { return mode == LCE_GRADS ? 1 << 30 : mode == LCE_LONG_GRADS ? kGradSteps : 16; }
// Registers: the epilogue's threads hold 128 sums each while the issuing warps need few.  The
// kernel starts with 168 per thread, and 88*128 + 208*256 = 168*384.
constexpr int kIssueRegs = 88, kEpilogueRegs = 208;
constexpr int kBoxBytes = 32 * 128;                 // an epilogue warp's box: 32 rows of 128 bytes
constexpr int kOffBox = kRingBytes, kOffBar = kOffBox + kEpiWarps * kBoxBytes;
constexpr int kNumBars = 2 * kMaxStages + 5;
constexpr int kSmemBytes = kOffBar + kNumBars * 8 + 16;
// Up to here tiles of 128 rows on single CTAs (losses over 128000 words of 4096: 4 rows 159 us, 199 on
// pairs; 128 rows 172 and 181; 200 rows 205 and 185).
constexpr int kNarrowRows = 128;
constexpr uint32_t kTmemCols = 512;

// A tile's time in K steps, for sharing out the work: the epilogue's, where the K loop is shorter.
// A single CTA's K step waits for memory, a pair's for the tensor cores.  (Steps of 7 rows, 88000 words of
// 2560: 342 us, with 10 for single CTAs 396, with 2 352; of 400 rows, 32000 words of 2048: 193 us, with 5
// for pairs 212, with 20 205.)
constexpr int kLeastSingle = 4, kLeastPair = 10;
__host__ __device__ constexpr int tile_cost(int cg, int steps)
{
    return (steps > (cg == 1 ? kLeastSingle : kLeastPair) ? steps : cg == 1 ? kLeastSingle : kLeastPair) + 1;
}

struct VocabArgs {
    LceProduct a;
    uint32_t *err;
    uint64_t wait_ns;
    int bn;            // columns per tile
    int a_box;         // rows that a load of A brings (STATS, DLOGITS)
    int group;         // STATS, DLOGITS: row tiles that share a sweep over the vocabulary
    int split_steps;   // DX: K steps per split
    int dx_parts;      // DX: parts of a split's sum, which are added in memory
};

// A tile: rows [m0, +128*CG), columns [n0, +bn), K steps [k0, k0 + nk).
struct Tile {
    int kind, m0, n0, k0, nk, slot;
    bool adds;   // to what is there
};
enum { TILE_LOGITS = 0, TILE_DX = 1, TILE_DW = 2 };

__device__ __forceinline__ int div_up(int a, int b) { return (a + b - 1) / b; }

// Which tiles this CTA or pair takes, the j-th of them by at(); the same in all of its roles.
template <int MODE, int CG>
struct Share {
    static constexpr int ROWS = 128 * CG;
    int cid, ncl;
    int row_tiles, col_tiles;
    int tiles, sweep;              // STATS, DLOGITS: all of them, and those of one sweep over the vocabulary
    int own, plane, steps;         // GRADS: DX tiles that are this pair's; tiles of a split; K steps of DW
    int nw, lead, others, ahead;   // DW tiles; those that this pair takes first, and how many pairs do; what they take in all
    int rest;                      // its place in the round

    __device__ __forceinline__ void init(const VocabArgs &p, int count, int cid_, int ncl_)
    {
        cid = cid_;
        ncl = ncl_;
        row_tiles = div_up(count, ROWS);
        if constexpr (!of_grads(MODE)) {
            col_tiles = div_up(p.a.words, p.bn);
            tiles = row_tiles * col_tiles;
            sweep = p.group * col_tiles;
        } else {
            // DX tiles in turn; the pairs that have one less take DW tiles for its
            // time before the rest of those goes round
            col_tiles = div_up(p.a.hidden, p.bn);
            plane = row_tiles * col_tiles;
            steps = div_up(count, BK);
            const int nd = p.a.dx ? p.a.splits * plane : 0, more = nd % ncl;   // `more` pairs have a DX tile more
            nw = p.a.dw ? div_up(p.a.words, ROWS) * col_tiles : 0;
            own = nd / ncl + (cid < more ? 1 : 0);
            lead = 0;
            if (more > 0) {
                const int cost = tile_cost(CG, steps);
                lead = min((tile_cost(CG, p.split_steps) + cost / 2) / cost, div_up(nw, ncl - more));
            }
            others = ncl - more;
            ahead = lead * others;
            rest = cid < more ? cid - more + ncl : cid - more;
            if (cid < more) lead = 0;
        }
    }

    __device__ __forceinline__ bool at(const VocabArgs &p, int j, Tile *t) const
    {
        if constexpr (!of_grads(MODE)) {
            const int i = cid + j * ncl;
            if (i >= tiles) return false;
            const int g = i / sweep, r = i - g * sweep, size = min(p.group, row_tiles - g * p.group), v = r / size;
            *t = {TILE_LOGITS, (g * p.group + r - v * size) * ROWS, v * p.bn, 0, div_up(p.a.hidden, BK), p.a.slot0 + 2 * v, false};
            return true;
        } else {
            if (j < own * p.dx_parts) {
                const int tile = j / p.dx_parts, part = j - tile * p.dx_parts, i = cid + tile * ncl;
                const int s = i / plane, r = i - s * plane, m = r / col_tiles;
                const int end = min((s + 1) * p.split_steps, div_up(p.a.words, BK)), k0 = s * p.split_steps + part * kDxSteps;
                const int nk = max(0, p.dx_parts == 1 ? end - k0 : min(kDxSteps, end - k0));
                *t = {TILE_DX, m * ROWS, (r - m * col_tiles) * p.bn, k0, nk, s, !p.a.first || part > 0};
                return true;
            }
            j -= own * p.dx_parts;
            const int i = j < lead ? j * others + rest : ahead + (j - lead) * ncl + rest;
            if (i >= nw) return false;
            const int m = i / col_tiles;
            *t = {TILE_DW, m * ROWS, (i - m * col_tiles) * p.bn, 0, steps, 0, p.a.accumulate != 0};
            return true;
        }
    }
};

// The box: row `lane`'s piece i of 16 bytes on the way in, row 4i + lane/8's piece
// lane%8 on the way out; the pieces are swizzled so that neither side meets a bank twice.
__device__ __forceinline__ void box_put(uint8_t *box, int lane, int i, uint4 v)
{
    *reinterpret_cast<uint4 *>(box + lane * 128 + ((i ^ (lane & 7)) * 16)) = v;
}
__device__ __forceinline__ uint4 box_get(const uint8_t *box, int row, int piece)
{
    return *reinterpret_cast<const uint4 *>(box + row * 128 + ((piece ^ (row & 7)) * 16));
}

// The first n of row `at`'s columns to where no 16-byte words lie: 32 of 32 bits one by one, or
// 64 of 16 bits in pairs that share a 32-bit word (an odd start leaves its first and
// its last column single).
__device__ __forceinline__ void put_single(float *dst, const uint8_t *box, int at, int n, bool add)
{
    const int lane = threadIdx.x & 31;
    if (lane >= n) return;
    const float v = *reinterpret_cast<const float *>(box + at * 128 + ((lane >> 2) ^ (at & 7)) * 16 + (lane & 3) * 4);
    dst[lane] = add ? dst[lane] + v : v;
}
__device__ __forceinline__ void put_pairs(uint16_t *dst, const uint8_t *box, int at, int n)
{
    auto value = [&](int i) {
        return *reinterpret_cast<const uint16_t *>(box + at * 128 + ((i >> 3) ^ (at & 7)) * 16 + (i & 7) * 2);
    };
    const int lane = threadIdx.x & 31, odd = (int)(reinterpret_cast<uintptr_t>(dst) >> 1) & 1, e = 2 * lane - odd;
    if (e >= 0 && e + 1 < n) *reinterpret_cast<uint32_t *>(dst + e) = value(e) | (uint32_t)value(e + 1) << 16;
    else if (e + 1 < n) dst[e + 1] = value(e + 1);
    else if (e < n) dst[e] = value(e);
    if (odd && lane == 0 && n == 64) dst[63] = value(63);
}

// ---------------------------------------------------------------- epilogues

// The columns [n0 + c, +32) of one row join its running maximum and sum of exponentials.
__device__ __forceinline__ void join_stats(const uint32_t (&r)[32], int left, float factor, float &top, float &sum)
{
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = j < left ? __uint_as_float(r[j]) : -INFINITY;
    float m[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int j = 4; j < 32; ++j) m[j & 3] = fmaxf(m[j & 3], v[j]);
    const float most = fmaxf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), top);
    const float base = most == -INFINITY ? 0.0f : most;
    // the difference before the factor: a sure word's exponential is one, however large its logit
    const float2 base2 = make_float2(base, base), factor2 = make_float2(factor, factor);
    float s[4] = {sum * ex2_approx((top - base) * factor), 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
        const float2 d = fmul2(fsub2(make_float2(v[j], v[j + 1]), base2), factor2);
        s[j & 2] += ex2_approx(d.x);
        s[(j & 2) + 1] += ex2_approx(d.y);
    }
    sum = (s[0] + s[1]) + (s[2] + s[3]);
    top = most;
}

// r[i] of a register array, i the same for no two lanes in general.
__device__ __forceinline__ float pick(const uint32_t (&r)[32], int i)
{
    uint32_t v = r[0];
#pragma unroll
    for (int j = 1; j < 32; ++j) v = j == i ? r[j] : v;
    return __uint_as_float(v);
}

template <int MODE, int CG>
__global__ void __launch_bounds__(kThreads, 1)
    vocab_umma_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                      const __grid_constant__ CUtensorMap map_x, const __grid_constant__ VocabArgs p)
{
    constexpr bool PAIR = CG == 2;
    constexpr int kStageBytes = stage_bytes(CG), kStages = kRingBytes / kStageBytes, kPartSteps = part_steps(MODE);
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kOffBar);
    uint64_t *empty = full + kStages;
    uint64_t *tfull = empty + kStages;
    uint64_t *tempty = tfull + 2;
    uint64_t *drain = tempty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int crank = PAIR ? (int)ptx::cluster_ctarank() : 0;
    const bool leader = crank == 0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(&full[i], 1);
            ptx::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&tfull[i], 1);
            ptx::mbar_init(&tempty[i], CG * kEpiWarps);   // one lane per epilogue warp of either CTA
        }
        ptx::mbar_init(drain, 1);
        ptx::mbar_init_fence();
        ptx::prefetch_tensormap(&map_a);
        ptx::prefetch_tensormap(&map_w);
        ptx::prefetch_tensormap(&map_x);
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
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    ptx::tc_fence_before();
    cta_sync();
    ptx::tc_fence_after();
    if constexpr (PAIR) ptx::cluster_sync();   // the peer's barriers exist
    const uint32_t tmem_base = *tmem_slot;
    bool sound = true;
    if ((ptx::smem_u32(smem) & 1023u) != 0) {
        sound = false;
        if (threadIdx.x == 0) atomicOr(p.err, TF_DEVERR_SMEM_ALIGN);
    }
    if constexpr (PAIR) {
        if (ptx::ld_shared_cluster_u32(ptx::mapa_shared(tmem_slot, (uint32_t)crank ^ 1u)) != tmem_base) {
            sound = false;
            if (threadIdx.x == 0) atomicOr(p.err, TF_DEVERR_PAIR_TMEM);
        }
    }
    const int count = *p.a.count;
    Share<MODE, CG> share;
    share.init(p, count, (int)blockIdx.x / CG, (int)gridDim.x / CG);

    // (one branch per warpgroup, which changes its registers as a whole)
    if (warp < kFirstEpiWarp) {
        if constexpr (MODE != LCE_GRADS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (sound && warp == 0) {
            // ------------------------------------------------------------ producer
            int stage = 0;
            uint32_t phase = 0, issued = 0, last_phase = 0;
            bool ok = true;
            const bool issuer = elect_one();
            const int half = p.bn / CG;   // columns of B that this CTA loads
            Tile t;
            for (int j = 0; ok && share.at(p, j, &t); ++j) {
                for (int kb = 0; kb < t.nk; ++kb) {
                    const bool got = ptx::mbar_wait(&empty[stage], phase ^ 1u, p.wait_ns);
                    if (!__all_sync(0xffffffffu, got)) {
                        ok = false;
                        break;
                    }
                    if (issuer) {
                        uint64_t *bar = &full[stage];
                        uint8_t *a_dst = smem + stage * kStageBytes, *b_dst = a_dst + kABytes;
                        const int k = (t.k0 + kb) * BK, row = t.m0 + crank * 128;
                        const uint32_t bar_cl = PAIR ? ptx::mapa_shared(bar, 0) : 0u;
                        auto load = [&](void *dst, const CUtensorMap *map, int c0, int c1) {
                            if constexpr (PAIR) ptx::tma_load_2d_pair(dst, map, bar_cl, c0, c1);
                            else ptx::tma_load_2d(dst, map, bar, c0, c1);
                        };
                        if constexpr (!of_grads(MODE)) {
                            if (leader) ptx::mbar_arrive_expect_tx(bar, (uint32_t)(CG * (p.a_box + half) * (BK * 2)));
                            load(a_dst, &map_a, k, row);
                            load(b_dst, &map_w, k, t.n0 + crank * half);
                        } else {
                            if (leader) ptx::mbar_arrive_expect_tx(bar, (uint32_t)(CG * (128 + half) * (BK * 2)));
                            const CUtensorMap *map_b = t.kind == TILE_DX ? &map_w : &map_x;
#pragma unroll
                            for (int i = 0; i < 2; ++i) {   // boxes of 64 rows (DX) or 64 words (DW)
                                const int m = row + 64 * i;
                                if (t.kind == TILE_DX) load(a_dst + i * kChunkBytes, &map_a, k, m);
                                else load(a_dst + i * kChunkBytes, &map_a, m, k);
                            }
                            for (int i = 0; i < half / 64; ++i)
                                load(b_dst + i * kChunkBytes, map_b, t.n0 + crank * half + 64 * i, k);
                        }
                    }
                    __syncwarp();
                    issued |= 1u << stage;
                    last_phase = (last_phase & ~(1u << stage)) | (phase << stage);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok && lane == 0) atomicOr(p.err, TF_DEVERR_PRODUCER_WAIT);
            // every copy has landed before the CTA exits (a pair's complete on the first CTA's barriers)
            for (int s = 0; s < kStages; ++s)
                if (leader && ((issued >> s) & 1u))
                    if (!ptx::mbar_wait<PAIR>(&full[s], (last_phase >> s) & 1u, p.wait_ns) && lane == 0)
                        atomicOr(p.err, TF_DEVERR_DRAIN_WAIT);
        } else if (sound && warp == 1) {
            // ------------------------------------------------------------ MMA issuer
            if (leader) {
                int stage = 0, b = 0;
                uint32_t phase = 0, taken = 0;   // taken: parity of the uses of either accumulator
                bool ok = true;
                const bool issuer = elect_one(), bf16 = p.a.dtype == TF_BF16;
                const uint32_t base = ptx::smem_u32(smem);
                Tile t;
                for (int j = 0; ok && share.at(p, j, &t); ++j) {
                    if (t.nk == 0) continue;
                    const bool a_mn = t.kind == TILE_DW, b_mn = of_grads(MODE);
                    const uint32_t id = idesc(128 * CG, p.bn, bf16, a_mn, b_mn);
                    const uint32_t a_step = a_mn ? desc_step(false) : desc_step(true), b_step = desc_step(!b_mn);
                    const uint32_t a_low = desc_low(base, !a_mn), b_low = desc_low(base + kABytes, !b_mn);
                    auto commit = [&](uint64_t *bar) {
                        if constexpr (PAIR) ptx::umma_commit_both(bar);
                        else ptx::umma_commit(bar);
                    };
                    for (int kb = 0; kb < t.nk; ++kb) {
                        const bool begins = kb % kPartSteps == 0, ends = kb == t.nk - 1 || kb % kPartSteps == kPartSteps - 1;
                        if (begins) {
                            const bool got = ptx::mbar_wait<PAIR>(&tempty[b], ((taken >> b) & 1u) ^ 1u, p.wait_ns);
                            if (!__all_sync(0xffffffffu, got)) {
                                ok = false;
                                break;
                            }
                        }
                        const bool got = ptx::mbar_wait(&full[stage], phase, p.wait_ns);
                        if (!__all_sync(0xffffffffu, got)) {
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after();
                        if (issuer) {
                            const uint32_t at = (uint32_t)stage * (kStageBytes >> 4), d = tmem_base + (uint32_t)(b * kTileN);
#pragma unroll
                            for (int k = 0; k < BK / UMMA_K; ++k) {
                                const uint64_t a = desc_of(a_low + at + k * a_step), bb = desc_of(b_low + at + k * b_step);
                                const uint32_t acc = k > 0 || !begins ? 1u : 0u;
                                if constexpr (PAIR) ptx::umma_bf16_pair(d, a, bb, id, acc);
                                else ptx::umma_bf16(d, a, bb, id, acc);
                            }
                            commit(&empty[stage]);
                            if (ends) commit(&tfull[b]);
                        }
                        __syncwarp();
                        if (ends) {
                            taken ^= 1u << b;
                            b ^= 1;
                        }
                        if (++stage == kStages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
                if (!ok && lane == 0) atomicOr(p.err, TF_DEVERR_MMA_WAIT);
                if (issuer) {   // (the lane that issued the MMAs)
                    if constexpr (PAIR) ptx::umma_commit_pair(ptx::smem_u32(drain));
                    else ptx::umma_commit(drain);
                }
                __syncwarp();
                if (!ptx::mbar_wait(drain, 0, p.wait_ns) && lane == 0) atomicOr(p.err, TF_DEVERR_DRAIN_WAIT);
            }
        }
    } else {
        if constexpr (MODE != LCE_GRADS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpilogueRegs));
        if (sound) {
            // ------------------------------------------------------------ epilogue
            // Warp w reads TMEM lanes 32*(w%4) .. +31, one row per lane, and one half of the columns.
            const int q = warp & 3, h = (warp - kFirstEpiWarp) >> 2;
            uint8_t *box = smem + kOffBox + (warp - kFirstEpiWarp) * kBoxBytes;
            const bool bf16 = p.a.dtype == TF_BF16;
            const int mid = (p.bn / 2 + 63) & ~63, c0 = h ? mid : 0, c1 = h ? p.bn : mid;   // this warp's columns of a tile
            const float mult = p.a.factor * (of_grads(MODE) ? __ldg(p.a.unit + 1) : 1.0f);
            int b = 0;
            uint32_t seen = 0;   // parity of the results of either accumulator
            bool ok = true;
            Tile t;
            auto pack = [&](uint32_t x, uint32_t y) {
                const float a = __uint_as_float(x), b = __uint_as_float(y);
                return bf16 ? Half2Of<__nv_bfloat16>::pack(a, b) : Half2Of<__half>::pack(a, b);
            };
            // 32 columns as 16-bit values into one half of the box's rows
            auto put_half = [&](const uint32_t (&r)[32], int part) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) w[k] = pack(r[8 * i + 2 * k], r[8 * i + 2 * k + 1]);
                    box_put(box, lane, part * 4 + i, make_uint4(w[0], w[1], w[2], w[3]));
                }
            };
            for (int j = 0; ok && share.at(p, j, &t); ++j) {
                const int row0 = t.m0 + crank * 128 + q * 32, row = row0 + lane;
                const int width = min(p.bn, (of_grads(MODE) ? p.a.hidden : p.a.words) - t.n0);
                // rows of this tile's M side: DLOGITS also writes the zeros behind them that dw's last K step reads
                const int rows = MODE == LCE_DLOGITS         ? (count + BK - 1) / BK * BK
                                 : t.kind == TILE_DW ? p.a.words
                                                     : count;
                const int left = row0 < rows ? min(width, c1) - c0 : 0;   // columns with results, up to 128
                int target = -1;
                float z = 0.0f, ca = 0.0f, cb = 0.0f;
                if constexpr (!of_grads(MODE)) {
                    if (row < count) {
                        target = __ldg(p.a.target + row) - p.a.v0 - t.n0 - c0;   // its place among this warp's columns
                        if constexpr (MODE == LCE_DLOGITS) {
                            z = __ldg(p.a.z + row);
                            ca = __ldg(p.a.ca + row);
                            cb = __ldg(p.a.cb + row);
                        }
                    }
                }
                // waits for the accumulator of the next part (or tile)
                auto await = [&]() {
                    const bool got = ptx::mbar_wait(&tfull[b], (seen >> b) & 1u, p.wait_ns);
                    if (!__all_sync(0xffffffffu, got)) return ok = false;
                    ptx::tc_fence_after();
                    seen ^= 1u << b;
                    return true;
                };
                // hands it back
                auto release = [&]() {
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (PAIR) ptx::mbar_arrive_cluster(ptx::mapa_shared(&tempty[b], 0));
                        else ptx::mbar_arrive(&tempty[b]);
                    }
                    b ^= 1;
                };
                const uint32_t columns = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)c0;
                uint32_t r[4][32];   // the sums of this row's columns
                // adds a tile's parts
                auto sum_parts = [&]() {
                    for (int k0 = 0; k0 < t.nk; k0 += kPartSteps) {
                        if (!await()) return;
                        const uint32_t taddr = columns + (uint32_t)(b * kTileN);
                        if (k0 == 0) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (32 * i < left) ptx::tmem_ld_32x32b_x32(taddr + (uint32_t)(32 * i), r[i]);
                            ptx::tmem_ld_wait();
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (32 * i >= left) break;
                                uint32_t v[32];
                                ptx::tmem_ld_32x32b_x32(taddr + (uint32_t)(32 * i), v);
                                ptx::tmem_ld_wait();
#pragma unroll
                                for (int k = 0; k < 32; k += 2) {
                                    const float2 old = make_float2(__uint_as_float(r[i][k]), __uint_as_float(r[i][k + 1]));
                                    const float2 sum = fadd2(old, make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])));
                                    r[i][k] = __float_as_uint(sum.x);
                                    r[i][k + 1] = __float_as_uint(sum.y);
                                }
                            }
                        }
                        release();
                    }
                };
                if constexpr (!of_grads(MODE)) {
                    sum_parts();
                    if (!ok) break;
                    if constexpr (MODE == LCE_STATS) {
                        float top = -INFINITY, sum = 0.0f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int c = 32 * i;
                            if (c >= left) break;
                            if (c + 32 <= left) join_stats(r[i], 32, p.a.factor, top, sum);
                            else join_stats(r[i], left - c, p.a.factor, top, sum);
                            const int at = target - c;
                            const bool hit = at >= 0 && at < 32 && target < left;
                            if (__any_sync(0xffffffffu, hit)) {
                                const float v = pick(r[i], at);
                                if (hit) p.a.at_target[row] = v;
                            }
                        }
                        if (row < count) p.a.part[(int64_t)(t.slot + h) * p.a.rows + row] = make_float2(top, sum);
                    } else {
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            if (64 * u >= left) break;
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const int i = 2 * u + half, c = 32 * i;
                                // lse before log2(e), so that a sure word's exponential is one, however large its logit
                                const float2 scale2 = make_float2(p.a.factor, p.a.factor), z2 = make_float2(-z, -z);
                                const float2 log2e2 = make_float2(kLog2e, kLog2e);
#pragma unroll
                                for (int k = 0; k < 32; k += 2) {
                                    const float2 l = make_float2(__uint_as_float(r[i][k]), __uint_as_float(r[i][k + 1]));
                                    const float2 d = fmul2(ffma2(l, scale2, z2), log2e2);
                                    r[i][k] = __float_as_uint(ex2_approx(d.x) * ca);
                                    r[i][k + 1] = __float_as_uint(ex2_approx(d.y) * ca);
                                }
                                const int at = target - c;
                                const bool hit = at >= 0 && at < 32 && target < left;
                                if (__any_sync(0xffffffffu, hit)) {
#pragma unroll
                                    for (int k = 0; k < 32; ++k)
                                        if (hit && k == at) r[i][k] = __float_as_uint(__uint_as_float(r[i][k]) - cb);
                                }
                                // columns behind the piece's words, and rows behind those that count, which
                                // dw's last K step reads: zeros
                                if (c + 32 > left || row0 + 32 > count) {
#pragma unroll
                                    for (int k = 0; k < 32; ++k) r[i][k] = row < count && c + k < left ? r[i][k] : 0u;
                                }
                                put_half(r[i], half);
                            }
                            __syncwarp();
                            const int piece = lane & 7, c = c0 + 64 * u + 8 * piece;
                            uint16_t *out = static_cast<uint16_t *>(p.a.dl) + t.n0 + c;
                            if (c < c1 && t.n0 + c < p.a.dl_pitch) {
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const int at = 4 * i + (lane >> 3);
                                    uint16_t *to = out + (int64_t)(row0 + at) * p.a.dl_pitch;
                                    if (row0 + at < p.a.rows) *reinterpret_cast<uint4 *>(to) = box_get(box, at, piece);
                                }
                            }
                            __syncwarp();
                        }
                    }
                } else {
                    const uint32_t taddr = columns + (uint32_t)(b * kTileN);
                    const bool dx = t.kind == TILE_DX;
                    const bool wide = dx || p.a.dw_f32;        // 32-bit results
                    const bool add = t.adds;
                    const int64_t pitch = dx ? p.a.dx_pitch : p.a.hidden;
                    uint8_t *out = dx ? reinterpret_cast<uint8_t *>(p.a.dx + (int64_t)t.slot * p.a.rows * p.a.dx_pitch)
                                      : static_cast<uint8_t *>(p.a.dw);
                    // rows that 16-byte words make up
                    const bool words = (reinterpret_cast<uintptr_t>(out) & 15u) == 0 && pitch % (wide ? 4 : 8) == 0;
                    // several parts are added first; one is read 64 columns at a time as they leave.  (Kernels that add
                    // parts have both halves of the loop apart, so that every sum has a register of its own.)
                    const bool parts = MODE == LCE_LONG_GRADS && t.nk > kPartSteps;
                    if (parts) {
                        sum_parts();
                        if (!ok) break;
                    } else if (t.nk > 0) {
                        if (!await()) break;
                        if (left <= 0) release();
                    }
                    constexpr int UNROLL = MODE == LCE_LONG_GRADS ? 2 : 1;
#pragma unroll UNROLL
                    for (int pass = 0; pass < 2; ++pass) {
                        const int u = 64 * pass, h0 = MODE == LCE_LONG_GRADS ? 2 * pass : 0, h1 = h0 + 1;
                        if (u >= left) break;
                        if (!parts && t.nk > 0) {
                            ptx::tmem_ld_32x32b_x32(taddr + (uint32_t)u, r[h0]);
                            ptx::tmem_ld_32x32b_x32(taddr + (uint32_t)(u + 32), r[h1]);
                            ptx::tmem_ld_wait();
                            if (u + 64 >= left) release();
                        } else if (!parts) {
#pragma unroll
                            for (int k = 0; k < 32; ++k) r[h0][k] = r[h1][k] = 0u;
                        }
                        if (t.nk == 0 && add) break;
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            r[h0][k] = __float_as_uint(__uint_as_float(r[h0][k]) * mult);
                            r[h1][k] = __float_as_uint(__uint_as_float(r[h1][k]) * mult);
                        }
                        if (!wide) {
                            put_half(r[h0], 0);
                            put_half(r[h1], 1);
                        }
                        const int per = wide ? 4 : 8, size = wide ? 4 : 2;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (i == 1 && (!wide || u + 32 >= left)) break;
                            if (wide) {
#pragma unroll
                                for (int k = 0; k < 8; ++k) {
                                    const uint32_t *v = &r[h0 + i][4 * k];
                                    box_put(box, lane, k, make_uint4(v[0], v[1], v[2], v[3]));
                                }
                            }
                            __syncwarp();
                            // the box's rows, of 128 bytes from column c on
                            const int c = t.n0 + c0 + u + 32 * i;
                            if (words) {
                                const int piece = lane & 7, col = c + per * piece;
                                uint8_t *dst = out + ((int64_t)(row0 + (lane >> 3)) * pitch + col) * size;
#pragma unroll
                                for (int k = 0; k < 8; ++k) {
                                    const int at = 4 * k + (lane >> 3);
                                    if (row0 + at >= rows || col >= pitch) continue;
                                    uint4 *to = reinterpret_cast<uint4 *>(dst + (int64_t)(4 * k) * pitch * size);
                                    uint4 v = box_get(box, at, piece);
                                    // dx's are added by the L2, for which no thread waits (dx alone, 64 rows, 128000 words
                                    // of 4096: 418 us, with loads 437); a sum's parts come from one thread, so in order
                                    if (add && dx) {
                                        asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(to),
                                                     "f"(__uint_as_float(v.x)), "f"(__uint_as_float(v.y)),
                                                     "f"(__uint_as_float(v.z)), "f"(__uint_as_float(v.w))
                                                     : "memory");
                                        continue;
                                    }
                                    if (add) {
                                        const uint4 o = *to;
                                        v.x = __float_as_uint(__uint_as_float(v.x) + __uint_as_float(o.x));
                                        v.y = __float_as_uint(__uint_as_float(v.y) + __uint_as_float(o.y));
                                        v.z = __float_as_uint(__uint_as_float(v.z) + __uint_as_float(o.z));
                                        v.w = __float_as_uint(__uint_as_float(v.w) + __uint_as_float(o.w));
                                    }
                                    *to = v;
                                }
                            } else {
                                const int n = (int)min((int64_t)(8 * per), pitch - c);   // columns of a row
                                for (int at = 0; at < min(32, rows - row0); ++at) {
                                    uint8_t *to = out + ((int64_t)(row0 + at) * pitch + c) * size;
                                    if (wide) put_single(reinterpret_cast<float *>(to), box, at, n, add);
                                    else put_pairs(reinterpret_cast<uint16_t *>(to), box, at, n);
                                }
                            }
                            __syncwarp();
                        }
                    }
                }
            }
            if (!ok && lane == 0) atomicOr(p.err, TF_DEVERR_EPILOGUE_WAIT);
        }
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
        auto kern = vocab_umma_kernel<MODE, CG>;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (e != cudaSuccess) return e;
        // the warpgroups' shares of the registers must not exceed what the kernel starts with
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, kern);
        if (e != cudaSuccess) return e;
        if (MODE != LCE_GRADS && kIssueRegs * 32 * kFirstEpiWarp + kEpilogueRegs * 32 * kEpiWarps > fa.numRegs * kThreads)
            return cudaErrorNotSupported;
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
            cfg.dynamicSmemBytes = kSmemBytes;
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

// K steps per split of dx's sums.
int split_steps(const LceProduct &a) { return ((a.words + BK - 1) / BK + a.splits - 1) / a.splits; }

template <int MODE, int CG>
cudaError_t launch_mode(const LceProduct &a, cudaStream_t st)
{
    constexpr int ROWS = 128 * CG;
    VocabArgs p = {};
    p.a = a;
    p.err = device_error_word();
    p.wait_ns = wait_limit_ns();
    if (!p.err) return cudaErrorInitializationError;
    const int row_tiles = (a.rows + ROWS - 1) / ROWS;
    int64_t tiles;
    if (of_grads(MODE)) {
        const int nh = (a.hidden + kTileN - 1) / kTileN, step = 64 * CG;   // equal widths, in whole boxes of either CTA
        p.bn = ((a.hidden + nh - 1) / nh + step - 1) / step * step;
        p.split_steps = split_steps(a);
        p.dx_parts = MODE == LCE_LONG_GRADS ? 1 : (p.split_steps + kDxSteps - 1) / kDxSteps;
        const int64_t cols = (a.hidden + p.bn - 1) / p.bn;
        tiles = ((a.dx ? (int64_t)a.splits * row_tiles : 0) + (a.dw ? (a.words + ROWS - 1) / ROWS : 0)) * cols;
    } else {
        p.bn = lce_word_tile(a.rows, a.words);
        p.a_box = CG == 2 || a.rows >= 128 ? 128 : (a.rows + 7) / 8 * 8;
        // rows whose tiles of x stay in L2 while the vocabulary goes past
        const int64_t fit = ((int64_t)32 << 20) / ((int64_t)ROWS * a.x_pitch * 2);
        p.group = fit < 1 ? 1 : fit > row_tiles ? row_tiles : (int)fit;
        tiles = (int64_t)row_tiles * ((a.words + p.bn - 1) / p.bn);
    }
    if (tiles == 0) return cudaSuccess;
    if (tiles >= (int64_t)1 << 31) return cudaErrorNotSupported;

    cudaError_t e = bind_context();
    if (e != cudaSuccess) return e;
    const CUtensorMapDataType type = a.dtype == TF_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    CUtensorMap ma, mw, mx;
    const int rows = a.rows > 0 ? a.rows : 1;   // (dw without rows: nothing is loaded)
    bool ok;
    if (of_grads(MODE)) {
        ok = encode_rows(&ma, type, a.dl, rows, a.words, a.dl_pitch, 64, 64) &&
             encode_rows(&mw, type, a.w, a.words, a.hidden, a.w_pitch, 64, 64) &&
             encode_rows(&mx, type, a.x, rows, a.hidden, a.x_pitch, 64, 64);
    } else {
        ok = encode_rows(&ma, type, a.x, rows, a.hidden, a.x_pitch, BK, p.a_box) &&
             encode_rows(&mw, type, a.w, a.words, a.hidden, a.w_pitch, BK, p.bn / CG);
        mx = ma;
    }
    if (!ok) return cudaErrorInvalidValue;

    int units = 0;
    e = resident<MODE, CG>(&units);
    if (e != cudaSuccess) return e;
    if (units > tiles) units = (int)tiles;
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
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 2 ? 2 : 1;
    return counted(cudaLaunchKernelEx(&cfg, vocab_umma_kernel<MODE, CG>, ma, mw, mx, p));
}

template <int MODE>
cudaError_t launch_rows(const LceProduct &a, cudaStream_t st)
{
    return a.rows <= kNarrowRows ? launch_mode<MODE, 1>(a, st) : launch_mode<MODE, 2>(a, st);
}

}  // namespace

int lce_row_tile(int64_t rows) { return rows <= kNarrowRows ? 128 : 256; }
int lce_units(int64_t rows) { return rows <= kNarrowRows ? sm_count() : sm_count() / 2; }

// As many waves of tiles as the widest take, of tiles as narrow as they then can be.
int lce_word_tile(int64_t rows, int64_t words)
{
    const bool narrow = rows <= kNarrowRows;
    const int64_t n = lce_units(rows), down = (rows + lce_row_tile(rows) - 1) / lce_row_tile(rows);
    const int64_t step = narrow ? 16 : 32;
    const int64_t waves = (down * ((words + kTileN - 1) / kTileN) + n - 1) / n, across = n * waves / down;
    const int64_t bn = ((words + across - 1) / across + step - 1) / step * step;
    return bn < 64 ? 64 : bn > kTileN ? kTileN : (int)bn;
}

// Splits of dx's sums: no longer than a CTA's (pair's) share of both gradients (301 rows,
// 10007 words of 1000: GRADS 22 us; with the most that fill two waves 33).
int lce_splits(int64_t rows, int64_t words, int64_t hidden)
{
    const int64_t tile = lce_row_tile(rows), across = (hidden + kTileN - 1) / kTileN;
    const int64_t steps = (words + BK - 1) / BK;
    const int64_t dx = (rows + tile - 1) / tile * across, dw = (words + tile - 1) / tile * across;
    const int cg = rows <= kNarrowRows ? 1 : 2;
    const int64_t share = (dx * tile_cost(cg, (int)steps) + dw * tile_cost(cg, (int)((rows + BK - 1) / BK))) / lce_units(rows);
    const int64_t s = (steps + share) / (share + 1);
    return s < 1 ? 1 : s > 16 ? 16 : (int)s;
}

cudaError_t launch_lce_product(int mode, const LceProduct &a, cudaStream_t st)
{
    if (mode == LCE_STATS) return launch_rows<LCE_STATS>(a, st);
    if (mode == LCE_DLOGITS) return launch_rows<LCE_DLOGITS>(a, st);
    const bool parts = a.dw && a.rows > kGradSteps * BK;
    return parts ? launch_rows<LCE_LONG_GRADS>(a, st) : launch_rows<LCE_GRADS>(a, st);
}

}  // namespace tf
