// Grouped products of operands that no tensor map can address (rows that are
// not multiples of 16 bytes, or unaligned bases):
//   FORWARD  y[m][n]     = act(sum_k x[m][k] w[e][n][k] + bias[e][n])   for m in group e
//   DGRAD    dx[m][k]    = (sum_n dy[m][n] w[e][n][k]) * act'(pre[m][k])
//   WGRAD    dw[e][n][k] = sum_{m in e} dy[m][n] x[m][k]
// Tensor cores all the same, with operands that threads bring: eight warps load
// 128-byte pieces of rows, two values per lane (a 4-byte load where the operand
// allows it, else two of 2 bytes), and put them into the swizzled tiles that
// the MMAs read; the first of them issues those, one K step behind.  Values outside a row, a group
// or the reduction become zeros on the way, so nothing there is read or counts.
// The side of the output that is contiguous in memory is the MMA's M side (n,
// k, and for WGRAD k too): a TMEM lane holds one value of every output row, and
// a warp's stores lie side by side.
//
// 128 x 128 tiles, two CTAs per SM, so that one loads while the other stores.
// Bound by the loads' way through the L1: a K step of both operands is 256
// pieces, the MMAs on it take 128 cycles.  16384 rows, 16 groups, bf16: forward
// 401 us for 2047 x 1001, 242 us (278 TFLOP/s) for 2046 x 1002, whose rows are
// whole words; on the CUDA cores either took 2.9 ms.  All of a K
// step's loads are under way at once; joining the values of a word as they come
// took 1343 and 306 us.  A ninth warp for the MMAs (96 registers instead of
// 128): 526 and 226 us.
#include <mutex>

#include "grouped.cuh"

namespace tf {
namespace {

using namespace grouped;

constexpr int TILE = 128, kStages = 3, kLoadWarps = 8, kThreads = 32 * kLoadWarps;
constexpr int kOperandBytes = TILE * BK * 2, kStageBytes = 2 * kOperandBytes;
constexpr int kSmemBytes = kStages * kStageBytes + 1024;   // (the ring starts on a multiple of 1024)
constexpr int kPerWarp = TILE / kLoadWarps;                // pieces of one operand per warp and K step
constexpr int kMaxPartRows = 1024;                         // WGRAD: rows per accumulation; dw adds the parts

// One operand's tile: `rows` x `cols` values from `src` on, rows `ld` apart.
struct Source {
    const uint16_t *src;
    int64_t ld;
    int rows, cols;
};

// A warp's pieces of the K step at k0: piece i = warp + 8j is row i of a K-major
// tile, values k0..k0+63, or row k0 + i%64 of an M- or N-major one, values
// 64*(i/64) and on.  Lane l holds the values 2l and 2l+1, as one word or as two.
struct Pieces {
    uint32_t lo[kPerWarp], hi[kPerWarp];
};

template <bool KMAJOR>
__device__ __forceinline__ void load_pieces(Pieces &v, const Source &s, int k0, int warp, int lane)
{
    const int r0 = KMAJOR ? warp : k0 + warp, c0 = (KMAJOR ? k0 : 0) + 2 * lane;
    const uint16_t *p = s.src + r0 * s.ld + c0;
    auto at = [&](int j, int &r, int &c) {
        const int dr = 8 * (KMAJOR ? j : j & 7), dc = KMAJOR ? 0 : 64 * (j >> 3);
        r = r0 + dr;
        c = c0 + dc;
        return p + dr * s.ld + dc;
    };
    // The same for all of the warp's pieces (rows 8 apart).  One loop for each way, so that its loads are all under way at once.
    const bool words = (reinterpret_cast<uintptr_t>(p) & 3u) == 0 &&
                       (s.cols % 2 == 0 || (KMAJOR ? k0 + 64 : TILE) <= s.cols);
    int r, c;
    if (words) {
#pragma unroll
        for (int j = 0; j < kPerWarp; ++j) {
            const uint16_t *q = at(j, r, c);
            v.lo[j] = r < s.rows && c < s.cols ? __ldg(reinterpret_cast<const uint32_t *>(q)) : 0u;
            v.hi[j] = 0;
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPerWarp; ++j) {
            const uint16_t *q = at(j, r, c);
            v.lo[j] = r < s.rows && c < s.cols ? __ldg(q) : 0u;
            v.hi[j] = r < s.rows && c + 1 < s.cols ? __ldg(q + 1) : 0u;
        }
    }
}

// Pieces warp + 8j, j < count, into the tile: 128-byte rows, 16-byte columns
// swizzled by the row's number modulo 8 (which is the warp's).
__device__ __forceinline__ void store_pieces(const Pieces &v, uint32_t tile, int count, int warp, int lane)
{
    const uint32_t at = tile + (uint32_t)(warp * 128 + (((lane >> 2) ^ warp) << 4) + (lane & 3) * 4);
#pragma unroll
    for (int j = 0; j < kPerWarp; ++j)
        if (j < count) asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + j * 1024), "r"(v.lo[j] | v.hi[j] << 16) : "memory");
}

// This lane's value of one TMEM column.
__device__ __forceinline__ float tmem_value(uint32_t taddr)
{
    uint32_t v;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(taddr));
    ptx::tmem_ld_wait();
    return __uint_as_float(v);
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads, 2) grouped_unaligned_kernel(const GroupedArgs a, uint32_t *err, uint64_t wait_ns)
{
    constexpr bool WG = MODE == GROUPED_WGRAD, A_KMAJOR = MODE == GROUPED_FORWARD, B_KMAJOR = !WG;
    __shared__ Schedule sch;
    __shared__ __align__(8) uint64_t full[kStages], empty[kStages], done, drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int dead;   // a wait has timed out: no more work, but every barrier of the CTA is still met
    extern __shared__ __align__(128) uint8_t dyn[];
    uint8_t *ring = dyn + (-ptx::smem_u32(dyn) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(&full[i], kLoadWarps);
            ptx::mbar_init(&empty[i], 1);
        }
        ptx::mbar_init(&done, 1);
        ptx::mbar_init(&drain, 1);
        ptx::mbar_init_fence();
        dead = 0;
    }
    if (warp == 0) {
        ptx::tmem_alloc(&tmem_slot, TILE);
        ptx::tmem_relinquish();
    }
    pdl_begin();
    const int M = MODE == GROUPED_FORWARD ? a.N : a.K, mt = (M + TILE - 1) / TILE;
    const int nt = WG ? (a.N + TILE - 1) / TILE : 0;
    ptx::tc_fence_before();
    make_schedule(sch, a.offsets, a.groups, a.rows, TILE, mt, err);
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const int64_t tiles = sch.bad ? 0 : WG ? (int64_t)a.groups * mt * nt : sch.tile[a.groups];

    auto wait = [&](uint64_t *bar, uint32_t parity, uint32_t why) {   // the whole warp
        if (__any_sync(0xffffffffu, *(volatile int *)&dead)) return false;
        const bool ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, wait_ns));
        if (!ok && lane == 0) {
            *(volatile int *)&dead = 1;
            atomicOr(err, why);
        }
        return ok;
    };

    int stage = 0;
    uint32_t phase = 0, done_phase = 0;
    const bool issuer = elect_one();
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        // output: M side [m0, +128), N side `cols` from n0 on
        int e, m0, n0, cols, parts = 1, len = 0;
        if (WG) {
            e = (int)(t / (mt * nt));
            const int r = (int)(t - (int64_t)e * (mt * nt)), rows = sch.row[e + 1] - sch.row[e];
            m0 = r % mt * TILE;
            n0 = r / mt * TILE;
            cols = min(TILE, a.N - n0);
            parts = max(1, (rows + kMaxPartRows - 1) / kMaxPartRows);
            len = ((rows + parts - 1) / parts + BK - 1) / BK * BK;
        } else {
            e = group_of_tile(sch, a.groups, (int)t);
            const int r = (int)t - sch.tile[e];
            m0 = r % mt * TILE;
            n0 = sch.row[e] + r / mt * TILE;
            cols = min(TILE, sch.row[e + 1] - n0);
        }
        // the MMA's N; whole boxes of 64 for an N-major operand
        const int w = WG ? (cols + 63) & ~63 : (cols + 15) & ~15;
        const uint16_t *we = reinterpret_cast<const uint16_t *>(a.w) + (int64_t)e * a.N * a.K;
        for (int part = 0; part < parts; ++part) {
            Source A, B;
            int red;
            if (WG) {
                const int first = sch.row[e] + part * len;
                red = min(len, sch.row[e + 1] - first);
                A = {reinterpret_cast<const uint16_t *>(a.x) + first * a.x_stride + m0, a.x_stride, red, M - m0};
                B = {reinterpret_cast<const uint16_t *>(a.dy) + first * a.dy_stride + n0, a.dy_stride, red, cols};
            } else {
                const void *tokens = A_KMAJOR ? a.x : a.dy;
                const int64_t ld = A_KMAJOR ? a.x_stride : a.dy_stride;
                red = A_KMAJOR ? a.K : a.N;
                A = {we + (A_KMAJOR ? (int64_t)m0 * a.K : m0), a.K, A_KMAJOR ? M - m0 : red, A_KMAJOR ? red : M - m0};
                B = {reinterpret_cast<const uint16_t *>(tokens) + n0 * ld, ld, cols, red};
            }
            const int steps = (red + BK - 1) / BK;
            const int pieces = WG ? w / 8 : (w - warp + 7) / 8;
            const uint32_t id = idesc(TILE, w, a.dtype == TF_BF16, !A_KMAJOR, !B_KMAJOR);
            int mma_stage = stage;
            uint32_t mma_phase = phase;
            auto multiply = [&](int k) {   // warp 0: the K step's MMAs
                if (wait(&full[mma_stage], mma_phase, TF_DEVERR_MMA_WAIT)) {
                    ptx::tc_fence_after();
                    const uint32_t tile = ptx::smem_u32(ring + mma_stage * kStageBytes);
                    const uint32_t al = desc_low(tile, A_KMAJOR), bl = desc_low(tile + kOperandBytes, B_KMAJOR);
                    if (issuer) {
#pragma unroll
                        for (int i = 0; i < BK / UMMA_K; ++i)
                            ptx::umma_bf16(tmem, desc_of(al + i * desc_step(A_KMAJOR)), desc_of(bl + i * desc_step(B_KMAJOR)),
                                           id, k > 0 || i > 0);
                        ptx::umma_commit(&empty[mma_stage]);
                        if (k == steps - 1) ptx::umma_commit(&done);
                    }
                    __syncwarp();
                }
                if (++mma_stage == kStages) {
                    mma_stage = 0;
                    mma_phase ^= 1u;
                }
            };
            for (int k = 0; k < steps; ++k) {
                Pieces va, vb;
                load_pieces<A_KMAJOR>(va, A, k * BK, warp, lane);
                load_pieces<B_KMAJOR>(vb, B, k * BK, warp, lane);
                if (warp == 0 && k > 0) multiply(k - 1);   // (one step behind, so as not to wait for the other warps)
                if (wait(&empty[stage], phase ^ 1u, TF_DEVERR_PRODUCER_WAIT)) {
                    const uint32_t tile = ptx::smem_u32(ring + stage * kStageBytes);
                    store_pieces(va, tile, kPerWarp, warp, lane);
                    store_pieces(vb, tile + kOperandBytes, pieces, warp, lane);
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&full[stage]);
                }
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (warp == 0 && steps > 0) multiply(steps - 1);
            const bool ready = steps > 0 && wait(&done, done_phase, TF_DEVERR_EPILOGUE_WAIT);
            if (steps > 0) done_phase ^= 1u;
            const bool add = WG && (a.accumulate || part > 0);
            if (ready || (WG && steps == 0 && !add)) {
                ptx::tc_fence_after();
                // warps w and w + 4 read TMEM lanes 32*(w%4) and on, each 64 of the columns
                const int m = m0 + (warp & 3) * 32 + lane;
                const float bias = MODE == GROUPED_FORWARD && a.bias && m < M ? __ldg(a.bias + (int64_t)e * M + m) : 0.0f;
#pragma unroll 1
                for (int c = (warp >> 2) * 64; c < min(cols, (warp >> 2) * 64 + 64); c += 32) {
                    uint32_t r[32];
                    if (steps > 0) {
                        ptx::tmem_ld_32x32b_x32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)c, r);
                        ptx::tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) r[j] = 0u;
                    }
                    float least = INFINITY;   // FORWARD: of the sums
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (c + j >= cols || m >= M) continue;
                        const int64_t row = n0 + c + j;
                        float v = __uint_as_float(r[j]);
                        if constexpr (MODE == GROUPED_FORWARD) {
                            v += bias;
                            least = fminf(least, v);
                            if (a.pre) reinterpret_cast<T *>(a.pre)[row * a.pre_stride + m] = Half2Of<T>::round(v);
                            reinterpret_cast<T *>(a.y)[row * a.y_stride + m] = Half2Of<T>::round(act_value<false>(a.act, v));
                        } else if constexpr (MODE == GROUPED_DGRAD) {
                            if (a.act != TF_ACT_NONE)
                                v *= act_slope<true>(a.act, Half2Of<T>::widen(reinterpret_cast<const T *>(a.pre)[row * a.pre_stride + m]));
                            reinterpret_cast<T *>(a.y)[row * a.y_stride + m] = Half2Of<T>::round(v);
                        } else {
                            float *dst = a.dw + ((int64_t)e * a.N + row) * a.K + m;
                            *dst = add ? *dst + v : v;
                        }
                    }
                    // far_value() in place of what lies there, the sums fetched once more (a second copy of the
                    // loop above took 433 us where this takes 395)
                    if (MODE == GROUPED_FORWARD && a.act != TF_ACT_NONE && __any_sync(0xffffffffu, least < far_from(a.act))) {
#pragma unroll 1
                        for (int j = 0; j < 32; ++j) {
                            const float v = tmem_value(tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(c + j)) + bias;
                            if (c + j < cols && m < M && v < far_from(a.act))
                                reinterpret_cast<T *>(a.y)[(n0 + c + j) * a.y_stride + m] = Half2Of<T>::round(act_value<true>(a.act, v));
                        }
                    }
                }
            }
            ptx::tc_fence_before();
            cta_sync();   // the accumulator has been read
            ptx::tc_fence_after();
        }
    }
    if (warp == 0) {
        if (*(volatile int *)&dead) {   // MMAs may still be reading the ring
            if (issuer) ptx::umma_commit(&drain);
            __syncwarp();
            if (!ptx::mbar_wait(&drain, 0, wait_ns) && lane == 0) atomicOr(err, TF_DEVERR_DRAIN_WAIT);
            __syncwarp();
        }
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, TILE);
    }
}

// dbias[e][n] = sum of dy[m][n] over group e's rows.  A CTA takes 64 columns of
// one group: VEC columns per thread (8: 16-byte loads), 64/VEC threads side by
// side, the others on rows of their own, four loads each in flight, sums in
// levels; the CTA's partial sums are added in order.  Bound by HBM: dy once.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) grouped_bias_grad_kernel(const GroupedArgs a, uint32_t *err)
{
    pdl_begin();
    constexpr int ACROSS = 64 / VEC, DOWN = 256 / ACROSS;
    __shared__ float red[DOWN][65];
    __shared__ int bad;
    if (threadIdx.x == 0) bad = 0;
    cta_sync();
    for (int i = threadIdx.x; i <= a.groups; i += blockDim.x) {
        const int v = a.offsets[i];
        if (v < 0 || v > a.rows || (i > 0 && a.offsets[i - 1] > v)) bad = 1;
    }
    cta_sync();
    if (bad) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(err, TF_DEVERR_OFFSETS);
        return;
    }
    const int e = blockIdx.y, q = threadIdx.x / ACROSS, c = (int)threadIdx.x % ACROSS * VEC, n = blockIdx.x * 64 + c;
    const int lo = a.offsets[e], hi = a.offsets[e + 1];
    const T *dy = reinterpret_cast<const T *>(a.dy) + n;
    constexpr int PAIRS = (VEC + 1) / 2;   // (of a single column the second value stays zero)
    float2 sum[PAIRS] = {};
    // (N is a multiple of VEC)
    sum_rows(sum, lo + q, n < a.N ? hi : lo, 4 * DOWN, [&](int m, float2 (&rows)[PAIRS]) {
        if constexpr (VEC == 8) {
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = m + i * DOWN < hi ? __ldg(reinterpret_cast<const uint4 *>(dy + (int64_t)(m + i * DOWN) * a.dy_stride))
                                         : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    rows[j] = i == 0 ? Half2Of<T>::unpack(w[j]) : fadd2(rows[j], Half2Of<T>::unpack(w[j]));
            }
        } else {
            rows[0] = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (m + i * DOWN < hi) rows[0].x += Half2Of<T>::widen(dy[(int64_t)(m + i * DOWN) * a.dy_stride]);
        }
    });
#pragma unroll
    for (int j = 0; j < VEC; ++j) red[q][c + j] = j % 2 ? sum[j / 2].y : sum[j / 2].x;
    cta_sync();
    if (threadIdx.x < 64 && blockIdx.x * 64 + threadIdx.x < (unsigned)a.N) {
        float t = 0.0f;
        for (int i = 0; i < DOWN; ++i) t += red[i][threadIdx.x];
        float *dst = a.dbias + (int64_t)e * a.N + blockIdx.x * 64 + threadIdx.x;
        *dst = a.accumulate ? *dst + t : t;
    }
}

// The kernel's shared-memory limit and carve-out, once per device.
cudaError_t allow_smem(const void *kern, bool (&known)[64])
{
    static std::mutex mu;
    int d = 0;
    cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess || d < 0 || d >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (known[d]) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    known[d] = e == cudaSuccess;
    return e;
}

template <typename T, int MODE>
cudaError_t launch_typed(const GroupedArgs &a, uint32_t *err, cudaStream_t st)
{
    static bool known[64];
    auto kern = grouped_unaligned_kernel<T, MODE>;
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), known);
    if (e != cudaSuccess) return e;
    const int64_t mt = ((MODE == GROUPED_FORWARD ? a.N : a.K) + TILE - 1) / TILE;
    const int64_t most = MODE == GROUPED_WGRAD ? (int64_t)a.groups * ((a.N + TILE - 1) / TILE) * mt
                                               : ((int64_t)a.rows / TILE + a.groups) * mt;
    const unsigned grid = (unsigned)(most < (int64_t)sm_count() * 2 ? most : (int64_t)sm_count() * 2);
    return launch_pdl(kern, dim3(grid), dim3(kThreads), kSmemBytes, st, a, err, wait_limit_ns());
}

}  // namespace

cudaError_t launch_grouped_unaligned(const GroupedArgs &a, int mode, cudaStream_t st)
{
    uint32_t *err = device_error_word();
    if (!err) return cudaErrorInitializationError;
    auto launch = [&](auto value) {
        using T = decltype(value);
        return mode == GROUPED_FORWARD ? launch_typed<T, GROUPED_FORWARD>(a, err, st)
               : mode == GROUPED_DGRAD ? launch_typed<T, GROUPED_DGRAD>(a, err, st)
                                       : launch_typed<T, GROUPED_WGRAD>(a, err, st);
    };
    return a.dtype == TF_BF16 ? launch(__nv_bfloat16()) : launch(__half());
}

cudaError_t launch_grouped_bias_grad(const GroupedArgs &a, cudaStream_t st)
{
    uint32_t *err = device_error_word();
    if (!err) return cudaErrorInitializationError;
    const dim3 grid((unsigned)((a.N + 63) / 64), (unsigned)a.groups);
    const bool vec = a.N % 8 == 0 && a.dy_stride % 8 == 0 && (reinterpret_cast<uintptr_t>(a.dy) & 15u) == 0;
    auto launch = [&](auto kern) { return launch_pdl(kern, grid, dim3(256), 0, st, a, err); };
    if (a.dtype == TF_BF16)
        return vec ? launch(grouped_bias_grad_kernel<__nv_bfloat16, 8>) : launch(grouped_bias_grad_kernel<__nv_bfloat16, 1>);
    return vec ? launch(grouped_bias_grad_kernel<__half, 8>) : launch(grouped_bias_grad_kernel<__half, 1>);
}

}  // namespace tf
