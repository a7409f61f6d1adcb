// Shared by the grouped-product kernels (rows sorted by group, every group
// with its own weights): the activation epilogues and their derivatives, the
// 16-bit storage types, and the tile schedule computed on the device from the
// row offsets, so that a call needs no copy of the offsets to the host.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx_sm100.cuh"
#include "train_internal.h"

namespace tf {
namespace grouped {

constexpr int kMaxGroups = (int)kGroupedMaxGroups;

// ---------------------------------------------------------------- 16-bit storage

template <typename T>
struct Half2Of;
template <>
struct Half2Of<__half> {
    __device__ static uint32_t pack(float a, float b)
    {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    __device__ static float2 unpack(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2 *>(&u)); }
    __device__ static uint32_t min2(uint32_t a, uint32_t b)
    {
        const __half2 h = __hmin2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    __device__ static __half round(float a) { return __float2half_rn(a); }
    __device__ static float widen(__half a) { return __half2float(a); }
};
template <>
struct Half2Of<__nv_bfloat16> {
    __device__ static uint32_t pack(float a, float b)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    __device__ static float2 unpack(uint32_t u)
    {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    __device__ static uint32_t min2(uint32_t a, uint32_t b)
    {
        const __nv_bfloat162 h = __hmin2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    __device__ static __nv_bfloat16 round(float a) { return __float2bfloat16_rn(a); }
    __device__ static float widen(__nv_bfloat16 a) { return __bfloat162float(a); }
};

// ---------------------------------------------------------------- activations

__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Q(t), the upper tail of the standard normal at t in [0, 12]: the fit of
// gelu_f32 (relative error below 1e-5 on [0, 6], below 2^-29 in value beyond:
// nothing beside 1, but see far_value()).
__device__ __forceinline__ float normal_tail(float t)
{
    const float v = fmaf(t, 1.0f / (TF_GELU_TMAX * 0.5f), -1.0f);
    float acc = TF_GELU_C7;
    acc = fmaf(acc, v, TF_GELU_C6);
    acc = fmaf(acc, v, TF_GELU_C5);
    acc = fmaf(acc, v, TF_GELU_C4);
    acc = fmaf(acc, v, TF_GELU_C3);
    acc = fmaf(acc, v, TF_GELU_C2);
    acc = fmaf(acc, v, TF_GELU_C1);
    acc = fmaf(acc, v, TF_GELU_C0);
    return ex2_approx(acc);
}

// Activation and slope far below zero, where they are numbers that only the
// exponents of bf16 hold: GELU below -6 by the scale of the tail's asymptotic
// series (gen_gelu_poly.py), SiLU below -80 as z e^z and (1 + z) e^z.  The
// exponentials are taken 2^32 too high, since ex2 flushes what an fp32 product
// still holds.  Relative error below 1e-4 down to the smallest bf16; at the
// clamps all is zero.  Such values are rare, so the epilogues look at the least
// of 32 values and leave these branches out where FAR is false (tested value by
// value they took 21.8 us instead of 17.5 for 4096 rows of 2048 x 512 with GELU).
constexpr float kFarScale = 32.0f, kFarUnscale = 1.0f / 4294967296.0f;
__host__ __device__ constexpr float far_from(int act) { return act == TF_ACT_GELU ? -TF_GELU_TMAX : -80.0f; }

// t*Q(t) = tail_scale(t, s) * s * kFarUnscale
__device__ __forceinline__ float tail_scale(float t, float &s, float &u)
{
    const float t2 = t * t;
    u = rcp_approx(t2);
    s = fmaf(fmaf(TF_GELU_FAR2, u, TF_GELU_FAR1), u, TF_GELU_FAR0);
    return ex2_approx(fmaf(t2, -0.5f * kLog2e, kFarScale - 1.3257480647f));   // log2 sqrt(2 pi)
}

template <int ACT>
__device__ __forceinline__ float far_value(float z)
{
    if constexpr (ACT == TF_ACT_GELU) {
        float s, u;
        const float e = tail_scale(fminf(-z, TF_GELU_TFAR), s, u);
        return -(e * s) * kFarUnscale;
    } else {
        const float v = fmaxf(z, -200.0f);
        return v * ex2_approx(fmaf(v, kLog2e, kFarScale)) * kFarUnscale;
    }
}

template <int ACT>
__device__ __forceinline__ float far_slope(float z)
{
    if constexpr (ACT == TF_ACT_GELU) {
        float s, u;
        const float t = fminf(-z, TF_GELU_TFAR), e = tail_scale(t, s, u);
        return e * t * fmaf(s, u, -1.0f) * kFarUnscale;
    } else {
        const float v = fmaxf(z, -200.0f);
        return (1.0f + v) * ex2_approx(fmaf(v, kLog2e, kFarScale)) * kFarUnscale;
    }
}

// The pre-activation is an fp32 sum of any size (it need not be a finite
// fp16), so the arguments are clamped where the function has reached its
// limit, which gives the limits at the infinities: |z| at 12 in
// GELU(z) = max(z, 0) - |z| Q(|z|), z at 100 in SiLU's slope, and those of
// far_value().  NaN stays NaN (min.NaN, max.NaN).
template <bool FAR>
__device__ __forceinline__ float act_value(int act, float z)
{
    if (act == TF_ACT_SILU) {
        if (FAR && z < far_from(TF_ACT_SILU)) return far_value<TF_ACT_SILU>(z);
        return silu_f32(z);
    }
    if (act == TF_ACT_GELU) {
        if (FAR && z < far_from(TF_ACT_GELU)) return far_value<TF_ACT_GELU>(z);
        const float t = min_nan(fabsf(z), TF_GELU_TCLAMP);
        return fmaf(-t, normal_tail(t), max_nan(z, 0.0f));
    }
    return z;
}

// d act/dz.  SiLU: s + z s (1 - s), s = sigmoid(z).  GELU: Phi(z) + z phi(z),
// that is h = Q(t) - t phi(t) for z < 0 and 1 - h for z >= 0, t = |z|.
template <bool FAR>
__device__ __forceinline__ float act_slope(int act, float z)
{
    if (act == TF_ACT_SILU) {
        if (FAR && z < far_from(TF_ACT_SILU)) return far_slope<TF_ACT_SILU>(z);
        const float v = min_nan(z, 100.0f);
        const float s = rcp_approx(1.0f + ex2_approx(-kLog2e * v));
        return fmaf(v * s, 1.0f - s, s);
    }
    if (act == TF_ACT_GELU) {
        if (FAR && z < far_from(TF_ACT_GELU)) return far_slope<TF_ACT_GELU>(z);
        const float t = min_nan(fabsf(z), TF_GELU_TCLAMP);
        const float phi = 0.3989422804f * ex2_approx(-0.5f * kLog2e * t * t);
        const float h = fmaf(-t, phi, normal_tail(t));
        return z >= 0.0f ? 1.0f - h : h;
    }
    return 1.0f;
}

// The same on pairs (packed fp32), with the activation a constant.
__device__ __forceinline__ float2 dup2(float a) { return make_float2(a, a); }

__device__ __forceinline__ float2 normal_tail2(float2 t)
{
    const float2 v = ffma2(t, dup2(1.0f / (TF_GELU_TMAX * 0.5f)), dup2(-1.0f));
    float2 acc = ffma2(dup2(TF_GELU_C7), v, dup2(TF_GELU_C6));
    acc = ffma2(acc, v, dup2(TF_GELU_C5));
    acc = ffma2(acc, v, dup2(TF_GELU_C4));
    acc = ffma2(acc, v, dup2(TF_GELU_C3));
    acc = ffma2(acc, v, dup2(TF_GELU_C2));
    acc = ffma2(acc, v, dup2(TF_GELU_C1));
    acc = ffma2(acc, v, dup2(TF_GELU_C0));
    return make_float2(ex2_approx(acc.x), ex2_approx(acc.y));
}

// f2 of a pair, with f1 in place of the values far below zero
template <int ACT, bool FAR, typename F1>
__device__ __forceinline__ float2 with_far(float2 z, float2 f2, F1 f1)
{
    if (FAR && z.x < far_from(ACT)) f2.x = f1(z.x);
    if (FAR && z.y < far_from(ACT)) f2.y = f1(z.y);
    return f2;
}

template <int ACT, bool FAR>
__device__ __forceinline__ float2 act_value2(float2 z)
{
    auto far = [](float v) { return far_value<ACT>(v); };
    if constexpr (ACT == TF_ACT_SILU) {
        return with_far<ACT, FAR>(z, silu_f32x2(z), far);
    } else if constexpr (ACT == TF_ACT_GELU) {
        const float2 t = make_float2(min_nan(fabsf(z.x), TF_GELU_TCLAMP), min_nan(fabsf(z.y), TF_GELU_TCLAMP));
        const float2 r = make_float2(max_nan(z.x, 0.0f), max_nan(z.y, 0.0f));
        return with_far<ACT, FAR>(z, ffma2(make_float2(-t.x, -t.y), normal_tail2(t), r), far);
    } else {
        return z;
    }
}

template <int ACT, bool FAR>
__device__ __forceinline__ float2 act_slope2(float2 z)
{
    if constexpr (ACT == TF_ACT_SILU) {
        return make_float2(act_slope<FAR>(TF_ACT_SILU, z.x), act_slope<FAR>(TF_ACT_SILU, z.y));
    } else if constexpr (ACT == TF_ACT_GELU) {
        const float2 t = make_float2(min_nan(fabsf(z.x), TF_GELU_TCLAMP), min_nan(fabsf(z.y), TF_GELU_TCLAMP));
        const float2 u = fmul2(fmul2(t, t), dup2(-0.5f * kLog2e));
        const float2 phi = make_float2(-0.3989422804f * ex2_approx(u.x), -0.3989422804f * ex2_approx(u.y));
        const float2 h = ffma2(t, phi, normal_tail2(t));
        const float2 f = make_float2(z.x >= 0.0f ? 1.0f - h.x : h.x, z.y >= 0.0f ? 1.0f - h.y : h.y);
        return with_far<ACT, FAR>(z, f, [](float v) { return far_slope<ACT>(v); });
    } else {
        return dup2(1.0f);
    }
}

// ---------------------------------------------------------------- column sums

// total += the sum over rows first, first + step, ... < end, where at(m, sum)
// sets `sum` to one step's rows' sum.  In three levels, of 64 steps, of 64 such sums
// and of those: in one level a long group's running sum outgrows its terms, and
// equal ones lose 2e-3 over 2^20 rows (1e-2 over 2^22).
template <int N, typename F>
__device__ __forceinline__ void sum_rows(float2 (&total)[N], int first, int end, int step, F at)
{
    constexpr int FAN = 64;
    auto into = [](float2 (&dst)[N], const float2 (&src)[N]) {
#pragma unroll
        for (int k = 0; k < N; ++k) dst[k] = fadd2(dst[k], src[k]);
    };
    for (int m = first; m < end;) {
        float2 mid[N] = {};
        for (int j = 0; j < FAN && m < end; ++j) {
            float2 low[N] = {};
            for (int i = 0; i < FAN && m < end; ++i, m += step) {
                float2 sum[N];
                at(m, sum);
                into(low, sum);
            }
            into(mid, low);
        }
        into(total, mid);
    }
}

// ---------------------------------------------------------------- tile schedule

// The groups' rows and the running count of their tiles, in shared memory.
// row[e] .. row[e+1] are group e's rows; tile[e] is the number of tiles before
// group e, each group taking ceil(rows/tile_rows) * col_tiles of them.
struct Schedule {
    int row[kMaxGroups + 1];
    int tile[kMaxGroups + 1];
    int bad;
};

// Fills the schedule with all threads of the CTA.  Offsets that fall, or that
// lie outside [0, rows], make the whole call do nothing: every CTA sees the
// same offsets and schedules no tile, and the error word says why.
__device__ __forceinline__ void make_schedule(Schedule &s, const int *__restrict__ offsets, int groups, int rows,
                                              int tile_rows, int col_tiles, uint32_t *err)
{
    if (threadIdx.x == 0) s.bad = 0;
    cta_sync();
    int wrong = 0;
    for (int i = threadIdx.x; i <= groups; i += blockDim.x) {
        const int v = offsets[i];
        s.row[i] = v;
        wrong |= v < 0 || v > rows || (i > 0 && offsets[i - 1] > v);
    }
    if (wrong) s.bad = 1;
    cta_sync();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int before = 0;
        for (int base = 0; base < groups; base += 32) {
            const int e = base + lane;
            int n = 0;
            if (e < groups && !s.bad) n = (s.row[e + 1] - s.row[e] + tile_rows - 1) / tile_rows * col_tiles;
            int sum = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += up;
            }
            if (e < groups) s.tile[e] = before + sum - n;
            before += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (lane == 0) {
            s.tile[groups] = before;
            if (s.bad && blockIdx.x == 0) atomicOr(err, TF_DEVERR_OFFSETS);
        }
    }
    cta_sync();
}

// The group that tile `t` < s.tile[groups] belongs to.
__device__ __forceinline__ int group_of_tile(const Schedule &s, int groups, int t)
{
    int lo = 0, hi = groups - 1;   // the last e with tile[e] <= t has rows: an empty group's successor starts at the same tile
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s.tile[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// ---------------------------------------------------------------- tensor-core operands

constexpr int BK = 64;                      // K step: one 128-byte swizzle row of 16-bit values
constexpr int UMMA_K = 16;
constexpr int kChunkBytes = 64 * BK * 2;    // one 64 x 64 box of an M- or N-major operand

// Shared-memory matrix descriptors (128-byte swizzle), as a low word that holds
// the address and a high word that does not change: advancing along K inside a
// tile, or to another stage, is one 32-bit addition.
//   K-major: rows of 64 values (128 bytes), eight of them an atom of 1024 bytes,
//     atoms stacked densely; 16 values along K are 32 bytes.
//   M- or N-major: boxes of 64 (M or N) x 64 (K) values, each a K row of 128
//     bytes; eight K rows are an atom (stride byte offset 1024), the next 64 M or
//     N values are a box further on (leading byte offset); 16 along K are 2048 bytes.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);   // stride offset, version 1, 128-byte swizzle

__device__ __forceinline__ uint32_t desc_low(uint32_t smem_addr, bool kmajor)
{
    return ((smem_addr & 0x3FFFFu) >> 4) | ((kmajor ? 1u : (uint32_t)(kChunkBytes >> 4)) << 16);
}
constexpr uint32_t desc_step(bool kmajor) { return (kmajor ? UMMA_K * 2 : UMMA_K * 128) >> 4; }

__device__ __forceinline__ uint64_t desc_of(uint32_t low)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(low), "r"(kDescHigh));
    return d;
}

// kind::f16 with fp32 accumulators; operands K-major unless said otherwise.
__device__ __forceinline__ uint32_t idesc(int m, int n, bool bf16, bool a_mmajor, bool b_nmajor)
{
    const uint32_t fmt = bf16 ? 1u : 0u;
    return (1u << 4) | (fmt << 7) | (fmt << 10) | ((a_mmajor ? 1u : 0u) << 15) | ((b_nmajor ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// One lane of the (converged) warp.  The roles that issue copies and MMAs run
// their loops with the whole warp and let one lane issue: in code that a single
// lane runs the compiler cannot keep what these instructions take in uniform
// registers, and a K step then takes its issuer ~600 cycles (the tensor cores
// 512 for the widest tile): 212 us against 189 for 16384 rows of 4096 x 2048.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

}  // namespace grouped
}  // namespace tf
