// Shared by the grouped-product kernels (rows sorted by group, every group
// with its own weights): the activation epilogues and their derivatives, the
// 16-bit storage types, and the tile schedule computed on the device from the
// row offsets, so that a call needs no copy of the offsets to the host.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

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
// gelu_f32 (relative error below 1e-5 on [0, 6], below 2^-29 in value beyond).
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

// The pre-activation is an fp32 sum of any size (it need not be a finite
// fp16), so both arguments are clamped where the function has reached its
// limit: |z| at 12 in GELU(z) = max(z, 0) - |z| Q(|z|), z at -100 in SiLU,
// which gives the limits at the infinities.  NaN stays NaN (min.NaN, max.NaN).
__device__ __forceinline__ float act_value(int act, float z)
{
    if (act == TF_ACT_SILU) {
        const float v = max_nan(z, -100.0f);
        return v * rcp_approx(1.0f + ex2_approx(-kLog2e * v));
    }
    if (act == TF_ACT_GELU) {
        const float t = min_nan(fabsf(z), TF_GELU_TCLAMP);
        return fmaf(-t, normal_tail(t), max_nan(z, 0.0f));
    }
    return z;
}

// d act/dz.  SiLU: s + z s (1 - s), s = sigmoid(z).  GELU: Phi(z) + z phi(z),
// that is h = Q(t) - t phi(t) for z < 0 and 1 - h for z >= 0, t = |z|.
__device__ __forceinline__ float act_slope(int act, float z)
{
    if (act == TF_ACT_SILU) {
        const float v = min_nan(max_nan(z, -100.0f), 100.0f);
        const float s = rcp_approx(1.0f + ex2_approx(-kLog2e * v));
        return fmaf(v * s, 1.0f - s, s);
    }
    if (act == TF_ACT_GELU) {
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

template <int ACT>
__device__ __forceinline__ float2 act_value2(float2 z)
{
    if constexpr (ACT == TF_ACT_SILU) {
        const float2 v = make_float2(max_nan(z.x, -100.0f), max_nan(z.y, -100.0f));
        return silu_f32x2(v);
    } else if constexpr (ACT == TF_ACT_GELU) {
        const float2 t = make_float2(min_nan(fabsf(z.x), TF_GELU_TCLAMP), min_nan(fabsf(z.y), TF_GELU_TCLAMP));
        const float2 r = make_float2(max_nan(z.x, 0.0f), max_nan(z.y, 0.0f));
        return ffma2(make_float2(-t.x, -t.y), normal_tail2(t), r);
    } else {
        return z;
    }
}

template <int ACT>
__device__ __forceinline__ float2 act_slope2(float2 z)
{
    if constexpr (ACT == TF_ACT_SILU) {
        return make_float2(act_slope(TF_ACT_SILU, z.x), act_slope(TF_ACT_SILU, z.y));
    } else if constexpr (ACT == TF_ACT_GELU) {
        const float2 t = make_float2(min_nan(fabsf(z.x), TF_GELU_TCLAMP), min_nan(fabsf(z.y), TF_GELU_TCLAMP));
        const float2 u = fmul2(fmul2(t, t), dup2(-0.5f * kLog2e));
        const float2 phi = make_float2(-0.3989422804f * ex2_approx(u.x), -0.3989422804f * ex2_approx(u.y));
        const float2 h = ffma2(t, phi, normal_tail2(t));
        return make_float2(z.x >= 0.0f ? 1.0f - h.x : h.x, z.y >= 0.0f ? 1.0f - h.y : h.y);
    } else {
        return dup2(1.0f);
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

}  // namespace grouped
}  // namespace tf
