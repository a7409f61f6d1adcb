// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   forward   y[i] = scale * table[token[i]]
//   backward  dtable[v] (+)= scale * sum over i with token[i] = v of dy[i]
//
// Both are bound by HBM.  The backward pass brings equal tokens together, so
// that every row of dtable is written once and in a fixed order of additions,
// which atomics would not give:
//   1  the keys (token, position) are sorted in chunks of 2048 in shared memory
//   2  32 sorted runs at a time become one: a key's place is the sum of its
//      places in all of them, found by binary search (keys are unique)
//   3  the sorted list is cut into pieces of equal length, whatever the words'
//      frequencies; a thread adds its columns of a piece's rows of dy and writes
//      a row of dtable where the word changes.  Words that cross a piece's ends
//      leave partial sums.  Other CTAs write the zeros of words that do not occur.
//   4  the partial sums of crossing words are added in order
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "lm_internal.h"

namespace tf {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float widen(T v);
template <>
__device__ __forceinline__ float widen(float v) { return v; }
template <>
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow(float v) { return v; }
template <>
__device__ __forceinline__ __half narrow(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow(float v) { return __float2bfloat16_rn(v); }

// VEC neighbouring values, loaded and stored as one word of up to 16 bytes.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
};

bool aligned_to(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// ---------------------------------------------------------------- forward

// A warp takes 32/lanes rows of `lanes` lanes each, UNROLL words per lane: enough
// loads under way to fill the memory's latency.
template <typename T, int VEC, int UNROLL>
__global__ void __launch_bounds__(kThreads) embed_kernel(const __grid_constant__ EmbedArgs a, int lanes, int chunks)
{
    pdl_begin();
    using P = Pack<T, VEC>;
    const int lane = threadIdx.x & 31, words = a.hidden / VEC;
    const int64_t warp = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t group = warp / chunks;
    const int c0 = (int)(warp - group * chunks) * lanes * UNROLL + lane % lanes;
    const int64_t i = group * (32 / lanes) + lane / lanes;
    if (i >= a.rows) return;
    const int64_t token = a.tokens.at(i);
    const bool inside = token >= 0 && token < a.vocab, none = token == a.padding;
    const bool reads = inside && !none;
    if (!inside && !none && c0 == 0) atomicOr(a.err, TF_DEVERR_INDEX);
    const P *src = reinterpret_cast<const P *>(static_cast<const T *>(a.table) + (reads ? token : 0) * a.hidden);
    P *dst = reinterpret_cast<P *>(static_cast<T *>(a.y) + i * a.y_stride);
    P v[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int c = c0 + u * lanes;
        if (reads && c < words) v[u] = src[c];
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int c = c0 + u * lanes;
        if (c >= words) break;
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[u].v[k] = narrow<T>(reads ? widen<T>(v[u].v[k]) * a.scale : 0.0f);
        dst[c] = v[u];
    }
}

template <typename T, int VEC>
cudaError_t launch_embed(const EmbedArgs &a, cudaStream_t st)
{
    constexpr int UNROLL = VEC == 1 ? 8 : 4;
    const int words = a.hidden / VEC;
    int lanes = 1;
    while (lanes < 32 && lanes < words) lanes *= 2;
    const int chunks = (words + lanes * UNROLL - 1) / (lanes * UNROLL);
    const int64_t groups = (a.rows + 32 / lanes - 1) / (32 / lanes);
    const int64_t blocks = (groups * chunks + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks >= (int64_t)1 << 31) return cudaErrorNotSupported;
    return launch_pdl(embed_kernel<T, VEC, UNROLL>, dim3((unsigned)blocks), dim3(kThreads), 0, st, a, lanes, chunks);
}

template <typename T>
cudaError_t embed_typed(const EmbedArgs &a, cudaStream_t st)
{
    auto fits = [&](int vec) {
        return a.hidden % vec == 0 && a.y_stride % vec == 0 && aligned_to(a.table, vec * sizeof(T)) &&
               aligned_to(a.y, vec * sizeof(T));
    };
    constexpr int FULL = 16 / (int)sizeof(T);
    if (fits(FULL)) return launch_embed<T, FULL>(a, st);
    if constexpr (sizeof(T) == 2)
        if (fits(2)) return launch_embed<T, 2>(a, st);
    return launch_embed<T, 1>(a, st);
}

// ---------------------------------------------------------------- backward: order

// A key holds the token in its upper and the row of dy in its lower half; tokens
// that have no gradient come last.
constexpr uint32_t kNone = 0xffffffffu;
constexpr int kSortThreads = 1024, kChunk = 2 * kSortThreads, kFanIn = 32;

__device__ __forceinline__ uint32_t word_of(uint64_t key) { return (uint32_t)(key >> 32); }

// Bitonic sort of a chunk in shared memory: a warp owns 64 neighbouring keys, so
// that steps of up to 32 need no barrier of the CTA.
__global__ void __launch_bounds__(kSortThreads) sort_chunks_kernel(const __grid_constant__ EmbedArgs a, uint64_t *out)
{
    pdl_begin();
    __shared__ uint64_t s[kChunk];
    const int64_t first = (int64_t)blockIdx.x * kChunk;
    const int n = (int)min((int64_t)kChunk, a.rows - first), t = threadIdx.x;
    int span = 64;
    while (span < n) span *= 2;
    for (int i = t; i < span; i += kSortThreads) {
        uint64_t key = ~0ull;
        if (i < n) {
            const int64_t token = a.tokens.at(first + i);
            const bool inside = token >= 0 && token < a.vocab, none = token == a.padding;
            if (!inside && !none) atomicOr(a.err, TF_DEVERR_INDEX);
            key = (uint64_t)(inside && !none ? (uint32_t)token : kNone) << 32 | (uint32_t)(first + i);
        }
        s[i] = key;
    }
    __syncthreads();
    for (int k = 2; k <= span; k *= 2) {
        for (int j = k / 2; j > 0; j /= 2) {
            if (t < span / 2) {
                const int i = 2 * t - (t & (j - 1));
                const uint64_t x = s[i], y = s[i + j];
                if ((x > y) == ((i & k) == 0)) {
                    s[i] = y;
                    s[i + j] = x;
                }
            }
            if (j > 32 || (j == 1 && k >= 64)) __syncthreads();
            else __syncwarp();
        }
    }
    for (int i = t; i < n; i += kSortThreads) out[first + i] = s[i];
}

// Keys of run [lo, hi) below `key`.
__device__ __forceinline__ int64_t below(const uint64_t *keys, int64_t lo, int64_t hi, uint64_t key)
{
    const int64_t start = lo;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (__ldg(keys + mid) < key) lo = mid + 1; else hi = mid;
    }
    return lo - start;
}

// Groups of up to kFanIn sorted runs of `len` keys become one run each.  Four
// searches at a time, whose loads do not wait for one another; neighbouring
// threads' keys take nearly the same path.
__global__ void __launch_bounds__(kThreads) merge_runs_kernel(const uint64_t *in, uint64_t *out, int64_t n, int64_t len)
{
    pdl_begin();
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    const uint64_t key = in[i];
    const int64_t run = i / len, group = run / kFanIn * kFanIn, base = group * len;
    int64_t place = i - run * len;
    for (int64_t r = group; r < group + kFanIn && r * len < n; r += 4) {
        int64_t lo[4], hi[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            lo[u] = min((r + u) * len, n);
            hi[u] = r + u < group + kFanIn && r + u != run ? min((r + u + 1) * len, n) : lo[u];
            place -= lo[u];
        }
        bool more = true;
        while (more) {
            uint64_t v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = lo[u] < hi[u] ? __ldg(in + ((lo[u] + hi[u]) >> 1)) : 0;
            more = false;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (lo[u] >= hi[u]) continue;
                const int64_t mid = (lo[u] + hi[u]) >> 1;
                if (v[u] < key) lo[u] = mid + 1; else hi[u] = mid;
                more |= lo[u] < hi[u];
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) place += lo[u];
    }
    out[base + place] = key;
}

// ---------------------------------------------------------------- backward: sums

constexpr int kSumThreads = 128;
constexpr int kFillRows = 64;      // rows of dtable per zeroing CTA
constexpr int kMinPiece = 32, kMaxPiece = 1024;
constexpr int kLevel = 64;         // rows added before their sum joins the piece's: long sums of equal terms keep their digits

struct SumArgs {
    const uint64_t *keys;
    const void *dy;
    float *dtable, *part;          // part: [pieces][2][pitch], of the words that go on before and behind the piece
    int64_t dy_stride, n, vocab, pitch;
    int hidden, accumulate, piece, pieces, lanes, sum_blocks;
    float scale;
};

template <int VEC>
__device__ __forceinline__ void put_row(float *dst, const float (&sum)[VEC], float scale, bool add)
{
    if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int k = 0; k < VEC; k += 4) {
            float4 v = make_float4(sum[k] * scale, sum[k + 1] * scale, sum[k + 2] * scale, sum[k + 3] * scale);
            float4 *p = reinterpret_cast<float4 *>(dst + k);
            if (add) {
                const float4 o = *p;
                v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
            }
            *p = v;
        }
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) dst[k] = add ? dst[k] + sum[k] * scale : sum[k] * scale;
    }
}

// The rows of dtable [v0, v0 + kFillRows) whose words do not occur become zero.
__device__ __forceinline__ void fill_zeros(const SumArgs &a, int64_t v0)
{
    __shared__ uint32_t seen[kFillRows];
    const int64_t v1 = min(v0 + kFillRows, a.vocab);
    if (threadIdx.x < kFillRows) {
        const uint64_t from = (uint64_t)(v0 + threadIdx.x) << 32;
        const int64_t at = below(a.keys, 0, a.n, from);
        seen[threadIdx.x] = at < a.n && word_of(__ldg(a.keys + at)) == (uint32_t)(v0 + threadIdx.x);
    }
    __syncthreads();
    const bool whole = a.hidden % 4 == 0 && (reinterpret_cast<uintptr_t>(a.dtable) & 15u) == 0;
    for (int64_t v = v0 + (threadIdx.x >> 5); v < v1; v += kSumThreads / 32) {
        if (seen[v - v0]) continue;
        float *row = a.dtable + v * a.hidden;
        if (whole)
            for (int c = threadIdx.x & 31; c < a.hidden / 4; c += 32)
                reinterpret_cast<float4 *>(row)[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        else
            for (int c = threadIdx.x & 31; c < a.hidden; c += 32) row[c] = 0.0f;
    }
}

// `lanes` threads per piece, each with VEC neighbouring columns of a slice of
// lanes*VEC; the CTA's other threads take further pieces.
template <typename T, int VEC>
__global__ void __launch_bounds__(kSumThreads) sum_pieces_kernel(const __grid_constant__ SumArgs a)
{
    pdl_begin();
    if ((int)blockIdx.x >= a.sum_blocks) {
        if (blockIdx.y == 0) fill_zeros(a, (int64_t)((int)blockIdx.x - a.sum_blocks) * kFillRows);
        return;
    }
    constexpr int UNROLL = 8;
    using P = Pack<T, VEC>;
    const int p = (int)blockIdx.x * (kSumThreads / a.lanes) + (int)threadIdx.x / a.lanes;
    const int c = ((int)blockIdx.y * a.lanes + (int)threadIdx.x % a.lanes) * VEC;
    if (p >= a.pieces || c >= a.hidden) return;
    const int64_t first = (int64_t)p * a.piece, end = min(first + a.piece, a.n);
    const T *dy = static_cast<const T *>(a.dy) + c;
    float sum[VEC] = {}, low[VEC] = {};
    int held = 0;
    uint32_t word = word_of(__ldg(a.keys + first));
    bool head = first > 0 && word_of(__ldg(a.keys + first - 1)) == word;   // the word goes on from the piece before
    auto flush = [&](bool goes_on) {
        if (word != kNone) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) sum[k] += low[k];
            if (head || goes_on)
                put_row<VEC>(a.part + ((int64_t)p * 2 + (head ? 0 : 1)) * a.pitch + c, sum, 1.0f, false);
            else
                put_row<VEC>(a.dtable + (int64_t)word * a.hidden + c, sum, a.scale, a.accumulate != 0);
        }
#pragma unroll
        for (int k = 0; k < VEC; ++k) sum[k] = low[k] = 0.0f;
        held = 0;
        head = false;
    };
    for (int64_t i = first; i < end; i += UNROLL) {
        uint64_t key[UNROLL];
        P v[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) key[u] = i + u < end ? __ldg(a.keys + i + u) : ~0ull;
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
            if (word_of(key[u]) != kNone) v[u] = *reinterpret_cast<const P *>(dy + (int64_t)(uint32_t)key[u] * a.dy_stride);
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            if (i + u >= end) break;
            if (word_of(key[u]) != word) {
                flush(false);
                word = word_of(key[u]);
            }
            if (word == kNone) continue;
#pragma unroll
            for (int k = 0; k < VEC; ++k) low[k] += widen<T>(v[u].v[k]);
            if (++held == kLevel) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    sum[k] += low[k];
                    low[k] = 0.0f;
                }
                held = 0;
            }
        }
    }
    flush(end < a.n && word_of(__ldg(a.keys + end)) == word);
}

constexpr int kJoinCols = 32, kJoinSplits = 8, kJoinPieces = 4;

// Words that cross the ends of pieces: the CTA of the piece where the word
// begins adds its partial sums, in kJoinSplits stretches that are joined in order.
__global__ void __launch_bounds__(kJoinCols * kJoinSplits) join_pieces_kernel(const __grid_constant__ SumArgs a)
{
    pdl_begin();
    __shared__ float4 red[kJoinSplits][kJoinCols];
    const int col = threadIdx.x % kJoinCols, split = threadIdx.x / kJoinCols;
    const int c = ((int)blockIdx.y * kJoinCols + col) * 4;
    for (int p = (int)blockIdx.x * kJoinPieces; p < min(((int)blockIdx.x + 1) * kJoinPieces, a.pieces - 1); ++p) {
        const int64_t first = (int64_t)p * a.piece, end = first + a.piece;   // (the next piece exists)
        const uint32_t word = word_of(__ldg(a.keys + end - 1));
        if (word == kNone || word_of(__ldg(a.keys + end)) != word) continue;
        if (p > 0 && word_of(__ldg(a.keys + first)) == word && word_of(__ldg(a.keys + first - 1)) == word) continue;
        const int64_t last = below(a.keys, 0, a.n, ((uint64_t)word + 1) << 32) - 1;   // its last key
        const int64_t count = last / a.piece - p + 1, per = (count + kJoinSplits - 1) / kJoinSplits;
        float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (c < a.hidden) {
            const float *src = a.part + c;
#pragma unroll 4
            for (int64_t q = split * per; q < min((split + 1) * per, count); ++q) {
                const float4 v = *reinterpret_cast<const float4 *>(src + ((p + q) * 2 + (q == 0 ? 1 : 0)) * a.pitch);
                t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
            }
        }
        red[split][col] = t;
        __syncthreads();
        if (split == 0 && c < a.hidden) {
            for (int s = 1; s < kJoinSplits; ++s) {
                const float4 v = red[s][col];
                t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
            }
            const float sum[4] = {t.x, t.y, t.z, t.w};
            float *dst = a.dtable + (int64_t)word * a.hidden + c;
            for (int k = 0; k < min(4, a.hidden - c); ++k)
                dst[k] = a.accumulate ? dst[k] + sum[k] * a.scale : sum[k] * a.scale;
        }
        __syncthreads();
    }
}

// Threads per piece and slices of a row, for VEC columns per thread.
int lanes_of(int words)
{
    int lanes = 1;
    while (lanes < kSumThreads && lanes < words) lanes *= 2;
    return lanes;
}

// Pieces that fill the SMs (32 CTAs each) where the list is long enough, of 32
// to 1024 keys.  Sized for 8 columns per thread, whatever the type, so that the
// workspace depends on the sizes alone.
int64_t piece_target(int64_t hidden)
{
    const int lanes = lanes_of((int)((hidden + 7) / 8));
    const int64_t slices = (hidden + 8 * lanes - 1) / (8 * lanes), per_block = kSumThreads / lanes;
    return (32 * 152 + slices - 1) / slices * per_block;
}
int64_t piece_of(int64_t rows, int64_t hidden)
{
    const int64_t most = piece_target(hidden), len = (rows + most - 1) / most;
    return len < kMinPiece ? kMinPiece : len > kMaxPiece ? kMaxPiece : len;
}
// (does not fall as rows grow)
int64_t most_pieces(int64_t rows, int64_t hidden)
{
    const int64_t most = piece_target(hidden), shortest = (rows + kMinPiece - 1) / kMinPiece,
                  longest = (rows + kMaxPiece - 1) / kMaxPiece;
    return shortest < most ? shortest : longest > most ? longest : most;
}
int64_t pitch_of(int64_t hidden) { return (hidden + 7) / 8 * 8; }
int64_t keys_bytes(int64_t rows) { return (rows * 8 + 255) / 256 * 256; }

template <typename T, int VEC>
cudaError_t launch_sums(const EmbedArgs &a, SumArgs s, cudaStream_t st)
{
    s.lanes = lanes_of(a.hidden / VEC);
    const int slices = (a.hidden + s.lanes * VEC - 1) / (s.lanes * VEC), per_block = kSumThreads / s.lanes;
    s.sum_blocks = (s.pieces + per_block - 1) / per_block;
    const int64_t fill = a.accumulate ? 0 : (a.vocab + kFillRows - 1) / kFillRows;
    return launch_pdl(sum_pieces_kernel<T, VEC>, dim3((unsigned)(s.sum_blocks + fill), (unsigned)slices), dim3(kSumThreads),
                      0, st, s);
}

template <typename T>
cudaError_t sums_typed(const EmbedArgs &a, const SumArgs &s, cudaStream_t st)
{
    auto fits = [&](int vec) {
        return a.hidden % vec == 0 && a.dy_stride % vec == 0 && aligned_to(a.dy, vec * sizeof(T)) &&
               (vec < 4 || aligned_to(a.dtable, 16));
    };
    constexpr int FULL = 16 / (int)sizeof(T);
    if (fits(FULL)) return launch_sums<T, FULL>(a, s, st);
    if constexpr (sizeof(T) == 2)
        if (fits(2)) return launch_sums<T, 2>(a, s, st);
    return launch_sums<T, 1>(a, s, st);
}

}  // namespace

cudaError_t launch_embedding_forward(const EmbedArgs &a, cudaStream_t st)
{
    if (a.dtype == TF_FP32) return embed_typed<float>(a, st);
    return a.dtype == TF_BF16 ? embed_typed<__nv_bfloat16>(a, st) : embed_typed<__half>(a, st);
}

// Two lists of keys, then the partial sums.
int64_t embedding_backward_workspace(int64_t rows, int64_t, int64_t hidden)
{
    return 2 * keys_bytes(rows) + most_pieces(rows, hidden) * 2 * pitch_of(hidden) * 4;
}

cudaError_t launch_embedding_backward(const EmbedArgs &a, cudaStream_t st)
{
    uint64_t *from = static_cast<uint64_t *>(a.ws), *to = from + keys_bytes(a.rows) / 8;
    SumArgs s = {};
    s.part = reinterpret_cast<float *>(static_cast<char *>(a.ws) + 2 * keys_bytes(a.rows));
    s.dy = a.dy; s.dtable = a.dtable; s.dy_stride = a.dy_stride; s.n = a.rows; s.vocab = a.vocab;
    s.pitch = pitch_of(a.hidden); s.hidden = a.hidden; s.accumulate = a.accumulate; s.scale = a.scale;
    s.piece = (int)piece_of(a.rows, a.hidden);
    s.pieces = (int)((a.rows + s.piece - 1) / s.piece);
    cudaError_t e = cudaSuccess;
    if (a.rows > 0) {
        const int64_t chunks = (a.rows + kChunk - 1) / kChunk;
        e = launch_pdl(sort_chunks_kernel, dim3((unsigned)chunks), dim3(kSortThreads), 0, st, a, from);
        for (int64_t len = kChunk; e == cudaSuccess && len < a.rows; len *= kFanIn) {
            e = launch_pdl(merge_runs_kernel, dim3((unsigned)((a.rows + kThreads - 1) / kThreads)), dim3(kThreads), 0, st,
                           static_cast<const uint64_t *>(from), to, a.rows, len);
            uint64_t *t = from;
            from = to;
            to = t;
        }
        if (e != cudaSuccess) return e;
    }
    s.keys = from;
    if (a.dtype == TF_FP32) e = sums_typed<float>(a, s, st);
    else e = a.dtype == TF_BF16 ? sums_typed<__nv_bfloat16>(a, s, st) : sums_typed<__half>(a, s, st);
    if (e != cudaSuccess || s.pieces < 2) return e;
    const unsigned across = (unsigned)((a.hidden + 4 * kJoinCols - 1) / (4 * kJoinCols));
    return launch_pdl(join_pieces_kernel, dim3((unsigned)((s.pieces - 1 + kJoinPieces - 1) / kJoinPieces), across),
                      dim3(kJoinCols * kJoinSplits), 0, st, s);
}

}  // namespace tf
