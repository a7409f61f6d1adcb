// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   forward   y[i] = scale * table[token[i]]
//   backward  dtable[v] (+)= scale * sum over i with token[i] = v of dy[i]
//
// Both are bound by HBM.  The backward pass brings equal tokens together, so
// that every row of dtable is written once and in a fixed order of additions,
// which atomics would not give:
//   1  a stable counting sort of (token, position): every CTA owns a range of the
//      vocabulary, reads all tokens (they are few beside the rows) and places those of
//      its range, so that no CTA waits for another
//   2  the sorted list is cut into pieces of equal length, whatever the words'
//      frequencies; a thread adds its columns of a piece's rows of dy and writes
//      a row of dtable where the word changes.  A word that goes on for less than a
//      piece is finished where it began; longer ones leave partial sums.  Other
//      CTAs write the zeros of words that do not occur.
//   3  the partial sums of the long words are added in order
#include <type_traits>

#include "grouped.cuh"
#include "lm_internal.h"
#include "ptx_sm100.cuh"

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
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 18;   // words per pass: the counters of 2^18/152 words and 32 warps fill the shared memory
constexpr int64_t kSortBlocks = 152;

__device__ __forceinline__ uint32_t word_of(uint64_t key) { return (uint32_t)(key >> 32); }

// One pass of the stable counting sort, by the digit (word >> shift) & mask: the
// first takes the tokens, a second one, for more than 2^18 words, the first one's
// keys.  A warp has a stretch of the list and counters of its own, so that places
// follow the order of the list: below this CTA's range, smaller digits, earlier
// warps, earlier in the warp.  16384 tokens take 10 us (sorting chunks and merging them took 32);
// a million 283, for which the SMs read all tokens from L2 twice, at 8.6 TB/s.
struct SortArgs {
    Indices tokens;
    const uint64_t *in;
    uint64_t *out;
    int *long_words;
    uint32_t *err;
    int64_t vocab;
    uint32_t padding;   // a word of the vocabulary, or kNone
    int n, shift, range;
    int64_t listed_padding;
};

template <bool FIRST, bool WIDE, bool ONLY>
__global__ void __launch_bounds__(kSortThreads) count_sort_kernel(const __grid_constant__ SortArgs a)
{
    pdl_begin();
    extern __shared__ uint32_t cnt[];   // [kSortWarps][range]
    __shared__ uint32_t warp_sums[kSortWarps], below_sums[kSortWarps];
    constexpr int UNROLL = 8;
    constexpr uint32_t mask = (1u << kDigitBits) - 1;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    // ONLY: the words themselves are the digits, and what is no word lies behind the last range
    const uint32_t d0 = blockIdx.x * (uint32_t)a.range;
    const uint32_t range = ONLY ? min((uint32_t)a.range, (uint32_t)a.vocab - d0) : (uint32_t)a.range;
    auto place_of = [&](uint32_t word) { return (ONLY ? word : (word >> a.shift) & mask) - d0; };
    const int seg = ((a.n + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    const int lo = min(a.n, warp * seg), hi = min(a.n, lo + seg);
    for (int i = t; i < kSortWarps * a.range; i += kSortThreads) cnt[i] = 0;
    if (blockIdx.x == 0 && t == 0) *a.long_words = 0;
    __syncthreads();
    uint32_t *mine = cnt + warp * a.range;
    // 32*UNROLL entries from i on: their words (kNone: not there) and, of keys, their rows
    auto load_from = [&](auto whole, int i, uint32_t (&word)[UNROLL], uint32_t (&row)[UNROLL]) {
        auto there = [&](int u) { return decltype(whole)::value || i + 32 * u < hi; };
        if constexpr (FIRST && !WIDE) {
#pragma unroll
            for (int u = 0; u < UNROLL; ++u)
                word[u] = there(u) ? static_cast<const uint32_t *>(a.tokens.p)[i + 32 * u] : kNone;
        } else {
            const uint2 *src = FIRST ? static_cast<const uint2 *>(a.tokens.p) : reinterpret_cast<const uint2 *>(a.in);
            uint2 v[UNROLL];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) v[u] = there(u) ? src[i + 32 * u] : make_uint2(kNone, kNone);
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {   // a token's halves, or a key's: its row and its word
                word[u] = !FIRST ? v[u].y : v[u].y == 0 ? v[u].x : kNone;
                row[u] = v[u].x;
            }
        }
        if (FIRST && (!ONLY || a.padding != kNone)) {
#pragma unroll
            for (int u = 0; u < UNROLL; ++u)
                if ((!ONLY && word[u] >= (uint32_t)a.vocab) || word[u] == a.padding) word[u] = kNone;
        }
    };
    auto load = [&](int i, uint32_t (&word)[UNROLL], uint32_t (&row)[UNROLL]) {
        if (i - lane + 32 * UNROLL <= hi) load_from(std::true_type(), i, word, row);
        else load_from(std::false_type(), i, word, row);
    };
    // which of this lane's entries are in the range, where 32 bits hold them: few are, and only those are looked at again
    const bool marked = seg <= 32 * 32;
    uint32_t low = 0, marks = 0;
    int step = 0;
    for (int i = lo + lane; i < hi; i += 32 * UNROLL, step += UNROLL) {
        uint32_t word[UNROLL], row[UNROLL];
        load(i, word, row);
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const uint32_t at = place_of(word[u]);
            const bool there = ONLY || word[u] != kNone;
            low += there && at + d0 < d0;
            if (there && at < range) {
                atomicAdd(mine + at, 1u);
                marks |= 1u << ((step + u) & 31);
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) low += __shfl_xor_sync(0xffffffffu, low, o);
    if (lane == 0) below_sums[warp] = low;
    if (FIRST)   // the CTAs look through the tokens together for those that are neither words nor the padding
        for (int64_t i = (int64_t)blockIdx.x * kSortThreads + t; i < a.n; i += (int64_t)gridDim.x * kSortThreads) {
            const int64_t token = a.tokens.at(i);
            if ((token < 0 || token >= a.vocab) && token != a.listed_padding) atomicOr(a.err, TF_DEVERR_INDEX);
        }
    __syncthreads();
    uint32_t base = below_sums[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) base += __shfl_xor_sync(0xffffffffu, base, o);
    // counters become places: a warp per 32 digits' sums, then a thread per digit
    for (int d = 0; d < a.range; d += kSortThreads) {
        const bool live = d + t < a.range;
        uint32_t sum = 0;
        if (live) {
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) sum += cnt[w * a.range + d + t];
        }
        uint32_t scan = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += up;
        }
        if (lane == 31) warp_sums[warp] = scan;
        __syncthreads();
        uint32_t before = warp_sums[lane], all = before;   // this lane's warp; those before this warp, and all
        before = lane < warp ? before : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            before += __shfl_xor_sync(0xffffffffu, before, o);
            all += __shfl_xor_sync(0xffffffffu, all, o);
        }
        uint32_t at = base + before + scan - sum;
        base += all;
        if (live) {
            for (int w = 0; w < kSortWarps; w += 8) {
                uint32_t n[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) n[k] = cnt[(w + k) * a.range + d + t];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    cnt[(w + k) * a.range + d + t] = at;
                    at += n[k];
                }
            }
        }
        __syncthreads();
    }
    // 32 entries from i0 on, of which this lane has one, in the order of the list
    auto put = [&](int i, uint32_t word, uint32_t row, bool in_range) {
        const unsigned active = __ballot_sync(0xffffffffu, in_range);
        if (active == 0) return;
        if (in_range) {
            const uint32_t at = place_of(word);
            const unsigned same = __match_any_sync(active, at);
            const uint32_t before = __popc(same & ((1u << lane) - 1u)), first = mine[at];
            a.out[first + before] = (uint64_t)word << 32 | (FIRST ? (uint32_t)i : row);
            __syncwarp(active);
            if (before == 0) mine[at] = first + __popc(same);
        }
        __syncwarp();
    };
    if (marked) {
        for (int i = lo + lane; i - lane < hi; i += 32, marks >>= 1) {
            const bool in_range = marks & 1u;
            uint64_t v = 0;
            if (in_range) {
                if constexpr (!FIRST) v = a.in[i];
                else v = WIDE ? static_cast<const uint64_t *>(a.tokens.p)[i] : static_cast<const uint32_t *>(a.tokens.p)[i];
            }
            put(i, FIRST ? (uint32_t)v : word_of(v), (uint32_t)v, in_range);
        }
    } else {
        for (int i = lo + lane; i - lane < hi; i += 32 * UNROLL) {
            uint32_t word[UNROLL], row[UNROLL];
            load(i, word, row);
#pragma unroll
            for (int u = 0; u < UNROLL; ++u)
                put(i + 32 * u, word[u], row[u], (ONLY || word[u] != kNone) && place_of(word[u]) < range);
        }
    }
    if (blockIdx.x == gridDim.x - 1)   // the rest have no gradient
        for (int64_t i = (int64_t)base + t; i < a.n; i += kSortThreads) a.out[i] = ~0ull;
}

// Keys of [lo, hi) below `key`.
__device__ __forceinline__ int64_t below(const uint64_t *keys, int64_t lo, int64_t hi, uint64_t key)
{
    const int64_t start = lo;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (__ldg(keys + mid) < key) lo = mid + 1; else hi = mid;
    }
    return lo - start;
}

// ---------------------------------------------------------------- backward: sums

constexpr int kSumThreads = 128;
constexpr int kFillRows = 64;      // rows of dtable per zeroing CTA
constexpr int kMinPiece = 8, kMaxPiece = 1024;
// Terms added before their sum joins the next level's: long sums of equal terms keep their digits.
constexpr int kLevel = 64;
constexpr int64_t kMostPieces = 32768;
// The ring's copies under way are waited for at least this long after a wait that ran out.
constexpr uint64_t kLeastDrainNs = 1000000000;

struct SumArgs {
    const uint64_t *keys;
    const void *dy;
    float *dtable, *part;          // part: [pieces][2][pitch], of long words that go on before and behind the piece
    int *long_words;               // their number, then the pieces that they begin in
    int64_t dy_stride, n, vocab, pitch;
    int hidden, accumulate, piece, pieces, lanes, sum_blocks;
    float scale;
    uint32_t *err;
    uint64_t wait_ns;
};

// low += v, two columns at a time where there are as many.
template <typename T, int VEC>
__device__ __forceinline__ void add_values(float (&low)[VEC], const Pack<T, VEC> &v)
{
    if constexpr (VEC == 1) {
        low[0] += widen<T>(v.v[0]);
    } else {
#pragma unroll
        for (int k = 0; k < VEC; k += 2) {
            float2 x;
            if constexpr (sizeof(T) == 2) x = grouped::Half2Of<T>::unpack(*reinterpret_cast<const uint32_t *>(&v.v[k]));
            else x = make_float2(v.v[k], v.v[k + 1]);
            const float2 t = fadd2(make_float2(low[k], low[k + 1]), x);
            low[k] = t.x;
            low[k + 1] = t.y;
        }
    }
}

// A row's columns.  Adding to what is there is left to the L2, which does not make
// the thread wait for the old values; every element of dtable gets one such
// addition in a call, so that their order does not matter.
template <int VEC>
__device__ __forceinline__ void put_row(float *dst, const float (&sum)[VEC], float scale, bool add)
{
    if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int k = 0; k < VEC; k += 4) {
            const float4 v = make_float4(sum[k] * scale, sum[k + 1] * scale, sum[k + 2] * scale, sum[k + 3] * scale);
            if (add)
                asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(dst + k), "f"(v.x), "f"(v.y), "f"(v.z),
                             "f"(v.w)
                             : "memory");
            else
                *reinterpret_cast<float4 *>(dst + k) = v;
        }
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            if (add) atomicAdd(dst + k, sum[k] * scale);
            else dst[k] = sum[k] * scale;
        }
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
// lanes*VEC; the CTA's other threads take further pieces.  RING: the rows come through
// shared memory by bulk copies, two batches of eight ahead, which keeps more of them under
// way than registers could (16384 rows of 4096 bf16 into 32000 words: 59 us, 74 with registers).
template <typename T, int VEC, bool RING>
__global__ void __launch_bounds__(kSumThreads, RING ? 6 : 5) sum_pieces_kernel(const __grid_constant__ SumArgs a)
{
    pdl_begin();
    if ((int)blockIdx.x >= a.sum_blocks) {
        if (blockIdx.y == 0) fill_zeros(a, (int64_t)((int)blockIdx.x - a.sum_blocks) * kFillRows);
        return;
    }
    constexpr int UNROLL = RING || VEC * sizeof(T) < 16 ? 8 : 4;
    using P = Pack<T, VEC>;
    const int member = (int)threadIdx.x % a.lanes, group = (int)threadIdx.x / a.lanes;
    const int p = (int)blockIdx.x * (kSumThreads / a.lanes) + group;
    const int slice = (int)blockIdx.y * a.lanes * VEC, c = slice + member * VEC;
    __shared__ __align__(128) P ring[RING ? 2 * UNROLL * kSumThreads : 1];
    __shared__ __align__(8) uint64_t full[kSumThreads / 32][2];
    __shared__ uint32_t words[kSumThreads / 32][2][UNROLL];
    if (RING) {
        if (threadIdx.x < kSumThreads / 32 * 2) {
            ptx::mbar_init(&full[threadIdx.x / 2][threadIdx.x % 2], 1);
            ptx::mbar_init_fence();
        }
        __syncthreads();
    }
    if (p >= a.pieces || (!RING && c >= a.hidden)) return;
    const bool live = c < a.hidden;   // (RING: the others take part in the barriers)
    const int first = p * a.piece, n = (int)a.n, end = min(first + a.piece, n);   // (n + 2*piece fits)
    const T *dy = static_cast<const T *>(a.dy) + c;
    auto word_at = [&](int i) { return i >= 0 && i < n ? word_of(__ldg(a.keys + i)) : kNone; };
    // A word that goes on behind the piece it begins in for `piece` rows or more is long: each
    // of its pieces leaves a partial sum.  Otherwise the piece that it begins in finishes it.
    uint32_t word = word_at(first);
    const uint32_t final = word_at(end - 1);
    const bool head = word != kNone && word_at(first - 1) == word;
    const bool head_long = head && (word_at(first + a.piece - 1) == word || word_at(first - a.piece - 1) == word);
    const bool tail = final != kNone && word_at(end) == final;
    const bool tail_long = tail && (word_at(end + a.piece - 1) == final || (head && final == word));
    const int limit = tail && !tail_long ? min(end + a.piece, n) : end;
    float sum[VEC] = {}, low[VEC] = {};
    int held = 0;
    bool at_head = head;
    auto flush = [&](bool goes_on) {
        if (live && word != kNone && (!at_head || head_long)) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) sum[k] += low[k];
            if (at_head || goes_on)
                put_row<VEC>(a.part + ((int64_t)p * 2 + (at_head ? 0 : 1)) * a.pitch + c, sum, 1.0f, false);
            else
                put_row<VEC>(a.dtable + (int64_t)word * a.hidden + c, sum, a.scale, a.accumulate != 0);
            if (goes_on && !at_head && c == 0) a.long_words[1 + atomicAdd(a.long_words, 1)] = p;
        }
#pragma unroll
        for (int k = 0; k < VEC; ++k) sum[k] = low[k] = 0.0f;
        held = 0;
        at_head = false;
    };
    const uint32_t skipped = head && !head_long ? word : kNone;   // finished by the piece before
    auto key_at = [&](int i) {
        const uint64_t key = i < limit ? __ldg(a.keys + i) : ~0ull;
        return i < end || word_of(key) == final ? key : ~0ull;
    };
    auto add_row = [&](uint32_t w, const P &v) {
        if (w != word) {
            flush(false);
            word = w;
        }
        if (w == skipped) return;
        add_values<T, VEC>(low, v);
        if (++held == kLevel) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                sum[k] += low[k];
                low[k] = 0.0f;
            }
            held = 0;
        }
    };
    if constexpr (RING) {
        const uint32_t bytes = (uint32_t)(min(a.lanes * VEC, a.hidden - slice) * (int)sizeof(T));
        // The piece's first warp asks for a batch: a row per lane.
        auto fetch = [&](int i, int half) {
            if (member >= 32) return;
            const uint64_t key = member < UNROLL ? key_at(i + member) : ~0ull;
            const uint32_t w = word_of(key);
            const bool wanted = w != kNone && w != skipped;
            const unsigned rows = __ballot_sync(0xffffffffu, wanted);
            if (member < UNROLL) words[group][half][member] = w;
            if (member == 0) ptx::mbar_arrive_expect_tx(&full[group][half], __popc(rows) * bytes);
            __syncwarp();
            const T *src = static_cast<const T *>(a.dy) + slice + (int64_t)(uint32_t)key * a.dy_stride;
            if (wanted)
                ptx::bulk_load(&ring[(half * UNROLL + member) * kSumThreads + group * a.lanes], src, bytes, &full[group][half]);
            __syncwarp();
        };
        // The piece's threads meet; whether any of them says that a wait ran out.
        auto meet = [&](bool lost) {
            if (a.lanes == 32) {
                const bool any = __any_sync(0xffffffffu, lost);
                __syncwarp();
                return any;
            }
            __syncwarp();
            uint32_t any;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                : "=r"(any)
                : "r"((uint32_t)lost), "r"(group + 1), "r"(a.lanes)
                : "memory");
            return any != 0;
        };
        fetch(first, 0);
        if (first + UNROLL < limit) fetch(first + UNROLL, 1);
        meet(false);
        int batch = 0;
        for (int i = first; i < limit; i += UNROLL, ++batch) {
            const int half = batch & 1;
            const bool got = ptx::mbar_wait(&full[group][half], (uint32_t)(batch >> 1) & 1u, a.wait_ns);
            if (got) {
#pragma unroll 1
                for (int u = 0; u < UNROLL; ++u) {
                    const uint32_t w = words[group][half][u];
                    if (w == kNone) break;   // (the last of the list, or of the word that went on)
                    add_row(w, ring[(half * UNROLL + u) * kSumThreads + threadIdx.x]);
                }
            }
            if (meet(!got)) {
                // All of the piece's threads leave: nothing more is asked for or written, and the
                // batches under way, this one and the next, land while the CTA still owns the ring.
                if (member == 0) {
                    atomicOr(a.err, TF_DEVERR_PRODUCER_WAIT);
                    const uint64_t ns = a.wait_ns > kLeastDrainNs ? a.wait_ns : kLeastDrainNs;
                    for (int k = batch; k <= batch + 1 && first + k * UNROLL < limit; ++k)
                        if (!ptx::mbar_wait(&full[group][k & 1], (uint32_t)(k >> 1) & 1u, ns))
                            atomicOr(a.err, TF_DEVERR_DRAIN_WAIT);
                }
                return;
            }
            // (the batch has been read)
            if (i + 2 * UNROLL < limit) fetch(i + 2 * UNROLL, half);
        }
    } else {
        uint64_t key[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) key[u] = key_at(first + u);
        for (int i = first; i < limit; i += UNROLL) {
            P v[UNROLL];
            uint32_t w[UNROLL];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                w[u] = word_of(key[u]);
                const T *src = dy + (int64_t)(uint32_t)key[u] * a.dy_stride;
                if (w[u] != kNone && w[u] != skipped) v[u] = *reinterpret_cast<const P *>(src);
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) key[u] = key_at(i + UNROLL + u);   // the next ones, while the rows are under way
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                if (w[u] == kNone) break;
                add_row(w[u], v[u]);
            }
        }
    }
    flush(tail_long);
}

constexpr int kJoinCols = 32, kJoinSplits = 8, kJoinThreads = kJoinCols * kJoinSplits;

// Long words: a CTA adds 128 columns of one word's partial sums, in kJoinSplits
// stretches that are joined in order.
__global__ void __launch_bounds__(kJoinThreads) join_pieces_kernel(const __grid_constant__ SumArgs a)
{
    pdl_begin();
    __shared__ float4 red[kJoinSplits][kJoinCols];
    const int col = threadIdx.x % kJoinCols, split = threadIdx.x / kJoinCols;
    const int across = (a.hidden + 4 * kJoinCols - 1) / (4 * kJoinCols), items = *a.long_words * across;
    for (int item = (int)blockIdx.x; item < items; item += (int)gridDim.x) {
        const int p = a.long_words[1 + item / across], c = (item % across * kJoinCols + col) * 4;
        const uint32_t word = word_of(__ldg(a.keys + (int64_t)(p + 1) * a.piece - 1));
        int count = 1;   // pieces: those behind p that begin with the word follow one another
        for (int q = p + 1;; q += kJoinThreads) {
            const int64_t at = (int64_t)(q + (int)threadIdx.x) * a.piece;
            const int n = __syncthreads_count(at < a.n && word_of(__ldg(a.keys + at)) == word);
            count += n;
            if (n < kJoinThreads) break;
        }
        const int per = (count + kJoinSplits - 1) / kJoinSplits;
        float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (c < a.hidden) {
            const float *src = a.part + (int64_t)p * 2 * a.pitch + c;
            const int end = min((split + 1) * per, count);
            for (int q0 = split * per; q0 < end; q0 += kLevel) {
                float4 low = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
                for (int q = q0; q < min(q0 + kLevel, end); ++q) {
                    const float4 v = *reinterpret_cast<const float4 *>(src + (2 * (int64_t)q + (q == 0 ? 1 : 0)) * a.pitch);
                    low.x += v.x; low.y += v.y; low.z += v.z; low.w += v.w;
                }
                t.x += low.x; t.y += low.y; t.z += low.z; t.w += low.w;
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

// Pieces that fill the SMs where the list is long enough (14 CTAs each, and no more pieces than a
// long word's join adds quickly), of 8 to 1024 keys.  Sized for 8 columns per thread,
// whatever the type, so that the workspace depends on the sizes alone.  (16384 rows of 4096 into
// 32000 words: 76.6 us, with 10 to 18 CTAs each 77-81, with 24 87.)
int64_t piece_target(int64_t hidden)
{
    const int lanes = lanes_of((int)((hidden + 7) / 8));
    const int64_t slices = (hidden + 8 * lanes - 1) / (8 * lanes), per_block = kSumThreads / lanes;
    const int64_t fill = (14 * 152 + slices - 1) / slices * per_block;
    return fill < kMostPieces ? fill : kMostPieces;
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
int64_t list_bytes(int64_t pieces) { return ((pieces + 1) * 4 + 255) / 256 * 256; }

template <typename T, int VEC>
cudaError_t launch_sums(const EmbedArgs &a, SumArgs s, cudaStream_t st)
{
    s.lanes = lanes_of(a.hidden / VEC);
    const int slices = (a.hidden + s.lanes * VEC - 1) / (s.lanes * VEC), per_block = kSumThreads / s.lanes;
    s.sum_blocks = (s.pieces + per_block - 1) / per_block;
    const int64_t fill = a.accumulate ? 0 : (a.vocab + kFillRows - 1) / kFillRows;
    const dim3 grid((unsigned)(s.sum_blocks + fill), (unsigned)slices);
    if constexpr (VEC * sizeof(T) == 16)
        if (s.lanes >= 32) {
            auto kern = sum_pieces_kernel<T, VEC, true>;
            const void *id = reinterpret_cast<const void *>(kern);
            int known = 0;
            if (!recall(id, FACT_CARVEOUT, &known)) {   // shared memory for as many CTAs as the registers allow
                const cudaError_t e = cudaFuncSetAttribute(id, cudaFuncAttributePreferredSharedMemoryCarveout,
                                                           cudaSharedmemCarveoutMaxShared);
                if (e != cudaSuccess) return e;
                remember(id, FACT_CARVEOUT, 1);
            }
            return launch_pdl(kern, grid, dim3(kSumThreads), 0, st, s);
        }
    return launch_pdl(sum_pieces_kernel<T, VEC, false>, grid, dim3(kSumThreads), 0, st, s);
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

// The keys (twice for two passes), the long words' list, then the partial sums.
int64_t embedding_backward_workspace(int64_t rows, int64_t vocab, int64_t hidden)
{
    const int passes = vocab > (int64_t)1 << kDigitBits ? 2 : 1;
    const int64_t pieces = most_pieces(rows, hidden);
    return rows == 0 ? 0 : passes * keys_bytes(rows) + list_bytes(pieces) + pieces * 2 * pitch_of(hidden) * 4;
}

cudaError_t launch_embedding_backward(const EmbedArgs &a, cudaStream_t st)
{
    const int passes = a.vocab > (int64_t)1 << kDigitBits ? 2 : 1;
    char *ws = static_cast<char *>(a.ws);
    uint64_t *keys = reinterpret_cast<uint64_t *>(ws), *first = keys + (passes - 1) * keys_bytes(a.rows) / 8;
    SumArgs s = {};
    s.keys = keys;
    s.long_words = reinterpret_cast<int *>(ws + passes * keys_bytes(a.rows));
    s.part = reinterpret_cast<float *>(ws + passes * keys_bytes(a.rows) + list_bytes(most_pieces(a.rows, a.hidden)));
    s.dy = a.dy; s.dtable = a.dtable; s.dy_stride = a.dy_stride; s.n = a.rows; s.vocab = a.vocab;
    s.pitch = pitch_of(a.hidden); s.hidden = a.hidden; s.accumulate = a.accumulate; s.scale = a.scale;
    s.piece = (int)piece_of(a.rows, a.hidden);
    s.pieces = (int)((a.rows + s.piece - 1) / s.piece);
    s.err = a.err;
    s.wait_ns = wait_limit_ns();
    cudaError_t e = cudaSuccess;
    for (int pass = 0; a.rows > 0 && e == cudaSuccess && pass < passes; ++pass) {
        const int64_t all = ((a.vocab - 1) >> (pass * kDigitBits)) + 1, most = (int64_t)1 << kDigitBits;
        const int64_t digits = all < most ? all : most, even = (digits + kSortBlocks - 1) / kSortBlocks;
        const int64_t range = even < 64 ? 64 : even;
        const dim3 grid((unsigned)((digits + range - 1) / range));
        SortArgs q = {};
        q.tokens = a.tokens; q.in = first; q.out = pass == 0 ? first : keys; q.long_words = s.long_words; q.err = a.err;
        q.vocab = a.vocab; q.listed_padding = a.padding;
        q.padding = a.padding >= 0 && a.padding < a.vocab ? (uint32_t)a.padding : kNone;
        q.n = (int)a.rows; q.shift = pass * kDigitBits; q.range = (int)range;
        auto kern = pass > 0     ? count_sort_kernel<false, false, false>
                    : passes > 1 ? (a.tokens.wide ? count_sort_kernel<true, true, false> : count_sort_kernel<true, false, false>)
                                 : (a.tokens.wide ? count_sort_kernel<true, true, true> : count_sort_kernel<true, false, true>);
        e = raise_smem_limit(reinterpret_cast<const void *>(kern));
        if (e == cudaSuccess) e = launch_pdl(kern, grid, dim3(kSortThreads), (size_t)(kSortWarps * range * 4), st, q);
    }
    if (e != cudaSuccess) return e;
    if (a.dtype == TF_FP32) e = sums_typed<float>(a, s, st);
    else e = a.dtype == TF_BF16 ? sums_typed<__nv_bfloat16>(a, s, st) : sums_typed<__half>(a, s, st);
    if (e != cudaSuccess || s.pieces < 2) return e;
    return launch_pdl(join_pieces_kernel, dim3((unsigned)(8 * sm_count())), dim3(kJoinThreads), 0, st, s);
}

}  // namespace tf
