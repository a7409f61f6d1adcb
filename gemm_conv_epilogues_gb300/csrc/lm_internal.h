// Internal declarations of the two ends of a language model, the embedding and
// the cross entropy over its vocabulary: what their entry points pass to the
// launchers.
#pragma once

#include "tf_internal.h"

namespace tf {

// Tokens and targets: int32 or int64, as the caller has them.
struct Indices {
    const void *p;
    int wide;
    __host__ __device__ int64_t at(int64_t i) const
    {
        return wide ? static_cast<const int64_t *>(p)[i] : static_cast<const int32_t *>(p)[i];
    }
};

struct EmbedArgs {
    Indices tokens;
    const void *table;   // forward
    void *y;
    const void *dy;      // backward
    float *dtable;
    void *ws;
    int64_t y_stride, dy_stride, rows, vocab, padding;
    int hidden, dtype, accumulate;
    float scale;
    uint32_t *err;
};
cudaError_t launch_embedding_forward(const EmbedArgs &a, cudaStream_t st);
int64_t embedding_backward_workspace(int64_t rows, int64_t vocab, int64_t hidden);
cudaError_t launch_embedding_backward(const EmbedArgs &a, cudaStream_t st);

// Cross entropy of logits = scale * x w^T, and its gradients.
struct LceArgs {
    Indices targets;
    const void *x, *w;
    float *loss, *lse;               // outputs of the forward pass; the backward pass reads lse
    const float *dloss, *dlse;
    void *dx, *dw;
    void *ws;
    int64_t x_stride, dx_stride, rows, vocab, ignore;
    int hidden, dtype, dw_dtype, accumulate;
    float scale;
    uint32_t *err;
};
constexpr int64_t kLceMaxRows = (int64_t)1 << 22, kLceMaxVocab = (int64_t)1 << 22, kLceMaxHidden = 65536;
int64_t lce_workspace(bool backward, int64_t rows, int64_t vocab, int64_t hidden);
cudaError_t launch_lce_forward(const LceArgs &a, cudaStream_t st);
cudaError_t launch_lce_backward(const LceArgs &a, cudaStream_t st);

// The products (k_vocab_umma.cu), over the rows that count, which the first
// kernel has brought together, and over one piece of the vocabulary.
enum { LCE_STATS = 0, LCE_DLOGITS = 1, LCE_GRADS = 2 };
struct LceProduct {
    const int *count;        // rows that count, on the device
    const int *target;       // theirs, in order
    const void *x, *w;       // [rows][x_pitch], [words][w_pitch]; pitches are multiples of 8
    float2 *part;            // STATS: (maximum, sum) per slot and row
    float *at_target;        // STATS: the target's sum
    const float *z, *ca, *cb;   // DLOGITS: lse, and what the probabilities and the target take
    const float *unit;       // GRADS: unit[1] is the unit of the gradients of the logits
    void *dl;                // [rows][dl_pitch]
    float *dx;               // GRADS: [splits][rows][dx_pitch], null where not wanted
    void *dw;                // this piece's rows, null where not wanted
    int64_t x_pitch, w_pitch, dl_pitch, dx_pitch;
    int rows, words, v0, hidden;
    int slot0, splits;
    int first;               // the first piece: dx is written, not added to
    float factor;            // scale * log2(e) for STATS, scale for DLOGITS and GRADS
    int dtype, dw_f32, accumulate;
};
int lce_word_tile(int64_t rows, int64_t words);   // words per tile of the logits
int lce_splits(int64_t rows, int64_t words, int64_t hidden);   // of dx's sums, at most 16
cudaError_t launch_lce_product(int mode, const LceProduct &a, cudaStream_t st);

}  // namespace tf
