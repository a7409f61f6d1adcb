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

}  // namespace tf
