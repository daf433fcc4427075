// Internal declarations of a model's two ends (include/e2ttt_tokens.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/e2ttt_tokens.h"

namespace e2ttt {

struct EmbedArgs {
    const void *tokens, *in;  // in: table (forward) or dout (backward)
    void* out;                // out, or dtable
    int64_t N, W;
    int V;
    int wide;        // 8-byte tokens
    int in_f32, out_f32;
    int vec;         // every row of both starts on 16 bytes
    float scale;
    // backward
    int* start;      // [V + 1] where each token's places begin in `order`
    int* order;      // [N] places, by token and then as they come
    float* part;     // [2 ceil(N / kEmbedPiece)][W] sums over pieces of rows with many places
};
// Places that a wave sums for one row; rows with more are cut into pieces.
constexpr int kEmbedPiece = 16;
hipError_t launch_embedding_forward(const EmbedArgs& a, hipStream_t s);
hipError_t launch_embedding_backward(const EmbedArgs& a, hipStream_t s);

struct SampleArgs {
    const void* logits;
    const float *u, *temperature, *top_p, *min_p;  // all but u may be null
    const int* top_k;
    int64_t* token;
    float* logprob;  // may be null
    int64_t rows, stride;
    int V, f32;
    float T, p, mp;
    int k;
};
hipError_t launch_sample(const SampleArgs& a, hipStream_t s);

}  // namespace e2ttt
