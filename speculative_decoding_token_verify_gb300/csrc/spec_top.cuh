// spec_top.cuh -- launch interface of the top-list kernel, shared by
// spec_top.cu and spec_beam.cu. Internal to the library.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace sr {

struct TopArgs {
    const void *z;
    long long batch_stride, row_stride;   // elements
    int B, K, V, M;
    float s, sL, rs;              // inverse temperature, s log2(e); how far a logit may exceed the sum's reference
    // the user's outputs (log-probabilities), or, for the beam step, raw logits
    // and the row's (maximum, sum) in stat
    float *val;                   // [B * K][M]
    int32_t *ids;                 // [B * K][M]
    float *lse;                   // [B * K] or null
    float2 *stat;                 // null: val gets log-probabilities
    // the beam step's rows that need no reading
    const float *scores;          // [B * K] or null
    const int32_t *finished;      // [B * K] or null
    int32_t *status;
};

// Enqueue on `stream`. Returns a cudaError_t.
cudaError_t launch_top(const TopArgs &a, int bf16, cudaStream_t stream);

}  // namespace sr
