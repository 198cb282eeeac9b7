// logprobs.cuh -- launch arguments of the log probabilities (logprobs.cu).  Not a
// public header.
#pragma once

#include "common.cuh"

namespace specv {

struct LogprobArgs {
    const void *logits;
    const int32_t *tokens, *rows;
    int B, N, M, V, top;
    float c, inv_t;        // log2(e) / T, 1 / T
    float *logprob, *entropy;
    int32_t *rank, *top_ids;
    float *top_logprobs;
    uint32_t *err;         // the workspace's error word
    int cluster;           // CTAs a row
};

int launch_logprobs(LogprobArgs &a, int dtype, cudaStream_t st);

}  // namespace specv
