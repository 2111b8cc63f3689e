// Internal declarations of sampling and of the walk along the samples (include/moetree.h).
#pragma once

#include "common.cuh"

namespace moe {
namespace sample {

struct Args {
    const void *logits;
    long long ld;
    int R, V, group;  // rows that share a request's settings
    const float *temperature, *top_p, *min_p;
    const int *top_k;
    const float *u;
    int *token;
    float *logprob;
};

// Tokens at most: sums of V weights of up to 2^43 stay below 2^62.
constexpr int kMaxV = 1 << 19;

cudaError_t launch_sample(const Args &a, int dtype, cudaStream_t s);

struct AcceptArgs {
    const int *token, *parent, *sampled, *row_start;
    int B, N, R, P;
    int *path, *n_accept, *emitted;
};
cudaError_t launch_accept(const AcceptArgs &a, cudaStream_t s);

}  // namespace sample
}  // namespace moe
