// Internal declarations of the layer for a few tokens (moe_few_forward).
#pragma once

#include "common.cuh"

namespace moe {
namespace few {

constexpr int kMaxRows = 16;

// Byte offsets in the workspace. The head is zero before the first call: the check word, the grid's
// count (kBarrier), and the scores of kMaxRows tokens (kScores).
struct WsLayout {
    size_t h;  // [R k] rows of gated activations: f32, or bf16 pairs (the value and its rest)
    size_t total;
};
constexpr size_t kBarrier = 1024, kScores = 4096;
constexpr size_t kHeadBytes = kScores + (size_t)kMaxRows * kMaxE * 8;
WsLayout ws_layout(const moe_layer_desc &L, int R);

// Two fp32 values whose sum stands for one of twice the bits.
struct Pair {
    float hi, lo;
};

struct Args {
    const void *x, *wr, *wg, *wu, *wd;
    const int *slot;
    void *y;
    float *logits;        // or null
    int *topk_idx;        // or null
    float *gates;         // or null
    void *h;
    int *flags;
    unsigned long long *barrier, *scores;
    int R, d, E, k, f, slots;
    int norm, residual;
    Pair inv_d;  // 1 / d
};
// Tokens that one launch takes.
int rows_at_once(const moe_layer_desc &L);
cudaError_t launch_few(const Args &a, int dtype, int max_ctas, cudaStream_t s);

}  // namespace few
}  // namespace moe
