// Internal declarations of the layer for a few tokens (moe_few_forward).
#pragma once

#include "common.cuh"

namespace moe {
namespace few {

constexpr int kMaxRows = 16;

// Byte offsets in the workspace. The head (check word, grid barrier) is zero before the first call.
struct WsLayout {
    size_t logits;  // f32 [R, E]
    size_t h;       // [R k] rows of gated activations: f32, or bf16 pairs (the value and its rest)
    size_t total;
};
constexpr size_t kHeadBytes = 4096;
WsLayout ws_layout(const moe_layer_desc &L, int R);

struct Args {
    const void *x, *wr, *wg, *wu, *wd;
    const int *slot;
    void *y;
    float *logits;        // [R, E]
    int *topk_idx;        // or null
    float *gates;         // or null
    void *h;
    int *flags, *barrier;
    int R, d, E, k, f, slots;
    int norm, residual;
};
// Tokens that one launch takes.
int rows_at_once(const moe_layer_desc &L);
cudaError_t launch_few(const Args &a, int dtype, int max_ctas, cudaStream_t s);

}  // namespace few
}  // namespace moe
