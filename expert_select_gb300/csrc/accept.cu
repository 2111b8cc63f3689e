// The walk of a verified draft tree along the tokens sampled at its nodes ("MoE and speculative
// decoding" blog: per round the accepted prefix is committed and the rest rolled back). From the root
// on, the child whose drafted token is the one sampled at its parent is accepted; the walk ends at a
// node without such a child. As each node's token is drawn from the target's distribution there, what
// is emitted is distributed as if no draft had been made.
//
// A warp per sequence: up to kNodes nodes are read once into shared memory (the walk's steps depend
// on one another, and each would wait for memory), larger trees are walked in memory. Bound by
// latency: 16 trees of 65 nodes move 12 KB.
#include "common.cuh"
#include "sample.cuh"

namespace moe {
namespace sample {
namespace {

constexpr int kWarps = 4, kNodes = 512;

__global__ void __launch_bounds__(kWarps * 32) accept_kernel(const AcceptArgs a) {
    __shared__ int s_parent[kWarps][kNodes], s_token[kWarps][kNodes], s_sampled[kWarps][kNodes];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x * kWarps + warp;
    if (b >= a.B) return;
    int r0 = b * a.N, n = a.N;
    if (a.row_start) {
        r0 = a.row_start[b];
        n = a.row_start[b + 1] - r0;
        // ranges that do not fit are cut
        if (r0 < 0 || r0 > a.R) n = 0;
        n = max(0, min(min(n, a.N), a.R - r0));
    }
    const int *parent = a.parent ? a.parent + r0 : nullptr, *token = a.token + r0,
              *sampled = a.sampled + r0;
    if (n <= kNodes) {
        for (int i = lane; i < n; i += 32) {
            s_parent[warp][i] = parent ? parent[i] : i - 1;
            s_token[warp][i] = token[i];
            s_sampled[warp][i] = sampled[i];
        }
        __syncwarp();
        parent = s_parent[warp];
        token = s_token[warp];
        sampled = s_sampled[warp];
    }
    int *path = a.path + (size_t)b * a.P, *out = a.emitted ? a.emitted + (size_t)b * a.P : nullptr;
    int taken = 0, node = n > 0 ? 0 : -1;
    while (node >= 0 && taken < a.P) {
        const int t = sampled[node];
        if (lane == 0) {
            path[taken] = node;
            if (out) out[taken] = t;
        }
        ++taken;
        int next = -1;
        for (int c0 = node + 1; c0 < n && t >= 0; c0 += 32) {
            const int c = c0 + lane;
            const bool hit = c < n && token[c] == t && (parent ? parent[c] : c - 1) == node;
            const uint32_t m = __ballot_sync(0xffffffffu, hit);
            if (m) {
                next = c0 + __ffs(m) - 1;
                break;
            }
        }
        node = next;
    }
    for (int j = taken + lane; j < a.P; j += 32) {
        path[j] = -1;
        if (out) out[j] = -1;
    }
    if (lane == 0) a.n_accept[b] = taken;
}

}  // namespace

cudaError_t launch_accept(const AcceptArgs &a, cudaStream_t s) {
    return launch_pdl(accept_kernel, dim3((a.B + kWarps - 1) / kWarps), dim3(kWarps * 32), 0, s, a);
}

}  // namespace sample
}  // namespace moe
