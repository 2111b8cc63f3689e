// Arguments of the kernels that write to the paged key/value cache.
#pragma once

#include <limits.h>

#include "attn.cuh"

namespace moe {
namespace cache {

using attn::FLAG_BAD_PAGE;
using attn::FLAG_BAD_SEQUENCE;

struct AppendArgs {
    const void *q, *k, *v, *wq, *wk;
    long long ldq, ldk, ldv;
    void *kp, *vp, *q_out;
    const int *table, *cache_len, *row_start, *depth;
    const float *inv_freq;
    float eps, rope_scale;
    int rot;
    int *flags;  // check word or null
    int B, N, R, H, Hkv, dh, page, n_pages, max_pages, cap;
    long long st_page, st_tok, st_head;  // elements
};

struct CommitArgs {
    void *kp, *vp;
    const int *table, *cache_len, *path, *n_accept;
    int *new_len, *flags;
    int B, P, Hkv, page, n_pages, max_pages, cap;
    int row_bytes;                       // of one head of one slot
    long long st_page, st_tok, st_head;  // bytes
};

cudaError_t launch_append(const AppendArgs &a, int dtype, cudaStream_t s);
cudaError_t launch_commit(const CommitArgs &a, cudaStream_t s);

}  // namespace cache
}  // namespace moe
