// Internal declarations of the cache's page upkeep (include/moetree.h, "pages").
#pragma once

#include "attn.cuh"
#include "common.cuh"

namespace moe {
namespace pages {

// A bit of the check word: not enough free pages.
enum : int { FLAG_NO_PAGES = 16 };

// Byte offsets in the workspace: the check word's head, then scratch of one call.
struct WsLayout {
    size_t list;   // int32 [n_pages]  free pages in ascending order, or the holes of a compaction
    size_t map;    // int32 [n_pages]  where each page goes
    size_t claim;  // int32 [B]        first entry of a fork's list that names a sequence
    size_t off;    // int32 [max(B, entries)]  free pages taken by the entries before
    size_t total;
};
WsLayout ws_layout(const moe_page_book &K);

struct CopyArgs {
    char *kp, *vp;
    const int *moves;  // [n, 3]
    const int *count;  // or null: n
    int n;
    int page, n_pages;
    int heads, row_bytes;                       // of a token's head
    long long st_page, st_tok, st_head;         // bytes
    int *flags;
};

cudaError_t launch_free(const moe_page_book &K, const int *seqs, const int *keep, int n, void *ws,
                        cudaStream_t s);
cudaError_t launch_reserve(const moe_page_book &K, int N, const int *n_new, void *ws,
                           cudaStream_t s);
cudaError_t launch_fork(const moe_page_book &K, const int *src, const int *dst, int n, int *moves,
                        void *ws, cudaStream_t s);
cudaError_t launch_compact(const moe_page_book &K, int *table_out, int *ref_out, int *moves,
                           int *counts, void *ws, cudaStream_t s);
cudaError_t launch_copy(const CopyArgs &a, cudaStream_t s);

}  // namespace pages
}  // namespace moe
