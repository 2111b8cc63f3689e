// Entry points of a decoding round beside the tree's layer and attention (see include/moetree.h): the
// layer for a few tokens, sampling, the walk along the samples, and the cache's pages. Argument
// checks and launches.
#include <algorithm>
#include <cmath>

#include "few.cuh"
#include "pages.cuh"
#include "sample.cuh"

namespace moe {
namespace {

bool book_ok(const moe_page_book *K) {
    if (!K || K->B < 1 || K->B > 65536 || K->max_pages < 1 || K->n_pages < 1 || K->page_size < 1)
        return false;
    if (K->n_pages > 1 << 24 || (long long)K->page_size * K->max_pages > 1 << 30) return false;
    return K->page_table && K->held && K->cache_len && K->ref;
}
bool ws_ok(const void *ws) { return ws && !((uintptr_t)ws & 255u); }

bool overlap(const void *p, size_t n, const void *q, size_t m) {
    return p && q && (uintptr_t)p < (uintptr_t)q + m && (uintptr_t)q < (uintptr_t)p + n;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_few_workspace_bytes(const moe_layer_desc *L, int R) {
    if (!desc_ok(L) || R < 1 || R > few::kMaxRows) return 0;
    return few::ws_layout(*L, R).total;
}

moe_status moe_few_forward(const moe_layer_desc *L, const void *x, const void *W_r,
                           const void *W_gate, const void *W_up, const void *W_down,
                           const int *slot_of_expert, int R, void *y, float *logits, int *topk_idx,
                           float *gates, void *workspace, const moe_run_opts *opts,
                           moe_stream_t stream) {
    if (!desc_ok(L) || R < 0) return MOE_ERR_ARG;
    if (R == 0) return MOE_OK;
    if (R > few::kMaxRows) return MOE_ERR_UNSUPPORTED;
    if (!x || !W_r || !W_gate || !W_up || !W_down || !y || !ws_ok(workspace)) return MOE_ERR_ARG;
    for (const void *p : {x, W_r, W_gate, W_up, W_down, (const void *)y})
        if (!aligned16(p)) return MOE_ERR_ARG;
    if (opts && (opts->ffn_max_ctas < 0 || opts->ffn_begin || opts->ffn_end || opts->select_begin))
        return MOE_ERR_ARG;
    // a token's row is read until its outputs are written, other tokens' rows at any time
    const size_t bytes = (size_t)R * L->d * elem_size(L->dtype);
    if (y != x && overlap(x, bytes, y, bytes)) return MOE_ERR_ARG;
    const few::WsLayout w = few::ws_layout(*L, R);
    few::Args a{};
    a.wr = W_r;
    a.wg = W_gate;
    a.wu = W_up;
    a.wd = W_down;
    a.slot = slot_of_expert;
    a.h = at<void>(workspace, w.h);
    a.flags = at<int>(workspace, 0);
    a.barrier = at<unsigned long long>(workspace, few::kBarrier);
    a.scores = at<unsigned long long>(workspace, few::kScores);
    a.d = L->d;
    a.E = L->E;
    a.k = L->k;
    a.f = L->f;
    a.slots = L->slots > 0 ? L->slots : L->E;
    a.norm = opts && opts->norm_input;
    a.inv_d.hi = (float)(1.0 / L->d);
    a.inv_d.lo = (float)(1.0 / L->d - (double)a.inv_d.hi);
    a.residual = opts && opts->residual;
    const int most = few::rows_at_once(*L);
    const size_t row = (size_t)L->d * elem_size(L->dtype);
    for (int r0 = 0; r0 < R; r0 += most) {
        a.R = std::min(most, R - r0);
        a.x = (const char *)x + r0 * row;
        a.y = (char *)y + r0 * row;
        a.logits = logits ? logits + (size_t)r0 * L->E : nullptr;
        a.topk_idx = topk_idx ? topk_idx + (size_t)r0 * L->k : nullptr;
        a.gates = gates ? gates + (size_t)r0 * L->k : nullptr;
        const cudaError_t err = few::launch_few(a, L->dtype, opts ? opts->ffn_max_ctas : 0,
                                                (cudaStream_t)stream);
        if (err != cudaSuccess) return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

moe_status moe_sample(const moe_sample_params *P, const void *logits, long long ld, const float *u,
                      int R, int *token, float *logprob, moe_stream_t stream) {
    if (!P || (P->dtype != MOE_DTYPE_F32 && P->dtype != MOE_DTYPE_BF16)) return MOE_ERR_ARG;
    if (P->V < 1 || R < 0 || P->param_rows < 1 || ld < P->V) return MOE_ERR_ARG;
    if (P->V > sample::kMaxV || R > 1 << 26) return MOE_ERR_UNSUPPORTED;
    if (R == 0) return MOE_OK;
    if (!logits || !u || !token || (uintptr_t)logits % elem_size(P->dtype)) return MOE_ERR_ARG;
    sample::Args a{};
    a.logits = logits;
    a.ld = ld;
    a.R = R;
    a.V = P->V;
    a.group = P->param_rows;
    a.temperature = P->temperature;
    a.top_k = P->top_k;
    a.top_p = P->top_p;
    a.min_p = P->min_p;
    a.u = u;
    a.token = token;
    a.logprob = logprob;
    return cuda_status(sample::launch_sample(a, P->dtype, (cudaStream_t)stream));
}

moe_status moe_tree_accept(const int *token, const int *parent, const int *sampled,
                           const int *row_start, int B, int N, int R, int P, int *path,
                           int *n_accept, int *emitted, moe_stream_t stream) {
    if (B < 0 || N < 0 || R < 0 || P < 1) return MOE_ERR_ARG;
    if (!row_start && (long long)B * N != R) return MOE_ERR_ARG;
    if (B == 0) return MOE_OK;
    if (!path || !n_accept || (R > 0 && (!token || !sampled))) return MOE_ERR_ARG;
    sample::AcceptArgs a{};
    a.token = token;
    a.parent = parent;
    a.sampled = sampled;
    a.row_start = row_start;
    a.B = B;
    a.N = N;
    a.R = R;
    a.P = P;
    a.path = path;
    a.n_accept = n_accept;
    a.emitted = emitted;
    return cuda_status(sample::launch_accept(a, (cudaStream_t)stream));
}

// -------------------------------------------------------------------- pages

size_t moe_pages_workspace_bytes(const moe_page_book *K) {
    return book_ok(K) ? pages::ws_layout(*K).total : 0;
}

moe_status moe_kv_reserve(const moe_page_book *K, int N, const int *n_new, void *workspace,
                          moe_stream_t stream) {
    if (!book_ok(K) || N < 0 || !ws_ok(workspace)) return MOE_ERR_ARG;
    return cuda_status(pages::launch_reserve(*K, N, n_new, workspace, (cudaStream_t)stream));
}

moe_status moe_kv_free(const moe_page_book *K, const int *seqs, const int *keep, int n,
                       void *workspace, moe_stream_t stream) {
    if (!book_ok(K) || n < 0 || !ws_ok(workspace)) return MOE_ERR_ARG;
    if (n == 0) return MOE_OK;
    if (!seqs) return MOE_ERR_ARG;
    return cuda_status(pages::launch_free(*K, seqs, keep, n, workspace, (cudaStream_t)stream));
}

moe_status moe_kv_fork(const moe_page_book *K, const int *src, const int *dst, int n, int *moves,
                       void *workspace, moe_stream_t stream) {
    if (!book_ok(K) || n < 0 || n > K->B || !ws_ok(workspace)) return MOE_ERR_ARG;
    if (n == 0) return MOE_OK;
    if (!src || !dst || !moves) return MOE_ERR_ARG;
    return cuda_status(pages::launch_fork(*K, src, dst, n, moves, workspace, (cudaStream_t)stream));
}

moe_status moe_kv_compact(const moe_page_book *K, int *table_out, int *ref_out, int *moves,
                          int *counts, void *workspace, moe_stream_t stream) {
    if (!book_ok(K) || !table_out || !ref_out || !counts || !ws_ok(workspace)) return MOE_ERR_ARG;
    if (K->n_pages > 1 && !moves) return MOE_ERR_ARG;
    // each output may be its input, and nothing else that is read
    const size_t table = (size_t)K->B * K->max_pages * 4, ref = (size_t)K->n_pages * 4,
                 seqs = (size_t)K->B * 4;
    if ((table_out != K->page_table && overlap(table_out, table, K->page_table, table)) ||
        (ref_out != K->ref && overlap(ref_out, ref, K->ref, ref)) ||
        overlap(table_out, table, K->ref, ref) || overlap(table_out, table, K->held, seqs) ||
        overlap(ref_out, ref, K->page_table, table) || overlap(ref_out, ref, K->held, seqs) ||
        overlap(table_out, table, ref_out, ref))
        return MOE_ERR_ARG;
    return cuda_status(pages::launch_compact(*K, table_out, ref_out, moves, counts, workspace,
                                             (cudaStream_t)stream));
}

moe_status moe_kv_copy_pages(const moe_cache_desc *C, void *k_pages, void *v_pages,
                             const int *moves, int n, const int *count, void *workspace,
                             moe_stream_t stream) {
    if (!cache_ok(C) || n < 0 || ((uintptr_t)workspace & 255u)) return MOE_ERR_ARG;
    if (n == 0) return MOE_OK;
    if (!k_pages || !v_pages || !aligned16(k_pages) || !aligned16(v_pages) || !moves)
        return MOE_ERR_ARG;
    const int e = (int)elem_size(C->dtype);
    if ((long long)C->page_size * C->H_kv * C->dh * e / 16 > 1 << 30) return MOE_ERR_UNSUPPORTED;
    pages::CopyArgs a{};
    a.kp = (char *)k_pages;
    a.vp = (char *)v_pages;
    a.moves = moves;
    a.count = count;
    a.n = n;
    a.page = C->page_size;
    a.n_pages = C->n_pages;
    a.heads = C->H_kv;
    a.row_bytes = C->dh * e;
    a.st_page = C->stride_page * e;
    a.st_tok = C->stride_tok * e;
    a.st_head = C->stride_head * e;
    a.flags = (int *)workspace;
    return cuda_status(pages::launch_copy(a, (cudaStream_t)stream));
}

}  // extern "C"
