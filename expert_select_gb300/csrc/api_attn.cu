// Entry points of the attention half of the block (see include/moetree.h): argument checks, the
// attention workspace's layout, and the launches.
#include <algorithm>
#include <cmath>

#include "attn.cuh"
#include "cache.cuh"

namespace moe {
namespace attn {

static size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Partial results: slots 0 and 1 of every CTA, for whichever kernel runs.
WsLayout ws_layout(int dh, long long rows_per_seq) {
    const size_t rows =
        std::max((size_t)kMaxCtas * std::min<long long>(kSimtRows, rows_per_seq),
                 (size_t)kTcMaxCtas * std::min<long long>(kTcRows, rows_per_seq));
    WsLayout w{};
    w.rec = kHeadBytes;
    w.ml = align256(w.rec + (size_t)kMaxCtas * 4 * sizeof(int));
    w.o = align256(w.ml + rows * 2 * 2 * sizeof(float));
    w.total = align256(w.o + rows * 2 * dh * sizeof(float));
    return w;
}

}  // namespace attn

namespace {

bool cache_ok(const moe_cache_desc *C) {
    if (!C || C->H_kv < 1 || C->H < C->H_kv || C->H % C->H_kv || C->H > 65536) return false;
    if (C->dh < 8 || C->dh % 8 || C->dh > 256) return false;
    if (C->dtype != MOE_DTYPE_F32 && C->dtype != MOE_DTYPE_BF16) return false;
    if (C->page_size < 1 || C->n_pages < 1 || C->max_pages < 1) return false;
    if ((long long)C->page_size * C->max_pages > (1ll << 30)) return false;
    for (long long st : {C->stride_page, C->stride_tok, C->stride_head})
        if (st < C->dh || st % 8 || st > (1ll << 36)) return false;
    if (C->window < 0 || C->sink_tokens < 0) return false;
    return C->scale > 0.f && std::isfinite(C->scale);
}

// Rows of a ragged or uniform block. N nodes of G heads each must fit an int.
bool block_ok(const moe_cache_desc *C, int B, int N, int R, const int *row_start) {
    if (B < 0 || N < 0 || R < 0) return false;
    if ((long long)N * (C->H / C->H_kv) > (1ll << 30)) return false;
    return row_start ? true : (long long)B * N == R;
}

// Whether the kernel for few rows takes a bf16 block. With up to 16 rows for a key/value head the
// work is reading the cache: on 1-64 sequences of 4k-60k slots it takes 12-166 us where the
// tcgen05 kernel takes 18-167 (1.0 to 1.7 times as long; 24 rows of 64 sequences: 108 against 72).
// With more rows it reads the cache once for every 16, but starts and ends sooner: up to 32 such
// blocks in all and 2^17 slots between them it is 1.03 to 1.6 times as fast (8 nodes of 8 heads,
// 4 key/value heads of 128: 2003 slots 14.5 against 21.0 us, 8003 slots 21.0 against 23.9, 16003
// slots 30.6 against 27.8; 4 sequences of 1003 slots, 64 blocks, 21.9 against 21.0). The lengths
// are not known here: the page table's capacity stands for them, so 8 nodes over 2003 slots
// with a table for 131072 take 20.7 us, not 14.4.
// With either kernel forced on 226 shapes of 24 to 264 rows, this one is never slower where the rule
// takes it, and the other is at least 5 % slower on 26 where the rule takes that: twelve without a
// window (up to 1.25 times: one sequence of 16-30k slots, some short ones of 500-1000), fourteen
// with a window of 128, where a limit of 32 blocks is too low (groups of 8 heads, 4 key/value
// heads of 128: 128 trees of 3 nodes 88.8 us against 45.9, of 5 nodes 90.5 against 66.4, of 8 92.8
// against 80.1; but of 16 nodes 97.9 against 155.8).
bool few_rows(const attn::Args &a) {
    const long long rows = (long long)a.N * a.G;
    if (rows <= attn::kFewRows) return true;
    const long long blocks = (long long)a.B * a.Hkv * ((rows + attn::kFewRows - 1) / attn::kFewRows);
    long long slots = a.cap;
    if (a.window > 0) slots = std::min(slots, (long long)a.window + a.sinks + a.N);
    return blocks <= 32 && blocks * slots <= 1 << 17;
}

// Do n bytes at p and m bytes at q share any?
bool overlap(const void *p, size_t n, const void *q, size_t m) {
    return p && q && (uintptr_t)p < (uintptr_t)q + m && (uintptr_t)q < (uintptr_t)p + n;
}
// Bytes from the first to the last of R rows of `width` elements, ld apart.
size_t span(int R, long long ld, int width, int dtype) {
    return ((size_t)(R - 1) * ld + width) * elem_size(dtype);
}

bool rows_ok(const void *p, long long ld, int width) {
    return p && aligned16(p) && ld >= width && ld % 8 == 0;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_attention_workspace_bytes(const moe_cache_desc *C, int B, int N) {
    if (!cache_ok(C) || B < 1 || N < 1) return 0;
    if ((long long)N * (C->H / C->H_kv) > (1ll << 30)) return 0;
    return attn::ws_layout(C->dh, (long long)N * (C->H / C->H_kv)).total;
}

moe_status moe_tree_attention(const moe_cache_desc *C, const void *q, long long ldq,
                              const void *k_pages, const void *v_pages, const int *page_table,
                              const int *cache_len, const int *row_start, const int *parent,
                              const float *sink_logit, int B, int N, int R, void *out, float *lse,
                              void *workspace, moe_stream_t stream) {
    if (!cache_ok(C) || !block_ok(C, B, N, R, row_start)) return MOE_ERR_ARG;
    if (B == 0 || N == 0 || R == 0) return MOE_OK;
    if (!rows_ok(q, ldq, C->H * C->dh) || !k_pages || !v_pages || !page_table || !cache_len ||
        !out || !workspace)
        return MOE_ERR_ARG;
    if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out) ||
        ((uintptr_t)workspace & 255u))
        return MOE_ERR_ARG;
    attn::Args a{};
    a.G = C->H / C->H_kv;
    // (sequence, block of rows) pairs are counted in an int
    if ((long long)B * (((long long)N * a.G + attn::kSimtRows - 1) / attn::kSimtRows) > (1 << 30))
        return MOE_ERR_UNSUPPORTED;
    // one CTA may still read q where another has written its rows
    const int row = C->H * C->dh;
    if (overlap(out, span(R, row, row, C->dtype), q, span(R, ldq, row, C->dtype)))
        return MOE_ERR_ARG;
    const attn::WsLayout w = attn::ws_layout(C->dh, (long long)N * a.G);
    a.q = q;
    a.ldq = ldq;
    a.k = k_pages;
    a.v = v_pages;
    a.table = page_table;
    a.cache_len = cache_len;
    a.row_start = row_start;
    a.parent = parent;
    a.sink = sink_logit;
    a.out = out;
    a.lse = lse;
    a.flags = at<int>(workspace, 0);
    a.rec = at<int>(workspace, w.rec);
    a.part_ml = at<float>(workspace, w.ml);
    a.part_o = at<float>(workspace, w.o);
    a.B = B;
    a.N = N;
    a.R = R;
    a.H = C->H;
    a.Hkv = C->H_kv;
    a.dh = C->dh;
    a.page = C->page_size;
    a.n_pages = C->n_pages;
    a.max_pages = C->max_pages;
    a.cap = C->page_size * C->max_pages;
    a.st_page = C->stride_page;
    a.st_tok = C->stride_tok;
    a.st_head = C->stride_head;
    a.window = C->window;
    a.sinks = C->sink_tokens;
    a.scale = C->scale;
    cudaStream_t s = (cudaStream_t)stream;
    if (!attn::tc_supported(a, C->dtype)) return cuda_status(attn::launch_simt(a, C->dtype, s));
    return cuda_status(few_rows(a) ? attn::launch_few(a, s) : attn::launch_tc(a, s));
}

moe_status moe_kv_append(const moe_cache_desc *C, const moe_rope_params *P, const void *q,
                         long long ldq, const void *k, long long ldk, const void *v, long long ldv,
                         void *k_pages, void *v_pages, const int *page_table,
                         const int *cache_len, const int *row_start, const int *depth, int B,
                         int N, int R, void *q_out, void *workspace, moe_stream_t stream) {
    if (!cache_ok(C) || !P || !block_ok(C, B, N, R, row_start)) return MOE_ERR_ARG;
    if (P->inv_freq && (P->rot_dim < 8 || P->rot_dim % 8 || P->rot_dim > C->dh ||
                        !std::isfinite(P->rope_scale)))
        return MOE_ERR_ARG;
    if (!(P->eps >= 0.f) || !std::isfinite(P->eps)) return MOE_ERR_ARG;
    if (B == 0 || N == 0 || R == 0) return MOE_OK;
    if (!q != !q_out || (q && (!rows_ok(q, ldq, C->H * C->dh) || !aligned16(q_out))))
        return MOE_ERR_ARG;
    if (q && q == q_out && ldq != (long long)C->H * C->dh) return MOE_ERR_ARG;
    if (!rows_ok(k, ldk, C->H_kv * C->dh) || !rows_ok(v, ldv, C->H_kv * C->dh) || !k_pages ||
        !v_pages || !aligned16(k_pages) || !aligned16(v_pages) || !page_table || !cache_len)
        return MOE_ERR_ARG;
    // rows are taken in no order: q_out may be q itself, row for row, and else nothing that is read
    const int qw = C->H * C->dh, kw = C->H_kv * C->dh;
    const size_t out_bytes = q ? span(R, qw, qw, C->dtype) : 0;
    if ((q != q_out && overlap(q_out, out_bytes, q, span(R, ldq, qw, C->dtype))) ||
        overlap(q_out, out_bytes, k, span(R, ldk, kw, C->dtype)) ||
        overlap(q_out, out_bytes, v, span(R, ldv, kw, C->dtype)))
        return MOE_ERR_ARG;
    if (!aligned16(P->q_weight) || !aligned16(P->k_weight) || ((uintptr_t)workspace & 255u))
        return MOE_ERR_ARG;
    cache::AppendArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.wq = P->q_weight;
    a.wk = P->k_weight;
    a.ldq = ldq;
    a.ldk = ldk;
    a.ldv = ldv;
    a.kp = k_pages;
    a.vp = v_pages;
    a.q_out = q_out;
    a.table = page_table;
    a.cache_len = cache_len;
    a.row_start = row_start;
    a.depth = depth;
    a.inv_freq = P->inv_freq;
    a.eps = P->eps;
    a.rope_scale = P->rope_scale;
    a.rot = P->inv_freq ? P->rot_dim : 0;
    a.flags = (int *)workspace;
    a.B = B;
    a.N = N;
    a.R = R;
    a.H = C->H;
    a.Hkv = C->H_kv;
    a.dh = C->dh;
    a.page = C->page_size;
    a.n_pages = C->n_pages;
    a.max_pages = C->max_pages;
    a.cap = C->page_size * C->max_pages;
    a.st_page = C->stride_page;
    a.st_tok = C->stride_tok;
    a.st_head = C->stride_head;
    return cuda_status(cache::launch_append(a, C->dtype, (cudaStream_t)stream));
}

moe_status moe_kv_commit(const moe_cache_desc *C, void *k_pages, void *v_pages,
                         const int *page_table, const int *cache_len, const int *path,
                         const int *n_accept, int B, int P, int *new_len, void *workspace,
                         moe_stream_t stream) {
    if (!cache_ok(C) || B < 0 || P < 0) return MOE_ERR_ARG;
    if (B == 0) return MOE_OK;
    if (!k_pages || !v_pages || !aligned16(k_pages) || !aligned16(v_pages) || !page_table ||
        !cache_len || (P > 0 && !path) || !n_accept || !new_len || ((uintptr_t)workspace & 255u))
        return MOE_ERR_ARG;
    const long long e = (long long)elem_size(C->dtype);
    cache::CommitArgs a{};
    a.kp = k_pages;
    a.vp = v_pages;
    a.table = page_table;
    a.cache_len = cache_len;
    a.path = path;
    a.n_accept = n_accept;
    a.new_len = new_len;
    a.flags = (int *)workspace;
    a.B = B;
    a.P = P;
    a.Hkv = C->H_kv;
    a.page = C->page_size;
    a.n_pages = C->n_pages;
    a.max_pages = C->max_pages;
    a.cap = C->page_size * C->max_pages;
    a.row_bytes = (int)(C->dh * e);
    a.st_page = C->stride_page * e;
    a.st_tok = C->stride_tok * e;
    a.st_head = C->stride_head * e;
    return cuda_status(cache::launch_commit(a, (cudaStream_t)stream));
}

moe_status moe_block_norm(const moe_layer_desc *L, const void *x, const void *branch,
                          const void *w_post, const void *gate, int gate_rows, float scale,
                          const void *w_pre, float eps, int R, void *h, void *hn,
                          moe_stream_t stream) {
    if (!desc_ok(L) || R < 0 || !(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(scale))
        return MOE_ERR_ARG;
    if (gate && gate_rows < 1) return MOE_ERR_ARG;
    if (R == 0) return MOE_OK;
    if (!x || (branch && !h) || (!h && !hn)) return MOE_ERR_ARG;
    if ((h && h == hn) || (!branch && (w_post || gate))) return MOE_ERR_ARG;
    for (const void *p : {x, branch, w_post, gate, w_pre, (const void *)h, (const void *)hn})
        if (!aligned16(p)) return MOE_ERR_ARG;
    // rows are taken in no order: an output may be an input row for row, else shares nothing
    const size_t all = span(R, L->d, L->d, L->dtype), row = span(1, 0, L->d, L->dtype);
    const size_t gates = gate ? row * (((size_t)R + gate_rows - 1) / gate_rows) : 0;
    auto over = [&](const void *o, const void *in, size_t n, bool by_rows) {
        return !(by_rows && o == in) && overlap(o, all, in, n);
    };
    for (const void *o : {(const void *)h, (const void *)hn})
        if (over(o, x, all, o == h || h != x) || over(o, branch, all, true) ||
            over(o, gate, gates, gate_rows == 1) || over(o, w_post, row, false) ||
            over(o, w_pre, row, false))
            return MOE_ERR_ARG;
    if (overlap(h, all, hn, all)) return MOE_ERR_ARG;
    return cuda_status(launch_block_norm(*L, x, branch, w_post, gate, gate_rows, scale, w_pre, eps,
                                         R, h, hn, (cudaStream_t)stream));
}

}  // extern "C"
