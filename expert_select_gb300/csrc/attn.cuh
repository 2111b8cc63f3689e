// Shared parts of the paged-attention kernels: arguments, the visibility rule, the division
// of the work over the CTAs of one launch, and the layout of the partial results.
//
// Sequence b has cache_len[b] committed tokens in cache slots 0 .. len - 1 (slot = position)
// and n new nodes in slots len .. len + n - 1. The query heads of one key/value head share
// its keys, so the rows of a work item are (node, head in group) pairs: row q of a sequence
// and key/value head h is node q / G, query head h G + q % G.
//
// The work of a launch is a list of items, one per (sequence, block of rows, key/value head),
// each a number of key tiles. All tiles of all items, in this order, are divided into equal
// ranges, one per CTA, whatever items they belong to: lengths that differ between the
// sequences of a batch, causal chunks and single long sequences all keep every SM busy to the
// end. An item inside one range is finished by its CTA; an item that a range boundary cuts
// leaves unnormalised partial results (O, running maximum, sum) that attn_combine merges.
// The lengths live in device memory, so every CTA finds its range by itself (attn_plan) and
// the launch has the same shape whatever they are (it can be captured into a graph).
#pragma once

#include "common.cuh"

namespace moe {
namespace attn {

constexpr int kMaxCtas = 640;         // CTAs of an attention launch at most
constexpr size_t kHeadBytes = 4096;   // head of the workspace: the check word (zeroed by the caller)
constexpr float kLog2e = 1.4426950408889634f;

// Bits of the check word, beside those of the layer calls.
enum : int { FLAG_BAD_PAGE = 4, FLAG_BAD_SEQUENCE = 8 };

struct Args {
    const void *q;
    long long ldq;
    const void *k, *v;
    const int *table, *cache_len, *row_start, *parent;
    const float *sink;
    void *out;
    float *lse;
    int *flags;      // check word
    int *rec;        // [kMaxCtas][4]: items that were cut (see attn_combine)
    float *part_o;   // [CTAs][2][prows][dh]
    float *part_ml;  // [CTAs][2][prows][2]
    int B, N, R, H, Hkv, G, dh;
    int page, n_pages, max_pages, cap;  // cap: cache slots of a sequence (max_pages * page)
    long long st_page, st_tok, st_head;
    int window, sinks;
    float scale;
    int rows;        // rows of an item (of the launched kernel)
    int prows;       // rows of a partial result: min(rows, N G)
    int qblocks;     // blocks of `rows` rows that N nodes take
    int min_units;   // units of work of a CTA's range at least (a tile's weight or more)
    int fixed;       // units that an item costs beside its tiles
    int whole;       // units up to which an item is not cut
};

struct Seq {
    int len, n, row0;  // committed tokens, new nodes, first row of q
    int L;             // cache slots in use: len + n, at most cap
};

// Sizes that contradict one another are cut to what the buffers hold.
__device__ __forceinline__ Seq sequence(const Args &a, int b, int *bad = nullptr) {
    Seq s;
    int n, r0;
    if (a.row_start) {
        r0 = a.row_start[b];
        n = a.row_start[b + 1] - r0;
        if (r0 < 0 || n < 0 || n > a.N || r0 > a.R - n) {
            if (bad) *bad = 1;
            n = r0 < 0 ? 0 : min(min(n, a.N), a.R - r0);
            if (n < 0) n = 0;
        }
    } else {
        r0 = b * a.N;
        n = a.N;
    }
    int len = a.cache_len[b];
    if (len < 0 || len > a.cap - n) {
        if (bad) *bad = 1;
        len = max(0, min(len, a.cap));
    }
    s.len = len;
    s.n = n;
    s.row0 = r0;
    s.L = min(len + n, a.cap);
    return s;
}

// The key tiles of rows [q0, q1) (q1 > q0) of a sequence: ns tiles from slot 0 (first tokens that
// stay visible), then the tiles from w0 on; nt in all.
struct Tiles {
    int ns, w0, nt;
    __device__ __forceinline__ int at(int t) const { return t < ns ? t : w0 + (t - ns); }
};
template <int BN>
__device__ __forceinline__ Tiles tiles_of(const Args &a, const Seq &s, int q0, int q1) {
    const int i0 = q0 / a.G, i1 = (q1 - 1) / a.G;
    const int kend = a.parent ? s.L : min(s.L, s.len + i1 + 1);
    Tiles t;
    t.ns = t.w0 = 0;
    const int all = (kend + BN - 1) / BN;
    if (a.window > 0) {
        // the oldest slot a window can reach (tree nodes may all be at the root's depth); at most the
        // last one: where lengths are cut to the table, rows past its end may see nothing, and an
        // item without tiles would not write their zeros
        const int lo = min(max(0, s.len + (a.parent ? 0 : i0) - a.window + 1), kend - 1);
        t.w0 = lo / BN;
        t.ns = min((int)(((long long)a.sinks + BN - 1) / BN), t.w0);
    }
    t.nt = t.ns + all - t.w0;
    return t;
}

// Tiles of an entry's items, and the weight of one. HEAVY: rows from which a tile costs the
// tensor-core kernel 4 units of work instead of 3 (1.0 us for two 128-row tiles, which share the
// copies of K and V, against 0.75 us for one); 0: every tile is one unit.
template <int BN, int HEAVY>
__device__ __forceinline__ int entry_tiles(const Args &a, int e, int *w, int *bad = nullptr) {
    const int b = e / a.qblocks, q0 = (e - b * a.qblocks) * a.rows;
    const Seq s = sequence(a, b, bad);
    const int rows = s.n * a.G;
    *w = HEAVY ? 3 : 1;
    if (q0 >= rows) return 0;
    const int q1 = min(rows, q0 + a.rows);
    if (HEAVY && q1 - q0 >= HEAVY) *w = 4;
    return tiles_of<BN>(a, s, q0, q1).nt;
}

// A CTA's range of work, from `off` units into the item (entry e, key/value head h), where entry
// e = sequence * qblocks + block of rows. An item of nt tiles of weight w has a.fixed + nt w units:
// the first a.fixed are what it costs beside its tiles (see attn_plan), then w for each tile. A
// tile belongs to one CTA: a boundary at unit u of the item lies before tile
// floor((u - a.fixed) / w), for the range that ends there and for the one that begins.
struct Range {
    int e, h;
    long long off;   // the range's first unit within the item
    long long left;  // units from there to the range's end
    int parts;       // if the item's second part begins this range: the parts of the item; else 0
};

// Block-wide exclusive sum of `v` (and the total), over kWarps warps; scratch: kWarps long longs.
template <int kWarps>
__device__ __forceinline__ long long block_scan(long long v, long long *scratch, long long *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp) before += scratch[i];
        all += scratch[i];
    }
    *total = all;
    return before + inc - v;
}

// Finds the CTA's range (block-wide; every thread gets it). scratch: 34 long longs of shared
// memory. Each thread sums a run of entries and a block scan places the runs; the threads whose
// runs hold the range's boundaries look them up.
//
// A piece of an item costs a CTA several tiles' time beside its tiles (query rows, the pipeline's
// start and end, the output, and a partial result that the combine has to read). So an item counts
// a.fixed units beside its tiles (64 trees over contexts of 0.2-8k tokens: without, the CTAs with
// the short sequences took 1.3 times the mean), and two rules keep pieces few:
//  - where every item can have round(item / quota) CTAs of its own, it gets them, in equal parts,
//    and a CTA has one piece (a few long items: one tree of 65 nodes over 4k tokens took 31 us so
//    and 38 us with ranges that cross items);
//  - else, ranges of equal length, but a boundary inside an item of at most a.whole units moves to
//    the item's start.
template <int BN, int HEAVY, int kThreads>
__device__ __forceinline__ Range attn_plan(const Args &a, int cta, int n_ctas, long long *scratch) {
    const int tid = threadIdx.x;
    constexpr int kWarps = kThreads / 32;
    static_assert(2 * kWarps <= 28, "scratch holds two sums per warp and the result");
    const int E = a.B * a.qblocks;
    const int per = (E + kThreads - 1) / kThreads;
    const int e0 = min(E, tid * per), e1 = min(E, e0 + per);
    long long sum = 0;
    int bad = 0, w = 1, nt = 0;
    for (int e = e0; e < e1; ++e) {
        nt = entry_tiles<BN, HEAVY>(a, e, &w, &bad);
        sum += nt > 0 ? a.Hkv * ((long long)nt * w + a.fixed) : 0;
    }
    if (bad) atomicOr(a.flags, FLAG_BAD_SEQUENCE);
    int *found = reinterpret_cast<int *>(scratch + 28);
    if (tid == 0) found[8] = 0;
    long long total;
    const long long run = block_scan<kWarps>(sum, scratch, &total);  // the run's first unit
    // (64-bit divisions take hundreds of cycles: only where the numbers need them)
    const bool small = total < (1ll << 30);
    const long long quota =
        max((long long)a.min_units, small ? (long long)(((unsigned)total + n_ctas - 1) / (unsigned)n_ctas)
                                          : (total + n_ctas - 1) / n_ctas);
    // scratch[28 ..]: the item, the offset in it, how far the two boundaries moved back, parts
    if (per == 1 && small) {
        const unsigned item = (unsigned)nt * w + a.fixed;
        const int k = min(max(1, (int)((item + quota / 2) / (unsigned)quota)), nt);  // CTAs per item
        long long ctas;
        const long long first = block_scan<kWarps>((long long)a.Hkv * k, scratch + 14, &ctas);
        if (ctas <= n_ctas) {
            if (cta >= first && cta < first + (long long)a.Hkv * k) {
                const int local = cta - (int)first, h = local / k, j = local - h * k;
                const int t0 = (int)((long long)nt * j / k), t1 = (int)((long long)nt * (j + 1) / k);
                found[0] = tid;
                found[1] = h;
                const long long u0 = t0 > 0 ? a.fixed + (long long)t0 * w : 0;
                scratch[29] = u0;
                scratch[30] = a.fixed + (long long)t1 * w - u0;
                found[8] = j == 1 ? k : 0;
            }
            __syncthreads();
            Range r{0, 0, 0, 0, 0};
            if (cta < ctas) r = {found[0], found[1], scratch[29], scratch[30], found[8]};
            return r;
        }
    }
    const long long start = quota * cta, end = start + quota;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const long long u = which ? end : start;
        if (u >= total || u < run || u >= run + sum) continue;
        long long at = run;
        for (int e = e0; e < e1; ++e) {
            if (per > 1) nt = entry_tiles<BN, HEAVY>(a, e, &w);
            const long long item = (long long)nt * w + a.fixed, all = nt > 0 ? a.Hkv * item : 0;
            if (u < at + all) {
                const long long off = u - at;
                const long long h = small ? (long long)((unsigned)off / (unsigned)item) : off / item;
                const long long in = off - h * item;
                if (which) {
                    scratch[31] = item <= a.whole ? in : 0;
                } else {
                    found[0] = e;
                    found[1] = (int)h;
                    scratch[29] = item <= a.whole ? 0 : in;
                    scratch[30] = item <= a.whole ? in : 0;
                    // the first boundary inside an item that leaves tiles before it
                    const int one = a.fixed + w;
                    if (item > a.whole && in >= one && in - quota < one)
                        found[8] = 1 + (int)((item - in + quota - 1) / quota);
                }
                break;
            }
            at += all;
        }
    }
    __syncthreads();
    Range r{0, 0, 0, 0, 0};
    if (start < total)
        r = {found[0], found[1], scratch[29],
             (end < total ? end - scratch[31] : total) - (start - scratch[30]), found[8]};
    return r;
}

// One piece of an item: its tiles t .. t + count - 1 of nt.
struct Segment {
    Seq s;
    Tiles tl;
    int e = -1;          // entry: the fields up to rows belong to it
    int b, h, q0, rows;  // rows [q0, q0 + rows) of the sequence
    int t, count;
    bool whole;
};

// The next segment of a range (false: none is left). Moves the range past it.
template <int BN, int HEAVY>
__device__ __forceinline__ bool next_segment(const Args &a, Range &r, Segment &g) {
    while (r.left > 0) {
        if (g.e != r.e) {  // (the next key/value head of an entry has the same rows and tiles)
            g.e = r.e;
            g.b = r.e / a.qblocks;
            g.q0 = (r.e - g.b * a.qblocks) * a.rows;
            g.s = sequence(a, g.b);
            g.rows = min(a.rows, g.s.n * a.G - g.q0);
            g.tl.nt = 0;
            if (g.rows > 0) g.tl = tiles_of<BN>(a, g.s, g.q0, g.q0 + g.rows);
        }
        if (g.tl.nt == 0) {
            // (past a sequence's rows all of its blocks are empty: in a batch of prompt chunks and
            // single tokens most sequences have one block of many)
            r.e = g.rows <= 0 ? (g.b + 1) * a.qblocks : r.e + 1;
            r.h = 0;
            r.off = 0;
            continue;
        }
        const bool heavy = HEAVY && g.rows >= HEAVY;
        const long long item = (long long)g.tl.nt * (HEAVY ? (heavy ? 4 : 3) : 1) + a.fixed;
        const long long end = min(item, r.off + r.left);
        auto tile = [&](long long unit) {  // tiles before a unit (items have < 2^32 units)
            const unsigned u = (unsigned)max(0ll, unit - a.fixed);
            return HEAVY ? (int)(heavy ? u / 4u : u / 3u) : (int)u;
        };
        g.h = r.h;
        g.t = tile(r.off);
        g.count = tile(end) - g.t;
        g.whole = g.t == 0 && g.count == g.tl.nt;
        r.left -= end - r.off;
        r.off = 0;
        if (end == item && ++r.h == a.Hkv) {
            r.h = 0;
            ++r.e;
        }
        if (g.count > 0) return true;
    }
    return false;
}

// A cut item leaves its partial result in slot 0 of a CTA whose range begins inside it and in
// slot 1 of the CTA whose range holds its first tile.
__device__ __forceinline__ size_t part_row(const Args &a, int cta, const Segment &g, int row) {
    return ((size_t)cta * 2 + (g.t == 0 ? 1 : 0)) * a.prows + row;
}

// Record for attn_combine: the item whose second part begins this CTA's range, and its parts.
__device__ __forceinline__ void write_record(const Args &a, int cta, const Range &r) {
    int *rec = a.rec + cta * 4;
    rec[0] = r.e;
    rec[1] = r.h;
    rec[2] = r.left > 0 ? r.parts : 0;
}

// Bits of visible slots among [k0, k0 + 32) for the query node `node`, at position pos.
// Chains: slots up to the node's own, in the window or among the first tokens. Trees: the
// committed slots and the node's ancestors, found by walking up its parents (each step goes to
// a lower node: a parent outside [0, node) is the top).
__device__ __forceinline__ uint32_t range_bits(int lo, int hi, int k0) {  // slots [lo, hi)
    const int x0 = max(lo - k0, 0), x1 = min(hi - k0, 32);
    if (x1 <= x0) return 0u;
    return (x1 == 32 ? 0xffffffffu : (1u << x1) - 1u) & ~((1u << x0) - 1u);
}
template <int WORDS>
__device__ __forceinline__ void visible_bits(const Args &a, const Seq &s, int node, int pos, int k0,
                                             uint32_t (&bits)[WORDS]) {
    const int hi = a.parent ? min(s.len, s.L) : min(pos + 1, s.L);
    const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
#pragma unroll
    for (int w = 0; w < WORDS; ++w) {
        const int kw = k0 + 32 * w;
        bits[w] = range_bits(lo, hi, kw);
        if (a.window > 0) bits[w] |= range_bits(0, min(a.sinks, hi), kw);
    }
    if (a.parent && k0 + 32 * WORDS > s.len) {
        int p = pos;
        for (int m = node; m >= 0 && s.len + m >= k0; --p) {
            const int j = s.len + m - k0;
            const bool in = a.window <= 0 || pos - p < a.window || p < a.sinks;
            if (in && j < 32 * WORDS && s.len + m < s.L) {
#pragma unroll
                for (int w = 0; w < WORDS; ++w)
                    if ((j >> 5) == w) bits[w] |= 1u << (j & 31);
            }
            const int up = a.parent[s.row0 + m];
            m = up < m ? up : -1;
        }
    }
}

// A node's position: its depth in the tree is only needed (and only walked) for a window.
__device__ __forceinline__ int node_position(const Args &a, const Seq &s, int node) {
    if (!a.parent) return s.len + node;
    int d = 0;
    if (a.window > 0) {
        for (int m = node;; ++d) {
            const int up = a.parent[s.row0 + m];
            if (up < 0 || up >= m) break;
            m = up;
        }
    }
    return s.len + d;
}

// May a row of nodes i0 .. i1 not see some of the BN slots from k0? (Never false wrongly.)
template <int BN>
__device__ __forceinline__ bool tile_masked(const Args &a, const Seq &s, int i0, int i1, int k0) {
    const int first_hidden = a.parent ? min(s.len, s.L) : min(s.len + i0 + 1, s.L);
    if (k0 + BN > first_hidden) return true;
    if (a.window <= 0) return false;
    const int max_pos = s.len + (a.parent ? s.n - 1 : i1);
    return k0 < max_pos - a.window + 1 && k0 + BN > a.sinks;
}

// No row of the sequence sees slots a .. b: older than every window (nodes' positions are s.len or
// later) and behind the first tokens. Their table entries may hold anything: a cache with a window
// gives such pages back.
__device__ __forceinline__ bool out_of_reach(const Args &a, const Seq &s, int from, int to) {
    return a.window > 0 && from >= a.sinks && to <= s.len - a.window;
}

// The page of slot j, or -1 if the table's entry is outside the pool.
__device__ __forceinline__ int page_of(const Args &a, int b, int j) {
    const int pg = a.table[(size_t)b * a.max_pages + j / a.page];
    return pg >= 0 && pg < a.n_pages ? pg : -1;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&t);
}

// The tensor-core kernels raise a row's running maximum only when it grows by more than this
// (log2): until then the unnormalised p is at most 2^8, which bf16 and the fp32 sums hold as well
// as values up to 1, and O needs no rescaling. The maximum a row ends with is a scale factor that
// the division by the sum takes out again.
constexpr float kRaise = 8.f;

// Factor that normalises an accumulated O, and the log of the denominator, from the running
// maximum m (base-2 logits) and sum l, with the head's sink logit (natural log units).
__device__ __forceinline__ float finish(float m, float l, const float *sink, int head, float *lse) {
    float mm = l > 0.f ? m : -INFINITY;
    float den = l;
    float f = 1.f;
    if (sink) {
        const float s2 = sink[head] * kLog2e;
        const float top = fmaxf(mm, s2);
        if (top > -INFINITY) {
            f = l > 0.f ? exp2f(mm - top) : 0.f;
            den = l * f + exp2f(s2 - top);
            mm = top;
        }
    }
    *lse = den > 0.f ? (mm + log2f(den)) * 0.6931471805599453f : (den == den ? -INFINITY : den);
    return den == 0.f ? 0.f : f / den;
}

template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

cudaError_t launch_simt(Args a, int dtype, cudaStream_t s);
cudaError_t launch_combine(const Args &a, int dtype, int n_ctas, cudaStream_t s);
cudaError_t launch_tc(Args a, cudaStream_t s);
cudaError_t launch_few(Args a, cudaStream_t s);
bool tc_supported(const Args &a, int dtype);
// rows of an item, and CTAs of the tensor-core kernel at most (one per SM)
constexpr int kSimtRows = 32, kTcRows = 256, kTcMaxCtas = 160, kFewRows = 16;

struct WsLayout {
    size_t rec, ml, o, total;
};
WsLayout ws_layout(int dh, long long rows_per_seq);  // rows_per_seq = N G

}  // namespace attn
}  // namespace moe
