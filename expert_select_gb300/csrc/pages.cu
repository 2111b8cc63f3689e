// Upkeep of a cache's pages: sequences that end, grow and fork, and a pool that is compacted. The
// bookkeeping (which page belongs to whom) is apart from the copies of keys and values, as one table
// serves all layers and each layer has pools of its own.
//
// A page is free where its count of holders is 0; new pages are the free ones of the lowest numbers,
// in the order of the sequences, so results do not depend on the order of threads. Finding them is a
// scan over the counts (4 bytes a page), and the bookkeeping of a call waits for it, so a call is
// one cluster of CTAs: each scans its slice, the slices' sums meet in distributed shared memory, and
// the call's phases are cluster barriers instead of launches.
//
// Measured: the end, fork, growth and copies of 4 of 16 sequences 19.4 to 21 us (the host's: four calls of 3.5 to
// 5; 12 replayed from a graph), of 128 of 512 sequences 22.5; compaction 13 to 15 at 1k pages (8.4 from a graph)
// and 173 at 16k, of which the copies take 154, at the HBM's rate.
#include <cooperative_groups.h>

#include <algorithm>

#include "pages.cuh"

namespace moe {
namespace pages {

static size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

WsLayout ws_layout(const moe_page_book &K) {
    WsLayout w{};
    w.list = 4096;
    w.map = align256(w.list + (size_t)K.n_pages * 4);
    w.claim = align256(w.map + (size_t)K.n_pages * 4);
    w.off = align256(w.claim + (size_t)K.B * 4);
    w.total = align256(w.off + (size_t)K.B * 4);
    return w;
}

namespace {

namespace cg = cooperative_groups;

constexpr int kThr = 1024, kWarps = kThr / 32;
constexpr int kCluster = 8;

struct Book {
    int *table, *held, *len, *ref;
    int B, max_pages, n_pages, page;
    int *flags, *list, *map, *claim, *off;
};

__device__ __forceinline__ void flag(const Book &k, int bit) {
    if (k.flags) atomicOr(k.flags, bit);
}

// A sequence whose numbers fit the table: 0 <= held <= max_pages, 0 <= len <= held pages.
__device__ __forceinline__ bool sane(const Book &k, int held, int len) {
    return held >= 0 && held <= k.max_pages && len >= 0 && (long long)len <= (long long)held * k.page;
}

// A barrier of the call's CTAs. (A cluster's costs more than a CTA's even where it has one CTA.)
__device__ __forceinline__ void call_sync() {
    cg::cluster_group cl = cg::this_cluster();
    if (cl.num_blocks() > 1)
        cl.sync();
    else
        __syncthreads();
}

// Sums of the block's threads before this one (exclusive, in thread order) and of all.
template <typename T> __device__ __forceinline__ T block_scan(T v, T *part, T *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
    }
    __syncthreads();  // (part may still be read from the scan before)
    if (lane == 31) part[warp] = s;
    __syncthreads();
    if (warp == 0) {
        T p = part[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T t = __shfl_up_sync(0xffffffffu, p, o);
            if (lane >= o) p += t;
        }
        part[lane] = p;
    }
    __syncthreads();
    *total = part[kWarps - 1];
    return s - v + (warp ? part[warp - 1] : 0);
}

// The same of values up to `cap`, sums cut at it: the value before a thread is then at least what makes
// the sum with its own exceed cap - 1.
__device__ __forceinline__ int capped_scan(int v, int cap, int *part, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s = min(s + t, cap);
    }
    __syncthreads();
    if (lane == 31) part[warp] = s;
    __syncthreads();
    int p = part[lane], all = 0;  // (every warp scans the warps' sums itself)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, p, o);
        if (lane >= o) p = min(p + t, cap);
    }
    all = __shfl_sync(0xffffffffu, p, 31);
    const int before = __shfl_sync(0xffffffffu, p, max(warp - 1, 0));
    *total = all;
    return min((warp ? before : 0) + s, cap) - v;
}

// The same of a value of each warp, over the cluster's. `mine` is read by the other CTAs.
template <typename T>
__device__ __forceinline__ T cluster_scan(T v, T *part, T *mine, T *total) {
    cg::cluster_group cl = cg::this_cluster();
    const int ctas = cl.num_blocks(), rank = cl.block_rank(), lane = threadIdx.x & 31;
    T sum;
    const T at = __shfl_sync(0xffffffffu, block_scan(lane == 0 ? v : T(0), part, &sum), 0);
    if (ctas == 1) {
        *total = sum;
        return at;
    }
    if (threadIdx.x == 0) *mine = sum;
    cl.sync();
    // (a lane for each CTA: the reads do not wait for one another)
    T all = lane < ctas ? *cl.map_shared_rank(mine, lane) : T(0), base = lane < rank ? all : T(0);
#pragma unroll
    for (int o = kCluster / 2; o >= 1; o >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, o);
        base += __shfl_xor_sync(0xffffffffu, base, o);
    }
    cl.sync();  // (`mine` may be written again)
    *total = __shfl_sync(0xffffffffu, all, 0);
    return __shfl_sync(0xffffffffu, base, 0) + at;
}

// The cluster's warps share the pages [lo, hi) in contiguous runs, in order. Every warp gets the
// number of pages before its run for which `pick` holds; total: of all. Called by all threads.
constexpr int kDeep = 8;  // loads on their way
struct Run {
    int lo, hi, before, total;
    int v[kDeep];  // a lane's first pages
};
template <class Pick>
__device__ __forceinline__ Run cluster_count(const int *ref, int lo, int hi, int *part, int *mine,
                                             Pick pick) {
    cg::cluster_group cl = cg::this_cluster();
    const int ctas = cl.num_blocks(), rank = cl.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = max(0, hi - lo), warps = ctas * kWarps;
    // runs of whole 128-byte lines
    const int per = ((n + warps - 1) / warps + 31) / 32 * 32;
    const long long first = lo + (long long)(rank * kWarps + warp) * per;
    Run r;
    r.lo = (int)min((long long)max(lo, hi), first);
    r.hi = (int)min((long long)max(lo, hi), first + per);
    int c = 0;
#pragma unroll
    for (int q = 0; q < kDeep; ++q) r.v[q] = ref[max(0, min(r.lo + 32 * q + lane, r.hi - 1))];
#pragma unroll
    for (int q = 0; q < kDeep; ++q) {
        const int p = r.lo + 32 * q + lane;
        c += p < r.hi && pick(p, r.v[q]);
    }
#pragma unroll 8
    for (int p = r.lo + 32 * kDeep + lane; p < r.hi; p += 32) c += pick(p, ref[p]);
    r.before = cluster_scan(__reduce_add_sync(0xffffffffu, c), part, mine, &r.total);
    return r;
}

// Calls put(page, how many picked ones are before it) for the picked pages of the warp's run that have
// fewer than `want` before them.
template <class Pick, class Put>
__device__ __forceinline__ void cluster_emit(const int *ref, const Run &r, int want, Pick pick, Put put) {
    const int lane = threadIdx.x & 31;
    int at = r.before;
    int v[kDeep];
#pragma unroll
    for (int q = 0; q < kDeep; ++q) v[q] = r.v[q];
#pragma unroll 1
    for (int p0 = r.lo; p0 < r.hi && at < want; p0 += 32 * kDeep) {
        if (p0 > r.lo) {
#pragma unroll
            for (int q = 0; q < kDeep; ++q) v[q] = ref[min(p0 + 32 * q + lane, r.hi - 1)];
        }
#pragma unroll
        for (int q = 0; q < kDeep; ++q) {
            const int p = p0 + 32 * q + lane;
            const bool on = p < r.hi && pick(p, v[q]);
            const uint32_t m = __ballot_sync(0xffffffffu, on);
            const int i = at + __popc(m & ((1u << lane) - 1));
            if (on && i < want) put(p, i, v[q]);
            at += __popc(m);
        }
    }
}

__device__ __forceinline__ bool is_free(int, int ref) { return ref <= 0; }

__device__ __forceinline__ Run count_free(const Book &k, int *part, int *mine) {
    return cluster_count(k.ref, 0, k.n_pages, part, mine, is_free);
}
// The first `want` free pages, ascending: in `here` (of kSmall), where one CTA makes the call and
// wants no more, else in k.list. To be read after a call_sync.
constexpr int kSmall = 1024;
__device__ __forceinline__ const int *list_free(const Book &k, const Run &r, int want, int *here) {
    int *list = cg::this_cluster().num_blocks() == 1 && want <= kSmall ? here : k.list;
    cluster_emit(k.ref, r, want, is_free, [&](int p, int i, int) { list[i] = p; });
    return list;
}

// ------------------------------------------------------------------ free

// A CTA for each entry of the list. Lowering `held` is what takes the pages: of two entries that
// name one sequence each releases the pages between its own mark and the one it found. The tokens are
// cut before, so that the numbers fit at any time, for who reads them in the other order.
__global__ void __launch_bounds__(128) free_kernel(Book k, const int *seqs, const int *keep) {
    __shared__ int s_old;
    pdl_wait();
    const int b = seqs[blockIdx.x], left = keep ? keep[blockIdx.x] : 0;
    if (b < 0 || b >= k.B || left < 0) {
        if (threadIdx.x == 0) flag(k, attn::FLAG_BAD_SEQUENCE);
        return;
    }
    const long long want_ll = ((long long)left + k.page - 1) / k.page;
    const int want = (int)min(want_ll, (long long)k.max_pages);
    if (threadIdx.x == 0) {
        const volatile int *held = k.held + b, *len = k.len + b;
        // (side by side first; what looks wrong then may be another entry's work)
        int h = *held, l = *len;
        if (!sane(k, h, l)) {
            h = *held;
            __threadfence();
            l = *len;
        }
        s_old = 0;
        if (sane(k, h, l)) {
            if (l > left) atomicMin(&k.len[b], left);
            __threadfence();
            s_old = atomicMin(&k.held[b], want);
        } else {
            flag(k, attn::FLAG_BAD_SEQUENCE);
        }
    }
    __syncthreads();
    const int old = s_old;
    for (int j = want + threadIdx.x; j < old; j += blockDim.x) {
        const int p = k.table[(size_t)b * k.max_pages + j];
        if (p < 0 || p >= k.n_pages || atomicSub(&k.ref[p], 1) <= 0) {
            if (p >= 0 && p < k.n_pages) atomicAdd(&k.ref[p], 1);  // nobody held it: stays free
            flag(k, attn::FLAG_BAD_PAGE);
        }
    }
}

// ------------------------------------------------------------------ reserve

__global__ void __launch_bounds__(kThr) reserve_kernel(Book k, int N, const int *n_new) {
    __shared__ int part[kWarps], mine, here[kSmall];
    pdl_wait();
    const int rank = cg::this_cluster().block_rank(), ctas = cg::this_cluster().num_blocks();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // pages that a sequence lacks, up to one more than there are
    auto lacks = [&](int held, int len, int more, bool tell) {
        // (len and page_size are 2^30 at most)
        const unsigned want = ((unsigned)len + (unsigned)more + (unsigned)k.page - 1) / (unsigned)k.page;
        if (!sane(k, held, len) || more < 0 || want > (unsigned)k.max_pages) {
            if (tell) flag(k, attn::FLAG_BAD_SEQUENCE);
            return 0;
        }
        return min(max(0, (int)want - held), k.n_pages + 1);
    };
    // How many the sequences before it lack (sums are cut at n_pages + 1: what lies behind is not served
    // anyway): every CTA counts for itself. The loads of the last sequences are on their way beside those
    // of the free pages.
    const int cap = k.n_pages + 1;
    int total = 0, b0 = 0;
    for (; b0 + kThr < k.B; b0 += kThr) {
        const int b = b0 + threadIdx.x;
        const int need = lacks(k.held[b], k.len[b], n_new ? n_new[b] : N, rank == 0);
        int sum;
        const int at = capped_scan(need, cap, part, &sum);
        if (rank == 0) k.off[b] = min(total + at, cap);
        total = min(total + sum, cap);
    }
    const int b = b0 + threadIdx.x, held = b < k.B ? k.held[b] : 0, len = b < k.B ? k.len[b] : 0;
    const int more = n_new ? b < k.B ? n_new[b] : 0 : N;
    const Run r = count_free(k, part, &mine);
    const int need = b < k.B ? lacks(held, len, more, rank == 0) : 0;
    int sum;
    const int at = min(total + capped_scan(need, cap, part, &sum), cap);
    total = min(total + sum, cap);
    const int have = r.total, want = min(total, k.n_pages);
    if (want == 0) return;
    const int *list = list_free(k, r, want, here);
    call_sync();
    auto serve = [&](int seq, int first, int held_, int need_, int from, int step) {
        for (int j = from; j < need_; j += step) {
            const int p = list[first + j];
            k.table[(size_t)seq * k.max_pages + held_ + j] = p;
            k.ref[p] = 1;
        }
    };
    // The last sequences: a thread for each, and a warp for what it lacks where that is more than a few.
    // The CTAs take turns by warps.
    const bool mine_to_do = warp % ctas == rank;
    const bool met = at + need <= have;
    if (mine_to_do && need > 0) {
        if (!met) flag(k, FLAG_NO_PAGES);
        if (met) {
            if (need <= 8) serve(b, at, held, need, 0, 1);
            k.held[b] = held + need;
        }
    }
    if (mine_to_do) {
        uint32_t many = __ballot_sync(0xffffffffu, met && need > 8);
        for (; many; many &= many - 1) {
            const int l = __ffs(many) - 1;
            serve(b0 + warp * 32 + l, __shfl_sync(0xffffffffu, at, l), __shfl_sync(0xffffffffu, held, l),
                  __shfl_sync(0xffffffffu, need, l), lane, 32);
        }
    }
    // those before them, a warp for each
    for (int q = rank * kWarps + warp; q < b0; q += ctas * kWarps) {
        const int held_q = k.held[q], first = k.off[q];
        const int need_q = lacks(held_q, k.len[q], n_new ? n_new[q] : N, false);
        __syncwarp();  // (held is written below)
        if (need_q == 0) continue;
        if (first + need_q > have) {
            if (lane == 0) flag(k, FLAG_NO_PAGES);
            continue;
        }
        serve(q, first, held_q, need_q, lane, 32);
        if (lane == 0) k.held[q] = held_q + need_q;
    }
}

// ------------------------------------------------------------------ fork

constexpr int kForkCols = 256;  // table entries of a warp's piece
constexpr int kFewForks = 256;  // entries that every CTA keeps in shared memory

struct Fork {
    int src, dst, len;
    int at;  // number of its page among those that the call takes; -1: no fork
};

// One entry's piece of a table row: full pages are shared, what is behind them gets a page of its own.
__device__ __forceinline__ void fork_piece(const Book &k, const Fork &f, int i, int piece, int have,
                                           const int *list, int *moves) {
    const int lane = threadIdx.x & 31;
    const int full = f.at < 0 ? 0 : f.len / k.page, tail = f.at < 0 ? -1 : f.len - full * k.page;
    const bool short_of = tail > 0 && f.at >= have;
    if (tail < 0 || short_of) {
        if (piece == 0 && lane < 3) moves[3 * i + lane] = lane == 2 ? 0 : -1;
        if (piece == 0 && lane == 0 && short_of) flag(k, FLAG_NO_PAGES);
        return;
    }
    const int *from = k.table + (size_t)f.src * k.max_pages;
    int *to = k.table + (size_t)f.dst * k.max_pages;
    const int end = min(full, (piece + 1) * kForkCols);
    const int old = piece == 0 && lane == 0 && tail > 0 ? from[full] : -1;
#pragma unroll 4
    for (int j = piece * kForkCols + lane; j < end; j += 32) {
        const int p = from[j];
        to[j] = p;
        if (p >= 0 && p < k.n_pages)
            atomicAdd(&k.ref[p], 1);
        else
            flag(k, attn::FLAG_BAD_PAGE);
    }
    if (piece || lane) return;
    int fresh = -1;
    if (tail > 0) {
        fresh = list[f.at];
        to[full] = fresh;
        k.ref[fresh] = 1;
    }
    moves[3 * i] = old;
    moves[3 * i + 1] = fresh;
    moves[3 * i + 2] = tail;
    k.held[f.dst] = full + (tail > 0);
    k.len[f.dst] = f.len;
}

// FEW: up to kFewForks entries. Every CTA works all of them out for itself, a thread for each, from three
// loads that wait for one another (the entry, its sequences, the table), beside which the counts are read.
template <bool FEW>
__global__ void __launch_bounds__(kThr)
fork_kernel(Book k, const int *src, const int *dst, int n, int *moves) {
    __shared__ int part[kWarps], mine;
    __shared__ Fork forks[FEW ? kFewForks : 1];
    __shared__ int here[FEW ? kSmall : 1], counts[kWarps];
    pdl_wait();
    cg::cluster_group cl = cg::this_cluster();
    const int rank = cl.block_rank(), ctas = cl.num_blocks();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gt = rank * kThr + threadIdx.x;
    auto in = [&](int b) { return b >= 0 && b < k.B; };
    const int pieces = (k.max_pages + kForkCols - 1) / kForkCols;
    const long long items = (long long)n * pieces;
    if constexpr (FEW) {
        const int t = threadIdx.x;
        int a = -1, b = -1;
        if (t < n) {
            a = src[t];
            b = dst[t];
            forks[t].src = a;
            forks[t].dst = b;
        }
        const Run r = count_free(k, part, &mine);
        int tail = -1;
        if (t < n && in(a) && in(b)) {
            const int held = k.held[a], len = k.len[a], empty = k.held[b];
            // the first entry that names a sequence as its target has it; a target is no source
            bool ok = true;
#pragma unroll 8
            for (int j = 0; j < n; ++j) {
                const int other = forks[j].dst;
                ok = ok && other != a && (j >= t || other != b);
            }
            if (ok && empty == 0 && sane(k, held, len)) {
                tail = len % k.page;
                forks[t].len = len;
            }
        }
        if (t < n && tail < 0 && rank == 0) flag(k, attn::FLAG_BAD_SEQUENCE);
        // entries that need a page, and how many do before each
        const uint32_t needs = __ballot_sync(0xffffffffu, tail > 0);
        if (lane == 0) counts[warp] = __popc(needs);
        __syncthreads();
        const int c = counts[lane];
        const int total = __reduce_add_sync(0xffffffffu, c);
        const int before = __reduce_add_sync(0xffffffffu, lane < warp ? c : 0);
        if (t < n) forks[t].at = tail < 0 ? -1 : before + __popc(needs & ((1u << lane) - 1));
        const int *list = list_free(k, r, min(total, k.n_pages), here);
        call_sync();
        for (long long it = rank * kWarps + warp; it < items; it += ctas * kWarps) {
            const int i = (int)(it / pieces), piece = (int)(it - (long long)i * pieces);
            fork_piece(k, forks[i], i, piece, r.total, list, moves);
        }
    } else {
        for (int i = gt; i < n; i += ctas * kThr) {
            if (in(src[i])) k.claim[src[i]] = n;
            if (in(dst[i])) k.claim[dst[i]] = n;
        }
        call_sync();
        for (int i = gt; i < n; i += ctas * kThr)
            if (in(dst[i])) atomicMin(&k.claim[dst[i]], i);
        call_sync();
        // An entry without its `at`. (A target is never a source, so what is read here of a source is not
        // written by the call.)
        auto entry = [&](int i) {
            Fork f{src[i], dst[i], 0, -1};
            if (!in(f.src) || !in(f.dst) || k.claim[f.dst] != i || k.claim[f.src] != n) return f;
            if (!sane(k, k.held[f.src], k.len[f.src])) return f;
            f.len = k.len[f.src];
            f.at = 0;
            return f;
        };
        int total = 0;
        for (int i0 = 0; i0 < n; i0 += kThr) {
            const int i = i0 + threadIdx.x;
            int tail = -1;
            if (i < n) {
                const Fork f = entry(i);
                if (f.at == 0 && k.held[f.dst] == 0) tail = f.len % k.page;
                if (tail < 0 && rank == 0) flag(k, attn::FLAG_BAD_SEQUENCE);
            }
            int sum;
            const int at = block_scan((int)(tail > 0), part, &sum);
            if (rank == 0 && i < n) k.off[i] = tail < 0 ? -1 : total + at;
            total += sum;
        }
        const Run r = count_free(k, part, &mine);
        cluster_emit(k.ref, r, min(total, k.n_pages), is_free, [&](int p, int i, int) { k.list[i] = p; });
        call_sync();
        for (long long it = rank * kWarps + warp; it < items; it += ctas * kWarps) {
            const int i = (int)(it / pieces), piece = (int)(it - (long long)i * pieces);
            const int at = k.off[i];
            Fork f{-1, -1, 0, -1};
            if (at >= 0) {
                f = entry(i);
                f.at = at;
            }
            fork_piece(k, f, i, piece, r.total, k.list, moves);
        }
    }
}

// ------------------------------------------------------------------ compact

// The table with its pages' new numbers: entries `first`, `first` + `step`, ..
template <typename I>
__device__ __forceinline__ void remap(const Book &k, int *table_out, I all, I first, I step) {
    for (I i = first; i < all; i += step) {
        const int b = (int)(i / (I)k.max_pages), j = (int)(i - (I)b * (I)k.max_pages);
        int p = k.table[i];
        const int held = k.held[b];
        if (j == 0 && (held < 0 || held > k.max_pages)) flag(k, attn::FLAG_BAD_SEQUENCE);
        if (j < held) {
            const int to = p >= 0 && p < k.n_pages ? k.map[p] : -1;
            if (to >= 0)
                p = to;
            else
                flag(k, attn::FLAG_BAD_PAGE);
        }
        table_out[i] = p;
    }
}

// entries: of the table, where the cluster renames them itself; else 0, and remap_kernel does.
__global__ void __launch_bounds__(kThr)
compact_kernel(Book k, int *table_out, int *ref_out, int *moves, int *counts, unsigned entries) {
    __shared__ int part[kWarps], mine;
    __shared__ long long pairs[kWarps], my_pair;
    pdl_wait();
    cg::cluster_group cl = cg::this_cluster();
    const int lane = threadIdx.x & 31, n = k.n_pages;
    auto is_used = [](int, int ref) { return ref > 0; };
    Run r = cluster_count(k.ref, 0, n, part, &mine, is_used);
    const int n_used = r.total;
    auto is_hole = [&](int p, int ref) { return p < n_used && ref <= 0; };
    auto is_high = [&](int p, int ref) { return p >= n_used && ref > 0; };
    // The run's holes below n_used and pages in use above it; what stays or is free is written at once.
    // (ref_out may be ref: a free page's count becomes 0, others' change behind the next barrier)
    int holes = 0, high = 0;
    auto look = [&](int p, int ref) {
        holes += is_hole(p, ref);
        high += is_high(p, ref);
        if (is_high(p, ref)) return;
        k.map[p] = ref > 0 ? p : -1;
        if (ref > 0 || p >= n_used) ref_out[p] = max(ref, 0);
    };
#pragma unroll
    for (int q = 0; q < kDeep; ++q) {
        const int p = r.lo + 32 * q + lane;
        if (p < r.hi) look(p, r.v[q]);
    }
#pragma unroll 4
    for (int p = r.lo + 32 * kDeep + lane; p < r.hi; p += 32) look(p, k.ref[p]);
    long long total;
    const long long before = cluster_scan((long long)__reduce_add_sync(0xffffffffu, high) << 32 |
                                              __reduce_add_sync(0xffffffffu, holes),
                                          pairs, &my_pair, &total);
    r.before = (int)(before & 0xffffffff);
    cluster_emit(k.ref, r, n, is_hole, [&](int p, int i, int) { k.list[i] = p; });
    call_sync();
    // pages at n_used and above go to the holes, in order
    r.before = (int)(before >> 32);
    cluster_emit(k.ref, r, n, is_high, [&](int p, int i, int ref) {
        const int to = k.list[i];
        k.map[p] = to;
        ref_out[to] = ref;
        ref_out[p] = 0;
        moves[3 * (size_t)i] = p;
        moves[3 * (size_t)i + 1] = to;
        moves[3 * (size_t)i + 2] = k.page;
    });
    if (cl.block_rank() == 0 && threadIdx.x == 0) {
        counts[0] = (int)(total >> 32);
        counts[1] = n_used;
    }
    if (entries) {
        call_sync();
        remap<unsigned>(k, table_out, entries, cl.block_rank() * kThr + threadIdx.x, cl.num_blocks() * kThr);
    }
}

__global__ void __launch_bounds__(256) remap_kernel(Book k, int *table_out) {
    pdl_wait();
    remap<long long>(k, table_out, (long long)k.B * k.max_pages, blockIdx.x * 256ll + threadIdx.x,
                     gridDim.x * 256ll);
}

// ------------------------------------------------------------------ copy

constexpr int kCopyThr = 256, kCopyVecs = 4;  // 16-byte vectors a thread holds
constexpr int kCopyPart = kCopyThr * kCopyVecs;

// A page is `rows` runs of consecutive bytes: one, where heads and tokens lie densely token by
// token; one a head, where a head's tokens do; else one a token and head. Work is cut into parts of
// kCopyPart vectors of one page and pool.
__global__ void __launch_bounds__(kCopyThr) copy_kernel(const CopyArgs a) {
    pdl_wait();
    const int n = a.count ? min(max(*a.count, 0), a.n) : a.n;
    const int vecs = a.row_bytes / 16, page_vecs = a.page * a.heads * vecs;
    const int parts = (page_vecs + kCopyPart - 1) / kCopyPart;
    const long long items = 2ll * n * parts;
    const bool by_token = a.st_head == a.row_bytes && a.st_tok == (long long)a.heads * a.row_bytes;
    const bool by_head = a.st_tok == a.row_bytes;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int part = (int)(it % parts), m = (int)(it / parts / 2);
        char *pool = (it / parts) & 1 ? a.vp : a.kp;
        const int src = a.moves[3 * (size_t)m], dst = a.moves[3 * (size_t)m + 1];
        const int tokens = a.moves[3 * (size_t)m + 2];
        if (tokens <= 0 || src == dst) continue;
        if (src < 0 || src >= a.n_pages || dst < 0 || dst >= a.n_pages || tokens > a.page) {
            if (a.flags && threadIdx.x == 0) atomicOr(a.flags, attn::FLAG_BAD_PAGE);
            continue;
        }
        const char *from = pool + src * a.st_page;
        char *to = pool + dst * a.st_page;
        const int all = tokens * a.heads * vecs;
        uint4 v[kCopyVecs];
        long long at[kCopyVecs];
#pragma unroll
        for (int q = 0; q < kCopyVecs; ++q) {
            const int i = part * kCopyPart + q * kCopyThr + threadIdx.x;
            at[q] = -1;
            if (i >= all) continue;
            if (by_token) {
                at[q] = 16ll * i;
            } else if (by_head) {
                const int run = tokens * vecs, h = i / run;
                at[q] = h * a.st_head + 16ll * (i - h * run);
            } else {
                const int row = i / vecs, t = row / a.heads;
                at[q] = t * a.st_tok + (row - t * a.heads) * a.st_head + 16ll * (i - row * vecs);
            }
            v[q] = *reinterpret_cast<const uint4 *>(from + at[q]);
        }
#pragma unroll
        for (int q = 0; q < kCopyVecs; ++q)
            if (at[q] >= 0) *reinterpret_cast<uint4 *>(to + at[q]) = v[q];
    }
}

Book book(const moe_page_book &K, void *ws) {
    const WsLayout w = ws_layout(K);
    Book k{};
    k.table = K.page_table;
    k.held = K.held;
    k.len = K.cache_len;
    k.ref = K.ref;
    k.B = K.B;
    k.max_pages = K.max_pages;
    k.n_pages = K.n_pages;
    k.page = K.page_size;
    k.flags = at<int>(ws, 0);
    k.list = at<int>(ws, w.list);
    k.map = at<int>(ws, w.map);
    k.claim = at<int>(ws, w.claim);
    k.off = at<int>(ws, w.off);
    return k;
}

// One cluster: of one CTA where the scan is short (its barriers are the CTA's own then).
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), bool wide, cudaStream_t s, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(wide ? kCluster : 1);
    cfg.blockDim = dim3(kThr);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = wide ? kCluster : 1;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// us by one CTA and by eight: reserving 2000 pages 3.4, 4.9; 8000: 3.6, 5.0; 16000: 4.8, 4.9; 25000: 6.7, 4.9; 65000:
// 11, 5.1; 32 forks 4.7, 6.1; 4.7, 6.1; 5.8, 6.4; 6.9, 6.6; 8.9, 6.6; plans of compaction 6.3, 8.9; 7.1, 9.1; 11, 10;
// 19, 11; 47, 14 (12000: 10.7, 9.6; from 8192 on a warp's pages are more than its registers hold).
constexpr int kWidePages = 16384, kWidePlan = 8192;
constexpr int kWideEntries = 32768;  // of a fork's tables

}  // namespace

cudaError_t launch_free(const moe_page_book &K, const int *seqs, const int *keep, int n, void *ws,
                        cudaStream_t s) {
    return launch_pdl(free_kernel, dim3(n), dim3(128), 0, s, book(K, ws), seqs, keep);
}

cudaError_t launch_reserve(const moe_page_book &K, int N, const int *n_new, void *ws,
                           cudaStream_t s) {
    return launch_cluster(reserve_kernel, K.n_pages > kWidePages, s, book(K, ws), N, n_new);
}

cudaError_t launch_fork(const moe_page_book &K, const int *src, const int *dst, int n, int *moves,
                        void *ws, cudaStream_t s) {
    const bool wide = K.n_pages > kWidePages || (long long)n * K.max_pages > kWideEntries;
    return launch_cluster(n <= kFewForks ? fork_kernel<true> : fork_kernel<false>, wide, s, book(K, ws), src,
                          dst, n, moves);
}

cudaError_t launch_compact(const moe_page_book &K, int *table_out, int *ref_out, int *moves,
                           int *counts, void *ws, cudaStream_t s) {
    const Book k = book(K, ws);
    const bool wide = K.n_pages > kWidePlan;
    const long long all = (long long)K.B * K.max_pages;
    // A few entries a thread cost less than a launch.
    const bool here = all <= 8ll * kThr * (wide ? kCluster : 1);
    const cudaError_t err = launch_cluster(compact_kernel, wide, s, k, table_out, ref_out, moves, counts,
                                           here ? (unsigned)all : 0u);
    if (err != cudaSuccess || here) return err;
    const int ctas = (int)std::min<long long>((all + 255) / 256, 8ll * std::max(1, device_sms()));
    return launch_pdl(remap_kernel, dim3(ctas), dim3(256), 0, s, k, table_out);
}

cudaError_t launch_copy(const CopyArgs &a, cudaStream_t s) {
    const long long parts =
        ((long long)a.page * a.heads * (a.row_bytes / 16) + kCopyPart - 1) / kCopyPart;
    const int ctas =
        (int)std::min<long long>(2 * parts * a.n, 8ll * std::max(1, device_sms()));
    return launch_pdl(copy_kernel, dim3(ctas), dim3(kCopyThr), 0, s, a);
}

}  // namespace pages
}  // namespace moe
