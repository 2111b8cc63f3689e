// Paged attention on the 5th-generation tensor cores: bf16, head size up to 128.
//
//   S = Q K^T (fp32, tensor memory),  P = 2^(c S - m) (bf16, tensor memory),  O += P V
//
// in one pass over the keys with a running maximum m and sum l per row (c = scale log2 e). An
// item is 256 rows (node, head in group) of one key/value head: a prompt chunk or a large tree
// fills both 128-row tiles, which then share every K and V tile ("two tiles"); where an item has
// at most 128 rows (16 nodes of a group of 8 heads; the last 8 rows of 65 such nodes) its one tile
// is computed over even key tiles by one half of the CTA and over odd ones by the other, and the
// halves are merged at the end ("one tile"). Either way two independent score tiles are in flight: while
// the tensor cores work for one, the CUDA cores exponentiate the other.
//
// One CTA per SM, 416 threads:
//   warps 0, 3   TMA producers of K and of V: tiles of 64 slots, each through a ring of stages;
//                a tile is gathered as boxes of gcd(page size, 64) slots, their pages looked up
//                a tile ahead (with 16-slot pages one warp spent 1.7 us on a tile's 16 copies)
//   warps 1, 12  MMA issuers of slots 0 and 1 (warp 1 also allocates TMEM)
//   warp 2       looks after V: clears what no row may see (see below)
//   warps 4-7, 8-11  softmax of slot 0 and slot 1: a thread per row, its 64 scores in registers
// (With 13 warps a thread has at most 128 registers; all are used, and 44-56 bytes spilled. Twelve
// warps would allow 168. The 13th, an issuing warp for each slot, took the 64 trees below from 523 to
// 502 us when it came and left the chunks as they were.)
//
// TMEM (512 columns): two buffers of S for each of slots 0 and 1 (64 columns each; P overwrites the
// first 32 of its S), O of slots 0 and 1 (128 each). With two buffers S of the next tile is there
// when a softmax warp is done with one: with one buffer of 128 keys each slot's chain S, softmax,
// P V took 2.1 us for 128 keys of both slots, twice the tensor cores' time. The second product
// reads P from tensor memory and V from shared memory as it was loaded (MN-major), so P never
// passes through shared memory.
//
// Measured (32 query and 4 key/value heads of 128, bf16): two chunks of 4096 tokens over 28k cached
// ones 3.3 ms, 1.2 PFLOP/s; there a tile pair takes 1750 cycles, where its products need 1090 at
// the nominal rate, and the SM clock falls from 2.0 to 1.66 GHz under the load (power). 64 trees of
// 65 nodes over 0.2-8k tokens 0.42 ms: 65 nodes of 8 heads are 520 rows, three items that each read
// the sequence's K and V (1.6 GB from HBM for 0.55 GB of cache), and a piece of an item costs
// about 10 us beside its tiles (query rows, the pipeline's start and end, the output). That fixed
// cost is most of what a window leaves: 4096 tokens over 4003 with a window of 128 (64/8 heads of
// 64) 140 us for 11 us of bytes, 64 trees of 65 nodes so 223 us for 14.
//
// A masked score is -inf, so its P is 0; but 0 x V is NaN where V is infinite or NaN. In tiles
// that hold masked slots (the last ones, and a window's first) warp 2 therefore clears the rows of
// V past the sequence's end and the non-finite elements of the others before the second product;
// rows that do see such an element get it back at the end (a slow path that only runs then).
//
// Every wait is bounded: after 2 s it sets the check bit and the CTA drains and leaves.
#include <limits.h>

#include <algorithm>

#include "attn.cuh"
#include "tmem.cuh"

namespace moe {
namespace attn {
namespace {

using namespace tc;

constexpr int kBN = 64;
constexpr int kThreads = 416;
constexpr int kHeavy = 129;      // rows from which an item has two tiles
constexpr int kMaxStages = 8;    // of K and of V each
constexpr int kCtlBytes = 2048;

struct Params {
    Args a;
    CUtensorMap kmap, vmap;
    int box;  // slots of a TMA box: gcd(page size, 64)
};

// Control block in shared memory. A parity tells only neighbouring phases of a barrier apart, so
// whoever waits must know the phase before to be over. K and V stages have barriers of their own
// and one producer each for that, and the two S buffers too: S of tile u + 2 comes after P V of
// tile u, so P V of tile u - 1 (the other buffer) may be outstanding when S of tile u is there.
// And each slot has a query barrier of its own, used only in pieces where the slot has tiles: the
// next such piece's rows are loaded after the slot's products of this one. (A barrier that both
// slots waited for in every piece could be two phases on before the issuing warp of a slot without
// tiles looked at it: in pieces of one key tile and at most 128 rows nothing else waits for that
// warp until the stages of K or V run out.)
struct Ctl {
    uint64_t kfull[kMaxStages], kempty[kMaxStages], vfull[kMaxStages], vempty[kMaxStages],
        vready[kMaxStages], s_full[2][2], p_full[2][2], pv_done[2][2], q_full[2], done[2];
    long long scratch[34];
    uint32_t tmem;
    volatile int abort;
    volatile int bad_page;  // a tile of this CTA had a page outside the pool
    volatile int bad_v;     // a masked tile of this CTA had non-finite V
    float ml[2][128];       // slot 1's maximum and sum, for the merge
};
static_assert(sizeof(Ctl) <= kCtlBytes, "control block");

__device__ __forceinline__ void softmax_bar() {  // the 256 threads of warps 4-11
    __syncwarp();
    asm volatile("bar.sync 1, 256;" ::: "memory");
}

// Position of a tile in the ring of K (or V) stages: counts up over the CTA's segments.
template <int NS> struct Slot {
    static __device__ __forceinline__ int stage(uint32_t pos) { return (int)(pos % NS); }
    static __device__ __forceinline__ uint32_t parity(uint32_t pos) { return (pos / NS) & 1u; }
};

// Adds the non-finite elements of V that a row sees to its O (slow; only where a masked tile held
// some, which took no part in the products).
__device__ __forceinline__ void give_back(const Args &a, const Segment &g, int node, int pos, int n,
                                       int chunks, uint32_t tO) {
    for (int x = 0; x < chunks; ++x) {
        uint32_t o[32];
        tmem_ld32(tO + x * 32u, o);
        for (int t = 0; t < n; ++t) {
            const int k0 = g.tl.at(g.t + t) * kBN;
            uint32_t bits[2];
            visible_bits<2>(a, g.s, node, pos, k0, bits);
#pragma unroll 1
            for (int j = 0; j < kBN; ++j) {
                const uint32_t wb = j < 32 ? bits[0] : bits[1];
                if (!((wb >> (j & 31)) & 1u)) continue;
                const int pg = page_of(a, g.b, k0 + j);
                if (pg < 0) continue;
                const __nv_bfloat16 *vr = (const __nv_bfloat16 *)a.v + (size_t)pg * a.st_page +
                                          (size_t)((k0 + j) % a.page) * a.st_tok +
                                          (size_t)g.h * a.st_head;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (x * 32 + i < a.dh) {
                        const float e = __bfloat162float(vr[x * 32 + i]);
                        const float v = __uint_as_float(o[i]);
                        if (!isfinite(e)) o[i] = __float_as_uint(isfinite(v) ? e : v + e);
                    }
            }
        }
        __syncwarp();
        tmem_st32(tO + x * 32u, o);
        tmem_wait_st();
    }
}

// Stages of K and of V each that fit beside the query tiles.
template <int DC> constexpr int stages() {
    return std::min(kMaxStages, (227 * 1024 - 1024 - kCtlBytes - 2 * DC * 16384) / (2 * DC * 8192));
}

template <int DC>  // 64-column chunks of the head size
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    Ctl &c = *reinterpret_cast<Ctl *>(gbase);
    constexpr uint32_t kTile = DC * 16384u;  // 128 query rows x 64 DC bf16
    constexpr uint32_t kKv = DC * 8192u;     // 64 slots x 64 DC bf16
    constexpr int NS = stages<DC>();
    using Ring = Slot<NS>;
    const uint32_t sQ = base + kCtlBytes, sK = sQ + 2 * kTile, sV = sK + NS * kKv;
    uint8_t *gQ = gbase + kCtlBytes, *gV = gQ + 2 * kTile + NS * kKv;
    const Args &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto bar = [&](uint64_t &b) { return smem_u32(&b); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(bar(c.kfull[s]), 1);
            mbar_init(bar(c.kempty[s]), 2);
            mbar_init(bar(c.vfull[s]), 1);
            mbar_init(bar(c.vempty[s]), 2);
            mbar_init(bar(c.vready[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            for (int x = 0; x < 2; ++x) {
                mbar_init(bar(c.s_full[i][x]), 1);
                mbar_init(bar(c.p_full[i][x]), 4);  // a lane of each warp
                mbar_init(bar(c.pv_done[i][x]), 1);
            }
            mbar_init(bar(c.q_full[i]), 8);  // a lane of each softmax warp
            mbar_init(bar(c.done[i]), 1);
        }
        c.abort = c.bad_page = c.bad_v = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&p.kmap);
        prefetch_map(&p.vmap);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_u32(&c.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    const uint32_t tmem = c.tmem;
    Range r = attn_plan<kBN, kHeavy, kThreads>(a, blockIdx.x, gridDim.x, c.scratch);
    if (threadIdx.x == 64) write_record(a, blockIdx.x, r);

    uint32_t issued = 0, last_par = 0;  // producer: stages with a load issued, parity of the last
    bool mma_issued = false;

    if (warp == 0 || warp == 3) {
        // -------------------------------------- producers: warp 0 of K, warp 3 of V
        const bool is_k = warp == 0;
        const CUtensorMap *map = is_k ? &p.kmap : &p.vmap;
        uint64_t *full = is_k ? c.kfull : c.vfull, *empty = is_k ? c.kempty : c.vempty;
        uint32_t rp = 0;
        bool ok = true;
        Segment g;
        while (ok && next_segment<kBN, kHeavy>(a, r, g)) {
            const int n = __shfl_sync(0xffffffffu, g.count, 0);
            // Pages of 64 boxes (one tile of single-slot boxes, 64 tiles of 64-slot ones), two a
            // lane; the next 64 boxes' are on their way while these are used. A box out of every
            // row's reach is not copied (its stage keeps what it held: those scores are masked, and
            // the keeper clears those rows of V).
            const int per_tile = kBN / p.box, in_use = (g.s.L + p.box - 1) / p.box;  // boxes
            int first = -1, in_page = 0;  // box of pg[0] of lane 0; slot in its page of the next box
            // boxes gone0 .. gone0 + gone - 1 are wholly out of reach (see out_of_reach)
            const int shift = __ffs(p.box) - 1;
            const int gone0 = (int)(((long long)a.sinks + p.box - 1) >> shift);
            const unsigned gone = a.window > 0 ? max(0, ((g.s.len - a.window + 1) >> shift) - gone0) : 0;
            auto needed = [&](int bx) { return bx < in_use && (unsigned)(bx - gone0) >= gone; };
            int pg[2], next[2];
            uint32_t good[2], there[2];
            auto look_up = [&](int from, int (&out)[2]) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int bx = from + lane + 32 * i;
                    out[i] = needed(bx) ? a.table[(size_t)g.b * a.max_pages + bx * p.box / a.page] : -1;
                }
            };
            auto take = [&](int from) {  // makes `next` current and looks further ahead
                first = from;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    pg[i] = next[i];
                    good[i] = __ballot_sync(0xffffffffu, pg[i] >= 0 && pg[i] < a.n_pages);
                    there[i] = __ballot_sync(0xffffffffu, needed(from + lane + 32 * i));
                }
                look_up(from + 64, next);
                if (good[0] != there[0] || good[1] != there[1]) {
                    if (lane == 0) {
                        c.bad_page = 1;
                        __threadfence_block();
                        atomicOr(a.flags, FLAG_BAD_PAGE);
                    }
                    __syncwarp();
                }
            };
            int box0 = -1;
            for (int t = 0; ok && t < n; ++t, ++rp) {
                const int bx = g.tl.at(g.t + t) * per_tile;
                const int st = Ring::stage(rp);
                if (bx != box0 || t == 0) in_page = bx * p.box % a.page;  // the tiles' first, or a jump
                box0 = bx + per_tile;
                if (t == 0 || bx < first || bx >= first + 128) {
                    look_up(bx, next);
                    take(bx);
                } else if (bx >= first + 64) {
                    take(first + 64);
                }
                const uint64_t ok64 = (((uint64_t)good[1] << 32) | good[0]) >> (bx - first);
                const uint64_t mask = per_tile == 64 ? ~0ull : (1ull << per_tile) - 1ull;
                const uint64_t todo = ok64 & mask;
                ok = mbar_wait(bar(empty[st]), Ring::parity(rp) ^ 1u, &c.abort, a.flags);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint32_t fb = bar(full[st]);
                if (lane == 0) mbar_expect_tx(fb, (uint32_t)__popcll(todo) * p.box * 128u * DC);
                __syncwarp();
                uint32_t dst = (is_k ? sK : sV) + (uint32_t)st * kKv;
                const int boxes = min(per_tile, in_use - bx);
                auto copy = [&](int page, int in) {
#pragma unroll
                    for (int h = 0; h < DC; ++h)
                        tma_load_4d_elect(dst + h * 8192u, map, h * 64, in, g.h, page, fb);
                };
                if (boxes == 4 && todo == 15ull) {
                    // 16-slot pages: four copies without a loop's bookkeeping (64 blocks of 16
                    // nodes over 4k tokens: 208 -> 198 us)
                    const int i = bx - first, src = i < 32 ? pg[0] : pg[1];
                    int page[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) page[x] = __shfl_sync(0xffffffffu, src, (i + x) & 31);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        copy(page[x], in_page);
                        dst += p.box * 128u;
                        in_page += p.box;
                        if (in_page >= a.page) in_page = 0;
                    }
                } else {
                    for (int x = 0; x < boxes; ++x) {
                        const int i = bx - first + x;
                        const int page = __shfl_sync(0xffffffffu, i < 32 ? pg[0] : pg[1], i & 31);
                        if ((todo >> x) & 1ull) copy(page, in_page);
                        dst += p.box * 128u;
                        in_page += p.box;
                        if (in_page >= a.page) in_page = 0;
                    }
                }
                issued |= 1u << st;
                last_par = (last_par & ~(1u << st)) | (Ring::parity(rp) << st);
            }
        }
        __syncwarp();
    } else if (warp == 1 || warp == 12) {
        // ----------------------------------------------------------- MMA issuer
        const uint32_t id_s = idesc_bf16(128, kBN), id_o = idesc_bf16(128, 64 * DC) | kIdescBMn;
        // A slot's products are issued by a warp of its own: what bounds a tile's time is this
        // warp's chain of waits and issues, not the products. (One warp for both slots took 2060
        // cycles for a pair of tiles whose products need 1090 at the nominal rate; votes and
        // divisions by the ring's length at every wait had made it 2400.) So stages and parities are
        // counted, and the waits' verdicts are looked at once a tile.
        const int slot = warp == 1 ? 0 : 1;
        uint32_t kst = 0, kph = 0, vst = 0, vph = 0, qph = 0;
        uint32_t u0 = 0;  // tiles of the slot before the segment
        bool ok = true;
        auto wait = [&](uint64_t &b, uint32_t par) {
            ok &= mbar_wait(bar(b), par, &c.abort, a.flags);
        };
        auto all_ok = [&]() { return __all_sync(0xffffffffu, ok) != 0; };
        const uint32_t k_lo = sw128_lo(sK, 16), v_lo = sw128_lo(sV, 8192);
        const uint32_t tS = tmem + slot * 128u, tO = tmem + 256u + slot * 128u;
        Segment g;
        while (all_ok() && next_segment<kBN, kHeavy>(a, r, g)) {
            const bool two = __shfl_sync(0xffffffffu, g.rows, 0) > 128;
            const int n = __shfl_sync(0xffffffffu, g.count, 0);
            const uint32_t q_lo = sw128_lo(sQ + (two ? (uint32_t)slot * kTile : 0u), 16);
            // u: the slot's tile count; its S buffer is u & 1, the buffer's use u >> 1
            auto score = [&](uint32_t u) {  // S from the current K stage
                const uint32_t k = k_lo + kst * (kKv >> 4), d = tS + (u & 1u) * 64u;
#pragma unroll
                for (int x = 0; x < 4 * DC; ++x)
                    mma_ss_elect(d, q_lo + (((x >> 2) * 16384u + (x & 3) * 32u) >> 4),
                                 k + (((x >> 2) * 8192u + (x & 3) * 32u) >> 4), id_s, x != 0);
                commit_elect(bar(c.s_full[slot][u & 1u]));
            };
            auto wait_k = [&]() {
                wait(c.kfull[kst], kph);
                __syncwarp();
                tc_fence_after();
            };
            // A stage is free when both issuing warps have passed it; a tile that is not this slot's
            // is passed at once (after its copy has landed: an arrival must not count for an
            // earlier use of the stage).
            auto free_k = [&](bool mine) {
                if (mine)
                    commit_elect(bar(c.kempty[kst]));
                else if (lane == 0)
                    mbar_arrive(bar(c.kempty[kst]));
                if (++kst == NS) {
                    kst = 0;
                    kph ^= 1u;
                }
            };
            auto free_v = [&](bool mine) {
                if (mine)
                    commit_elect(bar(c.vempty[vst]));
                else if (lane == 0)
                    mbar_arrive(bar(c.vempty[vst]));
                if (++vst == NS) {
                    vst = 0;
                    vph ^= 1u;
                }
            };
            auto output = [&](uint32_t u, bool first) {  // O += P V, current V stage
                wait(c.p_full[slot][u & 1u], (u >> 1) & 1u);
                __syncwarp();
                tc_fence_after();
                const uint32_t v = v_lo + vst * (kKv >> 4), pt = tS + (u & 1u) * 64u;
#pragma unroll
                for (int x = 0; x < kBN / 16; ++x)
                    mma_ts_elect(tO, pt + x * 8u, v + x * (2048u >> 4), id_o, !first || x != 0);
                commit_elect(bar(c.pv_done[slot][u & 1u]));
            };
            if (two || n > slot) {  // the slot has tiles
                wait(c.q_full[slot], qph);
                qph ^= 1u;
                __syncwarp();
                tc_fence_after();
                mma_issued = true;
            }
            // with two row tiles each slot takes every key tile, else the slots take them in turn;
            // S runs two of the slot's tiles ahead of P V
            const int ahead = two ? 2 : 4, sh = two ? 0 : 1;
            auto mine = [&](int t) { return two || (t & 1) == slot; };
            for (int t = 0; t < min(n, ahead); ++t) {
                wait_k();
                if (mine(t)) score(u0 + (t >> sh));
                free_k(mine(t));
            }
            for (int t = 0; t < n; ++t) {
                wait(c.vready[vst], vph);
                if (mine(t)) output(u0 + (t >> sh), t <= sh);
                __syncwarp();
                free_v(mine(t));
                if (t + ahead < n) {
                    wait_k();
                    if (mine(t)) score(u0 + (t >> sh) + 2);
                    free_k(mine(t));
                }
                if (!all_ok()) break;
            }
            u0 += two ? n : (n + 1 - slot) / 2;
        }
        __syncwarp();
    } else if (warp == 2) {
        // -------------------------------------------------------- keeper of V
        uint32_t rp = 0;
        bool ok = true;
        Segment g;
        while (ok && next_segment<kBN, kHeavy>(a, r, g)) {
            const int n = g.count;
            const int i0 = g.q0 / a.G, i1 = (g.q0 + g.rows - 1) / a.G;
            const int pos = i0 == i1 ? node_position(a, g.s, i0) : 0;
            for (int t = 0; ok && t < n; ++t, ++rp) {
                const int st = Ring::stage(rp);
                ok = __all_sync(0xffffffffu, mbar_wait(bar(c.vfull[st]), Ring::parity(rp), &c.abort,
                                                       a.flags));
                if (!ok) break;
                const int k0 = g.tl.at(g.t + t) * kBN;
                if (c.bad_page || tile_masked<kBN>(a, g.s, i0, i1, k0)) {
                    // rows that no query of the item sees are cleared whole: with one node all
                    // that it does not see, else what lies past the end, is out of every row's
                    // reach or has no page
                    uint32_t bits[2];
                    if (i0 == i1) {
                        visible_bits<2>(a, g.s, i0, pos, k0, bits);
                    } else {
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            const int kw = k0 + 32 * w;
                            bits[w] = range_bits(0, g.s.L, kw);
                            if (a.window > 0)
                                bits[w] &= ~range_bits(a.sinks, g.s.len - a.window + 1, kw);
                        }
                    }
                    uint8_t *tile = gV + (size_t)st * kKv;
#pragma unroll 1
                    for (int w = 0; w < 2; ++w) {
                        const int row = 32 * w + lane;
                        bool keep = (bits[w] >> lane) & 1u;
                        if (keep && c.bad_page) keep = page_of(a, g.b, k0 + row) >= 0;
                        if (keep && i0 == i1) continue;
#pragma unroll 1
                        for (int h = 0; h < DC; ++h)
#pragma unroll
                            for (int x = 0; x < 8; ++x) {
                                uint4 *q = reinterpret_cast<uint4 *>(tile + h * 8192 + row * 128 +
                                                                     ((x ^ (row & 7)) << 4));
                                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                                if (keep) {
                                    v = *q;
                                    uint32_t *e = reinterpret_cast<uint32_t *>(&v);
                                    bool bad = false;
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        if ((e[i] & 0x7f80u) == 0x7f80u) {
                                            e[i] &= 0xffff0000u;
                                            bad = true;
                                        }
                                        if ((e[i] & 0x7f800000u) == 0x7f800000u) {
                                            e[i] &= 0xffffu;
                                            bad = true;
                                        }
                                    }
                                    if (!bad) continue;
                                    c.bad_v = 1;
                                }
                                *q = v;
                            }
                    }
                    __threadfence_block();
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(bar(c.vready[st]));
            }
        }
    } else {
        // -------------------------------------------------------------- softmax
        // A failed wait leaves `dead` set: the thread then runs through its loops without
        // computing or storing, so that the barriers stay matched.
        const int slot = (warp - 4) >> 2, quad = warp & 3;
        const int trow = quad * 32 + lane;  // row of the slot's tile
        const int tid = threadIdx.x - 128;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t tO = tmem + 256u + slot * 128u + lanes;
        uint32_t u = 0;  // tiles of the slot so far
        bool dead = false;
        Segment g;
        while (next_segment<kBN, kHeavy>(a, r, g)) {
            const bool two = g.rows > 128;
            const int n = g.count;
            softmax_bar();  // the last segment's tiles and exchange buffer are done with
            {
                // 8 DC pieces of 16 B a row; a thread keeps its piece and takes every
                // (256 / (8 DC))th row, up to sixteen rows' loads in flight at a time
                constexpr int kStep = 256 / (8 * DC);
                const int rows = two ? 256 : 128, ch = tid % (8 * DC), first = tid / (8 * DC);
                const __nv_bfloat16 *q = (const __nv_bfloat16 *)a.q + (size_t)g.s.row0 * a.ldq +
                                         (size_t)g.h * a.G * a.dh + ch * 8;
                const int dn = kStep / a.G, dg = kStep - dn * a.G;  // a step in nodes and heads
                int node = (g.q0 + first) / a.G, hd = g.q0 + first - node * a.G;
                for (int y = first; y < rows; y += 16 * kStep) {
                    uint4 v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        v[i] = make_uint4(0u, 0u, 0u, 0u);
                        if (y + i * kStep < g.rows && ch * 8 < a.dh)
                            v[i] = __ldg(reinterpret_cast<const uint4 *>(
                                q + (size_t)node * a.ldq + (size_t)hd * a.dh));
                        node += dn;
                        hd += dg;
                        if (hd >= a.G) {
                            hd -= a.G;
                            ++node;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int row = y + i * kStep, rr = row & 127;
                        if (row < rows)
                            *reinterpret_cast<uint4 *>(gQ + (row >> 7) * kTile + (ch >> 3) * 16384 +
                                                       rr * 128 + (((ch & 7) ^ (rr & 7)) << 4)) =
                                v[i];
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(c.q_full[0]));
                    if (two || n > 1) mbar_arrive(bar(c.q_full[1]));
                }
            }
            const int row = two ? slot * 128 + trow : trow;  // row of the item
            const bool active = row - lane < g.rows;         // the warp has rows
            const int rr = min(row, g.rows - 1);
            const int node = (g.q0 + rr) / a.G;
            const int pos = node_position(a, g.s, node);
            const int s0 = two ? slot * 128 : 0;
            const int i0 = (g.q0 + min(s0, g.rows - 1)) / a.G,
                      i1 = (g.q0 + min(s0 + 127, g.rows - 1)) / a.G;
            const float cs = a.scale * kLog2e;
            float m = -INFINITY, l = 0.f;
            int tiles = 0;
            for (int t = two ? 0 : slot; t < n; t += two ? 1 : 2, ++tiles, ++u) {
                const int k0 = g.tl.at(g.t + t) * kBN;
                const uint32_t tS = tmem + slot * 128u + (u & 1u) * 64u + lanes;
                if (!mbar_wait(bar(c.s_full[slot][u & 1u]), (u >> 1) & 1u, &c.abort, a.flags))
                    dead = true;
                tc_fence_after();
                if (active && !__any_sync(0xffffffffu, dead)) {
                    uint32_t s[kBN];
                    tmem_ld64(tS, s);
                    if (tile_masked<kBN>(a, g.s, i0, i1, k0) || c.bad_page) {
                        uint32_t bits[2];
                        visible_bits<2>(a, g.s, node, pos, k0, bits);
                        if (c.bad_page) {
#pragma unroll
                            for (int w = 0; w < 2; ++w)
                                for (int x = 0; x < 32; ++x)
                                    if (((bits[w] >> x) & 1u) && page_of(a, g.b, k0 + 32 * w + x) < 0)
                                        bits[w] &= ~(1u << x);
                        }
#pragma unroll
                        for (int w = 0; w < 2; ++w)
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                if (!((bits[w] >> x) & 1u)) s[32 * w + x] = 0xff800000u;  // -inf
                    }
                    float mx[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mx[i] = fmaxf(__uint_as_float(s[i]), __uint_as_float(s[i + 4]));
#pragma unroll
                    for (int i = 8; i < kBN; i += 8)
#pragma unroll
                        for (int x = 0; x < 4; ++x)  // three-operand maxima
                            mx[x] = fmaxf(fmaxf(mx[x], __uint_as_float(s[i + x])),
                                          __uint_as_float(s[i + x + 4]));
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    const bool raise = (top - m) * cs > kRaise;  // m = -inf: yes, unless top is too
                    if (__any_sync(0xffffffffu, raise)) {
                        const float mn = fmaxf(m, top);
                        const float f = m == -INFINITY ? 0.f : ex2((m - mn) * cs);
                        m = mn;
                        l *= f;
                        if (tiles > 0) {
                            // S runs ahead: the last tile's product may still be adding to O
                            if (!mbar_wait(bar(c.pv_done[slot][(u - 1) & 1u]), ((u - 1) >> 1) & 1u,
                                           &c.abort, a.flags))
                                dead = true;
                            __syncwarp();
                            tc_fence_after();
#pragma unroll 1
                            for (int x = 0; x < 2 * DC; ++x) {
                                uint32_t o[32];
                                tmem_ld32(tO + x * 32u, o);
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                tmem_st32(tO + x * 32u, o);
                            }
                        }
                    }
                    const float sub = m == -INFINITY ? 0.f : -m * cs;
                    const uint64_t cs2 = pack2(cs, cs), sub2 = pack2(sub, sub);
                    uint64_t sum[2] = {0ull, 0ull};
                    uint32_t pk[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float2 e = unpack2(fma2(
                            pack2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), cs2,
                            sub2));
                        const float p0 = ex2(e.x), p1 = ex2(e.y);
                        sum[i & 1] = add2(sum[i & 1], pack2(p0, p1));
                        pk[i] = pack_bf16(p0, p1);
                    }
                    tmem_st32(tS, pk);
                    tmem_wait_st();
                    const float2 st = unpack2(add2(sum[0], sum[1]));
                    l += st.x + st.y;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(c.p_full[slot][u & 1u]));
            }
            if (tiles > 0 && !mbar_wait(bar(c.pv_done[slot][(u - 1) & 1u]), ((u - 1) >> 1) & 1u,
                                        &c.abort, a.flags))
                dead = true;
            tc_fence_after();
            const bool live = !__any_sync(0xffffffffu, dead);
            // one tile: slot 1 hands its part over through the query tiles' shared memory, a block
            // of 32 columns x 32 rows per warp
            float *xch = reinterpret_cast<float *>(gQ);
            const bool merge = !two && n > 1;
            if (merge) {
                softmax_bar();  // slot 0's last scores have read Q too
                if (slot == 1) {
                    c.ml[0][trow] = m;
                    c.ml[1][trow] = l;
                    if (active && live) {
#pragma unroll 1
                        for (int x = 0; x < 2 * DC; ++x) {
                            uint32_t o[32];
                            tmem_ld32(tO + x * 32u, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                xch[(x * 4 + quad) * 1024 + i * 32 + lane] = __uint_as_float(o[i]);
                        }
                    }
                }
                softmax_bar();
            }
            if (!active || !live || (!two && slot == 1)) {
                tc_fence_before();
                continue;
            }
            float f0 = 1.f, f1 = 0.f;
            if (merge) {
                const float m1 = c.ml[0][trow], l1 = c.ml[1][trow];
                const float top = fmaxf(m, m1), ref = top == -INFINITY ? 0.f : top;
                f0 = ex2((m - ref) * cs);
                f1 = ex2((m1 - ref) * cs);
                l = l * f0 + l1 * f1;
                m = top;
            }
            const float m2 = m * cs;  // base-2 logits
            const int qr = g.q0 + rr, head = g.h * a.G + (qr - node * a.G);
            const size_t orow = (size_t)(g.s.row0 + node) * a.H + head;
            float fin = 1.f;
            const bool mine = row < g.rows;
            if (g.whole) {
                float lse;
                fin = finish(m2, l, a.sink, head, &lse);
                if (mine && a.lse) a.lse[orow] = lse;
            } else if (mine) {
                *reinterpret_cast<float2 *>(a.part_ml + part_row(a, blockIdx.x, g, row) * 2) =
                    make_float2(m2, l);
            }
            // one verdict for the warp, whose lanes also meet here: the keeper may set the flag for a
            // later piece at any moment, and tensor memory is read by all lanes together
            if (__any_sync(0xffffffffu, c.bad_v)) {
                give_back(a, g, node, pos, n, 2 * DC, tO);
                f0 = fmaxf(f0, 1e-37f);  // what was given back must not vanish in the merge
            }
            const int first = row - lane, left = min(32, g.rows - first);
            // a row's columns are in one thread: turn the warp's blocks of 32 rows x 32 columns around
            // in 4 KB of shared memory (of this slot's query tile, or the exchange block that this
            // warp has just read), in swizzled 16-byte pieces, so that a store covers whole rows
            float *part = a.part_o + part_row(a, blockIdx.x, g, first) * a.dh;
#pragma unroll 1
            for (int x = 0; x < 2 * DC; ++x) {
                uint32_t o[32];
                tmem_ld32(tO + x * 32u, o);
                if (merge) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        o[i] = __float_as_uint(__uint_as_float(o[i]) * f0 +
                                               xch[(x * 4 + quad) * 1024 + i * 32 + lane] * f1);
                }
                uint8_t *turn =
                    gQ + (two ? slot * kTile + quad * 4096u : (x * 4 + quad) * 4096u);
                __syncwarp();
                if (g.whole) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            w[y] = pack_bf16(__uint_as_float(o[8 * i + 2 * y]) * fin,
                                             __uint_as_float(o[8 * i + 2 * y + 1]) * fin);
                        *reinterpret_cast<uint4 *>(turn + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    __syncwarp();
                    const int piece = lane & 3;
                    const bool col = x * 32 + piece * 8 < a.dh;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int ry = y * 8 + (lane >> 2);
                        const uint4 w = *reinterpret_cast<const uint4 *>(
                            turn + ry * 64 + ((piece ^ ((ry >> 1) & 3)) << 4));
                        const long long at = __shfl_sync(0xffffffffu, (long long)orow, ry);
                        if (ry < left && col)
                            *reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.out + at * a.dh + x * 32 +
                                                       piece * 8) = w;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4 *>(turn + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                            make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    __syncwarp();
                    const int piece = lane & 7;
                    const bool col = x * 32 + piece * 4 < a.dh;
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const int ry = y * 4 + (lane >> 3);
                        const uint4 w = *reinterpret_cast<const uint4 *>(
                            turn + ry * 128 + ((piece ^ (ry & 7)) << 4));
                        if (ry < left && col)
                            *reinterpret_cast<uint4 *>(part + (size_t)ry * a.dh + x * 32 +
                                                       piece * 4) = w;
                    }
                }
            }
            tc_fence_before();
        }
    }

    // ---- nothing may be in flight when the CTA frees its tensor memory and leaves ----
    __syncthreads();
    if ((warp == 0 || warp == 3) && lane == 0)
        for (int s = 0; s < NS; ++s)
            if (issued & (1u << s))
                mbar_wait(bar(warp == 0 ? c.kfull[s] : c.vfull[s]), (last_par >> s) & 1u, nullptr,
                          a.flags);
    if ((warp == 1 || warp == 12) && mma_issued) {
        uint64_t &d = c.done[warp == 1 ? 0 : 1];
        commit_elect(bar(d));
        mbar_wait(bar(d), 0, nullptr, a.flags);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem)
                     : "memory");
}

bool encode_pool(CUtensorMap *m, const void *base, const Args &a, int box) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)a.dh, (cuuint64_t)a.page, (cuuint64_t)a.Hkv,
                                (cuuint64_t)a.n_pages};
    const cuuint64_t st[3] = {(cuuint64_t)a.st_tok * 2, (cuuint64_t)a.st_head * 2,
                              (cuuint64_t)a.st_page * 2};
    const cuuint32_t bx[4] = {64, (cuuint32_t)box, 1, 1}, es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, st, bx, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DC> cudaError_t launch_dc(Params &p, int ctas, cudaStream_t s) {
    constexpr int smem = 1024 + kCtlBytes + (stages<DC>() + 2) * DC * 16384;
    const cudaError_t err = allow_smem(attn_tc_kernel<DC>, smem);
    if (err != cudaSuccess) return err;
    return launch_pdl(attn_tc_kernel<DC>, dim3(ctas), dim3(kThreads), smem, s, p);
}

}  // namespace

bool tc_supported(const Args &a, int dtype) {
    return dtype == MOE_DTYPE_BF16 && a.dh <= 128 && encode_fn() != nullptr;
}

cudaError_t launch_tc(Args a, cudaStream_t s) {
    const int nsm = device_sms();
    if (nsm <= 0) return cudaErrorInvalidDevice;
    const int ctas = std::min(nsm, kTcMaxCtas);
    a.rows = kTcRows;
    a.qblocks = (int)(((long long)a.N * a.G + kTcRows - 1) / kTcRows);
    a.prows = (int)std::min<long long>(a.rows, (long long)a.N * a.G);
    a.min_units = 24;
    a.fixed = 48;
    a.whole = 64;
    Params p{};
    p.a = a;
    p.box = 1;
    while (p.box < kBN && a.page % (2 * p.box) == 0) p.box *= 2;
    if (!encode_pool(&p.kmap, a.k, a, p.box) || !encode_pool(&p.vmap, a.v, a, p.box))
        return cudaErrorInvalidValue;
    cudaError_t err = a.dh <= 64 ? launch_dc<1>(p, ctas, s) : launch_dc<2>(p, ctas, s);
    if (err != cudaSuccess) return err;
    return launch_combine(a, MOE_DTYPE_BF16, ctas, s);
}

}  // namespace attn
}  // namespace moe
