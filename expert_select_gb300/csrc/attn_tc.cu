// Paged attention on the 5th-generation tensor cores: bf16, head size up to 128.
//
//   S = Q K^T (fp32, tensor memory),  P = 2^(c S - m) (bf16, tensor memory),  O += P V
//
// in one pass over the keys with a running maximum m and sum l per row (c = scale log2 e). An
// item is 256 rows (node, head in group) of one key/value head: a prompt chunk or a large tree
// fills both 128-row tiles, which then share every K and V tile ("two tiles"); where an item has
// at most 128 rows (single tokens: 8 rows of a group of 8 heads) its one tile is computed over
// even key tiles by one half of the CTA and over odd ones by the other, and the halves are
// merged at the end ("one tile"). Either way two independent score tiles are in flight: while
// the tensor cores work for one, the CUDA cores exponentiate the other.
//
// One CTA per SM, 384 threads:
//   warp 0       TMA producer: key tiles of 128 slots, K and V alternating, through a ring of
//                stages; a tile is gathered as boxes of gcd(page size, 128) slots, a lane per box,
//                each looking its page up
//   warp 1       TMEM allocator and MMA issuer (one lane)
//   warp 2       looks after V: clears what no row may see (see below)
//   warps 4-7, 8-11  softmax of slot 0 and slot 1: a thread per row, its 128 scores in registers
//
// TMEM (512 columns): S of slots 0 and 1 (128 each; P overwrites S's first 64), O of slots 0 and
// 1. The second product reads P from tensor memory and V from shared memory as it was loaded
// (MN-major), so P never passes through shared memory.
//
// A masked score is -inf, so its P is 0; but 0 x V is NaN where V is infinite or NaN. In tiles
// that hold masked slots (the last ones, and a window's first) warp 2 therefore clears the rows of
// V past the sequence's end and the non-finite elements of the others before the second product;
// rows that do see such an element get it back at the end (a slow path that only runs then).
//
// Every wait is bounded: after 2 s it sets the check bit and the CTA drains and leaves.
#include <algorithm>

#include "attn.cuh"
#include "tmem.cuh"

namespace moe {
namespace attn {
namespace {

using namespace tc;

constexpr int kBN = 128;
constexpr int kThreads = 384;
constexpr int kVq = 8;           // V-ready barriers in rotation: more than V tiles in the ring
constexpr int kMaxStages = 6;
constexpr int kCtlBytes = 2048;

struct Params {
    Args a;
    CUtensorMap kmap, vmap;
    int box;     // slots of a TMA box: gcd(page size, 128)
    int stages;
};

struct Ctl {  // control block in shared memory; barriers first
    uint64_t full[kMaxStages], empty[kMaxStages], vready[kVq], s_full[2], p_full[2], o_done[2],
        q_full, done;
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

// Positions of K and V tiles of a segment of n tiles in the ring's order: LA K tiles first, then
// V(t), K(t + LA) in turn.
__device__ __forceinline__ int k_pos(int t, int la) { return t < la ? t : 2 * t - la + 1; }
__device__ __forceinline__ int v_pos(int t, int la, int n) { return t + min(t + la, n); }

struct Ring {
    uint32_t base;  // ring position of the segment's first tile
    int stages;
    __device__ __forceinline__ int stage(uint32_t pos) const { return (int)(pos % stages); }
    __device__ __forceinline__ uint32_t parity(uint32_t pos) const { return (pos / stages) & 1u; }
};

template <int DC>  // 64-column chunks of the head size
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    Ctl &c = *reinterpret_cast<Ctl *>(gbase);
    constexpr uint32_t kTile = DC * 16384u;  // 128 rows x 64 DC bf16
    const uint32_t sQ = base + kCtlBytes, sRing = sQ + 2 * kTile;
    uint8_t *gQ = gbase + kCtlBytes, *gRing = gQ + 2 * kTile;
    const Args &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto bar = [&](uint64_t &b) { return smem_u32(&b); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(bar(c.full[s]), 1);
            mbar_init(bar(c.empty[s]), 1);
        }
        for (int i = 0; i < kVq; ++i) mbar_init(bar(c.vready[i]), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(c.s_full[i]), 1);
            mbar_init(bar(c.p_full[i]), 128);
            mbar_init(bar(c.o_done[i]), 1);
        }
        mbar_init(bar(c.q_full), 256);
        mbar_init(bar(c.done), 1);
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
    Range r = attn_plan<kBN, kThreads>(a, blockIdx.x, gridDim.x, c.scratch);
    if (threadIdx.x == 96) write_record<kBN>(a, blockIdx.x, r);
    Ring ring{0, p.stages};

    uint32_t issued = 0, last_par = 0;  // producer: stages with a load issued, parity of the last
    bool mma_issued = false;

    if (warp == 0) {
        // ------------------------------------------------------------- producer
        bool ok = true;
        while (ok && r.left > 0) {
            const Segment g = next_segment<kBN>(a, r);
            const int la = g.rows > 128 ? 1 : 2, n = g.count;
            for (int pos = 0, kt = 0, vt = 0; ok && pos < 2 * n; ++pos) {
                const bool is_k = kt < n && kt < vt + la;
                const int t = is_k ? kt++ : vt++;
                const int k0 = g.tl.at(g.t + t) * kBN;
                const uint32_t rp = ring.base + pos;
                const int st = ring.stage(rp);
                const int boxes = (min(kBN, g.s.L - k0) + p.box - 1) / p.box;
                int pg[4], good = 0;  // kBN / box <= 128 boxes, lane by lane
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int bx = lane + 32 * i;
                    pg[i] = bx < boxes ? page_of(a, g.b, k0 + bx * p.box) : -1;
                    good += __popc(__ballot_sync(0xffffffffu, pg[i] >= 0));
                }
                if (good < boxes && lane == 0) {
                    c.bad_page = 1;
                    __threadfence_block();
                    atomicOr(a.flags, FLAG_BAD_PAGE);
                }
                ok = mbar_wait(bar(c.empty[st]), ring.parity(rp) ^ 1u, &c.abort, a.flags);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint32_t fb = bar(c.full[st]);
                if (lane == 0) mbar_expect_tx(fb, (uint32_t)good * p.box * 128u * DC);
                __syncwarp();
                const CUtensorMap *map = is_k ? &p.kmap : &p.vmap;
                const uint32_t dst = sRing + (uint32_t)st * kTile;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (pg[i] >= 0) {
                        const int j = k0 + (lane + 32 * i) * p.box;
#pragma unroll
                        for (int h = 0; h < DC; ++h)
                            tma_load_4d(dst + h * 16384u + (uint32_t)(lane + 32 * i) * p.box * 128u,
                                        map, h * 64, j % a.page, g.h, pg[i], fb);
                    }
                issued |= 1u << st;
                last_par = (last_par & ~(1u << st)) | (ring.parity(rp) << st);
                __syncwarp();
            }
            ring.base += 2 * n;
        }
    } else if (warp == 1) {
        // ----------------------------------------------------------- MMA issuer
        if (lane == 0) {
            const uint32_t id_s = idesc_bf16(128, 128), id_o = idesc_bf16(128, 64 * DC) | kIdescBMn;
            uint32_t pcount[2] = {0, 0}, vcount = 0, seg = 0;
            bool ok = true;
            auto wait = [&](uint64_t &b, uint32_t par) {
                if (ok) ok = mbar_wait(bar(b), par, &c.abort, a.flags);
                tc_fence_after();
                return ok;
            };
            while (ok && r.left > 0) {
                const Segment g = next_segment<kBN>(a, r);
                const bool two = g.rows > 128;
                const int la = two ? 1 : 2, n = g.count;
                auto score = [&](int slot, int t) {  // S of a slot from K tile t
                    const uint32_t k = sRing + (uint32_t)ring.stage(ring.base + k_pos(t, la)) * kTile;
                    const uint32_t q = sQ + (two ? (uint32_t)slot * kTile : 0u);
#pragma unroll
                    for (int x = 0; x < 4 * DC; ++x) {
                        const uint32_t off = (x >> 2) * 16384u + (x & 3) * 32u;
                        mma_bf16(tmem + slot * 128u, sw128_desc(q + off), sw128_desc(k + off), id_s,
                                 x != 0);
                    }
                    mma_issued = true;
                    mma_commit(bar(c.s_full[slot]));
                };
                auto wait_k = [&](int t) {
                    const uint32_t rp = ring.base + k_pos(t, la);
                    return wait(c.full[ring.stage(rp)], ring.parity(rp));
                };
                auto free_k = [&](int t) {
                    mma_commit(bar(c.empty[ring.stage(ring.base + k_pos(t, la))]));
                };
                auto output = [&](int slot, int t, bool first) {  // O += P V tile t
                    const uint32_t v =
                        sRing + (uint32_t)ring.stage(ring.base + v_pos(t, la, n)) * kTile;
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        mma_bf16_ts(tmem + 256u + slot * 128u, tmem + slot * 128u + x * 8u,
                                    sw128_mn_desc(v + x * 2048u, 16384u), id_o, !first || x != 0);
                };
                auto wait_p = [&](int slot) { return wait(c.p_full[slot], pcount[slot]++ & 1u); };
                auto wait_v = [&]() {
                    const bool w = wait(c.vready[vcount % kVq], (vcount / kVq) & 1u);
                    ++vcount;
                    return w;
                };
                auto free_v = [&](int t) {
                    mma_commit(bar(c.empty[ring.stage(ring.base + v_pos(t, la, n))]));
                };
                if (!wait(c.q_full, seg++ & 1u)) break;
                if (two) {
                    if (!wait_k(0)) break;
                    score(0, 0);
                    score(1, 0);
                    free_k(0);
                    for (int t = 0; ok && t < n; ++t) {
                        const bool more = t + 1 < n;
                        if (!wait_v() || !wait_p(0)) break;
                        output(0, t, t == 0);
                        if (more) {
                            if (!wait_k(t + 1)) break;
                            score(0, t + 1);
                        } else {
                            mma_commit(bar(c.o_done[0]));
                        }
                        if (!wait_p(1)) break;
                        output(1, t, t == 0);
                        free_v(t);
                        if (more) {
                            score(1, t + 1);
                            free_k(t + 1);
                        } else {
                            mma_commit(bar(c.o_done[1]));
                        }
                    }
                } else {
                    for (int t = 0; t < min(n, 2); ++t) {
                        if (!wait_k(t)) break;
                        score(t, t);
                        free_k(t);
                    }
                    for (int t = 0; ok && t < n; ++t) {
                        const int slot = t & 1;
                        if (!wait_v() || !wait_p(slot)) break;
                        output(slot, t, t < 2);
                        free_v(t);
                        if (t + 2 < n) {
                            if (!wait_k(t + 2)) break;
                            score(slot, t + 2);
                            free_k(t + 2);
                        } else {
                            mma_commit(bar(c.o_done[slot]));
                        }
                    }
                }
                ring.base += 2 * n;
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        // -------------------------------------------------------- keeper of V
        uint32_t vcount = 0;
        bool ok = true;
        while (ok && r.left > 0) {
            const Segment g = next_segment<kBN>(a, r);
            const int la = g.rows > 128 ? 1 : 2, n = g.count;
            const int i0 = g.q0 / a.G, i1 = (g.q0 + g.rows - 1) / a.G;
            const int pos = i0 == i1 ? node_position(a, g.s, i0) : 0;
            for (int t = 0; ok && t < n; ++t) {
                const uint32_t rp = ring.base + v_pos(t, la, n);
                const int st = ring.stage(rp);
                ok = __all_sync(0xffffffffu,
                                mbar_wait(bar(c.full[st]), ring.parity(rp), &c.abort, a.flags));
                if (!ok) break;
                const int k0 = g.tl.at(g.t + t) * kBN;
                if (c.bad_page || tile_masked<kBN>(a, g.s, i0, i1, k0)) {
                    // rows that no query of the item sees are cleared whole: with one node all
                    // that it does not see, else what lies past the end or has no page
                    uint32_t bits[4];
                    if (i0 == i1) {
                        visible_bits<4>(a, g.s, i0, pos, k0, bits);
                    } else {
#pragma unroll
                        for (int w = 0; w < 4; ++w) bits[w] = range_bits(0, g.s.L, k0 + 32 * w);
                    }
                    uint8_t *tile = gRing + (size_t)st * kTile;
#pragma unroll 1
                    for (int w = 0; w < 4; ++w) {
                        const int row = 32 * w + lane;
                        bool keep = (bits[w] >> lane) & 1u;
                        if (keep && c.bad_page) keep = page_of(a, g.b, k0 + row) >= 0;
                        if (keep && i0 == i1) continue;
#pragma unroll 1
                        for (int h = 0; h < DC; ++h)
#pragma unroll
                            for (int x = 0; x < 8; ++x) {
                                uint4 *q = reinterpret_cast<uint4 *>(tile + h * 16384 + row * 128 +
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
                if (lane == 0) mbar_arrive(bar(c.vready[vcount % kVq]));
                ++vcount;
            }
            ring.base += 2 * n;
        }
    } else if (warp >= 4) {
        // -------------------------------------------------------------- softmax
        // A failed wait leaves `dead` set: the thread then runs through its loops without
        // computing or storing, so that the barriers stay matched.
        const int slot = (warp - 4) >> 2, quad = warp & 3;
        const int trow = quad * 32 + lane;  // row of the slot's tile
        const int tid = threadIdx.x - 128;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t tS = tmem + slot * 128u + lanes, tO = tmem + 256u + slot * 128u + lanes;
        uint32_t scount = 0, ocount = 0;
        bool dead = false;
        while (r.left > 0) {
            const Segment g = next_segment<kBN>(a, r);
            const bool two = g.rows > 128;
            const int n = g.count;
            softmax_bar();  // the last segment's tiles and exchange buffer are done with
            {
                const int rows = two ? 256 : 128;
                const __nv_bfloat16 *q = (const __nv_bfloat16 *)a.q;
                for (int i = tid; i < rows * 8 * DC; i += 256) {
                    const int row = i / (8 * DC), ch = i % (8 * DC);
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (row < g.rows && ch * 8 < a.dh) {
                        const int qr = g.q0 + row, node = qr / a.G;
                        v = __ldg(reinterpret_cast<const uint4 *>(
                            q + (size_t)(g.s.row0 + node) * a.ldq +
                            (size_t)(g.h * a.G + qr - node * a.G) * a.dh + ch * 8));
                    }
                    const int rr = row & 127;
                    *reinterpret_cast<uint4 *>(gQ + (row >> 7) * kTile + (ch >> 3) * 16384 +
                                               rr * 128 + (((ch & 7) ^ (rr & 7)) << 4)) = v;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(bar(c.q_full));
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
            for (int t = two ? 0 : slot; t < n; t += two ? 1 : 2, ++tiles) {
                const int k0 = g.tl.at(g.t + t) * kBN;
                if (!mbar_wait(bar(c.s_full[slot]), scount & 1u, &c.abort, a.flags)) dead = true;
                ++scount;
                tc_fence_after();
                if (active && !__any_sync(0xffffffffu, dead)) {
                    uint32_t s[128];
                    tmem_ld128(tS, s);
                    if (tile_masked<kBN>(a, g.s, i0, i1, k0) || c.bad_page) {
                        uint32_t bits[4];
                        visible_bits<4>(a, g.s, node, pos, k0, bits);
                        if (c.bad_page) {
#pragma unroll
                            for (int w = 0; w < 4; ++w)
                                for (int x = 0; x < 32; ++x)
                                    if (((bits[w] >> x) & 1u) && page_of(a, g.b, k0 + 32 * w + x) < 0)
                                        bits[w] &= ~(1u << x);
                        }
#pragma unroll
                        for (int w = 0; w < 4; ++w)
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                if (!((bits[w] >> x) & 1u)) s[32 * w + x] = 0xff800000u;  // -inf
                    }
                    float mx[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx[i] = __uint_as_float(s[i]);
#pragma unroll
                    for (int i = 4; i < 128; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(s[i]));
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    const bool raise = (top - m) * cs > kRaise;  // m = -inf: yes, unless top is too
                    if (__any_sync(0xffffffffu, raise)) {
                        const float mn = fmaxf(m, top);
                        const float f = m == -INFINITY ? 0.f : ex2((m - mn) * cs);
                        m = mn;
                        l *= f;
                        if (tiles > 0) {
#pragma unroll 1
                            for (int x = 0; x < 2 * DC; ++x) {
                                uint32_t o[32];
                                tmem_ld32(tO + x * 32u, o);
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                tmem_st32(tO + x * 32u, o);
                            }
                            tmem_wait_st();
                        }
                    }
                    const float sub = m == -INFINITY ? 0.f : m * cs;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        uint32_t pk[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int j = x * 64 + 2 * i;
                            const float p0 = ex2(fmaf(__uint_as_float(s[j]), cs, -sub));
                            const float p1 = ex2(fmaf(__uint_as_float(s[j + 1]), cs, -sub));
                            sum[(2 * i) & 3] += p0;
                            sum[(2 * i + 1) & 3] += p1;
                            pk[i] = pack_bf16(p0, p1);
                        }
                        tmem_st32(tS + x * 32u, pk);
                    }
                    tmem_wait_st();
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                }
                tc_fence_before();
                mbar_arrive(bar(c.p_full[slot]));
            }
            if (tiles > 0) {
                if (!mbar_wait(bar(c.o_done[slot]), ocount & 1u, &c.abort, a.flags)) dead = true;
                ++ocount;
                tc_fence_after();
            }
            const bool live = !__any_sync(0xffffffffu, dead);
            // one tile: slot 1 hands its part over through the query tiles' shared memory (column
            // by column, a thread per row)
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
                                xch[(x * 32 + i) * 128 + trow] = __uint_as_float(o[i]);
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
            const size_t prow = g.whole ? 0 : part_row(a, blockIdx.x, g, rr);
            if (g.whole) {
                float lse;
                fin = finish(m2, l, a.sink, head, &lse);
                if (mine && a.lse) a.lse[orow] = lse;
            } else if (mine) {
                a.part_ml[prow * 2] = m2;
                a.part_ml[prow * 2 + 1] = l;
            }
            const bool fix = c.bad_v != 0;
#pragma unroll 1
            for (int x = 0; x < 2 * DC; ++x) {
                uint32_t o[32];
                tmem_ld32(tO + x * 32u, o);
                float v[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(o[i]);
                if (merge) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        v[i] = v[i] * f0 + xch[(x * 32 + i) * 128 + trow] * f1;
                }
                if (fix) {
                    // give back the non-finite elements of V that this row sees
                    for (int t = 0; t < n; ++t) {
                        const int k0 = g.tl.at(g.t + t) * kBN;
                        uint32_t bits[4];
                        visible_bits<4>(a, g.s, node, pos, k0, bits);
#pragma unroll 1
                        for (int j = 0; j < kBN; ++j) {
                            const uint32_t wb = j < 64 ? (j < 32 ? bits[0] : bits[1])
                                                       : (j < 96 ? bits[2] : bits[3]);
                            if (!((wb >> (j & 31)) & 1u)) continue;
                            const int pg = page_of(a, g.b, k0 + j);
                            if (pg < 0) continue;
                            const __nv_bfloat16 *vr =
                                (const __nv_bfloat16 *)a.v + (size_t)pg * a.st_page +
                                (size_t)((k0 + j) % a.page) * a.st_tok + (size_t)g.h * a.st_head;
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (x * 32 + i < a.dh) {
                                    const float e = __bfloat162float(vr[x * 32 + i]);
                                    if (!isfinite(e) && isfinite(v[i])) v[i] = e;
                                    else if (!isfinite(e)) v[i] += e;
                                }
                        }
                    }
                }
                if (!mine) continue;
                if (g.whole) {
                    __nv_bfloat16 *out = (__nv_bfloat16 *)a.out + orow * a.dh + x * 32;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (x * 32 + i * 8 < a.dh)
                            *reinterpret_cast<uint4 *>(out + i * 8) = make_uint4(
                                pack_bf16(v[i * 8] * fin, v[i * 8 + 1] * fin),
                                pack_bf16(v[i * 8 + 2] * fin, v[i * 8 + 3] * fin),
                                pack_bf16(v[i * 8 + 4] * fin, v[i * 8 + 5] * fin),
                                pack_bf16(v[i * 8 + 6] * fin, v[i * 8 + 7] * fin));
                } else {
                    float *out = a.part_o + prow * a.dh + x * 32;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (x * 32 + i * 4 < a.dh)
                            *reinterpret_cast<float4 *>(out + i * 4) =
                                make_float4(v[i * 4], v[i * 4 + 1], v[i * 4 + 2], v[i * 4 + 3]);
                }
            }
            tc_fence_before();
        }
    }

    // ---- nothing may be in flight when the CTA frees its tensor memory and leaves ----
    __syncthreads();
    if (warp == 0 && lane == 0)
        for (int s = 0; s < p.stages; ++s)
            if (issued & (1u << s))
                mbar_wait(bar(c.full[s]), (last_par >> s) & 1u, nullptr, a.flags);
    if (warp == 1 && lane == 0 && mma_issued) {
        mma_commit(bar(c.done));
        mbar_wait(bar(c.done), 0, nullptr, a.flags);
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
    constexpr int kTile = DC * 16384;
    constexpr int budget = 227 * 1024 - 1024 - kCtlBytes;  // less the alignment slack
    p.stages = std::min(kMaxStages, budget / kTile - 2);
    const int smem = 1024 + kCtlBytes + (p.stages + 2) * kTile;
    const cudaError_t err = cudaFuncSetAttribute(
        attn_tc_kernel<DC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    return launch_pdl(attn_tc_kernel<DC>, dim3(ctas), dim3(kThreads), smem, s, p);
}

}  // namespace

bool tc_supported(const Args &a, int dtype) {
    if (dtype != MOE_DTYPE_BF16 || a.dh > 128) return false;
    int dev = 0, major = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
        return false;
    return major >= 10 && encode_fn() != nullptr;
}

cudaError_t launch_tc(Args a, cudaStream_t s) {
    int dev = 0, nsm = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess)
        err = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    const int ctas = std::min(nsm, kTcMaxCtas);
    a.rows = kTcRows;
    a.qblocks = (int)(((long long)a.N * a.G + kTcRows - 1) / kTcRows);
    a.prows = (int)std::min<long long>(a.rows, (long long)a.N * a.G);
    a.min_tiles = 2;
    Params p{};
    p.a = a;
    p.box = 1;
    while (p.box < kBN && a.page % (2 * p.box) == 0) p.box *= 2;
    if (!encode_pool(&p.kmap, a.k, a, p.box) || !encode_pool(&p.vmap, a.v, a, p.box))
        return cudaErrorInvalidValue;
    err = a.dh <= 64 ? launch_dc<1>(p, ctas, s) : launch_dc<2>(p, ctas, s);
    if (err != cudaSuccess) return err;
    return launch_combine(a, MOE_DTYPE_BF16, ctas, s);
}

}  // namespace attn
}  // namespace moe
