// Paged attention for few rows: bf16, head size up to 128, items of at most 16 rows (single
// tokens, or a few nodes, of a group of query heads).
//
// The work is reading the cache: per key and key/value head 4 dh bytes against 64 dh operations,
// a sixteenth of what the tensor cores could do meanwhile. So the kernel is built for bytes in
// flight and for short items, not for the product's rate: every warp works on its own. A CTA
// of four warps takes tiles of 64 slots, warp w their slots 16 w .. 16 w + 15; it copies its K and
// V rows into its own ring of stages with cp.async (rows found through the page table, a lane
// per row), runs ahead of itself by the ring's length, over the ends of items too, and
// keeps its own running maximum, sum and O for its share of the keys (m16n8k16 products: S has
// two 8-key tiles, whose exponentials in registers are already the A operand of P V). The four
// warps' parts are merged when the CTA's piece of the item ends.
//
// Measured: one token over 131k slots (4 key/value heads of 128, bf16, 268 MB) 51 us with the
// combine (5.2 TB/s over the whole call; 39.5 us at the copy bandwidth); 128 tokens with a window
// of 128 slots (1024 items of 3-4 tiles) 28 us. Against the tcgen05 kernel, 8 rows of 4
// key/value heads of 128: one token over 60001 slots 31.8 us to 39.9, 64 of them over up to 4003
// slots 64.0 to 73.5. TMA boxes of 16 slots instead of cp.async were no faster (131k slots: 53 us).
#include <limits.h>

#include <algorithm>

#include "attn.cuh"
#include "tc.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kBN = 64;     // slots of a tile
constexpr int kWarps = 4;   // 16 slots each
constexpr int kThr = 32 * kWarps;
constexpr int kLight = 0;  // every tile is one unit of work

template <int DC> struct Shape {
    static constexpr int kRow = DC * 128;           // bytes of a row in shared memory
    static constexpr int kHalf = 16 * kRow;         // K (or V) of a stage
    static constexpr int kCtas = DC == 1 ? 3 : 2;   // per SM
    static constexpr int kStages = 3;
    static constexpr int kRing = kStages * 2 * kHalf;
    static constexpr int kXch = 2 * 16 * DC * 64 * 4;  // two warps' O
    static constexpr int kSmem = kWarps * kRing + kXch;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void ldsm(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

struct Cursor {
    Range r;
    Segment g;
    int t;
    bool on;
    __device__ __forceinline__ void start(const Args &a, const Range &range) {
        r = range;
        t = 0;
        on = next_segment<kBN, kLight>(a, r, g);
    }
    __device__ __forceinline__ void step(const Args &a) {
        if (++t < g.count) return;
        t = 0;
        on = next_segment<kBN, kLight>(a, r, g);
    }
};

template <int DC>
__global__ void __launch_bounds__(kThr, Shape<DC>::kCtas) attn_few_kernel(const Args a) {
    using S = Shape<DC>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long scratch[34];
    __shared__ uint32_t s_pages[kWarps][S::kStages];  // slots of a stage that have a page
    __shared__ float s_ml[kWarps][2][16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    const Range range = attn_plan<kBN, kLight, kThr>(a, blockIdx.x, gridDim.x, scratch);
    if (threadIdx.x == 0) write_record(a, blockIdx.x, range);
    const uint32_t ring = tc::smem_u32(smem) + warp * S::kRing;
    uint8_t *gring = smem + warp * S::kRing;
    float *xch = reinterpret_cast<float *>(smem + kWarps * S::kRing);
    const __nv_bfloat16 *kp = (const __nv_bfloat16 *)a.k, *vp = (const __nv_bfloat16 *)a.v;

    Cursor ld, cp;
    ld.start(a, range);
    cp.start(a, range);
    int lstage = 0;
    // the page of the lane's row in the tile that is copied next, looked up a tile ahead
    // (INT_MIN: the slot is past the sequence's end or out of every row's reach)
    int page = INT_MIN, slot = 0;
    auto look_up = [&]() {
        page = INT_MIN;
        if (!ld.on) return;
        slot = ld.g.tl.at(ld.g.t + ld.t) * kBN + warp * 16 + (lane & 15);
        if (slot < ld.g.s.L && !out_of_reach(a, ld.g.s, slot, slot))
            page = max(a.table[(size_t)ld.g.b * a.max_pages + slot / a.page], -1);
    };
    look_up();
    auto issue = [&]() {  // copies the warp's 16 slots of the next tile, if there is one
        if (ld.on) {
            const bool ok = page >= 0 && page < a.n_pages;
            if (!ok && page != INT_MIN) atomicOr(a.flags, FLAG_BAD_PAGE);
            const long long off =
                ok ? (long long)page * a.st_page + (long long)(slot % a.page) * a.st_tok +
                         (long long)ld.g.h * a.st_head
                   : 0ll;
            ld.step(a);
            look_up();
            const uint32_t have = __ballot_sync(0xffffffffu, ok) & 0xffffu;
            if (lane == 0) s_pages[warp][lstage] = have;
            const uint32_t dst = ring + lstage * 2 * S::kHalf;
            if (have) {
#pragma unroll
                for (int i = 0; i < 4 * DC; ++i) {
                    const int idx = lane + 32 * i, row = idx / (8 * DC), ch = idx % (8 * DC);
                    const long long o = __shfl_sync(0xffffffffu, off, row) + ch * 8;
                    const bool there = ((have >> row) & 1u) && ch * 8 < a.dh;
                    const uint32_t at = dst + row * S::kRow + ((ch ^ (row & 7)) << 4);
                    cp16(at, kp + (there ? o : 0), there);
                    cp16(at + S::kHalf, vp + (there ? o : 0), there);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        lstage = lstage + 1 == S::kStages ? 0 : lstage + 1;
    };
#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) issue();

    const float cs = a.scale * kLog2e;
    const int r0 = lane >> 2, cq = (lane & 3) * 2;  // fragment rows r0, r0 + 8; first column
    uint32_t q[4 * DC][4];
    float o[8 * DC][4], m[2], l[2];
    int node[2], pos[2], i0 = 0, i1 = 0, stage = 0;
    while (cp.on) {
        const Segment &g = cp.g;
        if (cp.t == 0) {
            i0 = g.q0 / a.G;
            i1 = (g.q0 + g.rows - 1) / a.G;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int row = r0 + 8 * x, qr = g.q0 + min(row, g.rows - 1);
                node[x] = qr / a.G;
                pos[x] = node_position(a, g.s, node[x]);
                const __nv_bfloat16 *src = (const __nv_bfloat16 *)a.q +
                                           (size_t)(g.s.row0 + node[x]) * a.ldq +
                                           (size_t)(g.h * a.G + qr - node[x] * a.G) * a.dh;
#pragma unroll
                for (int k = 0; k < 4 * DC; ++k)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int col = k * 16 + y * 8 + cq;
                        q[k][2 * y + x] = row < g.rows && col < a.dh
                                              ? *reinterpret_cast<const uint32_t *>(src + col)
                                              : 0u;
                    }
                m[x] = -INFINITY;
                l[x] = 0.f;
            }
#pragma unroll
            for (int n = 0; n < 8 * DC; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        }
        issue();
        asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 1) : "memory");
        __syncwarp();
        // a piece of 16 slots without one to read (3 of 4 in a tile of a few first tokens) is done
        const uint32_t have = s_pages[warp][stage];
        if (have) {
            const uint32_t sk = ring + stage * 2 * S::kHalf, sv = sk + S::kHalf;
            const int k0 = g.tl.at(g.t + cp.t) * kBN + warp * 16;
            // ---- S = Q K^T, two tiles of 8 keys
            float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            {
                // matrices: keys 0-7 twice, 8-15 twice
                const int key = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
                for (int k = 0; k < 4 * DC; ++k) {
                    uint32_t b[4];
                    const int ch = 2 * k + ((lane >> 3) & 1);
                    ldsm(sk + key * S::kRow + ((ch ^ (key & 7)) << 4), b);
                    mma16(s[0], q[k], b[0], b[1]);
                    mma16(s[1], q[k], b[2], b[3]);
                }
            }
            // back: keys whose V is fixed up below
            uint32_t vis[2] = {0xffffu, 0xffffu}, back = 0u;
            if (have != 0xffffu || tile_masked<16>(a, g.s, i0, i1, k0)) {
                uint32_t some = 0u, all = 0xffffu;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t bits[1];
                    visible_bits<1>(a, g.s, node[x], pos[x], k0, bits);
                    vis[x] = bits[0] & have;
                    if (r0 + 8 * x < g.rows) {
                        some |= vis[x];
                        all &= vis[x];
                    }
                }
                some = __reduce_or_sync(0xffffffffu, some);
                all = __reduce_and_sync(0xffffffffu, all);
                // 0 x V is NaN where V is not finite: clear the rows that no query sees and the
                // non-finite elements of those that only some see (added back below)
#pragma unroll 1
                for (int i = 0; i < 4 * DC; ++i) {
                    const int idx = lane + 32 * i, row = idx / (8 * DC), ch = idx % (8 * DC);
                    if ((all >> row) & 1u) continue;
                    uint4 *at = reinterpret_cast<uint4 *>(gring + stage * 2 * S::kHalf + S::kHalf +
                                                          row * S::kRow + ((ch ^ (row & 7)) << 4));
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if ((some >> row) & 1u) {
                        v = *at;
                        uint32_t *e = reinterpret_cast<uint32_t *>(&v);
                        bool bad = false;
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            if ((e[w] & 0x7f80u) == 0x7f80u) {
                                e[w] &= 0xffff0000u;
                                bad = true;
                            }
                            if ((e[w] & 0x7f800000u) == 0x7f800000u) {
                                e[w] &= 0xffffu;
                                bad = true;
                            }
                        }
                        if (!bad) continue;
                        back |= 1u << row;
                    }
                    *at = v;
                }
                back = __reduce_or_sync(0xffffffffu, back);
                __syncwarp();
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (!((vis[x >> 1] >> (n * 8 + cq + (x & 1))) & 1u)) s[n][x] = -INFINITY;
            }
            // ---- running maximum; P
            float top[2], f[2] = {1.f, 1.f};
            bool raise = false;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float t = fmaxf(fmaxf(s[0][2 * x], s[0][2 * x + 1]),
                                fmaxf(s[1][2 * x], s[1][2 * x + 1]));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                top[x] = t;
                raise |= (t - m[x]) * cs > kRaise;
            }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float mn = fmaxf(m[x], top[x]);
                    f[x] = m[x] == -INFINITY ? 0.f : ex2((m[x] - mn) * cs);
                    m[x] = mn;
                    l[x] *= f[x];
                }
#pragma unroll
                for (int n = 0; n < 8 * DC; ++n) {
                    o[n][0] *= f[0];
                    o[n][1] *= f[0];
                    o[n][2] *= f[1];
                    o[n][3] *= f[1];
                }
            }
            const float sub[2] = {m[0] == -INFINITY ? 0.f : m[0] * cs,
                                  m[1] == -INFINITY ? 0.f : m[1] * cs};
            uint32_t p[4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float p0 = ex2(fmaf(s[n][2 * x], cs, -sub[x]));
                    const float p1 = ex2(fmaf(s[n][2 * x + 1], cs, -sub[x]));
                    l[x] += p0 + p1;
                    p[2 * n + x] = pack_bf16(p0, p1);
                }
            }
            // ---- O += P V
            {
                // keys 0-7, 8-15 of a column tile
                const int key = (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
                for (int n = 0; n < 4 * DC; ++n) {
                    uint32_t b[4];
                    const int ch = 2 * n + (lane >> 4);
                    ldsm_t(sv + key * S::kRow + ((ch ^ (key & 7)) << 4), b);
                    mma16(o[2 * n], p, b[0], b[1]);
                    mma16(o[2 * n + 1], p, b[2], b[3]);
                }
            }
            if (back) {
#pragma unroll 1
                for (int k = 0; k < 16; ++k) {
                    if (!((back >> k) & 1u)) continue;
                    const __nv_bfloat16 *v = vp + (long long)page_of(a, g.b, k0 + k) * a.st_page +
                                             (long long)((k0 + k) % a.page) * a.st_tok +
                                             (long long)g.h * a.st_head;
#pragma unroll
                    for (int n = 0; n < 8 * DC; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int col = n * 8 + cq + (x & 1);
                            if (col < a.dh && ((vis[x >> 1] >> k) & 1u)) {
                                const float e = __bfloat162float(v[col]);
                                if (!isfinite(e)) o[n][x] += e;
                            }
                        }
                }
            }
        }
        __syncwarp();
        stage = stage + 1 == S::kStages ? 0 : stage + 1;
        if (cp.t + 1 == g.count) {
            // ---- merge the four warps: scale to the common maximum, then 2 + 2 -> 1 + 1
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
                l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
                if ((lane & 3) == 0) {
                    s_ml[warp][0][r0 + 8 * x] = m[x];
                    s_ml[warp][1][r0 + 8 * x] = l[x];
                }
            }
            __syncthreads();
            float mt[2], lt[2], f[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int row = r0 + 8 * x;
                float t = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) t = fmaxf(t, s_ml[w][0][row]);
                mt[x] = t;
                const float ref = t == -INFINITY ? 0.f : t;
                lt[x] = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    lt[x] += s_ml[w][1][row] * ex2((s_ml[w][0][row] - ref) * cs);
                f[x] = ex2((m[x] - ref) * cs);
            }
#pragma unroll
            for (int n = 0; n < 8 * DC; ++n) {
                o[n][0] *= f[0];
                o[n][1] *= f[0];
                o[n][2] *= f[1];
                o[n][3] *= f[1];
            }
            // a warp's O as [column tile][lane] float4: no bank conflicts
            float4 *x4 = reinterpret_cast<float4 *>(xch);
            if (warp >= 2) {
#pragma unroll
                for (int n = 0; n < 8 * DC; ++n)
                    x4[(warp - 2) * 256 * DC + n * 32 + lane] =
                        make_float4(o[n][0], o[n][1], o[n][2], o[n][3]);
            }
            __syncthreads();
            if (warp < 2) {
#pragma unroll
                for (int n = 0; n < 8 * DC; ++n) {
                    const float4 v = x4[warp * 256 * DC + n * 32 + lane];
                    o[n][0] += v.x;
                    o[n][1] += v.y;
                    o[n][2] += v.z;
                    o[n][3] += v.w;
                }
            }
            if (warp == 1) {
                __syncwarp();
#pragma unroll
                for (int n = 0; n < 8 * DC; ++n)
                    x4[256 * DC + n * 32 + lane] = make_float4(o[n][0], o[n][1], o[n][2], o[n][3]);
            }
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int n = 0; n < 8 * DC; ++n) {
                    const float4 v = x4[256 * DC + n * 32 + lane];
                    o[n][0] += v.x;
                    o[n][1] += v.y;
                    o[n][2] += v.z;
                    o[n][3] += v.w;
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int row = r0 + 8 * x;
                    if (row >= g.rows) continue;
                    const int head = g.h * a.G + (g.q0 + row - node[x] * a.G);
                    if (g.whole) {
                        const size_t orow = (size_t)(g.s.row0 + node[x]) * a.H + head;
                        float lse;
                        const float fin = finish(mt[x] * cs, lt[x], a.sink, head, &lse);
                        __nv_bfloat16 *out = (__nv_bfloat16 *)a.out + orow * a.dh;
#pragma unroll
                        for (int n = 0; n < 8 * DC; ++n)
                            if (n * 8 < a.dh)
                                *reinterpret_cast<uint32_t *>(out + n * 8 + cq) =
                                    pack_bf16(o[n][2 * x] * fin, o[n][2 * x + 1] * fin);
                        if (a.lse && (lane & 3) == 0) a.lse[orow] = lse;
                    } else {
                        const size_t pr = part_row(a, blockIdx.x, g, row);
#pragma unroll
                        for (int n = 0; n < 8 * DC; ++n)
                            if (n * 8 < a.dh)
                                *reinterpret_cast<float2 *>(a.part_o + pr * a.dh + n * 8 + cq) =
                                    make_float2(o[n][2 * x], o[n][2 * x + 1]);
                        if ((lane & 3) == 0) {
                            a.part_ml[pr * 2] = mt[x] * cs;
                            a.part_ml[pr * 2 + 1] = lt[x];
                        }
                    }
                }
            }
        }
        cp.step(a);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int DC> cudaError_t launch_dc(const Args &a, int nsm, int *ctas, cudaStream_t s) {
    *ctas = std::min(kMaxCtas, Shape<DC>::kCtas * nsm);
    constexpr int smem = Shape<DC>::kSmem;
    const cudaError_t err = allow_smem(attn_few_kernel<DC>, smem);
    if (err != cudaSuccess) return err;
    return launch_pdl(attn_few_kernel<DC>, dim3(*ctas), dim3(kThr), smem, s, a);
}

}  // namespace

cudaError_t launch_few(Args a, cudaStream_t s) {
    const int nsm = device_sms();
    if (nsm <= 0) return cudaErrorInvalidDevice;
    int ctas = 0;
    a.rows = kFewRows;
    a.qblocks = (int)(((long long)a.N * a.G + kFewRows - 1) / kFewRows);
    a.prows = (int)std::min<long long>(a.rows, (long long)a.N * a.G);
    a.min_units = 2;
    a.fixed = 2;
    a.whole = 10;
    cudaError_t err = a.dh <= 64 ? launch_dc<1>(a, nsm, &ctas, s) : launch_dc<2>(a, nsm, &ctas, s);
    if (err != cudaSuccess) return err;
    return launch_combine(a, MOE_DTYPE_BF16, ctas, s);
}

}  // namespace attn
}  // namespace moe
