// Paged attention on the CUDA cores, for every type and head size: fp32, and bf16 head sizes
// that the tensor-core kernel does not take. Also the merge of cut items.
//
//   out[n, h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - max)  over visible slots j
//
// computed in one pass over the keys with a running maximum and sum. An item is 32 rows
// (node, head in group) of one key/value head; a CTA of 128 threads takes a tile of 32 keys at a
// time: K and V rows go through the page table into shared memory as fp32, each thread forms 4
// rows x 2 keys of the scores, 16 lanes share a row's maximum and sum, and each thread
// accumulates 4 rows x dh / 16 columns of O in registers.
//
// Measured: chunks of 4096 fp32 tokens over 1021 slots 24 TFLOP/s (16/2 heads of 64, 2.14 ms) and
// 29.5 (32/4 heads of 128, 6.98 ms); 5 trees of 33 nodes with a window of 200 slots 25 us, where a
// CTA waits for its few tiles (the issue slots are used to 0.28 while it runs). bf16 heads of 256 (16/8):
// a chunk of 4096 tokens over 4003 15.8 ms (25.7 TFLOP/s), 64 single tokens over 4003 3.0 ms (0.7
// TB/s): the tensor-core kernels end at 128, where their two S buffers and O of two tiles fill
// tensor memory.
#include <algorithm>

#include "attn.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kBN = 32;
constexpr int kThr = 128;
constexpr int kLight = 0;  // every tile is one unit of work

// NC: 64-column chunks of the head size (dh <= 64 NC).
template <int NC> constexpr int simt_smem() {
    // Q and K rows padded by 4 floats (the 8 lanes of a 16-byte phase read different banks)
    return (32 * (64 * NC + 4) * 2 + 32 * 64 * NC + 32 * 36) * 4;
}

template <typename T>
__device__ __forceinline__ void load_row(float *dst, const T *src, int col, bool ok) {
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (ok) Vec8<T>::load(src + col, v);
    *reinterpret_cast<float4 *>(dst + col) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(dst + col + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

template <typename T, int NC>
__global__ void __launch_bounds__(kThr) attn_simt_kernel(const Args a) {
    extern __shared__ float sm[];
    __shared__ long long scratch[34];
    constexpr int D = 64 * NC, LD = D + 4;
    float *sQ = sm, *sK = sQ + 32 * LD, *sV = sK + 32 * LD, *sP = sV + 32 * D;  // sP [key][36]
    const int tid = threadIdx.x, tr = tid >> 4, tk = tid & 15;
    pdl_wait();
    Range r = attn_plan<kBN, kLight, kThr>(a, blockIdx.x, gridDim.x, scratch);
    if (tid == 0) write_record(a, blockIdx.x, r);
    const T *q = (const T *)a.q, *kp = (const T *)a.k, *vp = (const T *)a.v;
    Segment g;
    while (next_segment<kBN, kLight>(a, r, g)) {
        __syncthreads();
        // query rows, scaled so that scores are base-2 logits
        for (int i = tid; i < 32 * (D / 8); i += kThr) {
            const int row = i / (D / 8), col = (i % (D / 8)) * 8;
            const int qr = g.q0 + row;
            const bool ok = row < g.rows && col < a.dh;
            const int node = qr / a.G;
            const T *src = q + (size_t)(g.s.row0 + (ok ? node : 0)) * a.ldq +
                           (size_t)(g.h * a.G + (ok ? qr - node * a.G : 0)) * a.dh;
            load_row<T>(sQ + row * LD, src, col, ok);
#pragma unroll
            for (int c = 0; c < 8; ++c) sQ[row * LD + col + c] *= a.scale * kLog2e;
        }
        float m[4], l[4], acc[4][NC][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int x = 0; x < 4; ++x) acc[i][c][x] = 0.f;
        }
        // the half-warp's four rows: lanes 0-3 of it look up their visible bits
        const int vrow = tr * 4 + (tk & 3);
        const bool vok = vrow < g.rows;
        const int vnode = (g.q0 + (vok ? vrow : 0)) / a.G;
        const int vpos = node_position(a, g.s, vnode);
        for (int t = g.t; t < g.t + g.count; ++t) {
            const int k0 = g.tl.at(t) * kBN;
            __syncthreads();
            int bad = 0;
            for (int i = tid; i < 32 * (D / 8); i += kThr) {
                const int key = i / (D / 8), col = (i % (D / 8)) * 8;
                const int j = k0 + key;
                bool ok = j < g.s.L && col < a.dh && !out_of_reach(a, g.s, j, j);
                size_t off = 0;
                if (ok) {
                    const int pi = j / a.page, pg = a.table[(size_t)g.b * a.max_pages + pi];
                    if (pg < 0 || pg >= a.n_pages) {
                        ok = false;
                        bad = 1;
                    } else {
                        off = (size_t)pg * a.st_page + (size_t)(j - pi * a.page) * a.st_tok +
                              (size_t)g.h * a.st_head;
                    }
                }
                load_row<T>(sK + key * LD, kp + off, col, ok);
                load_row<T>(sV + key * D, vp + off, col, ok);
            }
            if (bad) atomicOr(a.flags, FLAG_BAD_PAGE);
            // slots of a page outside the pool are not visible
            uint32_t pages_ok = 0xffffffffu;
            {
                const int j = k0 + (tid & 31);
                bool ok = true;
                if (j < g.s.L && !out_of_reach(a, g.s, j, j)) {
                    const int pg = a.table[(size_t)g.b * a.max_pages + j / a.page];
                    ok = pg >= 0 && pg < a.n_pages;
                }
                pages_ok = __ballot_sync(0xffffffffu, ok);
            }
            uint32_t bits[1] = {0u};
            if (vok) visible_bits<1>(a, g.s, vnode, vpos, k0, bits);
            bits[0] &= pages_ok;
            __syncthreads();
            float s[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i][0] = s[i][1] = 0.f;
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                const float4 ka = *reinterpret_cast<const float4 *>(sK + tk * LD + c);
                const float4 kb = *reinterpret_cast<const float4 *>(sK + (tk + 16) * LD + c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 qv = *reinterpret_cast<const float4 *>(sQ + (tr * 4 + i) * LD + c);
                    s[i][0] += qv.x * ka.x + qv.y * ka.y + qv.z * ka.z + qv.w * ka.w;
                    s[i][1] += qv.x * kb.x + qv.y * kb.y + qv.z * kb.z + qv.w * kb.w;
                }
            }
            float p[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t vb = __shfl_sync(0xffffffffu, bits[0], (tid & 16) + i);
                const bool on0 = (vb >> tk) & 1u, on1 = (vb >> (tk + 16)) & 1u;
                const float s0 = on0 ? s[i][0] : -INFINITY, s1 = on1 ? s[i][1] : -INFINITY;
                float mx = fmaxf(s0, s1);
#pragma unroll
                for (int o = 8; o >= 1; o >>= 1)
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float mn = fmaxf(m[i], mx);
                const float base = mn == -INFINITY ? 0.f : mn;
                const float f = exp2f(m[i] - base);
                p[i][0] = on0 ? exp2f(s0 - base) : 0.f;
                p[i][1] = on1 ? exp2f(s1 - base) : 0.f;
                float sum = p[i][0] + p[i][1];
#pragma unroll
                for (int o = 8; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                l[i] = l[i] * f + sum;
                m[i] = mn;
                if (f != 1.f) {
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int x = 0; x < 4; ++x) acc[i][c][x] *= f;
                }
            }
            // P goes to the 16 lanes of its rows (one warp) through shared memory, key-major
            *reinterpret_cast<float4 *>(sP + tk * 36 + tr * 4) =
                make_float4(p[0][0], p[1][0], p[2][0], p[3][0]);
            *reinterpret_cast<float4 *>(sP + (tk + 16) * 36 + tr * 4) =
                make_float4(p[0][1], p[1][1], p[2][1], p[3][1]);
            __syncwarp();
#pragma unroll 2
            for (int key = 0; key < kBN; ++key) {
                const float4 pv = *reinterpret_cast<const float4 *>(sP + key * 36 + tr * 4);
                const float pr[4] = {pv.x, pv.y, pv.z, pv.w};
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const float4 v =
                        *reinterpret_cast<const float4 *>(sV + key * D + c * 64 + tk * 4);
                    // a slot that the row does not see (p = 0) takes no part, whatever it holds
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (pr[i] != 0.f) {
                            acc[i][c][0] += pr[i] * v.x;
                            acc[i][c][1] += pr[i] * v.y;
                            acc[i][c][2] += pr[i] * v.z;
                            acc[i][c][3] += pr[i] * v.w;
                        }
                }
            }
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = tr * 4 + i;
            if (row >= g.rows) continue;
            if (g.whole) {
                const int qr = g.q0 + row, node = qr / a.G, head = g.h * a.G + (qr - node * a.G);
                const size_t orow = (size_t)(g.s.row0 + node) * a.H + head;
                float lse;
                const float f = finish(m[i], l[i], a.sink, head, &lse);
                T *o = (T *)a.out + orow * a.dh;
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const int col = c * 64 + tk * 4;
                    if (col < a.dh) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) o[col + x] = from_float<T>(acc[i][c][x] * f);
                    }
                }
                if (a.lse && tk == 0) a.lse[orow] = lse;
            } else {
                const size_t pr = part_row(a, blockIdx.x, g, row);
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const int col = c * 64 + tk * 4;
                    if (col < a.dh)
                        *reinterpret_cast<float4 *>(a.part_o + pr * a.dh + col) =
                            make_float4(acc[i][c][0], acc[i][c][1], acc[i][c][2], acc[i][c][3]);
                }
                if (tk == 0) {
                    a.part_ml[pr * 2] = m[i];
                    a.part_ml[pr * 2 + 1] = l[i];
                }
            }
        }
    }
}

// Merges the cut items. Record c is of the item whose second part begins CTA c's range (if any):
// its first part is in slot 1 of CTA c - 1, the others in slot 0 of CTAs c, c + 1, ...:
//   sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i,  M the largest m_i.
// Every block lists the records in use (a block per possible record and row group would be
// thousands that find nothing to do) and takes every gridDim.x-th group of rows of all items. WPR
// warps share a row (8 / WPR rows per group), warp w taking the parts w, w + WPR, ...: a single
// long sequence leaves a few rows in many parts, whose reads must not queue up behind one another;
// large items have many rows in few parts. Sums run in a fixed order.
template <typename T, int WPR, int NC>  // NC: 128-column chunks of the head size
__global__ void __launch_bounds__(256) attn_combine_kernel(const Args a, int n_ctas) {
    __shared__ float s_o[WPR > 1 ? 8 : 1][128 * NC], s_ml[8][2];
    constexpr int kAt = NC == 1 ? 10 : 5;  // parts whose loads are in flight together
    __shared__ int s_list[kMaxCtas], s_count[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp % WPR;
    pdl_wait();
    int n_items = 0;
    for (int c0 = 0; c0 < n_ctas; c0 += 256) {
        const int c = c0 + threadIdx.x;
        const bool used = c < n_ctas && a.rec[c * 4 + 2] != 0;
        const uint32_t mask = __ballot_sync(0xffffffffu, used);
        if (lane == 0) s_count[warp] = __popc(mask);
        __syncthreads();
        int at = n_items;
        for (int x = 0; x < 8; ++x) {
            if (x == warp && used) s_list[at + __popc(mask & ((1u << lane) - 1u))] = c;
            at += s_count[x];
        }
        n_items = at;
        __syncthreads();
    }
    const int groups = (a.prows + 8 / WPR - 1) / (8 / WPR);
    for (int work = blockIdx.x; work < n_items * groups; work += gridDim.x) {
        const int c = s_list[work / groups];
        const int4 rec = *reinterpret_cast<const int4 *>(a.rec + c * 4);
        const int e = rec.x, h = rec.y;
        const int b = e / a.qblocks, q0 = (e - b * a.qblocks) * a.rows;
        const Seq s = sequence(a, b);
        const int row = (work % groups) * (8 / WPR) + warp / WPR;
        const bool live = row < min(a.rows, s.n * a.G - q0);
        if (WPR == 1 && !live) continue;
        const int parts = live ? rec.z : 0;
        auto part = [&](int i) { return ((size_t)(c - 1 + i) * 2 + (i == 0)) * a.prows + row; };
        float acc[NC][4];  // columns 4 lane + 128 c
#pragma unroll
        for (int x = 0; x < NC; ++x) acc[x][0] = acc[x][1] = acc[x][2] = acc[x][3] = 0.f;
        float base = -INFINITY, l = 0.f;
        for (int i0 = w; i0 < parts; i0 += WPR * kAt) {
            float2 ml[kAt];
            float4 v[kAt][NC];
#pragma unroll
            for (int y = 0; y < kAt; ++y) {
                const int i = i0 + y * WPR;
                ml[y] = make_float2(-INFINITY, 0.f);
                if (i < parts) {
                    ml[y] = *reinterpret_cast<const float2 *>(a.part_ml + part(i) * 2);
#pragma unroll
                    for (int x = 0; x < NC; ++x) {
                        const int col = x * 128 + lane * 4;
                        v[y][x] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (col < a.dh)
                            v[y][x] = *reinterpret_cast<const float4 *>(a.part_o + part(i) * a.dh + col);
                    }
                }
            }
            float top = base;
#pragma unroll
            for (int y = 0; y < kAt; ++y)
                if (ml[y].y != 0.f) top = fmaxf(top, ml[y].x);  // (a part that saw nothing has sum 0)
            const float f = base == -INFINITY ? 0.f : exp2f(base - top);
            base = top;
            l *= f;
#pragma unroll
            for (int x = 0; x < NC; ++x)
#pragma unroll
                for (int z = 0; z < 4; ++z) acc[x][z] *= f;
            const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int y = 0; y < kAt; ++y) {
                const float wy = ml[y].y == 0.f ? 0.f : exp2f(ml[y].x - ref);
                if (wy == 0.f && ml[y].y == ml[y].y) continue;  // (a NaN sum goes through)
                l += wy * ml[y].y;
#pragma unroll
                for (int x = 0; x < NC; ++x) {
                    acc[x][0] += wy * v[y][x].x;
                    acc[x][1] += wy * v[y][x].y;
                    acc[x][2] += wy * v[y][x].z;
                    acc[x][3] += wy * v[y][x].w;
                }
            }
        }
        if constexpr (WPR > 1) {
#pragma unroll
            for (int x = 0; x < NC; ++x)
                *reinterpret_cast<float4 *>(&s_o[warp][x * 128 + lane * 4]) =
                    make_float4(acc[x][0], acc[x][1], acc[x][2], acc[x][3]);
            if (lane == 0) {
                s_ml[warp][0] = base;
                s_ml[warp][1] = l;
            }
            __syncthreads();
            if (w == 0 && live) {
                float top = base;
#pragma unroll
                for (int x = 1; x < WPR; ++x)
                    if (s_ml[warp + x][1] != 0.f) top = fmaxf(top, s_ml[warp + x][0]);
                const float ref = top == -INFINITY ? 0.f : top;
                const float f = base == -INFINITY ? 0.f : exp2f(base - ref);
                l *= f;
#pragma unroll
                for (int x = 0; x < NC; ++x)
#pragma unroll
                    for (int z = 0; z < 4; ++z) acc[x][z] *= f;
#pragma unroll
                for (int y = 1; y < WPR; ++y) {
                    const float ly = s_ml[warp + y][1];
                    const float wy = ly == 0.f ? 0.f : exp2f(s_ml[warp + y][0] - ref);
                    if (wy == 0.f && ly == ly) continue;
                    l += wy * ly;
#pragma unroll
                    for (int x = 0; x < NC; ++x) {
                        const float4 v =
                            *reinterpret_cast<const float4 *>(&s_o[warp + y][x * 128 + lane * 4]);
                        acc[x][0] += wy * v.x;
                        acc[x][1] += wy * v.y;
                        acc[x][2] += wy * v.z;
                        acc[x][3] += wy * v.w;
                    }
            }
            base = top;
            }
        }
        if (w == 0 && live) {
            const int qr = q0 + row, node = qr / a.G, head = h * a.G + (qr - node * a.G);
            const size_t orow = (size_t)(s.row0 + node) * a.H + head;
            float lse;
            const float f = finish(base, l, a.sink, head, &lse);
            T *out = (T *)a.out + orow * a.dh;
#pragma unroll
            for (int x = 0; x < NC; ++x) {
                const int col = x * 128 + lane * 4;
                if (col < a.dh) {
#pragma unroll
                    for (int z = 0; z < 4; ++z) out[col + z] = from_float<T>(acc[x][z] * f);
                }
        }
        if (a.lse && lane == 0) a.lse[orow] = lse;
        }
        if (WPR > 1) __syncthreads();  // the next group writes s_o again
    }
}

template <typename T, int NC> cudaError_t combine_nc(const Args &a, int n_ctas, cudaStream_t s) {
    const int sms = device_sms();
    if (a.prows <= kFewRows)
        return launch_pdl(attn_combine_kernel<T, 8, NC>, dim3(2 * sms), dim3(256), 0, s, a, n_ctas);
    return launch_pdl(attn_combine_kernel<T, 1, NC>, dim3(4 * sms), dim3(256), 0, s, a, n_ctas);
}
template <typename T> cudaError_t combine_t(const Args &a, int n_ctas, cudaStream_t s) {
    return a.dh <= 128 ? combine_nc<T, 1>(a, n_ctas, s) : combine_nc<T, 2>(a, n_ctas, s);
}

template <typename T, int NC>
cudaError_t launch_nc(const Args &a, int nsm, int *ctas, cudaStream_t s) {
    constexpr int smem = simt_smem<NC>();
    const cudaError_t err = allow_smem(attn_simt_kernel<T, NC>, smem);
    if (err != cudaSuccess) return err;
    // CTAs per SM that shared memory (228 KB, 1 KB of it per CTA) allows, at most four
    *ctas = std::min(kMaxCtas, nsm * std::max(1, std::min(4, (228 * 1024) / (smem + 2048))));
    return launch_pdl(attn_simt_kernel<T, NC>, dim3(*ctas), dim3(kThr), smem, s, a);
}

template <typename T> cudaError_t launch_t(const Args &a, int nsm, int *ctas, cudaStream_t s) {
    switch ((a.dh + 63) / 64) {
        case 1: return launch_nc<T, 1>(a, nsm, ctas, s);
        case 2: return launch_nc<T, 2>(a, nsm, ctas, s);
        case 3: return launch_nc<T, 3>(a, nsm, ctas, s);
        default: return launch_nc<T, 4>(a, nsm, ctas, s);
    }
}

}  // namespace

cudaError_t launch_combine(const Args &a, int dtype, int n_ctas, cudaStream_t s) {
    return dtype == MOE_DTYPE_BF16 ? combine_t<__nv_bfloat16>(a, n_ctas, s)
                                   : combine_t<float>(a, n_ctas, s);
}

cudaError_t launch_simt(Args a, int dtype, cudaStream_t s) {
    const int nsm = device_sms();
    if (nsm <= 0) return cudaErrorInvalidDevice;
    int ctas = 0;
    a.rows = kSimtRows;
    a.qblocks = (int)(((long long)a.N * a.G + kSimtRows - 1) / kSimtRows);
    a.prows = (int)std::min<long long>(a.rows, (long long)a.N * a.G);
    a.min_units = 2;
    a.fixed = 2;
    a.whole = 8;
    cudaError_t err = dtype == MOE_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a, nsm, &ctas, s)
                                  : launch_t<float>(a, nsm, &ctas, s);
    if (err != cudaSuccess) return err;
    return launch_combine(a, dtype, ctas, s);
}

}  // namespace attn
}  // namespace moe
