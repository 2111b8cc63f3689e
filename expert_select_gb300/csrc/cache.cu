// Writes to the paged key/value cache: the block's new rows (with q/k norms and rotary
// positions), and the move of an accepted path to the front of its block. Both are bound by
// memory (each row read and written once) and by launch latency when small.
#include <algorithm>

#include "cache.cuh"

namespace moe {
namespace cache {
namespace {

constexpr int kThr = 128;

// Two consecutive elements at p as fp32, and back.
__device__ __forceinline__ float2 load2(const __nv_bfloat16 *p) {
    const uint32_t u = *reinterpret_cast<const uint32_t *>(p);
    return make_float2(bf16_lo(u), bf16_hi(u));
}
__device__ __forceinline__ float2 load2(const float *p) {
    return *reinterpret_cast<const float2 *>(p);
}
__device__ __forceinline__ void store2(__nv_bfloat16 *p, float2 v) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.x, v.y);
}
__device__ __forceinline__ void store2(float *p, float2 v) { *reinterpret_cast<float2 *>(p) = v; }

// A CTA per row. The row's angles are formed once (pos * inv_freq in fp64, reduced to a
// fraction of a turn there: at position 10^6 an fp32 product would be off by up to 0.06 rad),
// then LPH lanes take a head at a time: unit u of a head is the elements (2u, 2u + 1) and their
// rotary partners rot / 2 further on (behind rot: two pairs that only pass through).
template <typename T, int LPH, int UPL>
__global__ void __launch_bounds__(kThr) append_kernel(const AppendArgs a) {
    __shared__ float2 cs[128];  // cos, sin of the rot / 2 <= 128 angles
    __shared__ int s_seq[2];
    pdl_wait();
    const int r = blockIdx.x, tid = threadIdx.x;
    // the row's sequence and node
    int b, n0, n;
    if (a.row_start) {
        if (tid == 0) {
            // the last sequence that starts at or before r (row_start ascends)
            int lo = 0, hi = a.B - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (a.row_start[mid] <= r) lo = mid; else hi = mid - 1;
            }
            s_seq[0] = lo;
        }
        __syncthreads();
        b = s_seq[0];
        n0 = a.row_start[b];
        n = a.row_start[b + 1] - n0;
    } else {
        b = r / a.N;
        n0 = b * a.N;
        n = a.N;
    }
    const int node = r - n0;
    const int len = a.cache_len[b];
    if (node < 0 || node >= n || node >= a.N) {  // not a row of any sequence
        if (tid == 0 && a.flags && r < a.row_start[a.B]) atomicOr(a.flags, FLAG_BAD_SEQUENCE);
        return;
    }
    const long long pos = (long long)len + (a.depth ? a.depth[r] : node);
    const long long slot = (long long)len + node;
    bool write = true;
    size_t dst = 0;
    if (len < 0 || slot >= a.cap) {
        write = false;
        if (tid == 0 && a.flags) atomicOr(a.flags, FLAG_BAD_SEQUENCE);
    } else {
        const int pi = (int)slot / a.page, pg = a.table[(size_t)b * a.max_pages + pi];
        if (pg < 0 || pg >= a.n_pages) {
            write = false;
            if (tid == 0 && a.flags) atomicOr(a.flags, FLAG_BAD_PAGE);
        } else {
            dst = (size_t)pg * a.st_page + (size_t)((int)slot - pi * a.page) * a.st_tok;
        }
    }
    const int half = a.inv_freq ? a.rot / 2 : 0;
    for (int i = tid; i < half; i += kThr) {
        double t = (double)pos * (double)a.inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
        t -= rint(t);
        float s, c;
        sincospif(2.f * (float)t, &s, &c);
        cs[i] = make_float2(c * a.rope_scale, s * a.rope_scale);
    }
    __syncthreads();

    const int sub = tid & (LPH - 1), first = tid / LPH;
    const int units = a.dh / 4, rot = 2 * half;
    const int q_heads = a.q ? a.H : 0;
    for (int i = first; i < q_heads + 2 * a.Hkv; i += kThr / LPH) {
        const bool is_q = i < q_heads, is_v = i >= q_heads + a.Hkv;
        const int h = is_q ? i : (is_v ? i - q_heads - a.Hkv : i - q_heads);
        const T *src = is_q ? (const T *)a.q + (size_t)r * a.ldq
                            : (is_v ? (const T *)a.v + (size_t)r * a.ldv
                                    : (const T *)a.k + (size_t)r * a.ldk);
        src += (size_t)h * a.dh;
        float2 x[UPL], y[UPL];
        int ca[UPL], cb[UPL];
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < UPL; ++j) {
            const int u = sub + j * LPH;
            if (u < units) {
                const int w = u - half / 2;
                ca[j] = w < 0 ? 2 * u : rot + 2 * w;
                cb[j] = ca[j] + (w < 0 ? half : (a.dh - rot) / 2);
                x[j] = load2(src + ca[j]);
                y[j] = load2(src + cb[j]);
                ss += x[j].x * x[j].x + x[j].y * x[j].y + y[j].x * y[j].x + y[j].y * y[j].y;
            }
        }
        const T *w = is_v ? nullptr : (const T *)(is_q ? a.wq : a.wk);
        float f = 1.f;
        if (w) {
            // the lanes of a head run together; the other half of the warp may be elsewhere
            const uint32_t group = LPH == 32 ? 0xffffffffu : 0xffffu << (tid & 16);
#pragma unroll
            for (int o = LPH / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(group, ss, o, LPH);
            f = 1.f / sqrtf(ss / (float)a.dh + a.eps);
        }
        T *out = is_q ? (T *)a.q_out + ((size_t)r * a.H + h) * a.dh
                      : (T *)(is_v ? a.vp : a.kp) + dst + (size_t)h * a.st_head;
        if (!is_q && !write) continue;
#pragma unroll
        for (int j = 0; j < UPL; ++j) {
            const int u = sub + j * LPH;
            if (u < units) {
                if (w) {
                    const float2 wx = load2(w + ca[j]), wy = load2(w + cb[j]);
                    x[j].x *= f * wx.x;
                    x[j].y *= f * wx.y;
                    y[j].x *= f * wy.x;
                    y[j].y *= f * wy.y;
                }
                if (!is_v && u < half / 2) {
                    const float2 c0 = cs[2 * u], c1 = cs[2 * u + 1];
                    const float2 p = x[j], q = y[j];
                    x[j].x = p.x * c0.x - q.x * c0.y;
                    y[j].x = q.x * c0.x + p.x * c0.y;
                    x[j].y = p.y * c1.x - q.y * c1.y;
                    y[j].y = q.y * c1.x + p.y * c1.y;
                }
                store2(out + ca[j], x[j]);
                store2(out + cb[j], y[j]);
            }
        }
    }
}

// A CTA per sequence, a thread per 16-byte piece of a slot (K and V of every head). Node
// path[j] >= j, and the path ascends, so slot j is never the source of a later move: pieces are
// read eight moves at a time and then written.
__global__ void __launch_bounds__(256) commit_kernel(const CommitArgs a) {
    __shared__ int s_bad;
    pdl_wait();
    const int b = blockIdx.x, tid = threadIdx.x;
    const int len = a.cache_len[b];
    int n = a.n_accept[b];
    if (tid == 0) s_bad = INT_MAX;
    __syncthreads();
    int flag = 0;
    if (n < 0 || n > a.P || len < 0) {
        flag = FLAG_BAD_SEQUENCE;
        n = len < 0 ? 0 : max(0, min(n, a.P));
    }
    const int *path = a.path + (size_t)b * a.P;
    const int *table = a.table + (size_t)b * a.max_pages;
    // the first node that is not above its predecessor or has no valid page ends the path
    for (int j = tid; j < n; j += blockDim.x) {
        const int m = path[j], prev = j > 0 ? path[j - 1] : -1;
        int f = 0;
        if (m <= prev || m < 0 || m >= a.cap - len) {
            f = FLAG_BAD_SEQUENCE;
        } else {
            const int ps = table[(len + m) / a.page], pd = table[(len + j) / a.page];
            if (ps < 0 || ps >= a.n_pages || pd < 0 || pd >= a.n_pages) f = FLAG_BAD_PAGE;
        }
        if (f) {
            flag |= f;
            atomicMin(&s_bad, j);
        }
    }
    if (flag && a.flags) atomicOr(a.flags, flag);
    __syncthreads();
    n = min(n, s_bad);
    const int per_head = a.row_bytes / 16;
    const int pieces = 2 * a.Hkv * per_head;
    for (int i = tid; i < pieces; i += blockDim.x) {
        const int which = i / (a.Hkv * per_head), w = i % (a.Hkv * per_head);
        const int h = w / per_head, c = w % per_head;
        char *pool = (char *)(which ? a.vp : a.kp) + (size_t)h * a.st_head + (size_t)c * 16;
        for (int j0 = 0; j0 < n; j0 += 8) {
            uint4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j0 + j < n) {
                    const int slot = len + path[j0 + j], pi = slot / a.page;
                    v[j] = *reinterpret_cast<const uint4 *>(pool + (size_t)table[pi] * a.st_page +
                                                            (size_t)(slot - pi * a.page) * a.st_tok);
                }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j0 + j < n && path[j0 + j] != j0 + j) {
                    const int slot = len + j0 + j, pi = slot / a.page;
                    *reinterpret_cast<uint4 *>(pool + (size_t)table[pi] * a.st_page +
                                               (size_t)(slot - pi * a.page) * a.st_tok) = v[j];
                }
        }
    }
    if (tid == 0) a.new_len[b] = len + n;
}

template <typename T> cudaError_t append_t(const AppendArgs &a, cudaStream_t s) {
    // 16 lanes hold a head of up to 64 elements, 32 lanes one of up to 128 (or 256)
    auto *k = a.dh <= 64    ? append_kernel<T, 16, 1>
              : a.dh <= 128 ? append_kernel<T, 32, 1>
                            : append_kernel<T, 32, 2>;
    return launch_pdl(k, dim3(a.R), dim3(kThr), 0, s, a);
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, int dtype, cudaStream_t s) {
    return dtype == MOE_DTYPE_BF16 ? append_t<__nv_bfloat16>(a, s) : append_t<float>(a, s);
}

cudaError_t launch_commit(const CommitArgs &a, cudaStream_t s) {
    const int pieces = 2 * a.Hkv * (a.row_bytes / 16);
    const int thr = std::min(256, ((pieces + 31) / 32) * 32);
    return launch_pdl(commit_kernel, dim3(a.B), dim3(thr), 0, s, a);
}

}  // namespace cache
}  // namespace moe
