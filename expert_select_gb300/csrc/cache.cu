// Writes to the paged key/value cache: the block's new rows (with q/k norms and rotary
// positions), and the move of an accepted path to the front of its block. Both are bound by
// memory (each row read and written once) and by launch latency when small. Measured: 6276 rows of
// 80 heads of 64 23.7 us (128.5 MB, 5.4 TB/s, 0.8 of the copy bandwidth; half of the issue slots used;
// four rows a CTA took 26.2), 64 single tokens 4.2 us, 256 accepted paths 3.8 us.
#include <algorithm>

#include "cache.cuh"

namespace moe {
namespace cache {
namespace {

constexpr int kThr = 128;

// W elements in a row, as they lie in memory and as fp32.
template <typename T, int W> struct Run;
template <int W> struct Run<__nv_bfloat16, W> {
    uint32_t r[W / 2];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        if constexpr (W == 8) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p);
            r[0] = u.x; r[1] = u.y; r[2] = u.z; r[3] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            r[0] = u.x; r[1] = u.y;
        }
    }
    __device__ __forceinline__ void get(float v[W]) const {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            v[2 * i] = bf16_lo(r[i]);
            v[2 * i + 1] = bf16_hi(r[i]);
        }
    }
    __device__ __forceinline__ static void store(__nv_bfloat16 *p, const float v[W]) {
        uint32_t w[W / 2];
#pragma unroll
        for (int i = 0; i < W / 2; ++i) w[i] = attn::pack_bf16(v[2 * i], v[2 * i + 1]);
        if constexpr (W == 8)
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
};
template <int W> struct Run<float, W> {
    float r[W];
    __device__ __forceinline__ void load(const float *p) {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const float4 u = *reinterpret_cast<const float4 *>(p + 4 * i);
            r[4 * i] = u.x; r[4 * i + 1] = u.y; r[4 * i + 2] = u.z; r[4 * i + 3] = u.w;
        }
    }
    __device__ __forceinline__ void get(float v[W]) const {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = r[i];
    }
    __device__ __forceinline__ static void store(float *p, const float v[W]) {
#pragma unroll
        for (int i = 0; i < W / 4; ++i)
            *reinterpret_cast<float4 *>(p + 4 * i) =
                make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
};

// a + b (a in .x) with what the sum loses added to .y (two-sum: exact).
__device__ __forceinline__ float2 add_kept(float2 a, float b) {
    const float s = a.x + b, t = s - a.x;
    return make_float2(s, a.y + ((a.x - (s - t)) + (b - t)));
}

// Fraction of a turn (.x, within half a turn of 0, and .y, some 2^-24 of one) that pos * freq
// radians leave. 1 / (2 pi) is taken as the sum of two fp32 values and the product with pos, cut into
// parts below 2^15 and 2^16 that are exact in fp32, with its rounding error; what the sum of the
// parts' fractions loses is kept in .y. Of the turns pos freq / (2 pi) at most 2^-45 are lost in all
// (emulated on the CPU: 1.5e-9 turns at positions up to 10^6, 3e-8 up to 2^24), where
// a plain fp32 product is off by up to 0.06 rad at 10^6 and the fraction as one fp32 value by
// 6e-8 turns.
__device__ __forceinline__ float2 turns(int pos, float freq) {
    constexpr double kInv = 0.15915494309189533577;  // 1 / (2 pi)
    constexpr float hi = (float)kInv, lo = (float)(kInv - (double)hi);
    const float c = freq * hi, ce = fmaf(freq, hi, -c) + freq * lo;
    const float big = (float)(pos & ~0xffff), small = (float)(pos & 0xffff);
    const float b = big * c, s = small * c;
    const float be = fmaf(big, c, -b) + big * ce, se = fmaf(small, c, -s) + small * ce;
    float2 t = add_kept(make_float2(b - rintf(b), 0.f), s - rintf(s));
    t = add_kept(add_kept(t, be), se);
    t.x -= rintf(t.x);
    return t;
}

// A head's elements of one lane become x / sqrt(mean x^2 + eps), ss being the head's fp32 sum of
// squares. It serves unless it overflows, or is so small that squares lost below fp32's range
// count; then the head is scaled by a power of two first. group: the lanes of the head.
template <int W, int LPH>
__device__ __forceinline__ float head_scale(float (&vx)[W], float (&vy)[W], bool on, float ss, int dh,
                                            float eps, uint32_t group) {
    if ((ss < INFINITY && (ss > 1e-25f * (float)dh || eps > 1e-30f)) || ss != ss)
        return 1.f / sqrtf(ss / (float)dh + eps);
    float mx = 0.f;
    if (on) {
#pragma unroll
        for (int j = 0; j < W; ++j) mx = fmaxf(mx, fmaxf(fabsf(vx[j]), fabsf(vy[j])));
    }
#pragma unroll
    for (int o = LPH / 2; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(group, mx, o, LPH));
    if (mx == 0.f || mx == INFINITY) return mx == 0.f ? 1.f / sqrtf(eps) : 0.f;
    int ex;
    frexpf(mx, &ex);  // mx = f 2^ex, f in [0.5, 1)
    ex = max(ex, -126);
    // mean + eps = 2^(2 ex) (t / dh + eps 2^(-2 ex)), t of the head scaled by 2^-ex
    const double e2 = ldexp((double)eps, -2 * ex);
    if (e2 > 1e30) return 1.f / sqrtf(eps);  // the mean is far below eps
    const float down = ldexpf(1.f, -ex);
    float t = 0.f;
    if (on) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
            vx[j] *= down;
            vy[j] *= down;
            t = fmaf(vx[j], vx[j], fmaf(vy[j], vy[j], t));
        }
    }
#pragma unroll
    for (int o = LPH / 2; o >= 1; o >>= 1) t += __shfl_xor_sync(group, t, o, LPH);
    return 1.f / sqrtf(t / (float)dh + (float)e2);
}

// A CTA per row. The row's angles are formed once; LPH lanes take a head at a time, a lane
// W elements and their rotary partners rot / 2 further on (behind rot: two runs that only pass
// through). The next heads' elements are on their way while a pass is computed.
template <typename T, int W, int LPH>
__global__ void __launch_bounds__(kThr) append_kernel(const AppendArgs a) {
    __shared__ __align__(16) float s_cos[128], s_sin[128];  // of the rot / 2 <= 128 angles
    pdl_wait();
    const int r = blockIdx.x, tid = threadIdx.x;
    const int sub = tid & (LPH - 1), first = tid / LPH;
    const int half = a.inv_freq ? a.rot / 2 : 0, rot = 2 * half;
    const bool on = sub * 2 * W < a.dh, turned = sub * W < half;
    const int ca = turned ? sub * W : rot + (sub * W - half);
    const int cb = ca + (turned ? half : (a.dh - rot) / 2);
    const int q_heads = a.q ? a.H : 0, heads = q_heads + 2 * a.Hkv;
    Run<T, W> x, y;
    auto fetch = [&](int i) {
        if (i >= heads || !on) return;
        const T *src;
        if (i < q_heads)
            src = (const T *)a.q + (size_t)r * a.ldq + (size_t)i * a.dh;
        else if (i < q_heads + a.Hkv)
            src = (const T *)a.k + (size_t)r * a.ldk + (size_t)(i - q_heads) * a.dh;
        else
            src = (const T *)a.v + (size_t)r * a.ldv + (size_t)(i - q_heads - a.Hkv) * a.dh;
        x.load(src + ca);
        y.load(src + cb);
    };
    fetch(first);
    // the row's sequence and node; every thread looks them up (the loads are shared)
    int b, n0, n;
    if (a.row_start) {
        // the last sequence that starts at or before r (row_start ascends)
        int lo = 0, hi = a.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.row_start[mid] <= r) lo = mid; else hi = mid - 1;
        }
        b = lo;
        n0 = a.row_start[b];
        n = a.row_start[b + 1] - n0;
    } else {
        b = r / a.N;
        n0 = b * a.N;
        n = a.N;
    }
    const int node = r - n0;
    if (node < 0 || node >= n || node >= a.N) {  // not a row of any sequence
        if (tid == 0 && a.flags && r < a.row_start[a.B]) atomicOr(a.flags, FLAG_BAD_SEQUENCE);
        return;
    }
    const int len = a.cache_len[b];
    const int pos = len + (a.depth ? a.depth[r] : node);
    bool write = len >= 0 && len < a.cap - node;
    size_t dst = 0;
    if (!write) {
        if (tid == 0 && a.flags) atomicOr(a.flags, FLAG_BAD_SEQUENCE);
    } else {
        const int slot = len + node, pi = slot / a.page;
        const int pg = a.table[(size_t)b * a.max_pages + pi];
        if (pg < 0 || pg >= a.n_pages) {
            write = false;
            if (tid == 0 && a.flags) atomicOr(a.flags, FLAG_BAD_PAGE);
        } else {
            dst = (size_t)pg * a.st_page + (size_t)(slot - pi * a.page) * a.st_tok;
        }
    }
    for (int i = tid; i < half; i += kThr) {
        const float2 t = turns(pos, a.inv_freq[i]);
        float s, c;
        sincospif(2.f * t.x, &s, &c);
        const float d = 6.2831853071795865f * t.y;  // (its square is below 2^-40)
        s_cos[i] = fmaf(-s, d, c) * a.rope_scale;
        s_sin[i] = fmaf(c, d, s) * a.rope_scale;
    }
    __syncthreads();

    for (int i = first; i < heads; i += kThr / LPH) {
        const bool is_q = i < q_heads, is_v = i >= q_heads + a.Hkv;
        const int h = is_q ? i : (is_v ? i - q_heads - a.Hkv : i - q_heads);
        float vx[W], vy[W];
        x.get(vx);
        y.get(vy);
        fetch(i + kThr / LPH);
        const T *w = is_v ? nullptr : (const T *)(is_q ? a.wq : a.wk);
        if (w) {
            float ss = 0.f;
            if (on) {
#pragma unroll
                for (int j = 0; j < W; ++j) ss = fmaf(vx[j], vx[j], fmaf(vy[j], vy[j], ss));
            }
            // the lanes of a head run together; the others of the warp may be elsewhere
            const uint32_t group =
                LPH == 32 ? 0xffffffffu : ((1u << LPH) - 1u) << (tid & 31 & ~(LPH - 1));
#pragma unroll
            for (int o = LPH / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(group, ss, o, LPH);
            const float f = head_scale<W, LPH>(vx, vy, on, ss, a.dh, a.eps, group);
            if (on) {
                Run<T, W> wx, wy;
                float fx[W], fy[W];
                wx.load(w + ca);
                wy.load(w + cb);
                wx.get(fx);
                wy.get(fy);
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    vx[j] *= f * fx[j];
                    vy[j] *= f * fy[j];
                }
            }
        }
        if (!on || (!is_q && !write)) continue;
        if (turned && !is_v) {
#pragma unroll
            for (int j = 0; j < W; j += 4) {
                const float4 c4 = *reinterpret_cast<const float4 *>(s_cos + ca + j);
                const float4 s4 = *reinterpret_cast<const float4 *>(s_sin + ca + j);
                const float cz[4] = {c4.x, c4.y, c4.z, c4.w}, sz[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const float p = vx[j + z], q = vy[j + z];
                    vx[j + z] = p * cz[z] - q * sz[z];
                    vy[j + z] = q * cz[z] + p * sz[z];
                }
            }
        }
        T *out = is_q ? (T *)a.q_out + ((size_t)r * a.H + h) * a.dh
                      : (T *)(is_v ? a.vp : a.kp) + dst + (size_t)h * a.st_head;
        Run<T, W>::store(out + ca, vx);
        Run<T, W>::store(out + cb, vy);
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
        // (m < j: behind a bad node the path may ascend again from a low one, and slot len + j
        // need not lie in the table; an ascending path has m >= j)
        if (m <= prev || m < j || m >= a.cap - len) {
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
    // 8 elements and their partners to a lane where both halves of a head, and what lies behind the
    // rotated part, are multiples of 8 elements; else 4
    const bool wide = a.dh % 16 == 0 && a.rot % 16 == 0;
    auto *k = wide ? (a.dh <= 64    ? append_kernel<T, 8, 4>
                      : a.dh <= 128 ? append_kernel<T, 8, 8>
                                    : append_kernel<T, 8, 16>)
                   : (a.dh <= 64    ? append_kernel<T, 4, 8>
                      : a.dh <= 128 ? append_kernel<T, 4, 16>
                                    : append_kernel<T, 4, 32>);
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
