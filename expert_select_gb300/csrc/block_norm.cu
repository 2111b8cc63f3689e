// The norms and the residual between the two halves of a decoder block in one pass:
//   u = w_post (.) branch / rms(branch);  h = x + scale gate (.) u;  hn = w_pre (.) h / rms(h)
// Each input is read and each output written once; the row stays in registers between the two
// sums of squares. Bound by memory: 4 R d elements.
#include <algorithm>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kMaxThr = 512;  // 8-element pieces: one a thread up to 4096 columns, else two

// An 8-element piece as it lies in memory (bf16: 16 bytes, fp32: 32), and its four pairs as fp32.
template <typename T> struct Piece;
template <> struct Piece<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        a = *reinterpret_cast<const uint4 *>(p);
    }
    __device__ __forceinline__ void get(uint64_t v[4]) const {
        v[0] = pack2(bf16_lo(a.x), bf16_hi(a.x));
        v[1] = pack2(bf16_lo(a.y), bf16_hi(a.y));
        v[2] = pack2(bf16_lo(a.z), bf16_hi(a.z));
        v[3] = pack2(bf16_lo(a.w), bf16_hi(a.w));
    }
    __device__ __forceinline__ static void store(__nv_bfloat16 *p, const uint64_t v[4]) {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 f = unpack2(v[q]);
            const __nv_bfloat162 t = __floats2bfloat162_rn(f.x, f.y);
            w[q] = *reinterpret_cast<const uint32_t *>(&t);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Piece<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = *reinterpret_cast<const float4 *>(p);
        b = *(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void get(uint64_t v[4]) const {
        v[0] = pack2(a.x, a.y);
        v[1] = pack2(a.z, a.w);
        v[2] = pack2(b.x, b.y);
        v[3] = pack2(b.z, b.w);
    }
    __device__ __forceinline__ static void store(float *p, const uint64_t v[4]) {
        const float2 x = unpack2(v[0]), y = unpack2(v[1]), z = unpack2(v[2]), w = unpack2(v[3]);
        reinterpret_cast<float4 *>(p)[0] = make_float4(x.x, x.y, y.x, y.y);
        reinterpret_cast<float4 *>(p)[1] = make_float4(z.x, z.y, w.x, w.y);
    }
};

// Sum (MAX false) or largest value over the CTA; every thread gets it. part: two buffers of 16
// floats used in turn, so that one barrier per reduction is enough.
template <bool MAX> __device__ __forceinline__ float cta_reduce(float v, float (*part)[16], int &turn) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const float w = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? fmaxf(v, w) : v + w;
    }
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    float *p = part[turn];
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    float t = lane < warps ? p[lane] : 0.f;  // (0 is neutral: maxima here are of absolute values)
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) {
        const float w = __shfl_xor_sync(0xffffffffu, t, o);
        t = MAX ? fmaxf(t, w) : t + w;
    }
    return __shfl_sync(0xffffffffu, t, 0);
}

// 1 / sqrt(mean v^2 + eps) of the row. The fp32 sum of squares serves unless it overflows, or is so
// small that squares lost below fp32's range count against eps too; then the row is scaled by a
// power of two first (v is left scaled: the factor is the scaled row's).
template <int NV>
__device__ __forceinline__ float row_scale(uint64_t (&v)[NV][4], int nv, int d, float eps,
                                           float (*part)[16], int &turn) {
    uint64_t s2 = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (i < nv) {
#pragma unroll
            for (int q = 0; q < 4; ++q) s2 = fma2(v[i][q], v[i][q], s2);
        }
    const float2 sp = unpack2(s2);
    const float s = cta_reduce<false>(sp.x + sp.y, part, turn);
    if ((s < INFINITY && (s > 1e-25f * (float)d || eps > 1e-30f)) || s != s)
        return rsqrtf(s * (1.f / (float)d) + eps);
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (i < nv) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 f = unpack2(v[i][q]);
                mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
        }
    mx = cta_reduce<true>(mx, part, turn);
    if (mx == 0.f || mx == INFINITY) return mx == 0.f ? 1.f / sqrtf(eps) : 0.f;
    int ex;
    frexpf(mx, &ex);  // mx = f 2^ex, f in [0.5, 1)
    // mean + eps = 2^(2 ex) (t / d + eps 2^(-2 ex)), t of the row scaled by 2^-ex
    const double e2 = ldexp((double)eps, -2 * ex);
    if (e2 > 1e30) return 1.f / sqrtf(eps);  // the mean is far below eps
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (i < nv) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float2 f = unpack2(v[i][q]);
                f.x = ldexpf(f.x, -ex);
                f.y = ldexpf(f.y, -ex);
                t = fmaf(f.x, f.x, fmaf(f.y, f.y, t));
                v[i][q] = pack2(f.x, f.y);
            }
        }
    t = cta_reduce<false>(t, part, turn);
    return 1.f / sqrtf(t / (float)d + (float)e2);
}

// A CTA takes every gridDim.x-th row. The rows of x, branch and gate come through a ring of two
// stages in shared memory; each thread copies with cp.async the pieces that it alone reads, so the
// ring needs no barrier, and x and branch may be the buffers that h and hn go to. The weights are
// read again for every row (from L1).
template <typename T, int NV>
__global__ void __launch_bounds__(kMaxThr)
block_norm_kernel(const T *x, const T *branch, const T *__restrict__ w_post,
                  const T *__restrict__ gate, int gate_rows, float scale,
                  const T *__restrict__ w_pre, float eps, int R, int d, T *h, T *hn) {
    constexpr int kStages = 2;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float part[2][16];
    int turn = 0;
    const int step = blockDim.x * 8, c0 = threadIdx.x * 8;
    const int nv = c0 < d ? (d - c0 + step - 1) / step : 0;
    T *ring = reinterpret_cast<T *>(smem) + c0;  // [stage][x, branch, gate][d]
    pdl_wait();
    auto fetch = [&](int row, int stage) {
        if (row < R) {
            const T *src[3] = {x + (size_t)row * d + c0,
                               branch ? branch + (size_t)row * d + c0 : nullptr,
                               gate ? gate + (size_t)(row / gate_rows) * d + c0 : nullptr};
#pragma unroll
            for (int m = 0; m < 3; ++m)
                if (src[m]) {
                    const uint32_t to =
                        (uint32_t)__cvta_generic_to_shared(ring + (size_t)(stage * 3 + m) * d);
#pragma unroll
                    for (int i = 0; i < NV; ++i)
                        if (i < nv)
#pragma unroll
                            for (int y = 0; y < (int)sizeof(Piece<T>); y += 16)
                                asm volatile(
                                    "cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                        to + i * step * (int)sizeof(T) + y),
                                    "l"((const char *)(src[m] + i * step) + y)
                                    : "memory");
                }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int row = blockIdx.x;
#pragma unroll
    for (int y = 0; y < kStages - 1; ++y) fetch(row + y * (int)gridDim.x, y);
    int stage = 0;
    for (; row < R; row += gridDim.x, stage = (stage + 1) % kStages) {
        fetch(row + (kStages - 1) * (int)gridDim.x, (stage + kStages - 1) % kStages);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        auto piece = [&](int m, int i, uint64_t (&v)[4]) {
            reinterpret_cast<const Piece<T> *>(ring + (size_t)(stage * 3 + m) * d + i * step)->get(v);
        };
        auto weights = [&](const T *w, int i, uint64_t (&v)[4]) {
            Piece<T> p;
            p.load(w + c0 + i * step);
            p.get(v);
        };
        uint64_t v[NV][4];
        if (branch) {
            uint64_t u[NV][4];
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < nv) piece(1, i, u[i]);
            float r = 1.f;
            if (w_post) r = row_scale<NV>(u, nv, d, eps, part, turn);
            const uint64_t r2 = pack2(r, r), sc2 = pack2(scale, scale);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < nv) {
                    uint64_t w[4], gv[4];
                    if (w_post) weights(w_post, i, w);
                    if (gate) piece(2, i, gv);
                    piece(0, i, v[i]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint64_t t = u[i][q];
                        if (w_post) t = mul2(mul2(t, r2), w[q]);
                        if (gate) t = mul2(t, gv[q]);
                        v[i][q] = fma2(sc2, t, v[i][q]);
                    }
                }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < nv) piece(0, i, v[i]);
        }
        if (h) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < nv) Piece<T>::store(h + (size_t)row * d + c0 + i * step, v[i]);
        }
        if (!hn) continue;
        const float r = row_scale<NV>(v, nv, d, eps, part, turn);
        const uint64_t r2 = pack2(r, r);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i < nv) {
                uint64_t w[4];
                if (w_pre) weights(w_pre, i, w);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    v[i][q] = mul2(v[i][q], r2);
                    if (w_pre) v[i][q] = mul2(v[i][q], w[q]);
                }
                Piece<T>::store(hn + (size_t)row * d + c0 + i * step, v[i]);
            }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Many rows: a warp per row, no block barriers on the way. A CTA takes a run of consecutive rows,
// its warps row after row; rows of x and branch come through a ring of two stages that each warp
// fills for itself with cp.async, a row ahead; h stays in registers as fp32 (NV pieces a lane).
// w_post (.) gate and w_pre are kept in shared memory as fp32, formed again where the gate row
// changes. Instructions are what this one is short of: 15 to a pair of elements.
constexpr int kRowWarps = 8;

// Factors a, b so that v a b = v / sqrt(mean v^2 + eps) without leaving fp32's range (a is 1 but
// for rows at its ends); s: the lane's sum of squares, value(i, q): pair q of its piece i.
template <int NV, typename F>
__device__ __forceinline__ float2 warp_scale(F value, float s, int nv, int d, float eps) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((s < INFINITY && (s > 1e-25f * (float)d || eps > 1e-30f)) || s != s)
        return make_float2(1.f, rsqrtf(s * (1.f / (float)d) + eps));
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (i < nv)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 f = unpack2(value(i, q));
                mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (mx == 0.f || mx == INFINITY)
        return make_float2(1.f, mx == 0.f ? 1.f / sqrtf(eps) : 0.f);
    int ex;
    frexpf(mx, &ex);
    ex = max(ex, -126);
    const double e2 = ldexp((double)eps, -2 * ex);
    if (e2 > 1e30) return make_float2(1.f, 1.f / sqrtf(eps));
    const float down = ldexpf(1.f, -ex);
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (i < nv)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 f = unpack2(value(i, q));
                t = fmaf(f.x * down, f.x * down, fmaf(f.y * down, f.y * down, t));
            }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return make_float2(down, 1.f / sqrtf(t / (float)d + (float)e2));
}

template <typename T, int NV>
__global__ void __launch_bounds__(32 * kRowWarps)
row_norm_kernel(const T *x, const T *branch, const T *__restrict__ w_post,
                const T *__restrict__ gate, int gate_rows, float scale,
                const T *__restrict__ w_pre, float eps, int R, int d, T *h, T *hn) {
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *s_post = reinterpret_cast<float *>(smem), *s_pre = s_post + d;
    T *ring = reinterpret_cast<T *>(s_pre + d) + (size_t)warp * 4 * d;  // [stage][x, branch][d]
    const int c0 = lane * 8, nv = c0 < d ? (d - c0 + 255) / 256 : 0;
    const bool scaled = w_post || gate;
    pdl_wait();
    auto fetch = [&](int row, int end, int stage) {  // each lane copies the pieces it will read
        if (row < end) {
            const uint32_t dst =
                (uint32_t)__cvta_generic_to_shared(ring + (size_t)stage * 2 * d + c0);
            const char *sx = (const char *)(x + (size_t)row * d + c0);
            const char *sb = (const char *)(branch + (size_t)row * d + c0);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < nv)
#pragma unroll
                    for (int y = 0; y < (int)sizeof(Piece<T>); y += 16) {
                        const int at = i * 256 * (int)sizeof(T) + y;
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + at),
                                     "l"(sx + at)
                                     : "memory");
                        if (branch)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                             dst + d * (int)sizeof(T) + at),
                                         "l"(sb + at)
                                         : "memory");
                    }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto piece = [](const T *p, uint64_t (&v)[4]) { reinterpret_cast<const Piece<T> *>(p)->get(v); };
    // (the halves of 8-element pieces apart, so that a warp's 16-byte reads meet no bank twice)
    auto wide = [&](const float *p, int c, uint64_t (&v)[4]) {
        Piece<float> w;
        w.a = *reinterpret_cast<const float4 *>(p + c / 2);
        w.b = *reinterpret_cast<const float4 *>(p + d / 2 + c / 2);
        w.get(v);
    };
    auto keep = [&](float *p, int c, const uint64_t (&v)[4]) {
        const float2 e = unpack2(v[0]), f = unpack2(v[1]), g = unpack2(v[2]), z = unpack2(v[3]);
        *reinterpret_cast<float4 *>(p + c / 2) = make_float4(e.x, e.y, f.x, f.y);
        *reinterpret_cast<float4 *>(p + d / 2 + c / 2) = make_float4(g.x, g.y, z.x, z.y);
    };
    const uint64_t sc2 = pack2(scale, scale);
    const int r0 = (int)((long long)R * blockIdx.x / gridDim.x),
              r1 = (int)((long long)R * (blockIdx.x + 1) / gridDim.x);
    for (int g0 = r0; g0 < r1;) {  // rows g0 .. g1 - 1 share a gate row
        const int g1 = gate ? min(r1, (g0 / gate_rows + 1) * gate_rows) : r1;
        int row = g0 + warp, stage = 0;
        fetch(row, g1, 0);
        __syncthreads();
        for (int c = threadIdx.x * 8; c < d; c += blockDim.x * 8) {
            uint64_t v[4], w[4];
            Piece<T> p;
            if (scaled) {
                if (w_post) {
                    p.load(w_post + c);
                    p.get(v);
                }
                if (gate) {
                    p.load(gate + (size_t)(g0 / gate_rows) * d + c);
                    p.get(w);
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = w_post ? mul2(v[q], w[q]) : w[q];
                }
                keep(s_post, c, v);
            }
            if (w_pre) {
                p.load(w_pre + c);
                p.get(v);
                keep(s_pre, c, v);
            }
        }
        __syncthreads();
        for (; row < g1; row += kRowWarps, stage ^= 1) {
            fetch(row + kRowWarps, g1, stage ^ 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            const T *sx = ring + (size_t)stage * 2 * d + c0, *sb = sx + d;
            float2 r = make_float2(1.f, 1.f);
            if (w_post) {
                uint64_t s2 = 0ull;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (i < nv) {
                        uint64_t u[4];
                        piece(sb + i * 256, u);
#pragma unroll
                        for (int q = 0; q < 4; ++q) s2 = fma2(u[q], u[q], s2);
                    }
                const float2 f = unpack2(s2);
                r = warp_scale<NV>(
                    [&](int i, int q) {
                        uint64_t u[4];
                        piece(sb + i * 256, u);
                        return u[q];
                    },
                    f.x + f.y, nv, d, eps);
            }
            const uint64_t a2 = pack2(r.x, r.x), b2 = pack2(r.y, r.y);
            uint64_t v[NV][4], s2 = 0ull;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < nv) {
                    piece(sx + i * 256, v[i]);
                    if (branch) {
                        uint64_t u[4], w[4];
                        piece(sb + i * 256, u);
                        if (w_post) {
                            if (r.x != 1.f) {
#pragma unroll
                                for (int q = 0; q < 4; ++q) u[q] = mul2(u[q], a2);
                            }
#pragma unroll
                            for (int q = 0; q < 4; ++q) u[q] = mul2(u[q], b2);
                        }
                        if (scaled) {
                            wide(s_post, c0 + i * 256, w);
#pragma unroll
                            for (int q = 0; q < 4; ++q) u[q] = mul2(u[q], w[q]);
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) v[i][q] = fma2(sc2, u[q], v[i][q]);
                    }
                    if (h) Piece<T>::store(h + (size_t)row * d + c0 + i * 256, v[i]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) s2 = fma2(v[i][q], v[i][q], s2);
                }
            if (!hn) continue;
            const float2 f = unpack2(s2);
            r = warp_scale<NV>([&](int i, int q) { return v[i][q]; }, f.x + f.y, nv, d, eps);
            const uint64_t c2 = pack2(r.x, r.x), e2 = pack2(r.y, r.y);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < nv) {
                    if (r.x != 1.f) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) v[i][q] = mul2(v[i][q], c2);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[i][q] = mul2(v[i][q], e2);
                    if (w_pre) {
                        uint64_t w[4];
                        wide(s_pre, c0 + i * 256, w);
#pragma unroll
                        for (int q = 0; q < 4; ++q) v[i][q] = mul2(v[i][q], w[q]);
                    }
                    Piece<T>::store(hn + (size_t)row * d + c0 + i * 256, v[i]);
                }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        g0 = g1;
    }
}

template <typename T>
cudaError_t launch_t(int d, const void *x, const void *branch, const void *w_post,
                     const void *gate, int gate_rows, float scale, const void *w_pre, float eps,
                     int R, void *h, void *hn, cudaStream_t s) {
    const int nsm = device_sms();
    if (nsm <= 0) return cudaErrorInvalidDevice;
    auto run = [&](auto *k, int thr, size_t smem, int per_sm) {
        const cudaError_t e = allow_smem(k, 226 * 1024);
        if (e != cudaSuccess) return e;
        return launch_pdl(k, dim3(std::min(R, nsm * per_sm)), dim3(thr), smem, s, (const T *)x,
                          (const T *)branch, (const T *)w_post, (const T *)gate, gate_rows, scale,
                          (const T *)w_pre, eps, R, d, (T *)h, (T *)hn);
    };
    const int vecs = d / 8;
    // A warp per row where there are several rows for each of the SM's warps, room for their rings,
    // and gate rows that many rows share: 8192 x 2880 bf16 takes 42 us so (4.5 TB/s) and 57 us with
    // 384 threads a row, whose two block reductions are a chain of 2000 cycles; a few rows are done
    // sooner with up to 512 threads each (65 x 2048: 2.5 us). The rings and weights bound the width:
    // bf16 up to 3208 columns, fp32 up to 1696. 8192 rows with both norms and a gate, here: bf16 3200
    // 44.5 us, fp32 1600 37.5; in the other kernel bf16 4096 86 us (3.1 TB/s), 5120 82 (4.1), 6144 145
    // (2.8), fp32 2048 59 (4.6), 4096 128 (4.2).
    const size_t row_smem = (size_t)d * (8 + 4 * kRowWarps * sizeof(T));
    if (R >= 2 * kRowWarps * nsm && row_smem <= 226 * 1024 && (!gate || gate_rows >= 4 * kRowWarps)) {
        const int nv = (vecs + 31) / 32, thr = 32 * kRowWarps;
        // CTAs that an SM holds: by shared memory, at most two (registers)
        const int per_sm = nv <= 4 && 2 * (row_smem + 1024) <= 227 * 1024 ? 2 : 1;
        return nv <= 4   ? run(row_norm_kernel<T, 4>, thr, row_smem, per_sm)
               : nv <= 8 ? run(row_norm_kernel<T, 8>, thr, row_smem, per_sm)
                         : run(row_norm_kernel<T, 13>, thr, row_smem, per_sm);
    }
    const int nv = (vecs + kMaxThr - 1) / kMaxThr;
    const int thr = (((vecs + nv - 1) / nv + 31) / 32) * 32;
    const size_t smem = 2 * 3 * (size_t)d * sizeof(T);
    const int per_sm = (int)std::max<size_t>(
        1, std::min<size_t>((nv == 1 ? 896 : 640) / thr, 227 * 1024 / (smem + 1024)));
    return nv == 1 ? run(block_norm_kernel<T, 1>, thr, smem, per_sm)
                   : run(block_norm_kernel<T, 2>, thr, smem, per_sm);
}

}  // namespace

cudaError_t launch_block_norm(const moe_layer_desc &L, const void *x, const void *branch,
                              const void *w_post, const void *gate, int gate_rows, float scale,
                              const void *w_pre, float eps, int R, void *h, void *hn,
                              cudaStream_t s) {
    if (R <= 0) return cudaSuccess;
    return L.dtype == MOE_DTYPE_BF16
               ? launch_t<__nv_bfloat16>(L.d, x, branch, w_post, gate, gate_rows, scale, w_pre,
                                         eps, R, h, hn, s)
               : launch_t<float>(L.d, x, branch, w_post, gate, gate_rows, scale, w_pre, eps, R, h,
                                 hn, s);
}

}  // namespace moe
