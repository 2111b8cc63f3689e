// The norms and the residual between the two halves of a decoder block in one pass:
//   u = w_post (.) branch / rms(branch);  h = x + scale gate (.) u;  hn = w_pre (.) h / rms(h)
// Each input is read and each output written once; the row stays in registers between the two
// sums of squares. Bound by memory: 4 R d elements.
#include <algorithm>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kMaxVecs = 3;  // 8-element pieces of a thread: 256 threads x 3 x 8 = 6144 columns

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float v[8]) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
        w[q] = *reinterpret_cast<const uint32_t *>(&t);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, const float v[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
// An 8-element piece as it lies in memory (bf16: 16 bytes, fp32: 32).
template <typename T> struct Piece;
template <> struct Piece<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        a = *reinterpret_cast<const uint4 *>(p);
    }
    __device__ __forceinline__ void get(float v[8]) const {
        v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
        v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z); v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
    }
};
template <> struct Piece<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = *reinterpret_cast<const float4 *>(p);
        b = *(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void get(float v[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};

// Sum (MAX false) or largest value over the CTA; every thread gets it. part: two buffers of 8
// floats used in turn, so that one barrier per reduction is enough.
template <bool MAX> __device__ __forceinline__ float cta_reduce(float v, float (*part)[8], int &turn) {
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
    float t = p[0];
    for (int w = 1; w < warps; ++w) t = MAX ? fmaxf(t, p[w]) : t + p[w];
    return t;
}

// 1 / sqrt(mean v^2 + eps) of the row as r1 * r2 (two factors: the value itself may leave fp32's
// range). The fp32 sum of squares serves unless it overflows, or is so small that squares lost
// below fp32's range count against eps too; then the row is scaled by a power of two first.
template <int NV>
__device__ __forceinline__ float2 row_scale(const float (&v)[NV][8], int nv, int d, float eps,
                                            float (*part)[8], int &turn) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (i < nv) {
#pragma unroll
            for (int q = 0; q < 8; ++q) s = fmaf(v[i][q], v[i][q], s);
        }
    s = cta_reduce<false>(s, part, turn);
    if ((s < INFINITY && (s > 1e-25f * (float)d || eps > 1e-30f)) || s != s)
        return make_float2(1.f / sqrtf(s / (float)d + eps), 1.f);
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (i < nv) {
#pragma unroll
            for (int q = 0; q < 8; ++q) mx = fmaxf(mx, fabsf(v[i][q]));
        }
    mx = cta_reduce<true>(mx, part, turn);
    if (mx == 0.f || mx == INFINITY) return make_float2(mx == 0.f ? 1.f / sqrtf(eps) : 0.f, 1.f);
    int ex;
    frexpf(mx, &ex);  // mx = f 2^ex, f in [0.5, 1)
    ex = max(ex, -120);
    const float down = ldexpf(1.f, -ex);  // exact: ex <= 128 gives 2^-128, a denormal: still exact
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (i < nv) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float w = ldexpf(v[i][q], -ex);
                t = fmaf(w, w, t);
            }
        }
    t = cta_reduce<false>(t, part, turn);
    // mean + eps = 2^(2 ex) (t / d + eps 2^(-2 ex))
    const double e2d = ldexp((double)eps, -2 * ex);
    if (e2d > 1e30) return make_float2(1.f / sqrtf(eps), 1.f);  // the mean is far below eps
    const float e2 = (float)e2d;
    return make_float2(1.f / sqrtf(t / (float)d + e2), down);
}

// A CTA takes every gridDim.x-th row; its weights stay in registers and the next row's x and
// branch are on their way while a row is reduced. (x and branch may be the buffers that h and hn
// go to, so they are read with plain loads, each element by the thread that writes it.)
template <typename T, int NV>
__global__ void __launch_bounds__(256)
block_norm_kernel(const T *x, const T *branch, const T *__restrict__ w_post,
                  const T *__restrict__ gate, int gate_rows, float scale,
                  const T *__restrict__ w_pre, float eps, int R, int d, T *h, T *hn) {
    __shared__ float part[2][8];
    int turn = 0;
    const int step = blockDim.x * 8, c0 = threadIdx.x * 8;
    const int nv = c0 < d ? (d - c0 + step - 1) / step : 0;
    Piece<T> px[NV], pb[NV], pg[NV], wp[NV], wn[NV];
    auto fetch = [&](int row) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i < nv) {
                px[i].load(x + (size_t)row * d + c0 + i * step);
                if (branch) pb[i].load(branch + (size_t)row * d + c0 + i * step);
                if (gate) pg[i].load(gate + (size_t)(row / gate_rows) * d + c0 + i * step);
            }
    };
    pdl_wait();
    int row = blockIdx.x;
    fetch(row);
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (i < nv) {
            if (w_post) wp[i].load(w_post + c0 + i * step);
            if (w_pre && hn) wn[i].load(w_pre + c0 + i * step);
        }
    for (; row < R; row += gridDim.x) {
        float v[NV][8], u[NV][8], gv[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i < nv) {
                px[i].get(v[i]);
                if (branch) pb[i].get(u[i]);
                if (gate) pg[i].get(gv[i]);
            }
        if (row + (int)gridDim.x < R) fetch(row + gridDim.x);
        if (branch) {
            float2 r = make_float2(1.f, 1.f);
            if (w_post) r = row_scale<NV>(u, nv, d, eps, part, turn);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < nv) {
                    float w[8];
                    if (w_post) wp[i].get(w);
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        float t = u[i][q];
                        if (w_post) t = t * r.y * r.x * w[q];
                        if (gate) t *= gv[i][q];
                        v[i][q] = fmaf(scale, t, v[i][q]);
                    }
                }
        }
        if (h) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < nv) store8(h + (size_t)row * d + c0 + i * step, v[i]);
        }
        if (!hn) continue;
        const float2 r = row_scale<NV>(v, nv, d, eps, part, turn);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i < nv) {
                float w[8];
                if (w_pre) wn[i].get(w);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float t = v[i][q] * r.y * r.x;
                    v[i][q] = w_pre ? t * w[q] : t;
                }
                store8(hn + (size_t)row * d + c0 + i * step, v[i]);
            }
    }
}

template <typename T>
cudaError_t launch_t(int d, const void *x, const void *branch, const void *w_post,
                     const void *gate, int gate_rows, float scale, const void *w_pre, float eps,
                     int R, void *h, void *hn, cudaStream_t s) {
    int dev = 0, nsm = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess)
        err = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    const int vecs = d / 8;
    const int nv = (vecs + 255) / 256;
    const int thr = (((vecs + nv - 1) / nv + 31) / 32) * 32;
    auto *k = nv == 1   ? block_norm_kernel<T, 1>
              : nv == 2 ? block_norm_kernel<T, 2>
                        : block_norm_kernel<T, kMaxVecs>;
    int per_sm = 1;
    err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, thr, 0);
    if (err != cudaSuccess) return err;
    return launch_pdl(k, dim3(std::min(R, nsm * std::max(1, per_sm))), dim3(thr), 0, s,
                      (const T *)x, (const T *)branch, (const T *)w_post, (const T *)gate,
                      gate_rows, scale, (const T *)w_pre, eps, R, d, (T *)h, (T *)hn);
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
