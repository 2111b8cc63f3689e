// The whole layer for a few tokens (single tokens of a few users, a short chain of drafted ones) in
// one launch: pre-norm, router, top-k, the experts, the gated sum and the residual.
//
// The work is reading the weights of the experts that the tokens choose, 3 d f elements each (8 of
// 9.4 MB for one token of the Qwen3-shaped layer, 11 us at the HBM's measured rate); the products are
// nothing beside it. What bounds a call is how soon after the router the weights stream, and that
// they keep streaming. So one CTA a SM stays for the whole call, and the steps are parted by two
// barriers over the grid (a cooperative launch: all CTAs run at once):
//   1. every CTA norms the tokens into its shared memory and forms the scores of an expert or two;
//   2. every CTA picks each token's experts from the scores, and takes an equal share of the rows
//      of W_gate and W_up over all chosen experts; the share's activations go to memory;
//   3. every CTA takes an equal share of W_down's rows (of output columns) over all chosen experts, so
//      that it alone sums what its columns get, in a fixed order.
// In both, the CTA's warps share the inner dimension of every row, so none of them waits for another's
// rows, and add up in shared memory. bf16 weights go from global memory straight into the operands of
// 16 x 8 x 16 products (the order of the inner index is free, so a lane's 16 bytes are two operands);
// tokens are the 8 columns. The activations times their gates are kept as a bf16 value and the bf16
// rest, which is fp32's accuracy to 2^-17. fp32 layers take fp32 products.
#include <algorithm>

#include "few.cuh"
#include "norm.cuh"

namespace moe {
namespace few {

static size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

WsLayout ws_layout(const moe_layer_desc &L, int R) {
    WsLayout w{};
    w.logits = kHeadBytes;
    w.h = align256(w.logits + (size_t)R * L.E * 4);
    w.total = align256(w.h + (size_t)R * L.k * L.f * 4);
    return w;
}

namespace {

constexpr int kThr = 512, kWarps = kThr / 32;
constexpr int kRedBytes = 16 * 1024;  // one buffer of the warps' partial sums

// Bytes between two tokens in shared memory: 64 bytes past whole lines, so that the 16-byte reads of
// two tokens' quarters of a line do not meet in a bank.
__host__ __device__ inline int token_stride(int d, int elem) { return (d * elem + 127) / 128 * 128 + 64; }

struct Plan {
    int n;                            // experts that some token chose
    short expert[kMaxE];              // ascending
    int slot[kMaxE];
    unsigned short tokens[kMaxE];     // by expert: a bit for each token
    unsigned char place[kMaxE][kMaxRows];  // by expert and token: the token's place of the expert
    float gate[kMaxRows][kMaxK];
    double part[kWarps];
    double scale[kMaxRows];
    int alive;
};

// 16 bytes that are read once, past L1.
__device__ __forceinline__ uint4 stream16(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 l2_16(const void *p) {
    uint4 v;
    asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// c += a b of a 16 x 16 and a 16 x 8 bf16 operand.
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 32 inner elements: a lane holds 8 of rows g (x) and g + 8 (y), and 8 of column g (b). Which inner
// index an operand's place stands for does not matter as long as both operands agree.
__device__ __forceinline__ void mma32(float (&c)[4], const uint4 &x, const uint4 &y, const uint4 &b) {
    mma(c, x.x, y.x, x.y, y.y, b.x, b.y);
    mma(c, x.z, y.z, x.w, y.w, b.z, b.w);
}

// Waits until all CTAs of the grid have come here; what they wrote before is visible then. bar: a
// count and a generation; the last to come sets the count back. Gives up after 2 s.
__device__ __forceinline__ bool grid_barrier(const Args &a, Plan &s) {
    __syncthreads();
    if (threadIdx.x == 0) {
        unsigned *count = (unsigned *)a.barrier, *gen = count + 32;
        unsigned was, got;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(was) : "l"(gen) : "memory");
        __threadfence();
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                     : "=r"(got)
                     : "l"(count)
                     : "memory");
        int alive = 1;
        if (got == gridDim.x - 1) {
            *count = 0;
            asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(gen), "r"(was + 1) : "memory");
        } else {
            unsigned long long t0, t;
            asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
            for (unsigned i = 0;; ++i) {
                unsigned now;
                asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(now) : "l"(gen) : "memory");
                if (now != was) break;
                if ((i & 255) == 255) {
                    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
                    if (t - t0 > 2000000000ull) {
                        atomicOr(a.flags, FLAG_WAIT_TIMEOUT);
                        alive = 0;
                        break;
                    }
                }
            }
        }
        s.alive = alive;
    }
    __syncthreads();
    return s.alive != 0;
}

// a + b with what the sum loses added to the rest (exact).
__device__ __forceinline__ void add_kept(float &hi, float &lo, float b) {
    const float s = hi + b, t = s - hi;
    lo += (hi - (s - t)) + (b - t);
    hi = s;
}

template <typename T> __device__ __forceinline__ void load8(const T *p, float v[8]);
template <> __device__ __forceinline__ void load8(const __nv_bfloat16 *p, float v[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
}
template <> __device__ __forceinline__ void load8(const float *p, float v[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Every token's scale 1 / sqrt(mean x^2 + eps). The squares' sum is carried as two fp32 values (bf16
// squares are exact in fp32, fp32 ones are split), or in fp64 where it leaves fp32's range; the root
// by two Newton steps in fp64, as a divide and a root there take dozens of its slow operations.
template <typename T>
__device__ __forceinline__ void norm_scales(const Args &a, Plan &s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int per = kWarps;  // warps a token
    while (per > 1 && kWarps / per < a.R) per /= 2;
    const int r = warp / per, w = warp % per;
    const T *x = reinterpret_cast<const T *>(a.x) + (size_t)r * a.d;
    double sum = 0.0;
    if (r < a.R) {
        float hi = 0.f, lo = 0.f;
        for (int c = (w * 32 + lane) * 8; c < a.d; c += per * 256) {
            float v[8];
            load8(x + c, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p = v[i] * v[i];
                if (sizeof(T) == 4) lo += fmaf(v[i], v[i], -p);
                add_kept(hi, lo, p);
            }
        }
        // (squares below 2^-100 may have lost bits, infinite ones everything)
        const bool fine = hi < 1e30f && (hi > 1e-25f || hi == 0.f);
        if (!__all_sync(0xffffffffu, fine)) {
            sum = 0.0;
            for (int c = (w * 32 + lane) * 8; c < a.d; c += per * 256) {
                float v[8];
                load8(x + c, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum = fma((double)v[i], (double)v[i], sum);
            }
        } else {
            sum = (double)hi + (double)lo;
        }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s.part[warp] = sum;
    __syncthreads();
    if (threadIdx.x < a.R) {
        double v = 0.0;
        for (int i = 0; i < per; ++i) v += s.part[threadIdx.x * per + i];
        v = v / (double)a.d + kNormEps;
        double y;
        if (v < 1e37) {
            y = (double)rsqrtf((float)v);
            y = y * fma(-0.5 * v * y, y, 1.5);
            y = y * fma(-0.5 * v * y, y, 1.5);
        } else {
            y = 1.0 / sqrt(v);
        }
        s.scale[threadIdx.x] = y;
    }
    __syncthreads();
}

// The tokens (normed where asked) go to shared memory.
template <typename T> __device__ __forceinline__ void stage_tokens(const Args &a, Plan &s, char *xs) {
    const int stride = token_stride(a.d, sizeof(T)), per = a.d / 8;
    if (a.norm) norm_scales<T>(a, s);
    for (int i = threadIdx.x; i < a.R * per; i += kThr) {
        const int r = i / per, c = (i - r * per) * 8;
        const T *src = reinterpret_cast<const T *>(a.x) + (size_t)r * a.d + c;
        T *dst = reinterpret_cast<T *>(xs + r * stride) + c;
        float v[8];
        load8(src, v);
        if (sizeof(T) == 2) {
            uint4 u = *reinterpret_cast<const uint4 *>(src);
            if (a.norm) {
                const double sc = s.scale[r];
                const float scf = __double2float_rn(sc);
                uint32_t q[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) q[j] = scaled_bf16(v[j], sc, scf);
                u = make_uint4(q[0] | q[1] << 16, q[2] | q[3] << 16, q[4] | q[5] << 16,
                               q[6] | q[7] << 16);
            }
            *reinterpret_cast<uint4 *>(dst) = u;
        } else {
            if (a.norm) {
                // the fp64 product, rounded once, from the scale as two fp32 values
                const double sc = s.scale[r];
                const float hi = __double2float_rn(sc), lo = (float)(sc - (double)hi);
                const bool plain = hi < 1e18f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float p = v[j] * hi, ap = fabsf(p);
                    v[j] = plain && ap > 1e-25f && ap < 1e37f ? p + (fmaf(v[j], hi, -p) + v[j] * lo)
                                                             : (float)((double)v[j] * sc);
                }
            }
            float4 *o = reinterpret_cast<float4 *>(dst);
            o[0] = make_float4(v[0], v[1], v[2], v[3]);
            o[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
    __syncthreads();
}

// A thread's 8 elements of a row, as they lie in memory.
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = stream16(p); }
    __device__ __forceinline__ void get(float v[8]) const {
        v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
        v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
    }
};
template <> struct Eight<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = stream16(p);
        b = stream16(p + 4);
    }
    __device__ __forceinline__ void get(float v[8]) const {
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z);
        v[3] = __uint_as_float(a.w); v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
        v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    }
};

// Scores of the CTA's experts, all tokens: the CTA's threads share an expert's row. first: the thread's
// elements of the CTA's first row, on their way since the start.
template <typename T>
__device__ __forceinline__ void router(const Args &a, const char *xs, float *red, Eight<T> first) {
    const int stride = token_stride(a.d, sizeof(T));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = blockIdx.x; e < a.E; e += gridDim.x) {
        const T *w = reinterpret_cast<const T *>(a.wr) + (size_t)e * a.d;
        float acc[kMaxRows];
#pragma unroll
        for (int r = 0; r < kMaxRows; ++r) acc[r] = 0.f;
        for (int c = threadIdx.x * 8; c < a.d; c += kThr * 8) {
            Eight<T> we = first;
            if (e != blockIdx.x || c >= kThr * 8) we.load(w + c);
            float wv[8];
            we.get(wv);
#pragma unroll
            for (int r = 0; r < kMaxRows; ++r) {
                if (r < a.R) {
                    float xv[8];
                    load8(reinterpret_cast<const T *>(xs + r * stride) + c, xv);
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[r] = fmaf(wv[i], xv[i], acc[r]);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < kMaxRows; ++r) {
            if (r < a.R) {
                float v = acc[r];
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (lane == 0) red[warp * kMaxRows + r] = v;
            }
        }
        __syncthreads();
        if (threadIdx.x < a.R) {
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) v += red[i * kMaxRows + threadIdx.x];
            a.logits[(size_t)threadIdx.x * a.E + e] = v;
        }
        __syncthreads();
    }
}

// Each token's k largest scores (ties to the lower expert), their softmax, and who chose whom.
__device__ __forceinline__ void choose(const Args &a, Plan &s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e < kMaxE; e += kThr) s.tokens[e] = 0;
    if (threadIdx.x == 0) s.n = 0;
    __syncthreads();
    if (warp < a.R) {
        const float *l = a.logits + (size_t)warp * a.E;
        uint32_t key[kMaxE / 32];
#pragma unroll
        for (int i = 0; i < kMaxE / 32; ++i) {
            const int e = i * 32 + lane;
            key[i] = 0;
            if (e < a.E) {
                const uint32_t b = __float_as_uint(__ldcg(l + e) + 0.f);
                key[i] = max(1u, b ^ ((int)b < 0 ? 0xffffffffu : 0x80000000u));
            }
        }
        float mine = -INFINITY, top = 0.f;  // lane j: the j-th chosen score
        int who = 0;
        for (int j = 0; j < a.k; ++j) {
            uint32_t best = 0;
#pragma unroll
            for (int i = 0; i < kMaxE / 32; ++i) best = max(best, key[i]);
            best = __reduce_max_sync(0xffffffffu, best);
            int e = kMaxE;
#pragma unroll
            for (int i = kMaxE / 32 - 1; i >= 0; --i)
                if (key[i] == best) e = i * 32 + lane;
            e = (int)__reduce_min_sync(0xffffffffu, (unsigned)e);
#pragma unroll
            for (int i = 0; i < kMaxE / 32; ++i)
                if (i * 32 + lane == e) key[i] = 0;
            const float v = __uint_as_float(best ^ ((int)best < 0 ? 0x80000000u : 0xffffffffu));
            if (j == 0) top = v;
            if (lane == j) {
                mine = v;
                who = e;
            }
        }
        const float p = lane < a.k ? expf(mine - top) : 0.f;
        float sum = p;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane < a.k) {
            const float g = p / sum;
            s.gate[warp][lane] = g;
            s.place[who][warp] = (unsigned char)lane;
            atomicOr(reinterpret_cast<unsigned *>(s.tokens) + who / 2,
                     1u << (warp + 16 * (who & 1)));
            if (blockIdx.x == 0) {
                if (a.topk_idx) a.topk_idx[warp * a.k + lane] = who;
                if (a.gates) a.gates[warp * a.k + lane] = g;
            }
        }
    }
    __syncthreads();
    if (warp == 0) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < kMaxE / 32; ++i) {
            const int e = i * 32 + lane;
            bool on = e < a.E && s.tokens[e];
            int slot = e;
            if (on && a.slot) slot = a.slot[e];
            if (on && (slot < 0 || slot >= a.slots)) {
                on = false;
                if (blockIdx.x == 0) atomicOr(a.flags, FLAG_BAD_EXPERT);
            }
            const uint32_t m = __ballot_sync(0xffffffffu, on);
            if (on) {
                const int at = n + __popc(m & ((1u << lane) - 1));
                s.expert[at] = (short)e;
                s.slot[at] = slot;
            }
            n += __popc(m);
        }
        if (lane == 0) s.n = n;
    }
    __syncthreads();
}

__device__ __forceinline__ float silu(float g) { return g / (1.f + expf(-g)); }

// The i-th token of a mask.
__device__ __forceinline__ int nth_token(unsigned mask, int i) {
    for (; i > 0; --i) mask &= mask - 1;
    return __ffs(mask) - 1;
}

// A gated activation of assignment (token, place), element j.
__device__ __forceinline__ void store_h(const Args &a, __nv_bfloat16 *, int row, int j, float v) {
    __nv_bfloat16 *h = reinterpret_cast<__nv_bfloat16 *>(a.h) + (size_t)row * 2 * a.f;
    const __nv_bfloat16 hi = __float2bfloat16(v);
    h[j] = hi;
    h[a.f + j] = __float2bfloat16(v - __bfloat162float(hi));
}
__device__ __forceinline__ void store_h(const Args &a, float *, int row, int j, float v) {
    reinterpret_cast<float *>(a.h)[(size_t)row * a.f + j] = v;
}

// Sums of the warps' partial results of `nj` rows and m tokens, the activations from them.
template <typename T>
__device__ __forceinline__ void finish_gate_up(const Args &a, const Plan &s, const float *red,
                                               int tiles, int e, int j0, int nj, unsigned mask, int m) {
    for (int o = threadIdx.x; o < nj * m; o += kThr) {
        const int i = o / nj, j = o - i * nj;
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float *p = red + ((size_t)(w * tiles + (j >> 3)) * 16 + (j & 7)) * m + i;
            g += p[0];
            u += p[8 * m];
        }
        const int r = nth_token(mask, i), place = s.place[e][r];
        store_h(a, (T *)nullptr, r * a.k + place, j0 + j, silu(g) * u * s.gate[r][place]);
    }
}

template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16(v); }
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ void store_y(const Args &a, int r, int col, float v) {
    const size_t at = (size_t)r * a.d + col;
    if (a.residual) v += to_float(reinterpret_cast<const T *>(a.x)[at]);
    reinterpret_cast<T *>(a.y)[at] = from_float<T>(v);
}

// ---- bf16 steps 2 and 3: a warp's weights come through a ring of its own ----
// An entry is 16 rows of 32 inner elements: every lane copies the two 16-byte operands that it will
// read itself, so a warp waits for no other thread. The copies of step 3's first entries, which do
// not depend on step 2, are on their way while the CTA ends step 2 and waits at the grid's barrier.

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool on) {
    const int n = on ? 16 : 0;  // (0: the 16 bytes become zeros, nothing is read)
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t p) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(p)
                 : "memory");
    return v;
}

// The entries of step 2: the CTA's share of the rows (pairs of a gate and an up row, over all chosen
// experts), in runs of one expert, tiles of 8 pairs, and the warp's part of the inner dimension.
struct GateUp {
    long long p, p1;
    int kc0, kc1, ui, j0, nj, tiles, tile, kc, m;
    const __nv_bfloat16 *wg, *wu;
    __device__ __forceinline__ void run(const Args &a, const Plan &s) {
        if (p >= p1) return;
        ui = (int)(p / a.f);
        j0 = (int)(p - (long long)ui * a.f);
        m = __popc(s.tokens[s.expert[ui]]);
        const int most = kRedBytes / (kWarps * 16 * 4 * m);
        nj = (int)min(min((long long)(a.f - j0), p1 - p), 8ll * most);
        tiles = (nj + 7) / 8;
        const size_t at = ((size_t)s.slot[ui] * a.f + j0) * a.d;
        wg = reinterpret_cast<const __nv_bfloat16 *>(a.wg) + at;
        wu = reinterpret_cast<const __nv_bfloat16 *>(a.wu) + at;
    }
    __device__ __forceinline__ void start(const Args &a, const Plan &s, int warp) {
        const long long pairs = (long long)s.n * a.f;
        p = pairs * blockIdx.x / gridDim.x;
        p1 = pairs * (blockIdx.x + 1) / gridDim.x;
        // (a warp without a part has one entry of zeros a tile)
        const int nk = (a.d + 31) / 32;
        kc0 = warp * nk / kWarps;
        kc1 = max(kc0 + 1, (warp + 1) * nk / kWarps);
        kc = kc0;
        tile = 0;
        run(a, s);
    }
    __device__ __forceinline__ bool more() const { return p < p1; }
    // (the inner elements behind a part of none belong to the next warp)
    __device__ __forceinline__ bool mine(const Args &a, int warp) const {
        return (warp + 1) * ((a.d + 31) / 32) / kWarps > kc0;
    }
    __device__ __forceinline__ bool last_of_tile() const { return kc + 1 == kc1; }
    __device__ __forceinline__ bool last_of_run() const { return last_of_tile() && tile + 1 == tiles; }
    __device__ __forceinline__ void next(const Args &a, const Plan &s) {
        if (++kc < kc1) return;
        kc = kc0;
        if (++tile < tiles) return;
        tile = 0;
        p += nj;
        run(a, s);
    }
    __device__ __forceinline__ void copy(const Args &a, uint32_t at, bool mine) const {
        const int lane = threadIdx.x & 31, j = tile * 8 + (lane >> 2), c = kc * 32 + 8 * (lane & 3);
        const bool on = mine && j < nj && c < a.d;
        const size_t row = on ? (size_t)j * a.d + c : 0;
        copy16(at, wg + row, on);
        copy16(at + 512, wu + row, on);
    }
};

// The entries of step 3: tiles of up to 16 of the CTA's output columns, and the warp's part of the
// inner dimension, which runs over all chosen experts.
struct Down {
    int c0, c1, tiles, tile, q0, q1, q, nk, ui, kc, first_ui, first_kc, b0, b1;
    __device__ __forceinline__ void columns() {
        b0 = c0 + (c1 - c0) * tile / tiles;
        b1 = c0 + (c1 - c0) * (tile + 1) / tiles;
    }
    __device__ __forceinline__ void start(const Args &a, const Plan &s, int warp) {
        c0 = (int)((long long)a.d * blockIdx.x / gridDim.x);
        c1 = (int)((long long)a.d * (blockIdx.x + 1) / gridDim.x);
        tiles = (c1 - c0 + 15) / 16;
        nk = (a.f + 31) / 32;
        const int all = s.n * nk;
        q0 = (int)((long long)all * warp / kWarps);
        q1 = (int)((long long)all * (warp + 1) / kWarps);
        first_ui = q0 / nk;
        first_kc = q0 - first_ui * nk;
        tile = 0;
        back();
        if (tiles) columns();
    }
    __device__ __forceinline__ void back() {
        q = q0;
        ui = first_ui;
        kc = first_kc;
    }
    __device__ __forceinline__ bool more() const { return q < q1 && tile < tiles; }
    __device__ __forceinline__ void step() {
        ++q;
        if (++kc == nk) {
            kc = 0;
            ++ui;
        }
    }
    __device__ __forceinline__ void next() {
        step();
        if (q < q1) return;
        back();
        if (++tile < tiles) columns();
    }
    __device__ __forceinline__ void copy(const Args &a, const Plan &s, uint32_t at) const {
        const int lane = threadIdx.x & 31, col = b0 + (lane >> 2), c = kc * 32 + 8 * (lane & 3);
        const __nv_bfloat16 *w = reinterpret_cast<const __nv_bfloat16 *>(a.wd) +
                                 (size_t)s.slot[ui] * a.d * a.f;
        const bool x = c < a.f && col < b1, y = c < a.f && col + 8 < b1;
        copy16(at, x ? w + (size_t)col * a.f + c : w, x);
        copy16(at + 512, y ? w + (size_t)(col + 8) * a.f + c : w, y);
    }
};

// NT: groups of 8 tokens; D: entries of a warp's ring.
template <int NT, int D> struct Ring {
    const Args &a;
    Plan &s;
    GateUp load1, use1;
    Down load2;
    bool mine1;
    uint32_t base;    // the lane's bytes of entry 0
    int put, take;    // entries

    __device__ __forceinline__ Ring(const Args &a_, Plan &s_, const char *ring) : a(a_), s(s_) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        base = (uint32_t)__cvta_generic_to_shared(ring) + warp * D * 1024 + lane * 16;
        put = take = 0;
        load1.start(a, s, warp);
        use1 = load1;
        mine1 = load1.mine(a, warp);
        load2.start(a, s, warp);
#pragma unroll 1
        for (int i = 0; i < D - 1; ++i) fill();
    }
    // The next entry's copies, of step 2 or, when they are all on their way, of step 3.
    __device__ __forceinline__ void fill() {
        const uint32_t at = base + put * 1024;
        if (load1.more()) {
            load1.copy(a, at, mine1);
            load1.next(a, s);
        } else if (load2.more()) {
            load2.copy(a, s, at);
            load2.next();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        put = put + 1 == D ? 0 : put + 1;
    }
    // The oldest entry's operands; its place is filled again by the next fill().
    __device__ __forceinline__ void get(uint4 &x, uint4 &y) {
        asm volatile("cp.async.wait_group %0;" ::"n"(D - 2) : "memory");
        const uint32_t at = base + take * 1024;
        x = shared16(at);
        y = shared16(at + 512);
        take = take + 1 == D ? 0 : take + 1;
    }

    __device__ __forceinline__ void gate_up(const char *xs, float *red) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
        const int stride = token_stride(a.d, 2);
        int buf = 0, run = -1;
        unsigned mask = 0;
        const char *x0 = nullptr, *x1 = nullptr;
        float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
        while (use1.more()) {
            const int m = use1.m;
            if (use1.ui != run) {  // this lane's columns: tokens g and g + 8 of the expert's
                run = use1.ui;
                mask = s.tokens[s.expert[run]];
                x0 = g < m ? xs + nth_token(mask, g) * stride : nullptr;
                x1 = g + 8 < m ? xs + nth_token(mask, g + 8) * stride : nullptr;
            }
            uint4 x, y, b = make_uint4(0, 0, 0, 0);
            const int c = use1.kc * 32 + 8 * t;
            const bool in = c < a.d;
            get(x, y);
            fill();
            if (in && x0) b = *reinterpret_cast<const uint4 *>(x0 + 2 * c);
            mma32(c0, x, y, b);
            if (NT > 1 && m > 8) {
                b = make_uint4(0, 0, 0, 0);
                if (in && x1) b = *reinterpret_cast<const uint4 *>(x1 + 2 * c);
                mma32(c1, x, y, b);
            }
            if (use1.last_of_tile()) {
                float *out = red + buf * (kRedBytes / 4);
                float *o = out + ((size_t)(warp * use1.tiles + use1.tile) * 16 + g) * m;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int col = 2 * t + q;
                    if (col < m) {
                        o[col] = c0[q];
                        o[8 * m + col] = c0[2 + q];
                    }
                    if (NT > 1 && col + 8 < m) {
                        o[col + 8] = c1[q];
                        o[8 * m + col + 8] = c1[2 + q];
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) c0[i] = c1[i] = 0.f;
                if (use1.last_of_run()) {
                    __syncthreads();
                    finish_gate_up<__nv_bfloat16>(a, s, out, use1.tiles, s.expert[run], use1.j0,
                                                  use1.nj, mask, m);
                    buf ^= 1;  // (a buffer is written again after the CTA's next barrier)
                }
            }
            use1.next(a, s);
        }
    }

    // The activations that an entry's columns are multiplied with.
    __device__ __forceinline__ void activations(int ui, int kc, uint4 (&hi)[NT], uint4 (&lo)[NT]) const {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = kc * 32 + 8 * (lane & 3);
        const int e = s.expert[ui];
        const unsigned mask = s.tokens[e];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            hi[n] = lo[n] = make_uint4(0, 0, 0, 0);
            const int r = g + 8 * n;
            if (c < a.f && (mask >> r & 1)) {
                const __nv_bfloat16 *p = reinterpret_cast<const __nv_bfloat16 *>(a.h) +
                                         (size_t)(r * a.k + s.place[e][r]) * 2 * a.f + c;
                hi[n] = l2_16(p);
                lo[n] = l2_16(p + a.f);
            }
        }
    }

    __device__ __forceinline__ void down(float *red) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
        Down use;
        use.start(a, s, warp);
        for (; use.tile < use.tiles;) {
            float acc[NT][4], sum[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][i] = sum[n][i] = 0.f;
            const int b0 = use.b0, b1 = use.b1;
            // activations are asked for two entries ahead
            Down ahead = use;
            uint4 hi[2][NT], lo[2][NT];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (ahead.q < use.q1) activations(ahead.ui, ahead.kc, hi[i], lo[i]);
                ahead.step();
            }
            while (use.q < use.q1) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (use.q < use.q1) {
                        uint4 x, y;
                        get(x, y);
                        fill();
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma32(acc[n], x, y, hi[i][n]);
                            mma32(acc[n], x, y, lo[i][n]);
                        }
                        if (ahead.q < use.q1) activations(ahead.ui, ahead.kc, hi[i], lo[i]);
                        ahead.step();
                        const int ui = use.ui;
                        use.step();
                        if (use.ui != ui || use.q == use.q1) {
                            // the expert's sums count for the tokens that chose it only (its
                            // weights may hold what times zero is not zero)
                            const unsigned mask = s.tokens[s.expert[ui]];
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    if (mask >> (n * 8 + 2 * t + (j & 1)) & 1) sum[n][j] += acc[n][j];
                                    acc[n][j] = 0.f;
                                }
                        }
                    }
                }
            }
            use.back();
            if (++use.tile < use.tiles) use.columns();
            __syncthreads();  // (the tile before is read out)
            float *o = red + (size_t)warp * 16 * kMaxRows;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[(g + 8 * (i >> 1)) * kMaxRows + n * 8 + 2 * t + (i & 1)] = sum[n][i];
            __syncthreads();
            for (int i = threadIdx.x; i < (b1 - b0) * a.R; i += kThr) {
                const int r = i / (b1 - b0), col = i - r * (b1 - b0);
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) v += red[(size_t)(w * 16 + col) * kMaxRows + r];
                store_y<__nv_bfloat16>(a, r, b0 + col, v);
            }
        }
    }
};

// fp32: a warp takes a pair of rows at a time.
__device__ __forceinline__ void gate_up(const Args &a, const Plan &s, const char *xs) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int stride = token_stride(a.d, 4);
    const long long pairs = (long long)s.n * a.f;
    const long long p0 = pairs * blockIdx.x / gridDim.x, p1 = pairs * (blockIdx.x + 1) / gridDim.x;
    for (long long p = p0 + warp; p < p1; p += kWarps) {
        const int ui = (int)(p / a.f), j = (int)(p - (long long)ui * a.f), e = s.expert[ui];
        const size_t at = ((size_t)s.slot[ui] * a.f + j) * a.d;
        const float *wg = reinterpret_cast<const float *>(a.wg) + at;
        const float *wu = reinterpret_cast<const float *>(a.wu) + at;
        // four tokens at a time (the weights are in L1 after the first)
        for (unsigned mask = s.tokens[e]; mask;) {
            int tok[4], n = 0;
            float ga[4] = {0.f, 0.f, 0.f, 0.f}, ua[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                tok[i] = mask ? __ffs(mask) - 1 : 0;
                n += mask != 0;
                mask &= mask - 1;
            }
#pragma unroll 4
            for (int c = lane * 4; c < a.d; c += 128) {
                const float4 gv = __ldg(reinterpret_cast<const float4 *>(wg + c));
                const float4 uv = __ldg(reinterpret_cast<const float4 *>(wu + c));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i < n) {
                        const float4 x = *reinterpret_cast<const float4 *>(xs + tok[i] * stride + 4 * c);
                        ga[i] += gv.x * x.x + gv.y * x.y + gv.z * x.z + gv.w * x.w;
                        ua[i] += uv.x * x.x + uv.y * x.y + uv.z * x.z + uv.w * x.w;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i >= n) continue;
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) {
                    ga[i] += __shfl_xor_sync(0xffffffffu, ga[i], o);
                    ua[i] += __shfl_xor_sync(0xffffffffu, ua[i], o);
                }
                const int place = s.place[e][tok[i]];
                if (lane == 0)
                    store_h(a, (float *)nullptr, tok[i] * a.k + place, j,
                            silu(ga[i]) * ua[i] * s.gate[tok[i]][place]);
            }
        }
    }
}

// fp32: a warp takes a column and a token at a time (the weights are in L1 after the first).
__device__ __forceinline__ void down(const Args &a, const Plan &s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = (int)((long long)a.d * blockIdx.x / gridDim.x);
    const int c1 = (int)((long long)a.d * (blockIdx.x + 1) / gridDim.x);
    const float *h = reinterpret_cast<const float *>(a.h);
    for (int i = warp; i < (c1 - c0) * a.R; i += kWarps) {
        const int col = c0 + i / a.R, r = i % a.R;
        float v = 0.f;
        for (int ui = 0; ui < s.n; ++ui) {
            const int e = s.expert[ui];
            if (!(s.tokens[e] >> r & 1)) continue;
            const float *w = reinterpret_cast<const float *>(a.wd) + ((size_t)s.slot[ui] * a.d + col) * a.f;
            const float *p = h + (size_t)(r * a.k + s.place[e][r]) * a.f;
#pragma unroll 4
            for (int c = lane * 4; c < a.f; c += 128) {
                const float4 wv = __ldg(reinterpret_cast<const float4 *>(w + c));
                const float4 hv = __ldcg(reinterpret_cast<const float4 *>(p + c));
                v += wv.x * hv.x + wv.y * hv.y + wv.z * hv.z + wv.w * hv.w;
            }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) store_y<float>(a, r, col, v);
    }
}

constexpr int kPlanBytes = (sizeof(Plan) + 127) / 128 * 128;
constexpr int kSmem = 227 * 1024;
constexpr int kFixed = kPlanBytes + 2 * kRedBytes;
constexpr int ring_bytes(int D) { return D * kWarps * 1024; }

// D = 0: fp32.
template <typename T, int NT, int D>
__global__ void __launch_bounds__(kThr, 1) few_kernel(const Args a) {
    extern __shared__ __align__(128) char dyn[];
    Plan &s = *reinterpret_cast<Plan *>(dyn);
    float *red = reinterpret_cast<float *>(dyn + kPlanBytes);
    const char *ring = dyn + kFixed;
    char *xs = dyn + kFixed + ring_bytes(D);
    Eight<T> first{};
    if (blockIdx.x < a.E && threadIdx.x * 8 < a.d)
        first.load(reinterpret_cast<const T *>(a.wr) + (size_t)blockIdx.x * a.d + threadIdx.x * 8);
    stage_tokens<T>(a, s, xs);
    router<T>(a, xs, red, first);
    if (!grid_barrier(a, s)) return;
    choose(a, s);
    if constexpr (D > 0) {
        Ring<NT, D> r(a, s, ring);
        r.gate_up(xs, red);
        const bool alive = grid_barrier(a, s);
        if (alive) r.down(red);
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        gate_up(a, s, xs);
        if (!grid_barrier(a, s)) return;
        down(a, s);
    }
}

template <typename T, int NT, int D> cudaError_t launch(const Args &a, int max_ctas, cudaStream_t s) {
    const int sms = device_sms();
    if (sms < 1) return cudaErrorInvalidDevice;
    cudaError_t err = allow_smem(few_kernel<T, NT, D>, kSmem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(max_ctas > 0 ? std::min(max_ctas, sms) : sms);
    cfg.blockDim = dim3(kThr);
    cfg.dynamicSmemBytes = (size_t)kFixed + ring_bytes(D) + (size_t)a.R * token_stride(a.d, sizeof(T));
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, few_kernel<T, NT, D>, a);
}

constexpr int kShallow = 4, kDeep = 8;

}  // namespace

int rows_at_once(const moe_layer_desc &L) {
    const int e = (int)elem_size(L.dtype);
    return std::min(kMaxRows, (kSmem - kFixed - (L.dtype == MOE_DTYPE_F32 ? 0 : ring_bytes(kShallow))) /
                                  token_stride(L.d, e));
}

cudaError_t launch_few(const Args &a, int dtype, int max_ctas, cudaStream_t s) {
    using bf16 = __nv_bfloat16;
    if (dtype == MOE_DTYPE_F32) return launch<float, 1, 0>(a, max_ctas, s);
    const bool deep = a.R * token_stride(a.d, 2) <= kSmem - kFixed - ring_bytes(kDeep);
    if (a.R <= 8)
        return deep ? launch<bf16, 1, kDeep>(a, max_ctas, s) : launch<bf16, 1, kShallow>(a, max_ctas, s);
    return deep ? launch<bf16, 2, kDeep>(a, max_ctas, s) : launch<bf16, 2, kShallow>(a, max_ctas, s);
}

}  // namespace few
}  // namespace moe
