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
// rest, which is fp32's accuracy to 2^-17. (With a third part, all 24 bits: one token 26.4 -> 27.0 us, 16 tokens
// 142 -> 158, the wide experts below 123 -> 137, and 1.8 of a thousand outputs there round to another
// bf16 neighbour than in 64 bits instead of 3.0; what is left are the tensor unit's fp32 sums.) fp32 layers take
// fp32 products.
//
// Measured, calls in a row with other weights each: one token of the Qwen3-shaped layer 26.5 us (6 until
// the first weights are asked for, 3 between the last of step 2 and the first of step 3), 16 tokens
// 134 to 146 by the experts they choose (0.8 of the HBM's measured rate; CTAs end step 2 over 13 us), 4 tokens of
// d = f = 2880, 32 experts, top-4 114 to 134 (0.78), 3 tokens of an fp32 layer of d 520 15.
#include <algorithm>

#include "few.cuh"

namespace moe {
namespace few {

static size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

WsLayout ws_layout(const moe_layer_desc &L, int R) {
    WsLayout w{};
    w.h = kHeadBytes;
    w.total = align256(w.h + (size_t)R * L.k * L.f * 4);
    return w;
}

namespace {

constexpr int kThr = 512, kWarps = kThr / 32;
// One buffer of the warps' partial sums: 16 rows of a token of every warp take 1 KB.
__host__ __device__ constexpr int red_bytes(int R) { return R <= 8 ? 8 * 1024 : 16 * 1024; }

// Bytes between two tokens in shared memory: 64 bytes past whole lines, so that the 16-byte reads of
// two tokens' quarters of a line do not meet in a bank.
__host__ __device__ constexpr int token_stride(int d, int elem) { return (d * elem + 127) / 128 * 128 + 64; }

struct Plan {
    int n;                            // experts that some token chose
    short expert[kMaxE];              // ascending
    int slot[kMaxE];
    unsigned short tokens[kMaxE];     // by expert: a bit for each token
    unsigned char place[kMaxE][kMaxRows];  // by expert and token: the token's place of the expert
    float gate[kMaxRows][kMaxK];
    Pair part[kWarps], scale[kMaxRows];
    double wide_scale[kMaxRows];
    int wide[kMaxRows];
    int pair0, pair1;                 // the CTA's share of the pairs of rows of step 2
    int col0, col1;                   // its output columns
    uint32_t word[kMaxE / 32];
    unsigned long long launch;
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

// The head of the workspace holds a word that counts the CTAs that have ended step 2 (low 16 bits)
// and the launches so far (the rest), and the scores of step 1, each beside the number of the launch that
// wrote it: who reads a score waits for the word itself, not for a barrier and then for the word.
__device__ __forceinline__ unsigned long long load_relaxed(const unsigned long long *p) {
    unsigned long long v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ unsigned long long load_acquire(const unsigned long long *p) {
    unsigned long long v;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ unsigned long long now_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}
constexpr unsigned long long kPatience = 2000000000ull;  // a wait gives up after 2 s

// Waits until all CTAs of the grid have come here; what they wrote before is visible then.
__device__ __forceinline__ bool grid_barrier(const Args &a, Plan &s, unsigned long long launch) {
    __syncthreads();
    if (threadIdx.x == 0) {
        unsigned long long was;
        __threadfence();
        asm volatile("atom.acq_rel.gpu.global.add.u64 %0, [%1], 1;"
                     : "=l"(was)
                     : "l"(a.barrier)
                     : "memory");
        if ((was & 0xffff) == gridDim.x - 1) {
            // the next launch's number; who still waits takes either as the sign
            atomicAdd(a.barrier, 0x10000ull - gridDim.x);
        } else {
            const unsigned long long t0 = now_ns();
            for (unsigned i = 1;; ++i) {
                const unsigned long long v = load_acquire(a.barrier);
                if (v >> 16 != launch || (v & 0xffff) == gridDim.x) break;
                if (i % 256 == 0 && now_ns() - t0 > kPatience) {
                    atomicOr(a.flags, FLAG_WAIT_TIMEOUT);
                    s.alive = 0;
                    break;
                }
            }
        }
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

// Every token's scale 1 / sqrt(mean x^2 + eps), from the tokens in shared memory. Sums and the scale
// are carried as pairs (2^-45; bf16 squares are exact in fp32, fp32 ones have a rest), as fp64
// operations take tens of cycles each here; a row whose squares leave fp32's range takes them.
template <typename T>
__device__ __forceinline__ void norm_scales(const Args &a, Plan &s, const char *xs) {
    const int stride = token_stride(a.d, sizeof(T));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int per = kWarps;  // warps a token
    while (per > 1 && kWarps / per < a.R) per /= 2;
    const int r = warp / per, w = warp % per;
    const T *x = reinterpret_cast<const T *>(xs + r * stride);
    Pair sum{0.f, 0.f};
    if (r < a.R) {
        // two sums side by side, two to an instruction
        const uint64_t minus = pack2(-1.f, -1.f);
        uint64_t hi = 0, lo = 0;
#pragma unroll 1
        for (int c = (w * 32 + lane) * 8; c < a.d; c += per * 256) {
            float v[8];
            load8(x + c, v);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const uint64_t q = pack2(v[i], v[i + 1]), p = mul2(q, q);
                if (sizeof(T) == 4) lo = add2(lo, fma2(q, q, mul2(p, minus)));
                // s = hi + p, and what it loses (exact)
                const uint64_t s2 = add2(hi, p), t2 = fma2(hi, minus, s2);
                lo = add2(lo, add2(fma2(fma2(t2, minus, s2), minus, hi), fma2(t2, minus, p)));
                hi = s2;
            }
        }
        const float2 h2 = unpack2(hi), l2 = unpack2(lo);
        sum = Pair{h2.x, l2.x + l2.y};
        add_kept(sum.hi, sum.lo, h2.y);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const float hi = __shfl_xor_sync(0xffffffffu, sum.hi, o), lo = __shfl_xor_sync(0xffffffffu, sum.lo, o);
        add_kept(sum.hi, sum.lo, hi);
        sum.lo += lo;
    }
    if (lane == 0) s.part[warp] = sum;
    __syncthreads();
    if (threadIdx.x < a.R) {
        Pair v{0.f, 0.f};
        for (int i = 0; i < per; ++i) {
            add_kept(v.hi, v.lo, s.part[threadIdx.x * per + i].hi);
            v.lo += s.part[threadIdx.x * per + i].lo;
        }
        // (squares below 2^-100 may have lost bits, infinite ones everything)
        const bool wide = !(v.hi < 1e30f && (v.hi > 1e-25f || v.hi == 0.f));
        s.wide[threadIdx.x] = wide;
        // mean + eps
        Pair m;
        m.hi = v.hi * a.inv_d.hi;
        m.lo = fmaf(v.hi, a.inv_d.hi, -m.hi) + fmaf(v.hi, a.inv_d.lo, v.lo * a.inv_d.hi);
        add_kept(m.hi, m.lo, (float)kNormEps);
        m.lo += (float)(kNormEps - (double)(float)kNormEps);
        // a Newton step from the fp32 root: y (1 + e / 2 + 3 e^2 / 8), e = 1 - m y^2
        const float y = rsqrtf(m.hi), q = __fmul_rn(y, y), qe = fmaf(y, y, -q);
        const float p = __fmul_rn(m.hi, q), pe = fmaf(m.hi, q, -p) + fmaf(m.hi, qe, m.lo * q);
        const float e = (1.f - p) - pe;
        // (the pair's first is the scale rounded to fp32)
        const float more = y * e * fmaf(0.375f, e, 0.5f), hi = y + more;
        s.scale[threadIdx.x] = Pair{hi, more - (hi - y)};
    }
    __syncthreads();
    if (r < a.R && w == 0 && s.wide[r]) {
        double t = 0.0;
        for (int c = lane * 8; c < a.d; c += 256) {
            float v[8];
            load8(x + c, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) t = fma((double)v[i], (double)v[i], t);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (lane == 0) s.wide_scale[r] = 1.0 / sqrt(t / (double)a.d + kNormEps);
    }
    __syncthreads();
}

// v times a scale in fp64, rounded once to bf16 (a call, so that no other element takes the fp64
// instructions).
__device__ __noinline__ uint32_t scaled_wide(float v, double sc) {
    return __bfloat16_as_ushort(__double2bfloat16((double)v * sc));
}
// An fp32 product with the scale's first part is off by a step and a half at most: half a step for its own
// rounding, and v times the second part, which is half a step of the first's or less. So where it lies two
// steps or more from the middle of two bf16 values its rounding is the answer.
__device__ __forceinline__ bool near_middle(float p) { return ((__float_as_uint(p) + 0x8001u) & 0xffffu) <= 2u; }
// Elsewhere what the product lacks decides (good to 2^-45 of the product, as the scale is).
__device__ __noinline__ uint32_t scaled_middle(float v, Pair sc) {
    const float p = v * sc.hi;
    if (!(fabsf(p) > 1e-25f)) return scaled_wide(v, (double)sc.hi + (double)sc.lo);
    const uint32_t b = __float_as_uint(p);
    const float past = p - __uint_as_float((b & 0xffff0000u) | 0x8000u);  // exact
    const float t = past + (fmaf(v, sc.hi, -p) + v * sc.lo);
    if (t == 0.f) return (b >> 16) + (b >> 16 & 1u);
    return (b >> 16) + ((t > 0.f) == (p > 0.f) ? 1u : 0u);
}
__device__ __forceinline__ void scale16(uint4 *p, Pair sc, const double *wide) {
    const uint4 w = *p;
    float v[8];
    load8(reinterpret_cast<const __nv_bfloat16 *>(&w), v);
    uint32_t q[4];
    bool middle = false;
    const uint64_t by = pack2(sc.hi, sc.hi);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 x = unpack2(mul2(pack2(v[2 * j], v[2 * j + 1]), by));
        middle |= near_middle(x.x) || near_middle(x.y);
        const __nv_bfloat162 b = __floats2bfloat162_rn(x.x, x.y);
        q[j] = reinterpret_cast<const uint32_t &>(b);
    }
    if (middle || wide) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t one = j & 1 ? q[j / 2] >> 16 : q[j / 2] & 0xffffu;
            if (wide)
                one = scaled_wide(v[j], *wide);
            else if (near_middle(v[j] * sc.hi))
                one = scaled_middle(v[j], sc);
            q[j / 2] = j & 1 ? (q[j / 2] & 0xffffu) | one << 16 : (q[j / 2] & 0xffff0000u) | one;
        }
    }
    *p = make_uint4(q[0], q[1], q[2], q[3]);
}
__device__ __noinline__ float scaled_wide_f32(float v, double sc) { return (float)((double)v * sc); }
__device__ __forceinline__ float scaled(float v, Pair sc) {
    const float p = v * sc.hi, ap = fabsf(p);
    // (where the product's rest may lie below fp32's range)
    if (!(ap > 1e-25f && ap < 1e37f)) return scaled_wide_f32(v, (double)sc.hi + (double)sc.lo);
    return p + (fmaf(v, sc.hi, -p) + v * sc.lo);
}

// The tokens go to shared memory, normed where asked.
template <typename T> __device__ __forceinline__ void stage_tokens(const Args &a, Plan &s, char *xs) {
    constexpr int kN = 16 / sizeof(T);
    const int stride = token_stride(a.d, sizeof(T)), per = a.d / kN, all = a.R * per;
#pragma unroll 4
    for (int i = threadIdx.x; i < all; i += kThr) {
        const int r = i / per, c = i - r * per;
        *reinterpret_cast<uint4 *>(xs + r * stride + 16 * c) =
            *(reinterpret_cast<const uint4 *>(a.x) + i);
    }
    __syncthreads();
    if (!a.norm) return;
    norm_scales<T>(a, s, xs);
    for (int i = threadIdx.x; i < all; i += kThr) {
        const int r = i / per, c = i - r * per;
        T *p = reinterpret_cast<T *>(xs + r * stride) + c * kN;
        const Pair sc = s.scale[r];
        const double *wide = s.wide[r] ? s.wide_scale + r : nullptr;
        if constexpr (sizeof(T) == 2) {
            scale16(reinterpret_cast<uint4 *>(p), sc, wide);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                p[j] = wide ? scaled_wide_f32(p[j], *wide) : scaled(p[j], sc);
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
__device__ __forceinline__ void router(const Args &a, const char *xs, float *red, Eight<T> first,
                                       uint32_t tag) {
    const int stride = token_stride(a.d, sizeof(T));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = blockIdx.x; e < a.E; e += gridDim.x) {
        const T *w = reinterpret_cast<const T *>(a.wr) + (size_t)e * a.d;
        // four tokens at a time: code that runs once waits for its instructions
#pragma unroll 1
        for (int r0 = 0; r0 < a.R; r0 += 4) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
            for (int c = threadIdx.x * 8; c < a.d; c += kThr * 8) {
                Eight<T> we = first;
                if (e != blockIdx.x || c >= kThr * 8) we.load(w + c);
                float wv[8];
                we.get(wv);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (r0 + q < a.R) {
                        float xv[8];
                        load8(reinterpret_cast<const T *>(xs + (r0 + q) * stride) + c, xv);
#pragma unroll
                        for (int i = 0; i < 8; ++i) acc[q] = fmaf(wv[i], xv[i], acc[q]);
                    }
                }
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[q] += __shfl_xor_sync(0xffffffffu, acc[q], o);
            if (lane < 4 && r0 + lane < a.R)
                red[warp * kMaxRows + r0 + lane] =
                    lane == 0 ? acc[0] : lane == 1 ? acc[1] : lane == 2 ? acc[2] : acc[3];
        }
        __syncthreads();
        if (threadIdx.x < a.R) {
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) v += red[i * kMaxRows + threadIdx.x];
            const unsigned long long word = (unsigned long long)tag << 32 | __float_as_uint(v);
            asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(a.scores + threadIdx.x * kMaxE + e),
                         "l"(word)
                         : "memory");
            if (a.logits) a.logits[(size_t)threadIdx.x * a.E + e] = v;
        }
        __syncthreads();
    }
}

// Each token's k largest scores (ties to the lower expert), their softmax, and who chose whom.
__device__ __forceinline__ void choose(const Args &a, Plan &s, uint32_t tag) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp < a.R) {
        const unsigned long long *l = a.scores + warp * kMaxE, t0 = now_ns();
        uint32_t key[kMaxE / 32];
#pragma unroll
        for (int i = 0; i < kMaxE / 32; ++i) key[i] = 0;
        for (unsigned tries = 1;; ++tries) {
            bool here = true;
#pragma unroll
            for (int i = 0; i < kMaxE / 32; ++i) {
                const int e = i * 32 + lane;
                if (e < a.E && key[i] == 0) {
                    const unsigned long long w = load_relaxed(l + e);
                    if ((uint32_t)(w >> 32) == tag) {
                        const uint32_t b = __float_as_uint(__uint_as_float((uint32_t)w) + 0.f);
                        key[i] = max(1u, b ^ ((int)b < 0 ? 0xffffffffu : 0x80000000u));
                    } else {
                        here = false;
                    }
                }
            }
            if (__all_sync(0xffffffffu, here)) break;
            if (tries % 256 == 0 && __any_sync(0xffffffffu, now_ns() - t0 > kPatience)) {
                if (lane == 0) {
                    atomicOr(a.flags, FLAG_WAIT_TIMEOUT);
                    s.alive = 0;
                }
                break;
            }
        }
        float mine = -INFINITY, top = 0.f;  // lane j: the j-th chosen score
        int who = 0;
        // the lane's keys in descending order (ties to the lower expert), so that what is next is at hand
        int id[kMaxE / 32];
#pragma unroll
        for (int i = 0; i < kMaxE / 32; ++i) id[i] = i * 32 + lane;
        const int held = (a.E + 31) / 32;
#pragma unroll
        for (int n = 1; n < kMaxE / 32; ++n) {
            if (n >= held) break;
#pragma unroll
            for (int i = n; i > 0; --i) {
                const bool up = key[i] > key[i - 1];
                const uint32_t k0 = up ? key[i] : key[i - 1], k1 = up ? key[i - 1] : key[i];
                const int i0 = up ? id[i] : id[i - 1], i1 = up ? id[i - 1] : id[i];
                key[i - 1] = k0;
                key[i] = k1;
                id[i - 1] = i0;
                id[i] = i1;
            }
        }
#pragma unroll 1
        for (int j = 0; j < a.k; ++j) {
            const uint32_t best = __reduce_max_sync(0xffffffffu, key[0]);
            const int e = (int)__reduce_min_sync(0xffffffffu, key[0] == best ? (unsigned)id[0] : (unsigned)kMaxE);
            if (e == id[0]) {
#pragma unroll
                for (int i = 0; i + 1 < kMaxE / 32; ++i) {
                    key[i] = key[i + 1];
                    id[i] = id[i + 1];
                }
                key[kMaxE / 32 - 1] = 0;
            }
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
    // a warp for 32 experts
    const int e = threadIdx.x;
    int slot = e;
    bool on = e < a.E && s.tokens[e];
    if (on && a.slot) slot = a.slot[e];
    if (on && (slot < 0 || slot >= a.slots)) {
        on = false;
        if (blockIdx.x == 0) atomicOr(a.flags, FLAG_BAD_EXPERT);
    }
    const uint32_t m = __ballot_sync(0xffffffffu, on);
    if (warp < kMaxE / 32 && lane == 0) s.word[warp] = m;
    __syncthreads();
    int before = 0, n = 0;
#pragma unroll
    for (int i = 0; i < kMaxE / 32; ++i) {
        const int c = __popc(s.word[i]);
        if (i < warp) before += c;
        n += c;
    }
    if (on) {
        const int at = before + __popc(m & ((1u << lane) - 1));
        s.expert[at] = (short)e;
        s.slot[at] = slot;
    }
    // (what needs divisions is computed once: 256 experts of 6144 pairs on a thousand CTAs fit 32 bits)
    if (threadIdx.x == 0) {
        s.n = n;
        const unsigned pairs = n * a.f;
        s.pair0 = (int)(pairs * blockIdx.x / gridDim.x);
        s.pair1 = (int)(pairs * (blockIdx.x + 1) / gridDim.x);
    } else if (threadIdx.x == 32) {
        s.col0 = (int)((unsigned)a.d * blockIdx.x / gridDim.x);
        s.col1 = (int)((unsigned)a.d * (blockIdx.x + 1) / gridDim.x);
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
    __nv_bfloat16 hi = __float2bfloat16(v);
    float rest = v - __bfloat162float(hi);
    if (fabsf(rest) == INFINITY || fabsf(v) == INFINITY) {
        // beyond bf16's largest: that and the rest; an infinity has none
        hi = __float2bfloat16_rz(v);
        rest = fabsf(v) == INFINITY ? 0.f : v - __bfloat162float(hi);
    }
    h[j] = hi;
    h[a.f + j] = __float2bfloat16(rest);
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

// n: 16, or 0: the 16 bytes become zeros and nothing is read.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int n) {
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

// Step 2's work: the CTA's share of the pairs (a gate and an up row) over all chosen experts, in runs of
// one expert whose partial sums fit a buffer, of tiles of 8 pairs.
struct Run {
    int ui, j0, nj, tiles, m;
    unsigned mask;
    __device__ __forceinline__ Run(const Args &a, const Plan &s, int p, int p1) {
        ui = (int)((unsigned)p / (unsigned)a.f);
        j0 = p - ui * a.f;
        mask = s.tokens[s.expert[ui]];
        m = __popc(mask);
        // tiles that fit a buffer: red_bytes() / (1 KB m)
        const int most = (a.R <= 8 ? 8u : 16u) / (unsigned)m;
        nj = min(min(a.f - j0, p1 - p), 8 * most);
        tiles = (nj + 7) / 8;
    }
};
// The warp's part of n groups of 32 inner elements.
__device__ __forceinline__ int part(int n, int warp) { return (int)((unsigned)(n * warp) / kWarps); }
__device__ __forceinline__ int groups(int n) { return (n + 31) / 32; }
// Step 3's work: the CTA's output columns, in tiles of up to 16.
struct Columns {
    int c0, c1, tiles;
    __device__ __forceinline__ explicit Columns(const Plan &s) {
        c0 = s.col0;
        c1 = s.col1;
        tiles = (c1 - c0 + 15) / 16;
    }
    __device__ __forceinline__ int at(int tile) const {
        return tiles == 1 ? (tile ? c1 : c0) : c0 + (int)((unsigned)((c1 - c0) * tile) / (unsigned)tiles);
    }
};

// What a warp copies, entry after entry: first step 2's, then step 3's. A segment is a run of entries
// along the inner dimension of the same 16 rows; inside it a lane's addresses only advance. Step 3's
// entries have the activations of the same inner elements in a second ring.
template <int D> struct Feed {
    const Args &a;
    const Plan &s;
    uint32_t base, put;      // the lane's bytes of entry 0, offset of the next entry
    // The same of the activations' ring: an entry has the values and the rests of as many columns as
    // there may be, 64 bytes each.
    uint32_t h_base, h_put;
    // the segment, as the lane sees it
    const __nv_bfloat16 *x, *y, *h;  // two rows of weights, and of activations
    int c, end, left;                // inner element, where the rows end, entries left
    int nx, ny, nh;                  // bytes of a copy, or 0
    // where the segments come from
    int pair, pair1, tile, tiles, nj, ui, j0, q;
    bool down, done;

    __device__ __forceinline__ Feed(const Args &a_, const Plan &s_, const char *ring, const char *h_ring)
        : a(a_), s(s_) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        base = (uint32_t)__cvta_generic_to_shared(ring) + warp * D * 1024 + lane * 16;
        put = 0;
        h_base = (uint32_t)__cvta_generic_to_shared(h_ring) + warp * D * slot() + (lane >> 2) * 128 +
                 (lane & 3) * 16;
        h_put = 0;
        pair = s.pair0;
        pair1 = s.pair1;
        nj = tiles = left = 0;
        tile = -1;
        down = done = false;
        segment();
    }
    __device__ __forceinline__ uint32_t slot() const { return min(a.R, 8) * 128; }
    // Activations of the lane's column of an expert, from element c on: the expert's g-th token's.
    __device__ __forceinline__ const __nv_bfloat16 *activations(int ui, int col, int c) const {
        const int e = s.expert[ui];
        const unsigned mask = s.tokens[e];
        const int r = nth_token(mask, col < __popc(mask) ? col : 0);
        return reinterpret_cast<const __nv_bfloat16 *>(a.h) +
               (size_t)(r * a.k + s.place[e][r]) * 2 * a.f + c;
    }
    __device__ __forceinline__ int columns(int ui) const { return __popc(s.tokens[s.expert[ui]]); }
    // The next segment (left > 0), or done.
    __device__ __forceinline__ void segment() {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
        if (!down) {
            const int k0 = part(groups(a.d), warp), k1 = part(groups(a.d), warp + 1);
            if (++tile >= tiles) {
                pair += nj;
                tile = 0;
                if (pair >= pair1 || k0 == k1) {  // (a warp without a part has no entries)
                    down = true;
                    q = part(s.n * groups(a.f), warp);
                    tiles = Columns(s).tiles;
                } else {
                    const Run r(a, s, pair, pair1);
                    tiles = r.tiles;
                    nj = r.nj;
                    ui = r.ui;
                    j0 = r.j0;
                }
            }
            if (!down) {
                const int j = tile * 8 + g;
                const bool on = j < nj;
                nx = ny = on ? 16 : 0;
                c = k0 * 32 + 8 * t;
                end = a.d;
                left = k1 - k0;
                const size_t at = ((size_t)s.slot[ui] * a.f + j0 + (on ? j : 0)) * a.d + c;
                x = reinterpret_cast<const __nv_bfloat16 *>(a.wg) + at;
                y = reinterpret_cast<const __nv_bfloat16 *>(a.wu) + at;
                return;
            }
        }
        const int nk = groups(a.f), q0 = part(s.n * nk, warp), q1 = part(s.n * nk, warp + 1);
        if (q >= q1) {
            q = q0;
            ++tile;
        }
        if (q0 == q1 || tile >= tiles) {
            done = true;
            return;
        }
        const Columns cols(s);
        const int e = q / nk, k0 = q - e * nk, col = cols.at(tile) + g, last = cols.at(tile + 1);
        left = min(nk - k0, q1 - q);
        q += left;
        nx = col < last ? 16 : 0;
        ny = col + 8 < last ? 16 : 0;
        c = k0 * 32 + 8 * t;
        end = a.f;
        x = reinterpret_cast<const __nv_bfloat16 *>(a.wd) +
            ((size_t)s.slot[e] * a.d + (nx ? col : 0)) * a.f + c;
        y = ny ? x + 8ll * a.f : x;
        h = activations(e, g, c);
        nh = g < columns(e) ? 16 : 0;
    }
    template <bool H> __device__ __forceinline__ void fill() {
        if (!done) {
            const bool in = c < end;
            copy16(base + put, x, in ? nx : 0);
            copy16(base + put + 512, y, in ? ny : 0);
            if (H) {
                if (in && nh) {
                    copy16(h_base + h_put, h, 16);
                    copy16(h_base + h_put + 64, h + a.f, 16);
                }
                h_put = h_put + slot() == D * slot() ? 0 : h_put + slot();
            }
            x += 32;
            y += 32;
            h += 32;
            c += 32;
            if (--left == 0) segment();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        put = put + 1024 == D * 1024 ? 0 : put + 1024;
    }
    // The activations of the entries of step 3 that were copied before there were any.
    __device__ __forceinline__ void catch_up() {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
        const int nk = groups(a.f), q0 = part(s.n * nk, warp), q1 = part(s.n * nk, warp + 1);
        int todo = min(D - 1, (q1 - q0) * Columns(s).tiles);
        const int none = D - 1 - todo;
#pragma unroll 1
        while (todo > 0) {  // (again from q0 where the warp's part is shorter than the ring)
#pragma unroll 1
            for (int q = q0; q < q1 && todo > 0;) {
                const int e = q / nk, n = min(min(nk - (q - e * nk), q1 - q), todo);
                const bool on = g < columns(e);
                int c = (q - e * nk) * 32 + 8 * t;
                const __nv_bfloat16 *p = activations(e, g, c);
#pragma unroll 1
                for (int i = 0; i < n; ++i, c += 32, p += 32) {
                    if (on && c < a.f) {
                        copy16(h_base + h_put, p, 16);
                        copy16(h_base + h_put + 64, p + a.f, 16);
                    }
                    h_put = h_put + slot() == D * slot() ? 0 : h_put + slot();
                    asm volatile("cp.async.commit_group;" ::: "memory");
                }
                q += n;
                todo -= n;
            }
        }
        // (as many groups as there are entries before an entry is waited for)
#pragma unroll 1
        for (int i = 0; i < none; ++i) asm volatile("cp.async.commit_group;" ::: "memory");
    }
};

// Steps 2 and 3. NT: groups of 8 tokens; D: entries of a warp's ring.
template <int NT, int D> struct Experts {
    const Args &a;
    Plan &s;
    Feed<D> feed;
    uint32_t take;

    __device__ __forceinline__ Experts(const Args &a_, Plan &s_, const char *ring, const char *h_ring)
        : a(a_), s(s_), feed(a_, s_, ring, h_ring), take(0) {
#pragma unroll 1
        for (int i = 0; i < D - 1; ++i) feed.template fill<false>();
    }
    // The oldest entry's address; its place is filled again by the next fill().
    __device__ __forceinline__ uint32_t get() {
        asm volatile("cp.async.wait_group %0;" ::"n"(D - 2) : "memory");
        const uint32_t at = feed.base + take;
        take = take + 1024 == D * 1024 ? 0 : take + 1024;
        return at;
    }

    __device__ __forceinline__ void gate_up(const char *xs, float *red) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
        const int stride = token_stride(a.d, 2);
        const int k0 = part(groups(a.d), warp), k1 = part(groups(a.d), warp + 1);
        const int p1 = s.pair1;
        int buf = 0;
#pragma unroll 1
        for (int p = s.pair0; p < p1;) {
            const Run r(a, s, p, p1);
            const int m = r.m;
            float *out = red + buf * (red_bytes(a.R) / 4);
            // this lane's columns: tokens g and g + 8 of the expert's
            const char *x0 = g < m ? xs + nth_token(r.mask, g) * stride : nullptr;
            const char *x1 = g + 8 < m ? xs + nth_token(r.mask, g + 8) * stride : nullptr;
#pragma unroll 1
            for (int tile = 0; tile < r.tiles; ++tile) {
                float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
                int c = k0 * 32 + 8 * t;
#pragma unroll 1
                for (int k = k0; k < k1; ++k, c += 32) {
                    const uint32_t at = get();
                    const uint4 x = shared16(at), y = shared16(at + 512);
                    uint4 b = make_uint4(0, 0, 0, 0);
                    if (x0 && c < a.d) b = *reinterpret_cast<const uint4 *>(x0 + 2 * c);
                    feed.template fill<false>();
                    mma32(c0, x, y, b);
                    if (NT > 1 && m > 8) {
                        b = make_uint4(0, 0, 0, 0);
                        if (x1 && c < a.d) b = *reinterpret_cast<const uint4 *>(x1 + 2 * c);
                        mma32(c1, x, y, b);
                    }
                }
                float *o = out + ((size_t)(warp * r.tiles + tile) * 16 + g) * m;
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
            }
            __syncthreads();
            finish_gate_up<__nv_bfloat16>(a, s, out, r.tiles, s.expert[r.ui], r.j0, r.nj, r.mask, m);
            buf ^= 1;  // (a buffer is written again after the CTA's next barrier)
            p += r.nj;
        }
    }

    __device__ __forceinline__ void down(float *red) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
        float *mine = red + (size_t)warp * 16 * a.R;
        const Columns cols(s);
        const int nk = groups(a.f), q0 = part(s.n * nk, warp), q1 = part(s.n * nk, warp + 1);
        feed.catch_up();
        uint32_t h_take = 0;
#pragma unroll 1
        for (int tile = 0; tile < cols.tiles; ++tile) {
            const int b0 = cols.at(tile), b1 = cols.at(tile + 1);
            for (int i = lane; i < 16 * a.R; i += 32) mine[i] = 0.f;
            __syncwarp();
            int ui = q0 / nk;
#pragma unroll 1
            for (int q = q0; q < q1; ++ui) {
                const int last = min(q1, (ui + 1) * nk);
                const unsigned mask = s.tokens[s.expert[ui]];
                const int m = __popc(mask);
                // products with the values and with their rests (two chains), and of tokens past the 8th
                float hi[4] = {0.f, 0.f, 0.f, 0.f}, lo[4] = {0.f, 0.f, 0.f, 0.f};
                float more[4] = {0.f, 0.f, 0.f, 0.f};
                int c = (q - ui * nk) * 32 + 8 * t;
#pragma unroll 1
                for (; q < last; ++q, c += 32) {
                    const uint32_t at = get();
                    const uint4 x = shared16(at), y = shared16(at + 512);
                    uint4 u = make_uint4(0, 0, 0, 0), v = u;
                    if (g < m && c < a.f) {
                        u = shared16(feed.h_base + h_take);
                        v = shared16(feed.h_base + h_take + 64);
                    }
                    h_take = h_take + feed.slot() == D * feed.slot() ? 0 : h_take + feed.slot();
                    feed.template fill<true>();
                    mma32(hi, x, y, u);
                    mma32(lo, x, y, v);
                    if (NT > 1 && m > 8) {
                        // (an expert of more than 8 tokens: the others' are read here and now)
                        const __nv_bfloat16 *p = feed.activations(ui, g + 8, c);
                        u = v = make_uint4(0, 0, 0, 0);
                        if (g + 8 < m && c < a.f) {
                            u = l2_16(p);
                            v = l2_16(p + a.f);
                        }
                        mma32(more, x, y, u);
                        mma32(more, x, y, v);
                    }
                }
                // the warp's part of the expert is done: its columns are tokens
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int col = 2 * t + k;
                    if (col < m) {
                        float *o = mine + g * a.R + nth_token(mask, col);
                        o[0] += hi[k] + lo[k];
                        o[8 * a.R] += hi[2 + k] + lo[2 + k];
                    }
                    if (NT > 1 && col + 8 < m) {
                        float *o = mine + g * a.R + nth_token(mask, col + 8);
                        o[0] += more[k];
                        o[8 * a.R] += more[2 + k];
                    }
                }
                __syncwarp();
            }
            __syncthreads();
            for (int i = threadIdx.x; i < (b1 - b0) * a.R; i += kThr) {
                const int r = i / (b1 - b0), col = i - r * (b1 - b0);
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) v += red[(size_t)(w * 16 + col) * a.R + r];
                store_y<__nv_bfloat16>(a, r, b0 + col, v);
            }
            __syncthreads();  // (the sums are read before the next tile's)
        }
    }
};

// ---- fp32 steps 2 and 3: rows times tokens in registers, 32 sums a lane ----
// A weight is read once for up to 4, 8 or 16 tokens, a token once for 8, 4 or 2 rows. Measured: 13 tokens,
// 7 experts of 1104 x 1088, top-6 76 us (floor 15; a warp and a row for each token 111), 14 tokens, 83
// experts of 904 x 336, top-8 74 (34; 161), one token, 68 of 1504 x 2608, top-4 52 (28; 56). Bound by the
// loads' latency: 16 warps with 8 loads each on their way. Asking L2 for the next rows ahead: 82 to 100.
// A lane's 32 sums are summed over the warp and shared out: lane i gets the i-th (31 shuffles).
__device__ __forceinline__ float sum_out(float (&v)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float keep = lane & o ? v[i + o] : v[i], give = lane & o ? v[i] : v[i + o];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    return v[0];
}
__device__ __forceinline__ void add_product(float &s, const float4 &a, const float4 &b) {
    s = fmaf(a.x, b.x, s);
    s = fmaf(a.y, b.y, s);
    s = fmaf(a.z, b.z, s);
    s = fmaf(a.w, b.w, s);
}

// P pairs of rows (np of them are there) times T tokens at a time.
template <int P, int T>
__device__ __forceinline__ void gate_up_pairs(const Args &a, const Plan &s, const char *xs, int ui, int j0,
                                              int np) {
    static_assert(P * T == 16, "32 sums, gate's in the lower half of the warp");
    const int lane = threadIdx.x & 31, e = s.expert[ui], stride = token_stride(a.d, 4);
    const size_t at = ((size_t)s.slot[ui] * a.f + j0) * a.d;
    const float *wg = reinterpret_cast<const float *>(a.wg) + at;
    const float *wu = reinterpret_cast<const float *>(a.wu) + at;
    for (unsigned mask = s.tokens[e]; mask;) {
        const unsigned group = mask;
        const int n = min(T, __popc(mask));
        int x[T];
#pragma unroll
        for (int t = 0; t < T; ++t) {
            x[t] = mask ? (__ffs(mask) - 1) * stride : 0;
            mask &= mask - 1;
        }
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.f;
        // (8 loads of weights on their way)
        constexpr int U = 4 / P;
#pragma unroll 1
        for (int c = lane * 4; c < a.d; c += 128 * U) {
            float4 w[U][2 * P];
#pragma unroll
            for (int k = 0; k < U; ++k)
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const size_t row = (size_t)(i < np ? i : 0) * a.d + (c + 128 * k < a.d ? c + 128 * k : c);
                    w[k][i] = __ldg(reinterpret_cast<const float4 *>(wg + row));
                    w[k][P + i] = __ldg(reinterpret_cast<const float4 *>(wu + row));
                }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (c + 128 * k >= a.d) break;
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    if (t >= n) break;
                    const float4 q = *reinterpret_cast<const float4 *>(xs + x[t] + 4 * (c + 128 * k));
#pragma unroll
                    for (int i = 0; i < 2 * P; ++i) add_product(v[i * T + t], w[k][i], q);
                }
            }
        }
        const float g = sum_out(v), u = __shfl_down_sync(0xffffffffu, g, 16);
        const int i = lane / T, t = lane % T;
        if (i < np && t < n) {
            const int r = nth_token(group, t), place = s.place[e][r];
            store_h(a, (float *)nullptr, r * a.k + place, j0 + i, silu(g) * u * s.gate[r][place]);
        }
    }
}

// The warps take groups of up to 4 pairs of an expert in turn: weights are read once for 4 tokens, and
// tokens once for 8 rows. More tokens take fewer rows, and so do short shares.
__device__ __forceinline__ void gate_up(const Args &a, const Plan &s, const char *xs) {
    const int warp = threadIdx.x >> 5, p1 = s.pair1;
    const int each = (p1 - s.pair0 + kWarps - 1) / kWarps;  // pairs a warp
    int turn = 0;
#pragma unroll 1
    for (int p = s.pair0; p < p1;) {
        const int ui = (int)((unsigned)p / (unsigned)a.f), end = min(p1, (ui + 1) * a.f);
        const int m = __popc((unsigned)s.tokens[s.expert[ui]]);
        const int size = each == 1 ? 1 : m <= 4 && each > 2 ? 4 : 2;
        const int n = (end - p + size - 1) / size;
#pragma unroll 1
        for (int g = (warp - turn) & (kWarps - 1); g < n; g += kWarps) {
            const int at = p + g * size, j0 = at - ui * a.f, np = min(size, end - at);
            if (size == 4)
                gate_up_pairs<4, 4>(a, s, xs, ui, j0, np);
            else if (size == 2)
                gate_up_pairs<2, 8>(a, s, xs, ui, j0, np);
            else
                gate_up_pairs<1, 16>(a, s, xs, ui, j0, np);
        }
        turn += n;
        p = end;
    }
}

// C columns times T tokens: the warps share the inner dimension over all chosen experts, in chunks of 128.
template <int C, int T>
__device__ __forceinline__ void down_columns(const Args &a, const Plan &s, int c0, int nc, int ui, int k0,
                                             int k1, float *mine) {
    static_assert(C * T == 32, "32 sums");
    const int lane = threadIdx.x & 31, e = s.expert[ui];
    const float *w0 = reinterpret_cast<const float *>(a.wd) + ((size_t)s.slot[ui] * a.d + c0) * a.f;
    for (unsigned mask = s.tokens[e]; mask;) {
        const unsigned group = mask;
        const int n = min(T, __popc(mask));
        int row[T];
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int r = mask ? __ffs(mask) - 1 : __ffs(group) - 1;
            row[t] = (r * a.k + s.place[e][r]) * a.f;
            mask &= mask - 1;
        }
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.f;
#pragma unroll 1
        for (int c = k0 * 128 + lane * 4; c < min(a.f, k1 * 128); c += 128) {
            // (all loads before the first branch, as it would part them: places without a token read the
            // first one's activations)
            float4 w[C], q[T];
#pragma unroll
            for (int i = 0; i < C; ++i)
                w[i] = __ldg(reinterpret_cast<const float4 *>(w0 + (size_t)(i < nc ? i : 0) * a.f + c));
#pragma unroll
            for (int t = 0; t < T; ++t)
                q[t] = __ldcg(reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(a.h) + row[t] + c));
#pragma unroll
            for (int t = 0; t < T; ++t) {
                if (t >= n) break;
#pragma unroll
                for (int i = 0; i < C; ++i) add_product(v[i * T + t], w[i], q[t]);
            }
        }
        const float sum = sum_out(v);
        const int i = lane / T, t = lane % T;
        if (i < nc && t < n) mine[i * a.R + nth_token(group, t)] += sum;
        __syncwarp();
    }
}

__device__ __forceinline__ void down(const Args &a, const Plan &s, float *red) {
    constexpr int kCols = 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nk = (a.f + 127) / 128, q0 = part(s.n * nk, warp), q1 = part(s.n * nk, warp + 1);
    float *mine = red + warp * kCols * a.R;
#pragma unroll 1
    for (int c0 = s.col0; c0 < s.col1; c0 += kCols) {
        const int nc = min(kCols, s.col1 - c0);
        for (int i = lane; i < kCols * a.R; i += 32) mine[i] = 0.f;
        __syncwarp();
#pragma unroll 1
        for (int q = q0; q < q1;) {
            const int ui = q / nk, last = min(q1, (ui + 1) * nk), k0 = q - ui * nk, k1 = last - ui * nk;
            if (__popc((unsigned)s.tokens[s.expert[ui]]) <= 4) {
                down_columns<8, 4>(a, s, c0, nc, ui, k0, k1, mine);
            } else {
#pragma unroll 1
                for (int h = 0; h < nc; h += 4)
                    down_columns<4, 8>(a, s, c0 + h, min(4, nc - h), ui, k0, k1, mine + h * a.R);
            }
            q = last;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < nc * a.R; i += kThr) {
            const int col = i / a.R, r = i - col * a.R;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += red[(w * kCols + col) * a.R + r];
            store_y<float>(a, r, c0 + col, v);
        }
        __syncthreads();  // (the sums are read before the next columns')
    }
}

constexpr int kPlanBytes = (sizeof(Plan) + 127) / 128 * 128;
constexpr int kSmem = 227 * 1024;
constexpr __host__ __device__ int fixed_bytes(int R) { return kPlanBytes + 2 * red_bytes(R); }
__host__ __device__ constexpr int ring_bytes(int D) { return D * kWarps * 1024; }
// Shared memory of a launch; step 3's activations take the tokens' place.
constexpr int smem_bytes(int R, int d, int elem, int D) {
    return fixed_bytes(R) + ring_bytes(D) + std::max(D * kWarps * std::min(R, 8) * 128, R * token_stride(d, elem));
}

// D = 0: fp32.
template <typename T, int NT, int D>
__global__ void __launch_bounds__(kThr, 1) few_kernel(const Args a) {
    extern __shared__ __align__(128) char dyn[];
    Plan &s = *reinterpret_cast<Plan *>(dyn);
    float *red = reinterpret_cast<float *>(dyn + kPlanBytes);
    const char *ring = dyn + fixed_bytes(a.R);
    char *xs = dyn + fixed_bytes(a.R) + ring_bytes(D);
    pdl_wait();
    Eight<T> first{};
    if (blockIdx.x < a.E && threadIdx.x * 8 < a.d)
        first.load(reinterpret_cast<const T *>(a.wr) + (size_t)blockIdx.x * a.d + threadIdx.x * 8);
    if (threadIdx.x < kMaxE) s.tokens[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
        // (no CTA counts this launch as ended before this one has come to the barrier)
        s.launch = load_relaxed(a.barrier) >> 16;
        s.alive = 1;
    }
    stage_tokens<T>(a, s, xs);
    const unsigned long long launch = s.launch;
    const uint32_t tag = (uint32_t)launch + 1;
    router<T>(a, xs, red, first, tag);
    choose(a, s, tag);
    if (!s.alive) return;
    if constexpr (D > 0) {
        Experts<NT, D> r(a, s, ring, xs);
        r.gate_up(xs, red);
        const bool alive = grid_barrier(a, s, launch);
        if (alive) r.down(red);
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        gate_up(a, s, xs);
        if (!grid_barrier(a, s, launch)) return;
        down(a, s, red);
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
    cfg.dynamicSmemBytes = smem_bytes(a.R, a.d, sizeof(T), D);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, few_kernel<T, NT, D>, a);
}

// Rings as deep as shared memory holds: at one or two tokens 10 entries a warp (of the 12 that it has of step 3
// in the Qwen3-shaped layer, 9 are on their way before the grid's barrier), up to 6 tokens 7, with more 5, and 4 from 9
// long tokens on (16 of more than 3392 elements).
static_assert(smem_bytes(2, kMaxD, 2, 10) <= kSmem && smem_bytes(6, kMaxD, 2, 7) <= kSmem &&
              smem_bytes(8, kMaxD, 2, 5) <= kSmem && smem_bytes(9, kMaxD, 2, 4) <= kSmem);
template <int NT, int D> cudaError_t launch_ring(const Args &a, int max_ctas, cudaStream_t s) {
    return launch<__nv_bfloat16, NT, D>(a, max_ctas, s);
}

}  // namespace

int rows_at_once(const moe_layer_desc &L) {
    const int e = (int)elem_size(L.dtype);
    int R = kMaxRows;
    while (R > 1 && smem_bytes(R, L.d, e, L.dtype == MOE_DTYPE_F32 ? 0 : 4) > kSmem) --R;
    return R;
}

static_assert(kHeadBytes == MOE_FEW_HEAD_BYTES, "the header says how much is zeroed");

cudaError_t launch_few(const Args &a, int dtype, int max_ctas, cudaStream_t s) {
    if (dtype == MOE_DTYPE_F32) return launch<float, 1, 0>(a, max_ctas, s);
    auto fits = [&](int D) { return smem_bytes(a.R, a.d, 2, D) <= kSmem; };
    if (a.R <= 8)
        return fits(10)  ? launch_ring<1, 10>(a, max_ctas, s)
               : fits(7) ? launch_ring<1, 7>(a, max_ctas, s)
                         : launch_ring<1, 5>(a, max_ctas, s);
    return fits(5) ? launch_ring<2, 5>(a, max_ctas, s) : launch_ring<2, 4>(a, max_ctas, s);
}

}  // namespace few
}  // namespace moe
