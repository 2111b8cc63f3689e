// Sampling of a token from each row of logits: temperature, top-k, top-p, min-p, and the inversion of
// the remaining tokens' distribution in the order of the tokens at a given random number.
//
//   w_i = 2^(-(l_max - l_i) log2(e) / T);  K = the k largest;  P = the shortest run of K in
//   descending order that holds at least p of K's weight;  M = those of w_i >= min_p;
//   token = the first i with sum_{j <= i, kept} w_j > u sum_{kept} w_j.
//
// A token of thousands follows from comparisons of sums of up to V weights, so sums that depend on the
// order of threads, or that are off by fp32's roundings, give another token every few thousand
// rows. Weights are therefore integers of 2^-43 (exp2 from a difference, a product and a
// polynomial carried as pairs of fp32 values; off by some 2^-42 relative, checked against 64 bits),
// and sums are 64-bit integers: exact, and the same in any order.
//
// A cluster of CTAs holds a row in shared memory, which reads it once.
//
// Every cut keeps the first tokens of the descending order, so what is kept lies among the largest
// ones, of which there are few as a rule: a bound from below on the last of them (for top-k, the k-th
// largest of the threads' own largest values, up to a bin; for min-p its own) lets a second pass collect
// them, and one CTA sorts them and does the rest. top-p needs the whole weight too; a sum of fp32
// exponentials, off by at most 2^-15, decides unless a cut lies within that.
// Where more is kept than a list holds (flat distributions, no cuts), cuts are found by histograms of
// the row's live values (weights that are not below 2^-43) over bins that descend with the value:
// counts for top-k, weights for top-p; the bin that a cut falls in is divided by the bits of the
// values until one value is left, and ties are taken in the order of the tokens.
#include <cooperative_groups.h>

#include <cfloat>

#include "sample.cuh"

namespace moe {
namespace sample {
namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kThr = 512, kWarps = kThr / 32;
constexpr int kBins = 1024, kPer = kBins / kThr;
constexpr int kMaxCluster = 8;
constexpr float kLive = 43.f;                   // octaves below the largest
constexpr float kBinScale = (kBins - 1) / kLive;
constexpr u64 kOne = 1ull << 43;                // the weight of the largest

// 2^(-j / 256) as two fp32 values.
struct Powers {
    float hi[256], lo[256];
};
constexpr Powers make_powers() {
    // 2^-(1/2), 2^-(1/4), .. 2^-(1/256)
    constexpr double root[8] = {0.70710678118654752440, 0.84089641525371454303,
                                0.91700404320467123175, 0.95760328069857364694,
                                0.97857206208770013451, 0.98922801319397548413,
                                0.99459942348363317565, 0.99729605608547012626};
    Powers t{};
    for (int j = 0; j < 256; ++j) {
        double v = 1.0;
        for (int b = 0; b < 8; ++b)
            if (j >> (7 - b) & 1) v *= root[b];
        t.hi[j] = (float)v;
        t.lo[j] = (float)(v - (double)t.hi[j]);
    }
    return t;
}
__device__ const Powers kPowers = make_powers();

// What the weights of a row depend on: the largest value, and log2(e) / T as two fp32 values.
struct Scale {
    float top, ch, cl;
};

// Octaves of a value below the largest, as the bins see it: it does not grow with the value.
__device__ __forceinline__ float octaves(const Scale &s, float l) { return (s.top - l) * s.ch; }
__device__ __forceinline__ bool is_live(const Scale &s, float l) { return octaves(s, l) < kLive; }

// The weight of a live value in units of 2^-43. The difference and its product with log2(e) / T are
// carried as two fp32 values; 2^-x is a table's 2^(-k/256) times e^q, |q| <= 2^-9 ln 2 and a
// little; the parts are turned into integers at 2^22 and 2^43.
__device__ __forceinline__ u64 weight(const Scale &s, float l, const float2 *powers) {
    constexpr float kBig = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
    constexpr double kLn2 = 0.69314718055994530942;
    constexpr float lh = (float)kLn2, ll = (float)(kLn2 - (double)lh);
    const float d = s.top - l, bb = d - s.top, e = (s.top - (d - bb)) - (l + bb);
    const float p = __fmul_rn(d, s.ch), pe = fmaf(d, s.ch, -p) + fmaf(d, s.cl, e * s.ch);
    const float kb = fmaf(p, 256.f, kBig);
    const int k = __float_as_int(kb) - 0x4b400000;
    const float r = fmaf(kb - kBig, -1.f / 256.f, p);  // exact
    const float q = __fmul_rn(-r, lh), ql = fmaf(-r, lh, -q) - fmaf(r, ll, pe * lh);
    const float more = fmaf(ql, q, ql) + q * q * fmaf(q, fmaf(q, 1.f / 24.f, 1.f / 6.f), 0.5f);
    const float eh = q + more, el = more - (eh - q);
    const float2 t = powers[k & 255];
    const float sc = __int_as_float((127 + 22 - (k >> 8)) << 23);
    const float a = t.x * sc, b = __fmul_rn(a, eh), al = t.y * sc;
    const float c = fmaf(a, eh, -b) + fmaf(a, el, fmaf(al, q, al));
    const float ai = a + 8388608.f, bi = b + kBig;
    const float rest = (a - (ai - 8388608.f)) + (b - (bi - kBig)) + c;
    const int hi = (__float_as_int(ai) - 0x4b000000) + (__float_as_int(bi) - 0x4b400000);
    const int lo = __float_as_int(fmaf(rest, 2097152.f, kBig)) - 0x4b400000;
    const long long w = ((long long)hi << 21) + lo;
    return w > 0 ? (u64)w : 0;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Values in the order of their keys (NaN and -0 do not occur).
__device__ __forceinline__ uint32_t key_of(float l) {
    const uint32_t b = __float_as_uint(l);
    return b ^ ((int)b < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key ^ ((int)key < 0 ? 0x80000000u : 0xffffffffu));
}

// A 16-byte block of a row.
template <typename T> struct Block;
template <> struct Block<float> {
    static constexpr int kN = 4;
    float4 v;
    __device__ __forceinline__ float get(int i) const {
        return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    }
    // NaN becomes -inf, +inf the largest finite value, -0 becomes 0
    __device__ __forceinline__ static float clean(float x) {
        return fminf(fmaxf(x, -INFINITY), FLT_MAX) + 0.f;
    }
    __device__ __forceinline__ void clean() {
        v.x = clean(v.x);
        v.y = clean(v.y);
        v.z = clean(v.z);
        v.w = clean(v.w);
    }
    __device__ __forceinline__ float top() const {
        return fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
    }
    __device__ __forceinline__ void edge(const float *p, int e, int V) {
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = e + i >= 0 && e + i < V ? p[e + i] : -INFINITY;
        v = make_float4(x[0], x[1], x[2], x[3]);
    }
};
template <> struct Block<__nv_bfloat16> {
    static constexpr int kN = 8;
    uint4 v;
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
        return i & 1 ? bf16_hi(w) : bf16_lo(w);
    }
    __device__ __forceinline__ static uint32_t clean(uint32_t x) {
        const uint32_t low = 0xff80ff80u, big = 0x7f7f7f7fu, zero = 0;
        __nv_bfloat162 t = __hmax2(reinterpret_cast<__nv_bfloat162 &>(x),
                                   reinterpret_cast<const __nv_bfloat162 &>(low));
        t = __hmin2(t, reinterpret_cast<const __nv_bfloat162 &>(big));
        t = __hadd2(t, reinterpret_cast<const __nv_bfloat162 &>(zero));
        return reinterpret_cast<uint32_t &>(t);
    }
    __device__ __forceinline__ void clean() {
        v.x = clean(v.x);
        v.y = clean(v.y);
        v.z = clean(v.z);
        v.w = clean(v.w);
    }
    __device__ __forceinline__ float top() const {
        const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&v);
        const __nv_bfloat162 m = __hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
    __device__ __forceinline__ void edge(const __nv_bfloat16 *p, int e, int V) {
        uint32_t x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = e + i >= 0 && e + i < V ? __bfloat16_as_ushort(p[e + i]) : 0xff80u;
        v = make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
    }
};

constexpr int kList = 512;           // tokens of a list
constexpr int kListK = 384;          // of them asked for (the bins' last may hold more)
constexpr int kGuess = 256;          // where only top-p cuts: as many of the largest are tried
constexpr float kSumError = 0x1p-15f;

struct Shared {
    float2 powers[256];
    union {
        struct {
            uint32_t lo[kBins], hi[kBins];
        };
        struct {
            uint32_t list_key[kList], list_index[kList];
            u64 sorted[kList];  // ~key, index: ascending
        };
    };
    u64 part[kWarps];
    float red_f[kWarps];
    uint32_t red_a[kWarps], red_b[kWarps];
    // read by the other CTAs of the cluster
    float top;
    uint32_t kmin, kmax, index;
    u64 wsum[kWarps];
    uint32_t ties[kWarps];
    uint32_t listed;
    float sum;
    int settled;
    // found by one thread
    int bin;
    u64 before;
    int owner;
    u64 own_w;
    uint32_t own_t;
    u64 target, z;
    float low;  // the least value that min-p keeps
};

// Sum of the block's threads before this one, in their order; the sum of all in *total.
__device__ __forceinline__ u64 block_scan(u64 v, u64 *part, u64 *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
    }
    __syncthreads();
    if (lane == 31) part[warp] = s;
    __syncthreads();
    u64 before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        const u64 p = part[i];
        if (i < warp) before += p;
        all += p;
    }
    *total = all;
    return before + s - v;
}

// log of the share that a token of logit l has of the sum z.
__device__ __forceinline__ float log_share(float l, float top, float temp, u64 z) {
    const float lz = z < 2 * kOne ? log1pf((float)(long long)(z - kOne) * 0x1p-43f)
                                  : logf((float)z * 0x1p-43f);
    return (l - top) / temp - lz;
}

// What is kept of a row: values of keys above `key`, and the first `ties` tokens of that key.
struct Cut {
    uint32_t key, ties;
};

template <typename T> struct Row {
    using B = Block<T>;
    const T *p;
    const B *held;     // the slice in shared memory, or null
    int V, shift;      // block j holds the tokens j kN - shift ..
    int b0, b1;        // blocks of this CTA's slice
    int w0, w1;        // of this warp
    __device__ __forceinline__ B from_memory(int j) const {
        B b;
        const int e = j * B::kN - shift;
        if (e >= 0 && e + B::kN <= V)
            b = *reinterpret_cast<const B *>(p + e);
        else
            b.edge(p, e, V);
        b.clean();
        return b;
    }
    __device__ __forceinline__ B block(int j) const { return held ? held[j - b0] : from_memory(j); }
    // f(value) for the warp's values of blocks that have one for which `any` of the largest holds;
    // whole warps call it
    template <class Any, class F> __device__ __forceinline__ void each(Any any, F f) const {
        const int lane = threadIdx.x & 31;
        for (int j0 = w0; j0 < w1; j0 += 32) {
            const int j = j0 + lane;
            const bool in = j < w1;
            B b;
            bool on = false;
            if (in) {
                b = block(j);
                on = any(b.top());
            }
            if (on) {
#pragma unroll
                for (int i = 0; i < B::kN; ++i) f(b.get(i));
            }
        }
    }
};

template <typename T> struct Sampler {
    Shared &sh;
    Row<T> row;
    Scale sc;
    Cut cut;
    cg::cluster_group cl;

    __device__ __forceinline__ u64 weigh(float l) const { return weight(sc, l, sh.powers); }
    // Live and not cut off (ties apart).
    __device__ __forceinline__ bool above(float l) const {
        return is_live(sc, l) && key_of(l) > cut.key;
    }

    __device__ __forceinline__ void clear() {
        for (int i = threadIdx.x; i < kBins; i += kThr) sh.lo[i] = sh.hi[i] = 0;
        __syncthreads();
    }
    template <bool W> __device__ __forceinline__ void add(int bin, float l) {
        if (!W) {
            atomicAdd(&sh.lo[bin], 1u);
            return;
        }
        const u64 w = weigh(l);
        const uint32_t low = (uint32_t)w, old = atomicAdd(&sh.lo[bin], low);
        const uint32_t high = (uint32_t)(w >> 32) + (old + low < old);
        if (high) atomicAdd(&sh.hi[bin], high);
    }
    // The cluster's histograms become their sum.
    __device__ __forceinline__ void share() {
        const int ctas = cl.num_blocks(), rank = cl.block_rank();
        __syncthreads();
        if (ctas == 1) return;
        cl.sync();
        const int per = kBins / ctas;
        for (int i = rank * per + threadIdx.x; i < (rank + 1) * per; i += kThr) {
            u64 v = 0;
            for (int c = 0; c < ctas; ++c) {
                const Shared *o = cl.map_shared_rank(&sh, c);
                v += (u64)o->hi[i] << 32 | o->lo[i];
            }
            for (int c = 0; c < ctas; ++c) {
                Shared *o = cl.map_shared_rank(&sh, c);
                o->lo[i] = (uint32_t)v;
                o->hi[i] = (uint32_t)(v >> 32);
            }
        }
        cl.sync();
    }
    // The bin in which the running sum reaches `target` (> 0): sh.bin, and the sum before it in
    // sh.before. False where it is not reached.
    __device__ __forceinline__ bool find(u64 target) {
        u64 v[kPer], own = 0, total;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int bin = threadIdx.x * kPer + i;
            v[i] = (u64)sh.hi[bin] << 32 | sh.lo[bin];
            own += v[i];
        }
        u64 at = block_scan(own, sh.part, &total);
        if (at < target && target <= at + own) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (at < target && target <= at + v[i]) {
                    sh.bin = threadIdx.x * kPer + i;
                    sh.before = at;
                }
                at += v[i];
            }
        }
        __syncthreads();
        return target <= total;
    }

    // Samples from a list of the row's largest tokens. own: the thread's largest value. False (for the
    // whole cluster) where the list does not hold all that may be kept.
    __device__ __forceinline__ bool from_list(const Args &a, int r, int k, float top_p,
                                              uint32_t low_key, float own, float u, float temp) {
        const int ctas = cl.num_blocks(), rank = cl.block_rank();
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const bool by_p = top_p < 1.f, whole = by_p && !k;  // top-p of the whole row's weight
        int last = kBins - 1;  // bins up to this one are listed
        if (k || !low_key) {
            clear();
            if (is_live(sc, own))
                atomicAdd(&sh.lo[min(kBins - 1, (int)(octaves(sc, own) * kBinScale))], 1u);
            share();
            if (find(k ? k : kGuess)) last = sh.bin;
            __syncthreads();  // (the list takes the bins' place)
        }
        float sum = 0.f;
        auto listed = [&](float l) {
            return is_live(sc, l) && min(kBins - 1, (int)(octaves(sc, l) * kBinScale)) <= last &&
                   (k || key_of(l) >= low_key);
        };
        for (int j0 = row.w0; j0 < row.w1; j0 += 32) {
            const int j = j0 + lane;
            if (j >= row.w1) continue;
            const Block<T> b = row.block(j);
            if (whole) {
                float part = 0.f;
#pragma unroll
                for (int i = 0; i < Block<T>::kN; ++i) part += exp2_approx(-octaves(sc, b.get(i)));
                sum += part;
            }
            if (listed(b.top())) {
#pragma unroll 1
                for (int i = 0; i < Block<T>::kN; ++i) {
                    const float l = b.get(i);
                    if (!listed(l)) continue;
                    const uint32_t at = atomicAdd(&sh.listed, 1u);
                    if (at < kList) {
                        sh.list_key[at] = key_of(l);
                        sh.list_index[at] = j * Block<T>::kN - row.shift + i;
                    }
                }
            }
        }
        if (whole) {
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) sh.red_f[warp] = sum;
            __syncthreads();
            if (threadIdx.x == 0) {
                for (int i = 1; i < kWarps; ++i) sum += sh.red_f[i];
                sh.sum = sum;
            }
        }
        cl.sync();
        int n = 0;
        for (int c = 0; c < ctas; ++c) n += (int)min(cl.map_shared_rank(&sh, c)->listed, kList + 1u);
        if (n > kList) {
            cl.sync();
            return false;
        }
        if (rank == 0) {
            // the lists of all CTAs, sorted
            u64 mine = ~0ull;
            float z_all = 0.f;
            int first = 0;
            for (int c = 0; c < ctas; ++c) {
                const Shared *o = cl.map_shared_rank(&sh, c);
                const int count = (int)o->listed, i = (int)threadIdx.x - first;
                if (i >= 0 && i < count) mine = (u64)~o->list_key[i] << 32 | o->list_index[i];
                first += count;
                if (whole) z_all += o->sum;
            }
            sh.sorted[threadIdx.x] = mine;
            __syncthreads();
            int at = 0;
            if ((int)threadIdx.x < n) {
#pragma unroll 4
                for (int i = 0; i < n; ++i) at += sh.sorted[i] < mine;
            }
            __syncthreads();
            if ((int)threadIdx.x < n) sh.sorted[at] = mine;
            __syncthreads();
            // token i of the order, its weight and that of those before it
            const int i = threadIdx.x;
            mine = i < n ? sh.sorted[i] : 0;
            const float l = value_of(~(uint32_t)(mine >> 32));
            const u64 w = i < n && (!k || i < k) ? weigh(l) : 0;
            u64 all;
            const u64 before = block_scan(w, sh.part, &all);
            bool kept = w > 0 && ~(uint32_t)(mine >> 32) >= low_key, sure = true;
            if (by_p) {
                if (whole) {
                    const double t = (double)top_p * (double)z_all * 0x1p43;
                    const double lo = t * (1.0 - (double)kSumError), hi = t * (1.0 + (double)kSumError);
                    // every border is on one side, and the last kept one is listed
                    sure = i == 0 || !kept || (double)before < lo || (double)before >= hi;
                    if (!low_key && (double)all < hi) sure = false;
                    kept = kept && (i == 0 || (double)before < t);
                } else {
                    const double t = (double)top_p * (double)all;
                    kept = kept && (i == 0 || before < (u64)ceil(t));
                }
            }
            const int keep = __syncthreads_count(kept);
            const bool fine = __syncthreads_and(sure);
            if (threadIdx.x == 0) sh.settled = fine;
            if (fine) {
                // in the order of the tokens
                u64 z, *weights = reinterpret_cast<u64 *>(sh.list_key);  // (the list has been read)
                weights[i] = w;
                block_scan(kept ? w : 0, sh.part, &z);
                if (kept) {
                    u64 at = 0;
#pragma unroll 4
                    for (int q = 0; q < keep; ++q)
                        if ((uint32_t)sh.sorted[q] < (uint32_t)mine) at += weights[q];
                    const double x = (double)u * (double)z;
                    const u64 target = min(z - 1, x > 0.0 ? (u64)x : 0ull);
                    if (at <= target && target < at + w) {
                        a.token[r] = (int)(uint32_t)mine;
                        if (a.logprob) a.logprob[r] = log_share(l, sc.top, temp, z);
                    }
                }
            }
        }
        cl.sync();
        const bool settled = cl.map_shared_rank(&sh, 0)->settled;
        cl.sync();
        return settled;
    }

    // The cut at which the running count (W: weight) of the values above cut.key reaches `target`
    // (> 0). False where it is not reached: nothing changes then. target_of gets the sum of all (W).
    template <bool W, class Target>
    __device__ __forceinline__ bool search(Target target_of) {
        clear();
        row.each([&](float m) { return above(m); }, [&](float l) {
            if (above(l)) add<W>(min(kBins - 1, (int)(octaves(sc, l) * kBinScale)), l);
        });
        share();
        u64 sum = 0;
        if (W) {  // the target depends on the sum
            u64 own = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int bin = threadIdx.x * kPer + i;
                own += (u64)sh.hi[bin] << 32 | sh.lo[bin];
            }
            block_scan(own, sh.part, &sum);
        }
        u64 target = target_of(sum);
        if (!find(target)) return false;
        const int first = sh.bin;
        target -= sh.before;
        // the keys that occur in the bin
        uint32_t kmin = 0xffffffffu, kmax = 0;
        row.each([&](float m) { return above(m); }, [&](float l) {
            if (above(l) && min(kBins - 1, (int)(octaves(sc, l) * kBinScale)) == first) {
                kmin = min(kmin, key_of(l));
                kmax = max(kmax, key_of(l));
            }
        });
        kmin = __reduce_min_sync(0xffffffffu, kmin);
        kmax = __reduce_max_sync(0xffffffffu, kmax);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) {
            sh.red_a[threadIdx.x >> 5] = kmin;
            sh.red_b[threadIdx.x >> 5] = kmax;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 0; i < kWarps; ++i) {
                kmin = min(kmin, sh.red_a[i]);
                kmax = max(kmax, sh.red_b[i]);
            }
            sh.kmin = kmin;
            sh.kmax = kmax;
        }
        cl.sync();
        for (int c = 0; c < (int)cl.num_blocks(); ++c) {
            const Shared *o = cl.map_shared_rank(&sh, c);
            kmin = min(kmin, o->kmin);
            kmax = max(kmax, o->kmax);
        }
        cl.sync();
        while (kmin < kmax) {
            const int shift = max(0, 32 - __clz(kmax - kmin) - 10);
            clear();
            row.each([&](float m) { return key_of(m) >= kmin; }, [&](float l) {
                const uint32_t key = key_of(l);
                if (key >= kmin && key <= kmax) add<W>((int)((kmax - key) >> shift), l);
            });
            share();
            find(target);
            target -= sh.before;
            kmax -= (uint32_t)sh.bin << shift;
            const uint32_t width = (1u << shift) - 1;
            if (kmax - kmin > width) kmin = kmax - width;
            if (shift == 0) break;
        }
        cut.key = kmax;
        // ties that are needed to reach the target
        if (W) {
            const u64 w = weigh(value_of(kmax));
            cut.ties = w ? (uint32_t)((target + w - 1) / w) : 1u;
        } else {
            cut.ties = (uint32_t)target;
        }
        return true;
    }
};

template <typename T>
__global__ void __launch_bounds__(kThr, 2) sample_kernel(const Args a, int held_blocks) {
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ __align__(16) Shared sh;
    using B = Block<T>;
    cg::cluster_group cl = cg::this_cluster();
    const int ctas = cl.num_blocks(), rank = cl.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = blockIdx.x / ctas;
    for (int i = threadIdx.x; i < 256; i += kThr)
        sh.powers[i] = make_float2(kPowers.hi[i], kPowers.lo[i]);
    pdl_wait();
    const int g = r / a.group;
    // (beyond these the weights are those of the largest alone, or equal)
    float temp = a.temperature ? a.temperature[g] : 1.f;
    if (temp > 0.f) temp = fminf(fmaxf(temp, 1e-30f), 1e30f);
    const int k = a.top_k ? a.top_k[g] : 0;
    const float top_p = a.top_p ? a.top_p[g] : 1.f, min_p = a.min_p ? a.min_p[g] : 0.f;
    const float u = a.u[r];

    Sampler<T> s{sh, {}, {}, {0, 0}, cl};
    Row<T> &row = s.row;
    row.p = reinterpret_cast<const T *>(a.logits) + (size_t)r * a.ld;
    row.V = a.V;
    row.shift = (int)(((uintptr_t)row.p / sizeof(T)) % B::kN);
    const int blocks = (a.V + row.shift + B::kN - 1) / B::kN, per = (blocks + ctas - 1) / ctas;
    row.b0 = min(blocks, rank * per);
    row.b1 = min(blocks, row.b0 + per);
    row.held = nullptr;
    const int wper = ((row.b1 - row.b0 + kWarps - 1) / kWarps + 31) / 32 * 32;
    row.w0 = min(row.b1, row.b0 + warp * wper);
    row.w1 = min(row.b1, row.w0 + wper);

    // the row's slice, and the largest value
    B *held = reinterpret_cast<B *>(dyn);
    const bool keep = per <= held_blocks;
    float top = -INFINITY;
#pragma unroll 4
    for (int j = row.w0 + lane; j < row.w1; j += 32) {
        const B b = row.from_memory(j);
        if (keep) held[j - row.b0] = b;
        top = fmaxf(top, b.top());
    }
    if (keep) row.held = held;
    const float own = top;  // the thread's largest
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) sh.red_f[warp] = top;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) top = fmaxf(top, sh.red_f[i]);
    if (threadIdx.x == 0) {
        sh.top = top;
        sh.index = 0xffffffffu;
        sh.owner = -1;
        sh.listed = 0;
    }
    cl.sync();
    for (int c = 0; c < ctas; ++c) top = fmaxf(top, cl.map_shared_rank(&sh, c)->top);

    if (top == -INFINITY) {  // nothing to sample from
        if (rank == 0 && threadIdx.x == 0) {
            a.token[r] = -1;
            if (a.logprob) a.logprob[r] = -INFINITY;
        }
        cl.sync();
        return;
    }
    if (!(temp > 0.f)) {  // the first of the largest
        for (int j = row.w0 + lane; j < row.w1; j += 32) {
            const B b = row.block(j);
            if (b.top() < top) continue;
            int first = 0;
            for (int i = B::kN - 1; i >= 0; --i)
                if (b.get(i) == top) first = i;
            atomicMin(&sh.index, (uint32_t)(j * B::kN - row.shift + first));
            break;
        }
        cl.sync();
        if (rank == 0 && threadIdx.x == 0) {
            uint32_t first = 0xffffffffu;
            for (int c = 0; c < ctas; ++c) first = min(first, cl.map_shared_rank(&sh, c)->index);
            a.token[r] = (int)first;
            if (a.logprob) a.logprob[r] = 0.f;
        }
        cl.sync();
        return;
    }

    const double c = 1.4426950408889634074 / (double)temp;
    s.sc.top = top;
    s.sc.ch = (float)c;
    s.sc.cl = (float)(c - (double)s.sc.ch);
    const bool by_k = k > 0 && k < a.V, by_p = top_p < 1.f, by_m = min_p > 0.f;
    if (by_m) {
        if (threadIdx.x == 0)
            sh.low = __double2float_ru((double)top + (double)temp * log((double)fminf(min_p, 1.f)));
        __syncthreads();
    }
    const uint32_t low_key = by_m ? key_of(sh.low + 0.f) : 0;
    if ((by_k && k <= kListK) || (!by_k && (by_m || by_p))) {
        const bool done = s.from_list(a, r, by_k ? k : 0, top_p, low_key, own, u, temp);
        if (done) return;
    }
    if (by_k) s.template search<false>([&](u64) { return (u64)k; });
    if (by_p) {
        const u64 w_tie = s.cut.ties ? s.weigh(value_of(s.cut.key)) : 0;
        u64 all = 0, target = 0;
        auto goal = [&](u64 above) {
            all = above;
            const double t = (double)top_p * (double)(above + w_tie * s.cut.ties);
            target = t >= 1.0 ? (u64)ceil(t) : 1;
            return target;
        };
        const Cut before = s.cut;
        if (!s.template search<true>(goal)) {  // the cut lies among the ties of top-k's
            if (before.ties && w_tie)
                s.cut.ties = min(before.ties, (uint32_t)((target - all + w_tie - 1) / w_tie));
        }
    }
    if (by_m && low_key - 1 >= s.cut.key) s.cut = Cut{low_key - 1, 0};

    // weights and ties of every warp, in the order of the tokens
    const u64 w_tie = s.cut.ties ? s.weigh(value_of(s.cut.key)) : 0;
    const Cut cut = s.cut;
    u64 sum = 0;
    uint32_t ties = 0;
    row.each([&](float m) { return is_live(s.sc, m) && key_of(m) >= cut.key; }, [&](float l) {
        if (!is_live(s.sc, l)) return;
        const uint32_t key = key_of(l);
        if (key > cut.key) sum += s.weigh(l);
        ties += key == cut.key;
    });
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    ties = __reduce_add_sync(0xffffffffu, ties);
    if (lane == 0) {
        sh.wsum[warp] = sum;
        sh.ties[warp] = ties;
    }
    cl.sync();
    {
        u64 w = 0, t = 0, all_w, all_t;
        if (threadIdx.x < kWarps * ctas) {
            const Shared *o = cl.map_shared_rank(&sh, threadIdx.x / kWarps);
            w = o->wsum[threadIdx.x % kWarps];
            t = o->ties[threadIdx.x % kWarps];
        }
        const u64 w0 = block_scan(w, sh.part, &all_w), t0 = block_scan(t, sh.part, &all_t);
        auto total = [&](u64 w, u64 t) { return w + w_tie * min(t, (u64)cut.ties); };
        const u64 z = total(all_w, all_t);
        const double x = (double)u * (double)z;
        const u64 target = min(z - 1, x > 0.0 ? (u64)x : 0ull);
        if (threadIdx.x < kWarps * ctas && total(w0, t0) <= target && target < total(w0 + w, t0 + t)) {
            sh.owner = threadIdx.x;
            sh.own_w = w0;
            sh.own_t = (uint32_t)t0;
            sh.target = target;
            sh.z = z;
        }
        __syncthreads();
    }
    if (sh.owner == rank * kWarps + warp) {
        const u64 target = sh.target;
        u64 w_at = sh.own_w, t_at = sh.own_t;
        auto total = [&](u64 w, u64 t) { return w + w_tie * min(t, (u64)cut.ties); };
        for (int j0 = row.w0; j0 < row.w1; j0 += 32) {
            const int j = j0 + lane;
            B b;
            u64 w = 0, t = 0;
            auto one = [&](float l, u64 &w, u64 &t) {
                if (!is_live(s.sc, l)) return;
                const uint32_t key = key_of(l);
                if (key > cut.key) w += s.weigh(l);
                t += key == cut.key;
            };
            if (j < row.w1) {
                b = row.block(j);
#pragma unroll
                for (int i = 0; i < B::kN; ++i) one(b.get(i), w, t);
            }
            u64 ws = w, ts = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 x = __shfl_up_sync(0xffffffffu, ws, o), y = __shfl_up_sync(0xffffffffu, ts, o);
                if (lane >= o) {
                    ws += x;
                    ts += y;
                }
            }
            const bool here = target < total(w_at + ws, t_at + ts);
            const uint32_t m = __ballot_sync(0xffffffffu, here);
            if (m) {
                if (lane == __ffs(m) - 1) {
                    w = w_at + ws - w;
                    t = t_at + ts - t;
                    for (int i = 0; i < B::kN; ++i) {
                        const float l = b.get(i);
                        one(l, w, t);
                        if (target < total(w, t)) {
                            a.token[r] = j * B::kN - row.shift + i;
                            if (a.logprob) a.logprob[r] = log_share(l, top, temp, sh.z);
                            break;
                        }
                    }
                }
                break;
            }
            w_at += __shfl_sync(0xffffffffu, ws, 31);
            t_at += __shfl_sync(0xffffffffu, ts, 31);
        }
    }
    cl.sync();  // (shared memory of CTAs that have ended is not to be read)
}

constexpr int kHeldBytes = 76 * 1024;  // of a row in a CTA: two CTAs share an SM

template <typename T> cudaError_t launch(const Args &a, cudaStream_t s) {
    const int blocks = (a.V + 2 * Block<T>::kN - 2) / Block<T>::kN;
    const int room = kHeldBytes / 16, sms = std::max(1, device_sms());
    // the CTAs that hold a row; more of them for few rows
    int ctas = 1;
    while (ctas < kMaxCluster && (blocks + ctas - 1) / ctas > room) ctas *= 2;
    while (ctas < kMaxCluster && (long long)a.R * ctas * 2 <= sms && blocks / ctas > 2 * kThr) ctas *= 2;
    const int per = (blocks + ctas - 1) / ctas;
    const int held = per <= room ? per : 0;
    cudaError_t err = allow_smem(sample_kernel<T>, kHeldBytes);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.R * ctas);
    cfg.blockDim = dim3(kThr);
    cfg.dynamicSmemBytes = (size_t)held * 16;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a, held);
}

}  // namespace

cudaError_t launch_sample(const Args &a, int dtype, cudaStream_t s) {
    return dtype == MOE_DTYPE_F32 ? launch<float>(a, s) : launch<__nv_bfloat16>(a, s);
}

}  // namespace sample
}  // namespace moe
