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
// polynomial carried as pairs of fp32 values; off by 1.3 units at most, checked against 64 bits),
// and sums are 64-bit integers: exact, and the same in any order.
//
// A row belongs to a CTA, or, where rows are few, to a cluster of CTAs that hold it in shared memory;
// else it is read again from L2.
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
//
// Measured for bf16 rows of 151936 with top-k 20 and top-p 0.9: one row 13.4 us (bound by the cluster's
// barriers), 1040 rows 85 (48 of it the HBM's; two CTAs an SM, and a row takes 8 to read and then 9 for its
// list); 192 rows of fp32 50257, a third of them without top-k, 75 to 80 (bound by the instructions of
// exact weights, and by the slowest rows).
#include <cooperative_groups.h>

#include <cfloat>

#include "sample.cuh"
#include "sample_keys.cuh"

namespace moe {
namespace sample {
namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kThr = 512, kWarps = kThr / 32;
constexpr int kBins = kRangeBins, kPer = kBins / kThr;
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

// The weights of two live values in units of 2^-43, two to an instruction. The difference and its product
// with log2(e) / T are carried as two fp32 values; 2^-x is a table's 2^(-k/256) times e^q, |q| <= 2^-9 ln 2
// and a little; the parts are turned into integers at 2^22 and 2^43. Bound by the fp32 pipe (40
// instructions), so what can be had negated or with an addend in one step is.
__device__ __forceinline__ void weight2(const Scale &s, float l0, float l1, const float2 *powers, u64 &w0,
                                        u64 &w1) {
    constexpr float kBig = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
    constexpr double kLn2 = 0.69314718055994530942;
    constexpr float lh = (float)kLn2, ll = (float)(kLn2 - (double)lh);
    auto both = [](float v) { return pack2(v, v); };
    const uint64_t minus = both(-1.f), l = pack2(l0, l1), top = both(s.top), ch = both(s.ch);
    const uint64_t d = fma2(l, minus, top), bb = add2(d, both(-s.top));
    const uint64_t e = fma2(add2(l, bb), minus, fma2(fma2(bb, minus, d), minus, top));
    const uint64_t p = mul2(d, both(-s.ch));  // -x
    const uint64_t pe = add2(fma2(d, ch, p), fma2(d, both(s.cl), mul2(e, ch)));
    const uint64_t kb = fma2(p, both(-256.f), both(kBig));
    const uint64_t r = fma2(add2(kb, both(-kBig)), both(1.f / 256.f), p);  // exact
    const uint64_t q = mul2(r, both(lh));
    const uint64_t ql = fma2(r, both(ll), fma2(pe, both(-lh), fma2(r, both(lh), mul2(r, both(-lh)))));
    const uint64_t poly = fma2(q, fma2(q, both(1.f / 24.f), both(1.f / 6.f)), both(0.5f));
    const uint64_t more = fma2(mul2(q, q), poly, fma2(ql, q, ql));
    const uint64_t eh = add2(q, more), el = fma2(fma2(q, minus, eh), minus, more);
    const float2 kf = unpack2(kb);
    const int k0 = __float_as_int(kf.x) - 0x4b400000, k1 = __float_as_int(kf.y) - 0x4b400000;
    const float2 t0 = powers[k0 & 255], t1 = powers[k1 & 255];
    // 2^(22 - (k >> 8))
    const uint64_t sc = pack2(__int_as_float((k0 & ~255) * -32768 + (149 << 23)),
                              __int_as_float((k1 & ~255) * -32768 + (149 << 23)));
    const uint64_t a = mul2(pack2(t0.x, t1.x), sc), al = mul2(pack2(t0.y, t1.y), sc);
    // a and a eh: their integers, and what is left of them (of a eh up to 2^-26)
    const uint64_t ai = add2(a, both(8388608.f)), bi = fma2(a, eh, both(kBig));
    const uint64_t ra = add2(a, fma2(ai, minus, both(8388608.f))), rb = fma2(a, eh, fma2(bi, minus, both(kBig)));
    const uint64_t rest = add2(add2(ra, rb), fma2(a, el, fma2(al, q, al)));
    const float2 af = unpack2(ai), bf = unpack2(bi), lo = unpack2(fma2(rest, both(2097152.f), both(kBig)));
    const int h0 = (__float_as_int(af.x) - 0x4b000000) + (__float_as_int(bf.x) - 0x4b400000);
    const int h1 = (__float_as_int(af.y) - 0x4b000000) + (__float_as_int(bf.y) - 0x4b400000);
    w0 = (u64)((long long)h0 * (1 << 21) + (__float_as_int(lo.x) - 0x4b400000));
    w1 = (u64)((long long)h1 * (1 << 21) + (__float_as_int(lo.y) - 0x4b400000));
}
// One of them: the same steps, so the same weight (0 where the value is not live).
__device__ __forceinline__ u64 weight(const Scale &s, float l, const float2 *powers) {
    u64 w, other;
    weight2(s, l, s.top, powers, w, other);
    return (long long)w > 0 ? w : 0;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T> __device__ __forceinline__ T from_value(float v);
template <> __device__ __forceinline__ float from_value(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_value(float v) { return __float2bfloat16(v); }

// A 16-byte block of a row.
template <typename T> struct Block;
template <> struct Block<float> {
    static constexpr int kN = 4;
    float4 v;
    __device__ __forceinline__ float get(int i) const {
        return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    }
    // the first value; the others move up
    __device__ __forceinline__ float take() {
        const float f = v.x;
        v.x = v.y;
        v.y = v.z;
        v.z = v.w;
        return f;
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
    // (by value: what a call gets the address of lives in memory)
    __device__ __noinline__ static uint4 edge(const float *p, int e, int V) {
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = e + i >= 0 && e + i < V ? p[e + i] : -INFINITY;
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
};
template <> struct Block<__nv_bfloat16> {
    static constexpr int kN = 8;
    uint4 v;
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
        return i & 1 ? bf16_hi(w) : bf16_lo(w);
    }
    __device__ __forceinline__ float take() {
        const float f = bf16_lo(v.x);
        v.x = __funnelshift_r(v.x, v.y, 16);
        v.y = __funnelshift_r(v.y, v.z, 16);
        v.z = __funnelshift_r(v.z, v.w, 16);
        v.w >>= 16;
        return f;
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
    __device__ __noinline__ static uint4 edge(const __nv_bfloat16 *p, int e, int V) {
        uint32_t x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = e + i >= 0 && e + i < V ? __bfloat16_as_ushort(p[e + i]) : 0xff80u;
        return make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
    }
};

constexpr int kList = kThr;             // tokens of a list, a thread for each
constexpr int kAsk = kList / 2;        // of them asked for (the last bin may hold more)
constexpr float kFar = 36.f;           // octaves from which values do not count in the fp32 sum
// The fp32 sum's relative error, whichever pass forms it. A term meets at most 282 additions (256 blocks of a
// thread that has 2^19 values alone with its CTA, a block's values, 24 of threads, warps and CTAs), 2^-24 each:
// 1.7 10^-5. Blocks of kFar octaves and more are left out: kMaxV 2^-36, 7.6 10^-6. Octaves have three roundings,
// and their mean over the weights is below 15 (V values x octaves down beside the largest: x V 2^-x / (1 + V 2^-x)):
// 1.9 10^-6, exp2 2.4 10^-7. 2.7 10^-5 < 2^-15. The sum made while a row is read has 106 additions at most (76 KB
// of blocks' largest values), but scales its terms three times more (what is scaled more often is too little), over
// 16 octaves more: 6.5 + 7.6 + 3.8 + 1 = 18.9 10^-6.
constexpr float kSumError = 0x1p-15f;

// A row, its settings, and where its results go.
struct Task {
    const void *inner, *low, *high;  // blocks (see Row)
    int blocks, shift;               // block j holds the tokens j kN - shift ..
    int b0, b1, per;                 // of this CTA's slice, and of a warp
    const void *tops;                // the blocks' largest values in shared memory, or null
    bool raw;
    float temp, top_p, u;
    int k;                 // 0: all
    uint32_t low_key;      // of min-p, or 0
    int *token;
    float *logprob;
};

// What is kept of a row: values of keys above `key`, and the first `ties` tokens of that key.
struct Cut {
    uint32_t key, ties;
};

struct Shared {
    Task task;
    Cut cut;
    u64 goal;      // what a search looks for
    float live;    // the least live value
    double below;  // how far min-p's least value lies from the largest (-inf: not asked for)
    u64 limit, limit_lo, limit_hi;
    uint4 ends[2];
    float2 powers[256];
    alignas(16) uint32_t lo[kBins];
    uint32_t hi[kBins];
    u64 list[kList];  // ~key, index: ascending
    u64 part[kWarps], scanned;
    Scale sc;
    // what a pass found, by warp
    float sums[kWarps];
    int ends_of[kMaxCluster];  // the lists', one after the other
    // read by the other CTAs of the cluster
    u64 wsum[kWarps];
    uint32_t ties[kWarps];
    float top, sum;
    uint32_t index;
    int listed, settled;
    // found by one thread
    int bin, owner;
    uint32_t edges[2];
    u64 before, own_w, target, z;
    uint32_t own_t;
    u64 part_w[kWarps], part_t[kWarps];
    int part_owner;
};

// A barrier of the row's CTAs. (A cluster's costs more than a CTA's even where it has one CTA.)
__device__ __forceinline__ void row_sync() {
    cg::cluster_group cl = cg::this_cluster();
    if (cl.num_blocks() > 1)
        cl.sync();
    else
        __syncthreads();
}

// Sum of the block's threads before this one, in their order; of all: sh.scanned. (What is used in
// several places is called: code that a row runs through once waits for its instructions.)
__device__ __noinline__ u64 block_scan(Shared &sh, u64 v) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 s = v;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const u64 t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
    }
    __syncthreads();
    if (lane == 31) sh.part[warp] = s;
    __syncthreads();
    if (warp == 0) {
        const u64 own = lane < kWarps ? sh.part[lane] : 0;
        u64 t = own;
#pragma unroll 1
        for (int o = 1; o < kWarps; o <<= 1) {
            const u64 x = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += x;
        }
        if (lane < kWarps) sh.part[lane] = t - own;
        if (lane == kWarps - 1) sh.scanned = t;
    }
    __syncthreads();
    return sh.part[warp] + s - v;
}

__device__ __noinline__ u64 weigh(const Shared &sh, float l) { return weight(sh.sc, l, sh.powers); }

__device__ __forceinline__ int bin_of(const Scale &sc, float l) {
    return min(kBins - 1, (int)(octaves(sc, l) * kBinScale));
}

// log of the share that a token of logit l has of the sum z, in fp32: off by a few steps (measured over mixed rows:
// 1.25 to 2 times the error of rounding the exact one). In fp64 one row's call took 13.4 -> 14.8 us and 16 trees of 65
// 96 -> 101; with what each step loses carried along 13.4 -> 13.75 for 1.1 times that error.
__device__ __noinline__ float log_share(float l, float top, float temp, u64 z) {
    const float lz = z < 2 * kOne ? log1pf((float)(long long)(z - kOne) * 0x1p-43f)
                                  : logf((float)z * 0x1p-43f);
    return (l - top) / temp - lz;
}

template <typename T> struct Row {
    using B = Block<T>;
    const B *inner;     // block j lies at inner + j, in memory or in shared memory
    const B *low, *high;  // (the first and the last one elsewhere, as they reach past the row)
    int high_j;
    int shift;          // block j holds the tokens j kN - shift ..
    int w0, w1;         // the warp's blocks
    bool raw;           // not cleaned
    __device__ __forceinline__ explicit Row(const Task &t) {
        inner = reinterpret_cast<const B *>(t.inner);
        low = reinterpret_cast<const B *>(t.low);
        high = reinterpret_cast<const B *>(t.high);
        high_j = t.blocks - 1;
        shift = t.shift;
        raw = t.raw;
        w0 = min(t.b1, t.b0 + (int)(threadIdx.x >> 5) * t.per);
        w1 = min(t.b1, w0 + t.per);
    }
    __device__ __forceinline__ const B *at(int j) const {
        const B *p = inner + j;
        p = j == 0 ? low : p;
        return j == high_j ? high : p;
    }
    // f(block, its number) for the warp's blocks, kDeep of them on their way at a time (the loads are
    // not conditional, so that none waits for another)
    template <int kDeep, class F> __device__ __forceinline__ void blocks(F f) const {
        const int lane = threadIdx.x & 31;
#pragma unroll 1
        for (int j0 = w0 + lane; j0 < w1; j0 += 32 * kDeep) {
            B b[kDeep];
#pragma unroll
            for (int q = 0; q < kDeep; ++q) b[q] = *at(min(j0 + 32 * q, w1 - 1));
            if (raw) {
#pragma unroll
                for (int q = 0; q < kDeep; ++q) b[q].clean();
            }
            f(b, j0, min(kDeep, (w1 - j0 + 31) / 32));
        }
    }
    __device__ __forceinline__ B block(int j) const {
        B b = *at(j);
        b.clean();
        return b;
    }
};

// What a pass over a row's slice does with its live values whose keys lie in lo .. hi:
enum : int {
    kCounts,       // counts them in bins by octave
    kCountKeys,    // counts them in bins (hi - key) >> arg
    kWeights,      // adds their weights in bins by octave
    kWeightKeys,   // adds their weights in bins (hi - key) >> arg
    kTake,         // appends those from lo on to the list
    kTakeAndSum,   // the same, and the fp32 sum of all weights
    kFinal         // the weight of those above lo, and how many are lo's
};

template <typename T, int kMode>
__device__ __noinline__ void pass(Shared &sh, uint32_t lo, uint32_t hi, int arg) {
    using B = Block<T>;
    const Row<T> row(sh.task);
    const Scale sc = sh.sc;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 wsum = 0;
    uint32_t ties = 0;
    float sum = 0.f;
    constexpr bool kTakes = kMode == kTake || kMode == kTakeAndSum;
    constexpr int kDeep = 8;
    // (keys below the least value's and above the largest's stand for no value)
    float least = lo > key_of(-INFINITY) ? value_of(lo) : -INFINITY;
    const float most = hi < key_of(INFINITY) ? value_of(hi) : INFINITY, cut = least;
    if (!kTakes) least = fmaxf(least, sh.live);
    if constexpr (kTakes) {
        row.template blocks<kDeep>([&](const auto &b, int j0, int n) {
            uint32_t todo = 0;  // blocks that hold a value to look at
#pragma unroll
            for (int q = 0; q < kDeep; ++q) {
                const float m = b[q].top();
                if (q >= n) continue;
                if (kMode == kTakeAndSum && octaves(sc, m) < kFar) {
                    float part = 0.f;
#pragma unroll
                    for (int i = 0; i < B::kN; ++i) part += exp2_approx(-octaves(sc, b[q].get(i)));
                    sum += part;
                }
                if (m >= least) todo |= 1u << q;
            }
#pragma unroll 1
            while (todo) {
                const int at_q = __ffs(todo) - 1;
                todo &= todo - 1;
                B one = b[0];
#pragma unroll
                for (int q = 1; q < kDeep; ++q)
                    if (at_q == q) one = b[q];
                uint32_t hits = 0;
#pragma unroll
                for (int i = 0; i < B::kN; ++i) hits |= one.get(i) >= least && one.get(i) <= most ? 1u << i : 0;
                int at = atomicAdd(&sh.listed, __popc(hits));
                const int token = (j0 + 32 * at_q) * B::kN - row.shift;
#pragma unroll 1
                for (int i = 0; hits; ++i, hits >>= 1) {
                    const float l = one.take();
                    if (!(hits & 1)) continue;
                    if (at < kList) sh.list[at] = (u64)~key_of(l) << 32 | (uint32_t)(token + i);
                    ++at;
                }
            }
        });
    } else {
        // blocks by their largest values, where these are at hand; the next one is on its way meanwhile
        constexpr int kMany = 16;
        const T *tops = reinterpret_cast<const T *>(sh.task.tops);
        const int b0 = sh.task.b0;
#pragma unroll 1
        for (int j0 = row.w0 + lane; j0 < row.w1; j0 += 32 * kMany) {
            uint32_t todo = 0;
#pragma unroll 4
            for (int q = 0; q < kMany; ++q) {
                const int j = j0 + 32 * q;
                if (j < row.w1 && (!tops || (float)tops[j - b0] >= least)) todo |= 1u << q;
            }
            B next;
            if (todo) next = *row.at(j0 + 32 * (__ffs(todo) - 1));
#pragma unroll 1
            while (todo) {
                B one = next;
                todo &= todo - 1;
                if (todo) next = *row.at(j0 + 32 * (__ffs(todo) - 1));
                if (row.raw) one.clean();
                uint32_t hits = 0;
#pragma unroll
                for (int i = 0; i < B::kN; ++i) hits |= one.get(i) >= least && one.get(i) <= most ? 1u << i : 0;
                if constexpr (kMode == kCounts || kMode == kCountKeys) {
#pragma unroll
                    for (int i = 0; i < B::kN; ++i) {
                        const float l = one.get(i);
                        if (hits >> i & 1)
                            atomicAdd(&sh.lo[kMode == kCounts ? bin_of(sc, l) : (int)((hi - key_of(l)) >> arg)], 1u);
                    }
                } else {
                    // (four at a time without a branch: each weight is a chain of some 25 steps)
#pragma unroll
                    for (int i = 0; i < B::kN; i += 4) {
                        if (!(hits >> i & 15)) continue;
                        u64 w[4];
                        weight2(sc, one.get(i), one.get(i + 1), sh.powers, w[0], w[1]);
                        weight2(sc, one.get(i + 2), one.get(i + 3), sh.powers, w[2], w[3]);
#pragma unroll
                        for (int o = 0; o < 4; ++o) {
                            const float l = one.get(i + o);
                            const bool on = hits >> (i + o) & 1;
                            if constexpr (kMode == kFinal) {
                                wsum += on && l > cut ? w[o] : 0;
                                ties += on && l == cut;
                            } else {
                                if (!on) continue;
                                const int bin = kMode == kWeightKeys ? (int)((hi - key_of(l)) >> arg) : bin_of(sc, l);
                                const uint32_t low = (uint32_t)w[o], old = atomicAdd(&sh.lo[bin], low);
                                const uint32_t high = (uint32_t)(w[o] >> 32) + (old + low < old);
                                if (high) atomicAdd(&sh.hi[bin], high);
                            }
                        }
                    }
                }
            }
        }
    }
    __syncwarp();
    if (kMode == kTakeAndSum) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) sh.sums[warp] = sum;
    }
    if (kMode == kFinal) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, o);
        ties = __reduce_add_sync(0xffffffffu, ties);
        if (lane == 0) {
            sh.wsum[warp] = wsum;
            sh.ties[warp] = ties;
        }
    }
    __syncthreads();
}

// Appends the values from lo on to the list: the blocks that have one are found by their largest values.
template <typename T> __device__ __noinline__ void take(Shared &sh, uint32_t lo) {
    using B = Block<T>;
    const Row<T> row(sh.task);
    const B *tops = reinterpret_cast<const B *>(sh.task.tops);
    const int b0 = sh.task.b0, n = (sh.task.b1 - b0 + B::kN - 1) / B::kN;
    const float least = value_of(lo);
#pragma unroll 1
    for (int i = threadIdx.x; i < n; i += kThr) {
        const B v = tops[i];
        uint32_t todo = 0;
#pragma unroll
        for (int q = 0; q < B::kN; ++q) todo |= v.get(q) >= least ? 1u << q : 0;
#pragma unroll 1
        for (; todo; todo &= todo - 1) {
            const int j = b0 + i * B::kN + __ffs(todo) - 1;
            B b = row.block(j);
            uint32_t hits = 0;
#pragma unroll
            for (int q = 0; q < B::kN; ++q) hits |= b.get(q) >= least ? 1u << q : 0;
            int at = atomicAdd(&sh.listed, __popc(hits));
            const int token = j * B::kN - row.shift;
#pragma unroll 1
            for (int q = 0; hits; ++q, hits >>= 1) {
                const float l = b.take();
                if (!(hits & 1)) continue;
                if (at < kList) sh.list[at] = (u64)~key_of(l) << 32 | (uint32_t)(token + q);
                ++at;
            }
        }
    }
    __syncthreads();
}

__device__ __forceinline__ void clear_bins(Shared &sh) {
    for (int i = threadIdx.x; i < kBins; i += kThr) sh.lo[i] = sh.hi[i] = 0;
    __syncthreads();
}

// The cluster's histograms become their sum.
__device__ __noinline__ void share_bins(Shared &sh) {
    cg::cluster_group cl = cg::this_cluster();
    const int ctas = cl.num_blocks(), rank = cl.block_rank();
    __syncthreads();
    if (ctas == 1) return;
    row_sync();
    const int per = kBins / ctas;
    for (int i = rank * per + threadIdx.x; i < (rank + 1) * per; i += kThr) {
        u64 v = 0;
#pragma unroll 4
        for (int c = 0; c < ctas; ++c) {
            const Shared *o = cl.map_shared_rank(&sh, c);
            v += (u64)o->hi[i] << 32 | o->lo[i];
        }
#pragma unroll 4
        for (int c = 0; c < ctas; ++c) {
            Shared *o = cl.map_shared_rank(&sh, c);
            o->lo[i] = (uint32_t)v;
            o->hi[i] = (uint32_t)(v >> 32);
        }
    }
    row_sync();
}

// The bin in which the running sum reaches `target` (> 0): sh.bin, and the sum before it in sh.before;
// sh.scanned: that of all. False where it is not reached.
__device__ __noinline__ bool find_bin(Shared &sh, u64 target) {
    u64 own = 0;
    const int bin0 = threadIdx.x * kPer;
#pragma unroll
    for (int i = 0; i < kPer; ++i) own += (u64)sh.hi[bin0 + i] << 32 | sh.lo[bin0 + i];
    u64 at = block_scan(sh, own);
    if (at < target && target <= at + own) {
        for (int i = 0; i < kPer; ++i) {
            const u64 v = (u64)sh.hi[bin0 + i] << 32 | sh.lo[bin0 + i];
            if (at < target && target <= at + v) {
                sh.bin = bin0 + i;
                sh.before = at;
            }
            at += v;
        }
    }
    __syncthreads();
    return target <= sh.scanned;
}

// The least key whose value is live and in bin b or one before it: bins descend with the value, so 32
// lanes divide what is left by 33 at a time.
__device__ __noinline__ uint32_t bin_edge(const Scale &sc, int b) {
    const int lane = threadIdx.x & 31;
    auto in = [&](uint32_t key) {
        const float l = value_of(key);
        return is_live(sc, l) && bin_of(sc, l) <= b;
    };
    uint32_t out = key_of(-FLT_MAX) - 1, at = key_of(sc.top);  // (out: not in)
    while (at - out > 1) {
        const uint32_t step = max(1u, (at - out) / 33);
        const uint32_t key = min(at, out + step * (lane + 1));
        const uint32_t m = __ballot_sync(0xffffffffu, in(key));
        const int first = m ? __ffs(m) - 1 : 32;
        const uint32_t from = out;
        if (first < 32) at = min(at, from + step * (first + 1));
        if (first > 0) out = min(at - 1, from + step * first);
    }
    return at;
}

// The least live value, for the passes that weigh or count.
__device__ __forceinline__ void set_live(Shared &sh) {
    if (threadIdx.x < 32) {
        const uint32_t edge = bin_edge(sh.sc, kBins - 1);
        if (threadIdx.x == 0) sh.live = value_of(edge);
    }
    __syncthreads();
}

// Lowers sh.cut to where the running count of the values above it reaches sh.goal (> 0), or (W) their
// running weight p times the weight of all of them and of the cut's ties. False where that is not
// reached: the cut stays, and sh.goal is what is wanted of its ties.
template <typename T, bool W> __device__ __noinline__ bool search(Shared &sh, double p) {
    cg::cluster_group cl = cg::this_cluster();
    u64 target = sh.goal;
    const Cut cut = sh.cut;
    uint32_t from = cut.key + 1;
    clear_bins(sh);
    if (!W && sh.task.tops) {
        // the goal-th of the blocks' largest values is a bound of what is looked for, up to a bin
        const T *tops = reinterpret_cast<const T *>(sh.task.tops);
        for (int i = threadIdx.x; i < sh.task.b1 - sh.task.b0; i += kThr)
            if ((float)tops[i] >= sh.live) atomicAdd(&sh.lo[bin_of(sh.sc, tops[i])], 1u);
        share_bins(sh);
        if (find_bin(sh, target)) from = max(from, bin_edge(sh.sc, sh.bin));
        __syncthreads();
        clear_bins(sh);
    }
    pass<T, W ? kWeights : kCounts>(sh, from, 0xffffffffu, 0);
    share_bins(sh);
    if (W) {
        u64 own = 0;
        for (int i = threadIdx.x; i < kBins; i += kThr) own += (u64)sh.hi[i] << 32 | sh.lo[i];
        block_scan(sh, own);
        const u64 tie = cut.ties ? weigh(sh, value_of(cut.key)) : 0;
        if (threadIdx.x == 0) {
            const double t = p * (double)(sh.scanned + tie * cut.ties);
            sh.goal = t >= 1.0 ? (u64)ceil(t) : 1;
        }
        __syncthreads();
        target = sh.goal;
        __syncthreads();
    }
    if (!find_bin(sh, target)) {
        if (threadIdx.x == 0) sh.goal = target - sh.scanned;
        __syncthreads();
        return false;
    }
    target -= sh.before;
    // the bin's keys; bf16 values' are 2^16 apart
    constexpr int kStep = sizeof(T) == 2 ? 16 : 0;
    const int bin = sh.bin;
    if (threadIdx.x < 64) {
        const uint32_t edge = threadIdx.x < 32 ? bin_edge(sh.sc, bin)
                              : bin            ? bin_edge(sh.sc, bin - 1) - 1
                                               : key_of(sh.sc.top);
        if ((threadIdx.x & 31) == 0) sh.edges[threadIdx.x / 32] = edge;
    }
    __syncthreads();
    KeyRange<kStep> keys(max(sh.edges[0], cut.key + 1), sh.edges[1]);
    for (bool more = keys.open(); more;) {
        const int shift = keys.shift();
        clear_bins(sh);
        pass<T, W ? kWeightKeys : kCountKeys>(sh, keys.min, keys.max, shift);
        share_bins(sh);
        find_bin(sh, target);
        target -= sh.before;
        more = keys.narrow(sh.bin, shift);
    }
    // ties that are needed to reach the target
    const u64 one = W ? weigh(sh, value_of(keys.max)) : 1;
    __syncthreads();
    if (threadIdx.x == 0) sh.cut = Cut{keys.max, one ? (uint32_t)((target + one - 1) / one) : 1u};
    __syncthreads();
    return true;
}

// Puts the first n of the list in ascending order: a thread counts what comes before its entry.
__device__ __noinline__ void sort_list(Shared &sh, int n) {
    const bool on = (int)threadIdx.x < n;
    const u64 mine = on ? sh.list[threadIdx.x] : 0;
    int at = 0;
    if (on) {
#pragma unroll 4
        for (int i = 0; i < n; ++i) at += sh.list[i] < mine;
    }
    __syncthreads();
    if (on) sh.list[at] = mine;
    __syncthreads();
}

__device__ __noinline__ void emit(const Shared &sh, int token, float l, u64 z) {
    *sh.task.token = token;
    if (sh.task.logprob) *sh.task.logprob = log_share(l, sh.sc.top, sh.task.temp, z);
}

__device__ __forceinline__ u64 aim(float u, u64 z) {
    const double x = (double)u * (double)z;
    return min(z - 1, x > 0.0 ? (u64)x : 0ull);
}

// The weight of the list's first n.
__device__ __noinline__ u64 list_weight(Shared &sh, int n) {
    u64 all = 0;
    for (int i = threadIdx.x; i < n; i += kThr) all += weigh(sh, value_of(~(uint32_t)(sh.list[i] >> 32)));
    block_scan(sh, all);
    all = sh.scanned;
    __syncthreads();
    return all;
}

// Borders (the weight before a token) below sh.limit are kept by top-p; in limit_lo .. limit_hi they
// cannot be told from it. z: the weight that top-p cuts, up to a relative error. One thread's fp64: it
// takes tens of cycles an instruction for every warp.
__device__ __noinline__ void set_limit(Shared &sh, double z, double error) {
    if (threadIdx.x == 0) {
        const double t = (double)sh.task.top_p * z;
        sh.limit = t >= 1.0 ? (u64)ceil(t) : 1;
        sh.limit_lo = error > 0.0 ? (u64)(t * (1.0 - error)) : sh.limit;
        sh.limit_hi = error > 0.0 ? (u64)(t * (1.0 + error)) + 1 : sh.limit;
    }
    __syncthreads();
}

// The cuts and the token from the sorted list of n tokens (top-k's at most); of_list: top-p is of their
// weight. False where a border cannot be told from top-p's limit.
__device__ __noinline__ bool choose(Shared &sh, int n, bool of_list) {
    const Task &ask = sh.task;
    const bool by_p = ask.top_p < 1.f;
    u64 limit = sh.limit, limit_lo = sh.limit_lo, limit_hi = sh.limit_hi;
    u64 *weights = reinterpret_cast<u64 *>(sh.lo);
    // a thread for each token adds up what it needs itself
    const int i = threadIdx.x;
    const bool on = i < n;
    const u64 e = on ? sh.list[i] : 0;
    const uint32_t key = ~(uint32_t)(e >> 32);
    const float l = value_of(key);
    const u64 w = on ? weigh(sh, l) : 0;
    if (on) weights[i] = w;
    __syncthreads();
    u64 before = 0;
    if (on) {
#pragma unroll 4
        for (int q = 0; q < i; ++q) before += weights[q];
    }
    if (of_list) {
        if (i == n - 1) sh.z = before + w;
        __syncthreads();
        set_limit(sh, (double)sh.z, 0.0);
        limit = limit_lo = limit_hi = sh.limit;
    }
    bool kept = w > 0 && key >= ask.low_key, sure = true;
    if (by_p && i > 0 && kept) {
        sure = before < limit_lo || before >= limit_hi;
        kept = before < limit;
    }
    const int keep = __syncthreads_count(kept);
    if (!__syncthreads_and(sure)) return false;
    if (i == keep - 1) {
        sh.z = before + w;
        sh.target = aim(ask.u, before + w);
    }
    __syncthreads();
    if (kept) {
        // in the order of the tokens
        const u64 target = sh.target;
        u64 at = 0;
#pragma unroll 4
        for (int q = 0; q < keep; ++q)
            if ((uint32_t)sh.list[q] < (uint32_t)e) at += weights[q];
        if (at <= target && target < at + w) emit(sh, (int)(uint32_t)e, l, sh.z);
    }
    return true;
}

// By one warp: the bin in which the running count reaches `want`, or the last: sh.bin. It looks at 128
// bins at a time and is done early where little is wanted.
__device__ __noinline__ void first_bin(Shared &sh, int want) {
    const int lane = threadIdx.x;
    uint32_t before = 0;
    int bin = kBins - 1;
#pragma unroll 1
    for (int b0 = 4 * lane; b0 < kBins; b0 += 128) {
        const uint4 v = *reinterpret_cast<const uint4 *>(sh.lo + b0);
        uint32_t s = v.x + v.y + v.z + v.w;
        const uint32_t own = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += x;
        }
        s += before;
        const uint32_t m = __ballot_sync(0xffffffffu, s >= (uint32_t)want);
        if (m) {
            if (lane == __ffs(m) - 1) {
                uint32_t at = s - own;
                bin = b0;
                if ((at += v.x) < (uint32_t)want) ++bin;
                if (bin == b0 + 1 && (at += v.y) < (uint32_t)want) ++bin;
                if (bin == b0 + 2 && (at += v.z) < (uint32_t)want) ++bin;
            }
            bin = __shfl_sync(0xffffffffu, bin, __ffs(m) - 1);
            break;
        }
        before = __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) sh.bin = bin;
}

// Samples from a list of the row's largest tokens: those that min-p leaves (want 0), or `want` of them
// and a few more. own: the thread's largest value. False (for the whole cluster) where the list does
// not hold all that may be kept.
template <typename T> __device__ __noinline__ bool from_list(Shared &sh, int want, float own, float sum) {
    const Task &ask = sh.task;
    cg::cluster_group cl = cg::this_cluster();
    const int ctas = cl.num_blocks(), rank = cl.block_rank();
    const bool whole = ask.top_p < 1.f && !ask.k;  // top-p of the whole row's weight
    int last = kBins - 1;                          // bins up to this one are listed
    int listed = 0, undecided = 0;
    if (threadIdx.x == 0) sh.listed = 0;
    if (want) {
        clear_bins(sh);
        // as many threads' largest values: at least as many values
        if (is_live(sh.sc, own)) atomicAdd(&sh.lo[bin_of(sh.sc, own)], 1u);
        // (each CTA's own as long as all their lists together are short)
        if (want * ctas > kAsk / 2)
            share_bins(sh);
        else
            __syncthreads();
        if (threadIdx.x < 32) first_bin(sh, want);
    }
    __syncthreads();
    if (want) last = sh.bin;
    // All values of those bins (and perhaps a few below them) are at least so large; min-p's least value
    // is one itself.
    float least = sh.sc.top - (float)(last + 1) * (1.0f + 0x1p-18f) / kBinScale / sh.sc.ch;
    uint32_t least_key = key_of(fmaxf(least, -FLT_MAX) + 0.f);
    if (!ask.k) least_key = max(least_key, ask.low_key);
    if (ask.tops) {
        if (whole) {
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if ((threadIdx.x & 31) == 0) sh.sums[threadIdx.x >> 5] = sum;
        }
        take<T>(sh, least_key);
    } else if (whole) {
        pass<T, kTakeAndSum>(sh, least_key, 0xffffffffu, 0);
    } else {
        pass<T, kTake>(sh, least_key, 0xffffffffu, 0);
    }
    if (whole && threadIdx.x == 0) {
        float all = 0.f;
        for (int i = 0; i < kWarps; ++i) all += sh.sums[i];
        sh.sum = all;
    }
    row_sync();
    if (rank == 0) {
        // a lane for each CTA reads how much it has listed
        const int lane = threadIdx.x & 31;
        int mine = 0, before;
        float z_all = 0.f;
        if (lane < ctas) {
            const Shared *o = cl.map_shared_rank(&sh, lane);
            mine = min(o->listed, kList + 1);
            z_all = whole ? o->sum : 0.f;
        }
        before = mine;
#pragma unroll
        for (int o = 1; o < kMaxCluster; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += x;
            z_all += __shfl_xor_sync(0xffffffffu, z_all, o);
        }
        int n = __shfl_sync(0xffffffffu, before, kMaxCluster - 1);
        z_all = __shfl_sync(0xffffffffu, z_all, 0);
        bool fine = n <= kList;
        if (threadIdx.x < ctas) sh.ends_of[lane] = before;
        __syncthreads();
        if (fine) {
            const int own = sh.listed;
            for (int i = own + threadIdx.x; i < n; i += kThr) {
                int c = 0, first = 0;
                for (int o = 1; o < ctas; ++o) {
                    const int x = sh.ends_of[o - 1];
                    if (i >= x) {
                        c = o;
                        first = x;
                    }
                }
                sh.list[i] = cl.map_shared_rank(&sh, c)->list[i - first];
            }
            __syncthreads();
            if (whole) {
                set_limit(sh, (double)z_all * 0x1p43, (double)kSumError);
                // (what top-p keeps last is to be listed)
                if (!ask.low_key) fine = list_weight(sh, n) >= sh.limit_hi;
            }
        }
        if (fine) {
            sort_list(sh, n);
            if (ask.k) n = min(n, ask.k);
            fine = choose(sh, n, ask.k && ask.top_p < 1.f);
            if (!fine) undecided = 1;
        }
        if (threadIdx.x == 0) sh.settled = fine ? 1 : undecided ? 2 : 0;
        listed = n;
    }
    row_sync();
    int settled = cl.map_shared_rank(&sh, 0)->settled;
    if (settled == 2) {
        // a border lies within the error of the fp32 sum: the row's weight as it is
        set_live(sh);
        pass<T, kFinal>(sh, 0, 0xffffffffu, 0);
        if (threadIdx.x < kWarps) {
            u64 sum = sh.wsum[threadIdx.x];
#pragma unroll
            for (int o = kWarps / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffu, sum, o);
            if (threadIdx.x == 0) sh.wsum[0] = sum;
        }
        row_sync();
        if (rank == 0) {
            u64 z = 0;
            for (int c = 0; c < ctas; ++c) z += cl.map_shared_rank(&sh, c)->wsum[0];
            set_limit(sh, (double)z, 0.0);
            choose(sh, listed, false);
        }
        settled = 1;
    }
    row_sync();
    return settled != 0;
}

// Samples from the row itself.
template <typename T> __device__ __noinline__ void from_row(Shared &sh) {
    using B = Block<T>;
    const Task &ask = sh.task;
    const Row<T> row(ask);
    cg::cluster_group cl = cg::this_cluster();
    const int ctas = cl.num_blocks(), rank = cl.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        sh.cut = Cut{0, 0};
        sh.goal = ask.k;
    }
    set_live(sh);
    if (ask.k) search<T, false>(sh, 0.0);
    if (ask.top_p < 1.f) {
        const Cut before = sh.cut;
        if (!search<T, true>(sh, (double)ask.top_p) && before.ties) {
            // the cut lies among the ties of top-k's
            const u64 tie = weigh(sh, value_of(before.key));
            if (threadIdx.x == 0 && tie)
                sh.cut.ties = min(before.ties, (uint32_t)((sh.goal + tie - 1) / tie));
            __syncthreads();
        }
    }
    Cut cut = sh.cut;
    if (ask.low_key && ask.low_key - 1 >= cut.key) cut = Cut{ask.low_key - 1, 0};

    // weights and ties of every warp, in the order of the tokens
    pass<T, kFinal>(sh, cut.key, 0xffffffffu, 0);
    row_sync();
    const u64 w_tie = cut.ties ? weigh(sh, value_of(cut.key)) : 0;
    auto total = [&](u64 w, u64 t) { return w + w_tie * min(t, (u64)cut.ties); };
    {
        u64 w = 0, t = 0;
        if (threadIdx.x < kWarps * ctas) {
            const Shared *o = cl.map_shared_rank(&sh, threadIdx.x / kWarps);
            w = o->wsum[threadIdx.x % kWarps];
            t = o->ties[threadIdx.x % kWarps];
        }
        const u64 w0 = block_scan(sh, w), all_w = sh.scanned;
        __syncthreads();
        const u64 t0 = block_scan(sh, t), all_t = sh.scanned;
        const u64 z = total(all_w, all_t);
        if (threadIdx.x == 0) sh.target = aim(ask.u, z);
        __syncthreads();
        const u64 goal = sh.target;
        if (total(w0, t0) <= goal && goal < total(w0 + w, t0 + t)) {
            sh.owner = threadIdx.x;
            sh.own_w = w0;
            sh.own_t = (uint32_t)t0;
            sh.z = z;
        }
        __syncthreads();
    }
    // The CTA whose warp holds the token: all its warps share that warp's blocks and add up their parts,
    // then the one that holds it adds up 32 blocks at a time.
    if (sh.owner >= 0 && sh.owner / kWarps == rank) {
        const Scale sc = sh.sc;
        const float least = cut.key > key_of(-INFINITY) ? value_of(cut.key) : -INFINITY;
        const u64 goal = sh.target;
        const int from = min(ask.b1, ask.b0 + sh.owner % kWarps * ask.per), to = min(ask.b1, from + ask.per);
        const int rounds = (to - from + 31) / 32, each = (rounds + kWarps - 1) / kWarps;
        const int j_from = from + warp * each * 32, j_to = min(to, j_from + each * 32);
        // a block's weight and ties
        auto block_sums = [&](const B &b, u64 &w, u64 &t) {
#pragma unroll 2
            for (int i = 0; i < B::kN; i += 2) {
                const float l0 = b.get(i), l1 = b.get(i + 1);
                u64 x, y;
                weight2(sc, l0, l1, sh.powers, x, y);
                if (l0 >= sh.live) {
                    if (l0 > least) w += x;
                    t += l0 == least;
                }
                if (l1 >= sh.live) {
                    if (l1 > least) w += y;
                    t += l1 == least;
                }
            }
        };
        u64 w_at = 0, t_at = 0;
#pragma unroll 1
        for (int turn = 0; turn < 2; ++turn) {
            u64 w_all = 0, t_all = 0;
            if (turn == 1 && sh.part_owner != warp) break;
#pragma unroll 1
            for (int j0 = j_from; j0 < j_to; j0 += 32) {
                const int j = j0 + lane;
                u64 w = 0, t = 0;
                B b;
                if (j < j_to) {
                    b = row.block(j);
                    block_sums(b, w, t);
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
                const uint32_t m = __ballot_sync(0xffffffffu, turn == 1 && goal < total(w_at + ws, t_at + ts));
                if (m) {
                    if (lane == __ffs(m) - 1) {
                        w = w_at + ws - w;
                        t = t_at + ts - t;
#pragma unroll 1
                        for (int i = 0; i < B::kN; ++i) {
                            const float l = b.take();
                            if (!(l >= sh.live)) continue;
                            if (l > least) w += weigh(sh, l);
                            t += l == least;
                            if (goal < total(w, t)) {
                                emit(sh, j * B::kN - row.shift + i, l, sh.z);
                                break;
                            }
                        }
                    }
                    break;
                }
                w_all += __shfl_sync(0xffffffffu, ws, 31);
                t_all += __shfl_sync(0xffffffffu, ts, 31);
                if (turn == 1) {
                    w_at += __shfl_sync(0xffffffffu, ws, 31);
                    t_at += __shfl_sync(0xffffffffu, ts, 31);
                }
            }
            if (turn == 1) break;
            if (lane == 0) {
                sh.part_w[warp] = w_all;
                sh.part_t[warp] = t_all;
            }
            __syncthreads();
            w_at = sh.own_w;
            t_at = sh.own_t;
            for (int i = 0; i < warp; ++i) {
                w_at += sh.part_w[i];
                t_at += sh.part_t[i];
            }
            if (lane == 0 && total(w_at, t_at) <= goal && goal < total(w_at + w_all, t_at + t_all))
                sh.part_owner = warp;
            __syncthreads();
        }
    }
    row_sync();  // (shared memory of CTAs that have ended is not to be read)
}

template <typename T>
__global__ void __launch_bounds__(kThr, 2) sample_kernel(const Args a, int held_blocks, int tops_blocks) {
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
    Task &t = sh.task;
    if (threadIdx.x == 0) {
        const int g = r / a.group;
        const T *p = reinterpret_cast<const T *>(a.logits) + (size_t)r * a.ld;
        t.shift = (int)(((uintptr_t)p / sizeof(T)) % B::kN);
        t.blocks = (a.V + t.shift + B::kN - 1) / B::kN;
        const int per = (t.blocks + ctas - 1) / ctas;
        t.b0 = min(t.blocks, rank * per);
        t.b1 = min(t.blocks, t.b0 + per);
        t.per = ((t.b1 - t.b0 + kWarps - 1) / kWarps + 31) / 32 * 32;
        // the row's ends reach into other memory: their blocks are made up
        const B *inner = reinterpret_cast<const B *>(p - t.shift);
        t.inner = inner;
        t.low = inner;
        t.high = inner + t.blocks - 1;
        if (t.shift) {
            sh.ends[0] = B::edge(p, -t.shift, a.V);
            t.low = sh.ends;
        }
        const int last = (t.blocks - 1) * B::kN - t.shift;
        if (last + B::kN > a.V) {
            sh.ends[1] = B::edge(p, last, a.V);
            t.high = sh.ends + 1;
        }
        if (t.blocks == 1 && t.shift) t.high = t.low;
        t.raw = true;
        // (beyond these the weights are those of the largest alone, or equal)
        t.temp = a.temperature ? a.temperature[g] : 1.f;
        if (t.temp > 0.f) t.temp = fminf(fmaxf(t.temp, 1e-30f), 1e30f);
        const int k = a.top_k ? a.top_k[g] : 0;
        t.k = k < a.V ? max(k, 0) : 0;
        const float p_ = a.top_p ? a.top_p[g] : 1.f;
        t.top_p = p_ < 1.f ? p_ : 1.f;
        t.u = a.u[r];
        t.token = a.token + r;
        t.logprob = a.logprob ? a.logprob + r : nullptr;
        sh.index = 0xffffffffu;
        sh.owner = -1;
        sh.part_owner = -1;
    } else if (threadIdx.x == 32) {
        float temp = a.temperature ? a.temperature[r / a.group] : 1.f;
        temp = fminf(fmaxf(temp, 1e-30f), 1e30f);
        const double c = 1.4426950408889634074 / (double)temp;
        sh.sc.ch = (float)c;
        sh.sc.cl = (float)(c - (double)sh.sc.ch);
    } else if (threadIdx.x == 64) {
        const float min_p = a.min_p ? a.min_p[r / a.group] : 0.f;
        float temp = a.temperature ? a.temperature[r / a.group] : 1.f;
        temp = fminf(fmaxf(temp, 1e-30f), 1e30f);
        sh.below = min_p > 0.f ? (double)temp * log((double)fminf(min_p, 1.f)) : -1.0 / 0.0;
    }
    __syncthreads();

    // the row's slice, and the largest value
    const Row<T> row(t);
    B *held = t.b1 - t.b0 <= held_blocks ? reinterpret_cast<B *>(dyn) - t.b0 : nullptr;
    T *tops = t.b1 - t.b0 <= tops_blocks
                  ? reinterpret_cast<T *>(dyn + (size_t)held_blocks * 16) - t.b0 : nullptr;
    // Beside it, where top-p is of the row's weight, the fp32 sum of the weights relative to a value that
    // the thread has seen; a larger one takes its place from 8 octaves on, so that what was added up
    // before hardly counts when it has been scaled down twice (its error: kSumError).
    const bool whole = tops && t.top_p < 1.f && !t.k && t.temp > 0.f;
    const float ch = sh.sc.ch;
    float top = -INFINITY, at = -INFINITY, sum = 0.f;
    row.template blocks<8>([&](const auto &b, int j0, int n) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (q >= n) continue;
            const float m = b[q].top();
            if (held) held[j0 + 32 * q] = b[q];
            if (tops) tops[j0 + 32 * q] = from_value<T>(m);
            if (whole && m > -INFINITY) {
                if (!((m - at) * ch < 8.f)) {
                    sum *= exp2_approx((at - m) * ch);
                    at = m;
                }
                if ((at - m) * ch < kFar) {
                    const uint64_t less = pack2(-at, -at), by = pack2(ch, ch);
                    uint64_t part = 0;
#pragma unroll
                    for (int i = 0; i < B::kN; i += 2) {
                        const float2 x = unpack2(mul2(add2(pack2(b[q].get(i), b[q].get(i + 1)), less), by));
                        part = add2(part, pack2(exp2_approx(x.x), exp2_approx(x.y)));
                    }
                    const float2 p2 = unpack2(part);
                    sum += p2.x + p2.y;
                }
            }
            top = fmaxf(top, m);
        }
    });
    const float own = top;  // the thread's largest
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) sh.sums[warp] = top;
    if (tops && threadIdx.x < B::kN) tops[t.b1 + threadIdx.x] = from_value<T>(-INFINITY);
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) top = fmaxf(top, sh.sums[i]);
    if (threadIdx.x == 0) {
        sh.top = top;
        t.tops = tops ? tops + t.b0 : nullptr;
        if (held) {
            t.inner = t.low = held;
            t.high = held + t.blocks - 1;
            t.raw = false;
        }
    }
    row_sync();
    if (ctas > 1) {  // (a lane for each CTA: the reads do not wait for one another)
        if (lane < ctas) top = fmaxf(top, cl.map_shared_rank(&sh, lane)->top);
#pragma unroll
        for (int o = kMaxCluster / 2; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = __shfl_sync(0xffffffffu, top, 0);
    }

    if (top == -INFINITY) {  // nothing to sample from
        if (rank == 0 && threadIdx.x == 0) {
            *t.token = -1;
            if (t.logprob) *t.logprob = -INFINITY;
        }
        row_sync();
        return;
    }
    if (!(t.temp > 0.f)) {  // the first of the largest
        if (own == top) {
            for (int j = row.w0 + lane; j < row.w1; j += 32) {
                B b = row.block(j);
                if (b.top() < top) continue;
                int i = 0;
                while (b.take() != top) ++i;
                atomicMin(&sh.index, (uint32_t)(j * B::kN - row.shift + i));
                break;
            }
        }
        row_sync();
        if (rank == 0 && threadIdx.x == 0) {
            uint32_t first = 0xffffffffu;
            for (int c = 0; c < ctas; ++c) first = min(first, cl.map_shared_rank(&sh, c)->index);
            *t.token = (int)first;
            if (t.logprob) *t.logprob = 0.f;
        }
        row_sync();
        return;
    }

    const bool by_m = sh.below > -1.0 / 0.0;
    if (threadIdx.x == 0) {
        sh.sc.top = top;
        t.low_key = by_m ? key_of(__double2float_ru((double)top + sh.below) + 0.f) : 0;
    }
    __syncthreads();
    // what is kept may fit a list: k tokens, or those that min-p leaves, or top-p's as a guess
    if (t.k ? t.k <= kAsk : by_m || t.top_p < 1.f)
        if (from_list<T>(sh, t.k ? t.k : by_m ? 0 : kAsk, own, whole && sum > 0.f ? sum * exp2_approx((at - top) * ch) : 0.f))
            return;
    from_row<T>(sh);
}

constexpr int kHeldBytes = 76 * 1024;  // of a row in a CTA: two CTAs share an SM

template <typename T> cudaError_t launch(const Args &a, cudaStream_t s) {
    const int blocks = (a.V + 2 * Block<T>::kN - 2) / Block<T>::kN;
    const int room = kHeldBytes / 16, sms = std::max(1, device_sms());
    // CTAs of a row, for rows long enough. Few rows take several; with more rows the cluster's barriers
    // cost more than what they save. Rows of bf16 151936, us by 1, 2, 4 and 8 CTAs a row: 16 rows with
    // top-k 20: 16.2, 15.9, 14.3, 14.5; 65: 18.3, 18.3, 18.4; 152: 19.8, 21.6, 46; 192: 24, 38, 51; 1040: 85, 132, 243.
    // Rows that no list serves gain from more CTAs up to where all of them run at once: without cuts 16 rows 73,
    // 45, 29, 27; 65: 74, 47, 47, 58; 152: 76, 76, 103; 192: 128, 108, 123; 304: 132, 139, 180. In batches of all
    // kinds they are waited for: 152: 194, 121, 95; 192: 195, 139, 111; 228: 292, 154, 132.
    // So with up to a row an SM two are taken, and up to one and a half where no list is to be expected (neither
    // top-k nor min-p is asked for) or a row's settings may be its own. What these are is on the device, so between one
    // and one and a half rows an SM with param_rows 1 a batch whose rows all have a list pays 14 us (top-k 20: 24 to
    // 38) for what a mixed one saves (40 to 137).
    const bool slow = a.group == 1 || (!a.top_k && !a.min_p);
    int ctas = a.R <= sms / 16 ? 8 : a.R <= sms / 2 ? 4 : a.R <= (slow ? 3 * sms / 2 : sms) ? 2 : 1;
    while (ctas > 1 && blocks / ctas < kThr) ctas /= 2;
    const int per = (blocks + ctas - 1) / ctas;
    const int held = per <= room ? per : 0;
    // the blocks' largest values, and a block of padding
    const int tops_bytes = (per + 2 * Block<T>::kN) * (int)sizeof(T) / 16 * 16;
    const bool tops = held || tops_bytes <= kHeldBytes;
    cudaError_t err = allow_smem(sample_kernel<T>, 2 * kHeldBytes);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.R * ctas);
    cfg.blockDim = dim3(kThr);
    cfg.dynamicSmemBytes = (size_t)held * 16 + (tops ? tops_bytes : 0);
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
    return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a, held, tops ? per : 0);
}

}  // namespace

cudaError_t launch_sample(const Args &a, int dtype, cudaStream_t s) {
    return dtype == MOE_DTYPE_F32 ? launch<float>(a, s) : launch<__nv_bfloat16>(a, s);
}

}  // namespace sample
}  // namespace moe
