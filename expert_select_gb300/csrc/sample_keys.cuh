// The order of logits as unsigned integers, and the division of a range of them (host and device: the
// tests run it on the host).
#pragma once

#include <stdint.h>
#include <string.h>

#ifdef __CUDACC__
#define MOE_KEYS_FN __host__ __device__ __forceinline__
#else
#define MOE_KEYS_FN inline
#endif

namespace moe {
namespace sample {

// Keys ascend with the values, and 0 and -0 have the same: every integer from -inf's key to +inf's stands
// for one value, with none for -0. So a key formed by adding or subtracting stands for the next value, and a
// range of values is a range of keys. Values of few bits (bf16) have keys of as many trailing zeros.
MOE_KEYS_FN uint32_t key_of(float l) {
    uint32_t b;
    memcpy(&b, &l, 4);
    return (int32_t)b < 0 ? 0u - b : b | 0x80000000u;
}
MOE_KEYS_FN float value_of(uint32_t key) {
    const uint32_t b = (int32_t)key < 0 ? key & 0x7fffffffu : 0u - key;
    float l;
    memcpy(&l, &b, 4);
    return l;
}

// Keys min .. max of which one is looked for, in bins of 2^shift() keys that descend with the key, of which
// there are kRangeBins at most. kStep: keys are multiples of 2^kStep.
constexpr int kRangeBins = 1024;
template <int kStep> struct KeyRange {
    uint32_t min, max;
    MOE_KEYS_FN KeyRange(uint32_t min_, uint32_t max_) : min(min_), max(max_ & ~((1u << kStep) - 1)) {}
    MOE_KEYS_FN bool open() const { return min < max; }
    // (for open ranges)
    MOE_KEYS_FN int shift() const {
        int bits = 0;
        for (uint32_t n = max - min; n >= (uint32_t)kRangeBins; n >>= 1) ++bits;
        return bits > kStep ? bits : kStep;
    }
    // It becomes one of its bins. False where that is a single key, which is max then.
    MOE_KEYS_FN bool narrow(int bin, int shift) {
        max -= (uint32_t)bin << shift;
        if (shift <= kStep) return false;
        const uint32_t width = (1u << shift) - 1;
        if (max > min && max - min > width) min = max - width;
        max &= ~((1u << kStep) - 1);
        return open();
    }
};

}  // namespace sample
}  // namespace moe
