// Rounding of normed elements, shared by the pre-norm kernel and the layer for a few tokens.
#pragma once

#include "common.cuh"

namespace moe {

// bf16(fp64(v * scale)), rounded to nearest even, for v an fp32 value. The fp32 product
// p = v * (float)scale lies within 2^-22.8 |p| of the fp64 product (one rounding of the
// scale to fp32 and one of the product, 2^-24 relative each); bf16 rounding midpoints are
// at least 2^-9 |p| apart, so when p is farther than 2^-21 |p| from the midpoint between
// its two bf16 neighbours, both products round to the same bf16 value and p's rounding is
// the answer. Otherwise (about one element in 4000, for zero, tiny or non-finite p, and for
// a scale whose fp32 rounding is not a normal number far from the range ends) the product
// is formed and rounded in fp64.
__device__ __forceinline__ uint32_t scaled_bf16(float v, double scale, float scale_f) {
    const float p = v * scale_f;
    const float ap = fabsf(p);
    if (scale_f >= 0x1p-100f && scale_f <= 0x1p+100f && ap >= 0x1p-100f && ap <= 0x1p+100f) {
        const __nv_bfloat16 lo = __float2bfloat16_rd(p), hi = __float2bfloat16_ru(p);
        const float flo = __bfloat162float(lo), fhi = __bfloat162float(hi);
        if (flo == fhi) return __bfloat16_as_ushort(lo);  // p is a bf16 value
        const float mid = 0.5f * (flo + fhi);              // exact: a 9-bit value
        const float dist = fabsf(p - mid);                 // exact (Sterbenz)
        if (dist > ap * 0x1p-21f) return __bfloat16_as_ushort(p < mid ? lo : hi);
    }
    return __bfloat16_as_ushort(__double2bfloat16((double)v * scale));
}

}  // namespace moe
