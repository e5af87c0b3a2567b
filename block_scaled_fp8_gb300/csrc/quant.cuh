// FP8 quantisation shared by the quantiser and the gated epilogues: the UE8M0 scale of a
// group and the E4M3 codes over it.
//
// The scale is the smallest power of two s with amax / s <= 448 (E4M3's largest value), 1 for a
// group of zeros.  With amax = 1.f 2^(E-127) that is 2^(E-127-8), or the next power above where
// 1.f > 1.75 (448 = 1.75 2^8): integer arithmetic on amax's bits, no logarithm and no rounding.
// Dividing by s is a multiplication by a power of two, so a code is one rounding of its value.
// NaN and infinities do not count for amax and become the NaN code: they stay visible, and the
// group's other values keep their scale.
#pragma once

#include <stdint.h>

#include "ptx.cuh"

namespace dg {

// Magnitude bits of v as the group's largest magnitude counts it (0 for NaN and infinities).
__device__ __forceinline__ uint32_t amax_bits(float v) {
    const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
    return b < 0x7F800000u ? b : 0u;
}

// Biased exponent (the UE8M0 byte) of the scale of a group with these amax bits: a fraction above
// 0.75 carries into the exponent.  127 for 0, and for a NaN (a group without a finite value).
__device__ __forceinline__ uint32_t ue8m0_of_amax(uint32_t bits) {
    const int e = static_cast<int>((bits + 0x1FFFFFu) >> 23) - 8;
    return bits - 1u >= 0x7F800000u ? 127u : static_cast<uint32_t>(max(e, 1));   // (at most 254 - 7)
}

// 1 / scale; the byte is at most 247, so this is a normal number.
__device__ __forceinline__ float inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// E4M3 codes of four values (none infinite) over one scale, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d, float inv) {
    return cvt_e4m3x2(a * inv, b * inv) | (cvt_e4m3x2(c * inv, d * inv) << 16);
}

}  // namespace dg
