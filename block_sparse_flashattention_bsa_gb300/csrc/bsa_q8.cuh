// bsa_q8.cuh -- rows of the 8-bit paged cache: D e4m3 codes and one e8m0 scale
// (a power of two, biased exponent 127) per row.
//
// Mathematics: a row y is held as code * 2^e with e the smallest integer in
// [kMinExp, kMaxExp] for which max |y| <= 448 * 2^e (448: the largest e4m3
// value).  A floating-point code loses nothing by a scale that is a power of
// two: the codes' relative step is the same, and code * 2^e is a bf16 number,
// exactly, so that the tensor cores work on the held values themselves and no
// scale is left to be applied to scores or weights.  kMinExp keeps 2^e times
// the smallest code a normal bf16 number, kMaxExp keeps 448 * 2^e finite in bf16.
#pragma once

#include <stdint.h>

#include "bsa_ptx.cuh"

namespace bsa {

constexpr int kMinExp = -100, kMaxExp = 118;

// The scale's exponent for a row's largest magnitude: max = 1.m * 2^x against 448 = 1.75 * 2^8.
__device__ __forceinline__ int row_exponent(float max) {
    const uint32_t b = __float_as_uint(max);
    return ::min(::max((int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0), kMinExp), kMaxExp);
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Two values to two e4m3 codes (nearest, ties to even, saturating; low byte: lo).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Codes to bf16 without a conversion instruction (there is none from e4m3): the
// code's exponent and mantissa bits, put at bf16's, stand for its value times
// 2^-120 (subnormal codes too), and a bf16 product with 2^(120 + e) gives
// code * 2^e exactly.  A NaN code comes out as 480 * 2^e.
__device__ __forceinline__ uint32_t spread_odd(uint32_t w) {  // bytes 1 and 3
    return (w & 0x80008000u) | ((w >> 4) & 0x07f007f0u);
}
__device__ __forceinline__ uint32_t spread_even(uint32_t w) {  // bytes 0 and 2
    return ((w << 8) & 0x80008000u) | ((w << 4) & 0x07f007f0u);
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// 2^(120 + e) of a scale byte as bf16 bits; exponents that one bf16 factor
// cannot reach (e above 7) need scale_rest() as a second one.  Bytes outside
// what is ever written (a slot that nothing was written to) give finite factors.
__device__ __forceinline__ uint32_t scale_first(uint32_t byte) {
    return (uint32_t)::min(::max((int)byte + 120, 127 + 120 + kMinExp), 254) << 7;
}
__device__ __forceinline__ uint32_t scale_rest(uint32_t byte) {
    return (uint32_t)(127 + ::min(::max((int)byte - 127 - 7, 0), kMaxExp - 7)) << 7;
}
constexpr uint32_t kOneStep = 127 + 7;  // scale bytes up to this need one factor

}  // namespace bsa
