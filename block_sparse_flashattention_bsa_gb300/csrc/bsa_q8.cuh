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

#include <cuda_fp16.h>
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

// Two e4m3 codes (the low or high half of w) as fp16, exactly.
__device__ __forceinline__ uint32_t codes_f16(uint32_t w, int high) {
    uint32_t r;
    if (high)
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "mov.b32 {lo, hi}, %1;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
            : "=r"(r)
            : "r"(w));
    else
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "mov.b32 {lo, hi}, %1;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
            : "=r"(r)
            : "r"(w));
    return r;
}
// The same in fp32.
__device__ __forceinline__ f2 codes_f32(uint32_t w, int high) {
    const uint32_t h = codes_f16(w, high);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return {f.x, f.y};
}

}  // namespace bsa
