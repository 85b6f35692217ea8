// paged.cuh -- the paged token cache's number formats and host checks, shared
// by its write and read paths (paged.cu) and its attention
// (paged_attention.cu).
#pragma once

#include "common.cuh"

namespace qvg {

// Scale byte of a group from the largest magnitude's bf16 bits (sign off):
// the smallest e with amax <= TOP 2^e.  TOP = 1.75 * 2^8 (e4m3) or 1.5 * 2^2
// (e2m1), so e is the exponent of amax less TOP's, plus one where amax's
// mantissa exceeds TOP's.  255: amax is an infinity or a NaN.
template <int BITS>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bf16) {
    constexpr int kExp = BITS == 8 ? 8 : 2, kMant = BITS == 8 ? 0x60 : 0x40;
    const int e = static_cast<int>(amax_bf16 >> 7) - kExp + (static_cast<int>(amax_bf16 & 0x7Fu) > kMant ? 1 : 0);
    return amax_bf16 >= 0x7F80u ? 255u : static_cast<uint32_t>(e < 1 ? 1 : e);
}

// 2^(byte - 127) (byte 255: infinity, which times a code of 0 is a NaN) and
// its reciprocal (bytes 1 .. 253).
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }
__device__ __forceinline__ float scale_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Two floats -> two e4m3 numbers (lo in the low byte), nearest even, within +-448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two floats -> two e2m1 numbers (lo in the low half byte).
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
        "cvt.u32.u8 %0, b;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}
// Two e4m3 numbers (the low 16 bits) -> two fp16 in one word.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t b) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(b)));
    return r;
}
// Two e2m1 numbers (the low 8 bits) -> two fp16 in one word.
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\t"
        "cvt.u8.u32 b, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
        : "=r"(r)
        : "r"(b));
    return r;
}

// Host: the shape checks of a cache (the buffers' too, unless `shape_only`).
qvg_status check_paged(const qvg_paged *c, bool shape_only);

}  // namespace qvg
