// rope.cuh -- rotary positions: the angle of a pair, shared by the rotation
// (rope.cu) and the cache's write path (paged.cu).
//
// Angles are kept in turns as 64-bit fractions.  A position moves pair i by
// step[i] / 2^64 turns, so position p stands at (p * step[i]) mod 2^64: one
// integer product, exact at any int32 position, where an fp32 product is off
// by 2^-24 of the angle itself (0.02 rad at position 300,000 of the fastest
// pair).  The top two bits (rounded) are the quadrant; the rest, at most an
// eighth of a turn either way, becomes a float with an error of 2^-28 turns
// at most and goes to sincospif.
#pragma once

#include "common.cuh"

namespace qvg {

// The plan as a kernel parameter (by value: no device memory).
struct RopeArgs {
    uint64_t step[QVG_ROPE_MAX_PAIRS];
    uint8_t axis[QVG_ROPE_MAX_PAIRS];
    int32_t pairs, axes, layout, transpose;
    float mscale;
};

// (mscale cos, mscale sin) of `position` at `step`.
__device__ __forceinline__ float2 rope_cos_sin(uint64_t step, int32_t position, float mscale, bool transpose) {
    const uint32_t turn = static_cast<uint32_t>((static_cast<uint64_t>(static_cast<int64_t>(position)) * step) >> 32);
    const uint32_t quad = (turn + 0x20000000u) >> 30;
    const int32_t rest = static_cast<int32_t>(turn - (quad << 30));
    float s, c;
    sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
    float co = (quad & 1u) ? s : c, si = (quad & 1u) ? c : s;
    co = ((quad + 1u) & 2u) ? -co : co;
    si = (quad & 2u) ? -si : si;
    return make_float2(mscale * co, transpose ? -mscale * si : mscale * si);
}

// The pair (x0, x1) turned by (cos, sin).  The products' roundings are spelt
// out: the rotation and the cache's write path give the same bits.
__device__ __forceinline__ float2 rope_turn(float x0, float x1, float c, float s) {
    return make_float2(fmaf(x0, c, -__fmul_rn(x1, s)), fmaf(x1, c, __fmul_rn(x0, s)));
}

// Host: whether a plan can be used with heads of d channels, and its
// by-value form.
bool rope_plan_ok(const qvg_rope_plan *plan, int d);
RopeArgs rope_args(const qvg_rope_plan *plan, bool transpose);

}  // namespace qvg
