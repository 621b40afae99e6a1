// RoPE angles of packed tokens at any position.
#pragma once

#include "common.cuh"

namespace relation {

// rope_sincos at any int32 position, which a float holds up to 2^24 only: above that the
// position is split into a multiple of 2^24 and the rest, both exact, and the multiple's
// fractional turn is added.  Each product's rounding error is a float of its own, so the
// angle is off by the frequency's own rounding, pos 2^-49 radians, and 4e-7.
__device__ __forceinline__ void position_sincos(int pos, float hi, float lo, float* s, float* c) {
    const int rest = pos % (1 << 24);
    if (rest == pos) {
        rope_sincos((float)pos, hi, lo, s, c);
        return;
    }
    float turns = 0.f;
    for (const float p : {(float)(pos - rest), (float)rest})
        for (const float f : {hi, lo}) {
            const float whole = p * f, err = fmaf(p, f, -whole);
            turns += (whole - rintf(whole)) + (err - rintf(err));
        }
    sincospif(2.f * (turns - rintf(turns)), s, c);
}

}  // namespace relation
