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

// The same to 1e-7, for rows that are rounded to fewer bits than a float of angle error would let stand: the turns are
// summed with what each addition loses, and that turns the pair by a little more.
__device__ __forceinline__ void position_sincos_fine(int pos, float hi, float lo, float* s, float* c) {
    float turns = 0.f, lost = 0.f;
    auto add = [&](float x) {
        const float t = turns + x, z = t - turns;
        lost += (turns - (t - z)) + (x - z);
        turns = t;
    };
    auto part = [&](float p) {
        for (const float f : {hi, lo}) {
            const float whole = p * f, err = fmaf(p, f, -whole);
            add(whole - rintf(whole));
            add(err - rintf(err));
        }
    };
    const int rest = pos % (1 << 24);
    part((float)rest);
    if (rest != pos) part((float)(pos - rest));
    float sn, cs;
    sincospif(2.f * (turns - rintf(turns)), &sn, &cs);
    const float more = 6.2831853f * lost;
    *s = fmaf(cs, more, sn);
    *c = fmaf(-sn, more, cs);
}

}  // namespace relation
