// la_gate.cuh - the gate of the gated linear recurrence: a and w = du/dx from
// the value g of a token and channel.
#pragma once

#include "la_common.cuh"

namespace la {

// e^g for the log gate.  A memory of T tokens has a about 1 - 1/T, and a
// rounding of a that is off to one side moves h by T times as much: fp32 e^g,
// whose error of an ulp need not be centred, was 6.6e-6 off over 5001 tokens
// with T up to 1000, where a correctly rounded a gives 4e-7.  Near 0, 1 +
// (e^g - 1) with the Taylor series of e^g - 1 up to g^7 / 7! (the next term is
// below 4e-10 for |g| <= 1/4) rounds once, at the last sum.
__device__ __forceinline__ float exp_gate(float g) {
    float p = 1.f / 5040.f;
    p = fmaf(p, g, 1.f / 720.f);
    p = fmaf(p, g, 1.f / 120.f);
    p = fmaf(p, g, 1.f / 24.f);
    p = fmaf(p, g, 1.f / 6.f);
    p = fmaf(p, g, 0.5f);
    p = fmaf(p * g, g, g);
    return fabsf(g) <= 0.25f ? 1.f + p : expf(g);
}

// GATE: a value of la_gate.  w is 1 - a for the sigmoid gate, without
// cancellation, and 1 for the others.
template <int GATE> __device__ __forceinline__ void gate_of(float g, float &a, float &w) {
    if (GATE == 2) {
        // the smaller of the two from the exponential, the larger as 1 minus it
        const float e = expf(-fabsf(g));
        const float lo = __fdividef(e, 1.f + e), hi = 1.f - lo;
        a = g >= 0.f ? hi : lo;
        w = g >= 0.f ? lo : hi;
        if (isnan(g)) a = w = g;
    } else {
        a = GATE == 1 ? exp_gate(g) : g;
        w = 1.f;
    }
}

}  // namespace la
