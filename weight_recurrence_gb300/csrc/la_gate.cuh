// la_gate.cuh - the gate of the gated linear recurrence: a and w = du/dx from
// the value g of a token and channel, for V neighbouring channels at a time.
#pragma once

#include "la_pair.cuh"

namespace la {

// V fp32 values, as pairs where V is even.
template <int V> struct Lanes {
    static_assert(V % 2 == 0, "");
    float2 p[V / 2];
    __device__ __forceinline__ float get(int v) const { return v % 2 ? p[v / 2].y : p[v / 2].x; }
    __device__ __forceinline__ void set(int v, float x) { (v % 2 ? p[v / 2].y : p[v / 2].x) = x; }
};
template <> struct Lanes<1> {
    float p[1];
    __device__ __forceinline__ float get(int) const { return p[0]; }
    __device__ __forceinline__ void set(int, float x) { p[0] = x; }
};

__device__ __forceinline__ float fma_pair(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float mul_pair(float a, float b) { return a * b; }
__device__ __forceinline__ float add_pair(float a, float b) { return a + b; }

template <int V> __device__ __forceinline__ Lanes<V> all(float x) {
    Lanes<V> r;
#pragma unroll
    for (int v = 0; v < V; v++) r.set(v, x);
    return r;
}
template <int V> __device__ __forceinline__ Lanes<V> fma(const Lanes<V> &a, const Lanes<V> &b, const Lanes<V> &c) {
    Lanes<V> r;
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; i++) r.p[i] = fma_pair(a.p[i], b.p[i], c.p[i]);
    return r;
}
template <int V> __device__ __forceinline__ Lanes<V> mul(const Lanes<V> &a, const Lanes<V> &b) {
    Lanes<V> r;
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; i++) r.p[i] = mul_pair(a.p[i], b.p[i]);
    return r;
}
template <int V> __device__ __forceinline__ Lanes<V> add(const Lanes<V> &a, const Lanes<V> &b) {
    Lanes<V> r;
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; i++) r.p[i] = add_pair(a.p[i], b.p[i]);
    return r;
}

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// x held within [-c, c]; NaN stays.
__device__ __forceinline__ float within(float x, float c) {
    float y;
    asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(c));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f, kMax = 3.402823466e38f;

// e^g as 2^t, t = g log2(e).  FINE: what t's rounding left out, d = g - t ln 2, is made
// good by e^d = 1 + d; without that e^g is off by another 2^-23 |g|, which is nothing
// to bf16 data, whose g has 8 bits and whose instructions have to be few.  GROW: e^g may
// be infinite, else g counts as 88 at most (1 / (1 + e^88) is under fp32's range).  It
// costs the fp32 calls up to 3 %: 3 x 5001 tokens of 333 channels, log gate, forward |
// backward 25.5 | 32.9 us, without 24.8 | 32.1; 5 x 3001 of 501, sigmoid, 31.6 | 47.3 and
// 31.0 | 46.4.
template <bool FINE, bool GROW, int V> __device__ __forceinline__ Lanes<V> exp_of(Lanes<V> g) {
    if constexpr (FINE) {
#pragma unroll
        for (int v = 0; v < V; v++) g.set(v, within(g.get(v), GROW ? 1e4f : 88.f));
    }
    const Lanes<V> t = mul(g, all<V>(-kLog2e));
    Lanes<V> e;
#pragma unroll
    for (int v = 0; v < V; v++) e.set(v, ex2_approx(-t.get(v)));
    if constexpr (FINE) {
        Lanes<V> f = e;
        if (GROW) {
#pragma unroll
            for (int v = 0; v < V; v++) f.set(v, fminf(e.get(v), kMax));   // inf + inf * d may be NaN
        }
        e = fma(f, fma(t, all<V>(kLn2), g), e);
    }
    return e;
}

// a = e^g of the log gate.  A memory of T tokens has a about 1 - 1/T, and a
// rounding of a that is off to one side moves h by T times as much: an fp32
// e^g, whose error of an ulp need not be centred, was 6.6e-6 off over 5001
// tokens with T up to 1000, where a correctly rounded a gives 4e-7.  Near 0, 1 +
// (e^g - 1) with the Taylor series of e^g - 1 up to g^7 / 7! (the next term is
// below 4e-10 for |g| <= 1/4) rounds once, at the last sum.  (The series for every
// g, after the whole powers of 2 are taken out: the same for fp32 data, 62.6 | 110 ->
// 65.5 | 105 and 61 | 93 -> 68 | 95 us for bf16.)
template <bool FINE, int V> __device__ __forceinline__ Lanes<V> exp_gate(const Lanes<V> &g) {
    Lanes<V> p = all<V>(1.f / 5040.f);
    p = fma(p, g, all<V>(1.f / 720.f));
    p = fma(p, g, all<V>(1.f / 120.f));
    p = fma(p, g, all<V>(1.f / 24.f));
    p = fma(p, g, all<V>(1.f / 6.f));
    p = fma(p, g, all<V>(0.5f));
    p = fma(mul(p, g), g, g);
    p = add(p, all<V>(1.f));
    const Lanes<V> e = exp_of<FINE, true, V>(g);
#pragma unroll
    for (int v = 0; v < V; v++)
        if (!(fabsf(g.get(v)) <= 0.25f)) p.set(v, e.get(v));
    return p;
}

// GATE: a value of la_gate.  w is 1 - a for the sigmoid gate, without
// cancellation, and 1 for the others.  The sigmoid has to be short: HBM
// delivers 3.9 values a clock and SM, and an SM issues 4 instructions a clock.
// w = 1 / (1 + e^g) is within 2^-21 of itself (bf16 data: 2^-21 (1 + |g|)); where a
// is the larger it is 1 - w, rounded once, so that an a next to 1 is not off to one
// side, where it is the smaller it is e^g w.
template <typename T, int GATE, int V>
__device__ __forceinline__ void gate_of(const Lanes<V> &g, Lanes<V> &a, Lanes<V> &w) {
    constexpr bool kFine = sizeof(T) == 4;
    if constexpr (GATE == 2) {
        const Lanes<V> e = exp_of<kFine, false, V>(g);
        w = add(e, all<V>(1.f));
#pragma unroll
        for (int v = 0; v < V; v++) w.set(v, rcp_approx(w.get(v)));
        a = fma(w, all<V>(-1.f), all<V>(1.f));
        const Lanes<V> small = mul(e, w);
#pragma unroll
        for (int v = 0; v < V; v++)
            if (g.get(v) < 0.f) a.set(v, small.get(v));
    } else {
        a = GATE == 1 ? exp_gate<kFine, V>(g) : g;
        w = all<V>(1.f);
    }
}

}  // namespace la
