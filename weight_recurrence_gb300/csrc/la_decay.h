// la_decay.h - linear attention with a decay for each head as sweeps: the one
// pattern that the forward pass and each of the three gradients are.
//
// A sweep reads rows x_i, y_i (width D) and z_i (width M) and carries a state
// (D x M).  With a = e^g, forwards:
//   out_i = c_intra sum_{j<=i} a^(i-j) (x_i.y_j) z_j + c_inter a^(i+1) x_i S
// and backwards in time, the state H entering behind the last of n tokens:
//   out_i = c_intra sum_{j>=i} a^(j-i) (x_i.y_j) z_j + c_inter a^(n-1-i) x_i H
// and the state after the sweep is
//   forwards   a^n S + c_state sum_j a^(n-1-j) y_j z_j
//   backwards  a^n H + c_state sum_j a^(j+1) y_j z_j
//
//            x     y     z     state                  c_intra c_inter c_state
//   out      q     k     v     S0 -> SN               scale   scale   1
//   dq       dout  v     k     S0 transposed          scale   scale   -
//   dv       k     q     dout  dSN -> dS0, backwards  scale   1       scale
//   dk       v     dout  q     dSN transposed, bw.    scale   1       -
//
// Few heads are cut into segments of tokens: a sweep over each segment gives
// its sum alone, a scan over the segments the state at each one's start, and
// the sweeps of all segments then run side by side.
#pragma once

#include "la_layer.h"

namespace la {

// What a state keeps over n tokens, a^n = x + y.  Next to 1 as 1 + (a^n - 1): a^n
// rounded would shorten (or lengthen) a long memory a little with every chunk.
// Else as a^n itself, which keeps its digits where it is small.
__device__ __forceinline__ float2 kept(float g, int n) {
    const float e = g * (float)n;
    return e > -0.5f ? make_float2(1.f, expm1f(e)) : make_float2(expf(e), 0.f);
}
__device__ __forceinline__ float keep(float2 a, float s) { return fmaf(a.y, s, a.x * s); }

// The same over many tokens of a state that grows, where a^n may be past fp32's range: a
// state of 0 stays 0, and a small one is not infinite before it has grown so far.  By
// a^(n/4) four times: where that too is infinite, so is the smallest number's growth.
__device__ __forceinline__ bool grows_far(float g, int n) { return g * (float)n > 80.f; }
__device__ __forceinline__ float keep_far(float g, int n, float s) {
    const float a = expf(0.25f * (g * (float)n));
    return s == 0.f ? s : s * a * a * a * a;
}

// The segment with a sequence's last token (0 where it has none).  The segments end below
// 2^31, but a token past one segment more would not.
__host__ __device__ constexpr int last_segment(int len, int seg_tokens) { return len > 0 ? (len - 1) / seg_tokens : 0; }
static_assert(last_segment(0, 128) == 0 && last_segment(128, 128) == 0 && last_segment(129, 128) == 1 &&
                  last_segment(2146435071, 7060736) == 303 && last_segment(2146435071, 2146435071) == 0,
              "lengths up to the largest");

struct DecaySweep {
    la_view x, y, z, out;      // out.data null: the state alone (x is not read)
    const float *start;        // state before the sweep, null: 0
    float *end;                // state after it, null: not wanted
    int D, M;                  // widths of x and y, of z and out
    int transposed;            // start and end lie as [M][D], else [D][M]
    int backwards;
    float c_intra, c_inter, c_state;
};

constexpr int kDecayMaxSweeps = 3;

struct DecayLaunch {
    DecaySweep sweep[kDecayMaxSweeps];
    int sweeps;
    const float *log_decay;
    const int *lens;
    int B, H, N;
    int segs, seg_tokens;      // segments of a sequence; tokens of one (a multiple of 128 if segs > 1)
    int sums;                  // every segment by itself: start 0, end at [B*H][segs][D*M]
    int starts;                // start at [B*H][segs][D*M]
    cudaStream_t stream;
};

// tensor cores (la_tc_decay.cu): bf16 rows on 16 byte boundaries
bool tc_decay_supported(const DecayLaunch &l, la_dtype dtype);
cudaError_t tc_decay(const DecayLaunch &l);

}  // namespace la
