// la_rotate.cu - norm of every head of the queries and keys and the rotation of
// their channels by the token's positions, in one pass, and its backward.
//
//   n = x rstd w,  rstd = 1/sqrt(mean(x^2) + eps);  pairs of n turned by the
//   token's angles;  backward: u = dy turned back,
//   dx = rstd (u w - xh avg(u w xh)),  dw = sum of u xh,  xh = x rstd
//
// Bound by HBM: every value is read once and written once.  A group of lanes
// keeps one token: it works out the token's angles once, in registers, and then
// walks over the heads, a head's pairs spread over the group, so that the sines
// cost a token's share of the heads and no table is read.  Neighbouring groups
// of a warp take neighbouring tokens, whose rows lie side by side.  The next
// heads' rows are on their way while some are worked on, the first ones while
// the angles are, and the weights lie in shared memory, which leaves the
// registers for it.  Measured (40 heads of 64 channels, 8 x 4096 tokens, bf16):
// forward 57 us, 5.9 of the copy's 6.8 TB/s, backward 90 us, 5.6 (without the
// rows ahead 71 and 122).  The bf16 backward takes pieces of 8 bytes, four heads
// ahead: with 16 the weights' sums leave room for one (107 us).  fp32 rows reach
// 6.4 TB/s both ways; rows by single values are bound by their instructions (16384
// tokens of 32 heads of 66 channels, bf16: 87 and 166 us, 1.6 and 1.3 TB/s; of 72
// channels, by 8 bytes, 51 and 77).
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "la_layer.h"
#include "la_pair.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = kRotateMaxD / 2;

struct RotArgs {
    const void *x[2], *dy[2];   // queries, keys
    void *y[2];                 // forward: y; backward: dx
    long long xb[2], xh[2], xn[2], yb[2], yh[2], yn[2], db[2], dh[2], dn[2];
    const float *w[2];
    int H[2];
    const int *pos;
    long long sa, sb, sn;
    const float *freq;
    int B, N, D, P;
    float eps;
    float *ws;                  // backward: [CTAs][2][D] or null
    int splits;                 // groups that share a token's heads
    int by_axis;                // positions on another axis than the first
    int half;                   // pairs P apart, else neighbours
    unsigned char axes[kMaxPairs];
};

// 2^128 / (2 pi), rounded down: its halves are turns a radian in 2^-64 and 2^-128
constexpr unsigned long long kTurnHigh = 0x28BE60DB9391054Aull, kTurnLow = 0x7F09D5F47D4D3770ull;

// f radians in 2^-64 turns, mod a turn, rounded down: f = m 2^e exactly, and the product of
// m with 1/(2 pi) to 128 bits is off by less than f 2^-128 turns.  An angle is then off by
// less than 2^-64 + |f| 2^-128 turns times its position: 2^-33 turns for the first at the
// last positions of 32 bits, as much for the second at |f| = 2^64.
__device__ __forceinline__ unsigned long long turns(float f) {
    const unsigned bits = __float_as_uint(f);
    const int field = (bits >> 23) & 255;
    const unsigned m = field ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
    const int e = (field ? field : 1) - 150;
    const unsigned __int128 low = (unsigned __int128)m * kTurnLow;
    const unsigned __int128 p = (unsigned __int128)m * kTurnHigh + (unsigned long long)(low >> 64);   // 2^-64 turns
    const unsigned long long rest = (unsigned long long)low;                                          // 2^-128
    unsigned long long t;
    if (e <= 0) t = e > -100 ? (unsigned long long)(p >> -e) : 0ull;
    else if (e < 64) t = (unsigned long long)p << e | rest >> (64 - e);
    else t = rest << (e - 64);   // at most 40
    return bits >> 31 ? 0ull - t : t;
}

// How a lane's V pairs lie in a head's row: kHalf, kAdjacent: V neighbouring pairs
// by pieces of V values, 16 bytes or (bf16, V = 4) 8; kAny: pairs a warp apart by single values.
enum Layout { kHalf, kAdjacent, kAny };
// CTAs that an SM holds: rows by pieces take the registers for their loads (three of
// them an SM: fp32 backward, 4 x 8192 tokens of 32 heads of 64, 126 -> 145 us), single values the
// warps (3 x 1234 tokens of 12 heads of 90 channels, two: 15 and 27 us, so 11 and 23).
constexpr int slots_of(Layout l, bool bwd) { return l != kAny ? 2 : bwd ? 3 : 4; }

// Channels of pair p: rotated pairs first, the channels behind them as pairs
// that do not turn.
__device__ __forceinline__ int first_of(int p, int P, bool half) { return half ? (p < P ? p : p + P) : 2 * p; }
__device__ __forceinline__ int second_of(int p, int P, int D, bool half) {
    return half ? (p < P ? p + P : p + D / 2) : 2 * p + 1;
}

// A lane's share of a row as it lies in memory: 2V values.
template <int bytes> struct Piece {
    using type = uint4;
};
template <> struct Piece<8> {
    using type = uint2;
};
template <typename T, Layout L, int V> struct Raw {
    typename Piece<V * sizeof(T)>::type w[2];
};
template <typename T, int V> struct Raw<T, kAny, V> {
    T v[2 * V];
};
// The first and the second values of its pairs, two pairs to a float2.
template <int V> struct Pairs {
    float2 a[V / 2], b[V / 2];
};

template <int V, Layout L> __device__ __forceinline__ int pair_of_lane(int lane, int i) {
    return L == kAny ? lane + 32 * i : V * lane + i;
}

// Two pairs (a, b), turned.
__device__ __forceinline__ void turn(float2 a, float2 b, float2 c, float2 s, float2 &ta, float2 &tb) {
    const float2 bs = mul_pair(b, s);
    ta = fma_pair(a, c, make_float2(-bs.x, -bs.y));
    tb = fma_pair(b, c, mul_pair(a, s));
}
// The same where pairs may not turn (x, y: whether they do), the channels behind the
// rotated ones: these leave as they came.  With cos 1 and sin 0 a value that is not
// finite would reach the other channel as 0 times itself, so a zero takes its place (of
// the sign that adds nothing to a zero of either).  By kernels of their own, as that
// costs registers (2 x 16384 tokens of 32 heads of 128, bf16, half of the channels: 86 ->
// 90 us forward, 142 -> 145 backward; in one kernel for both, rows that turn as a whole
// paid 1 to 4 % too).
__device__ __forceinline__ void turn_some(float2 a, float2 b, float2 c, float2 s, bool x, bool y, float2 &ta, float2 &tb) {
    const float2 bs = mul_pair(make_float2(x ? b.x : 0.f, y ? b.y : 0.f), s);
    const float2 as = mul_pair(make_float2(x ? a.x : -0.f, y ? a.y : -0.f), s);
    ta = fma_pair(a, c, make_float2(-bs.x, -bs.y));
    tb = fma_pair(b, c, as);
}
// A lane's pairs, turned; back: by the angles' negatives; ALL: every channel turns.
template <int V, Layout L, bool back, bool ALL>
__device__ __forceinline__ void turn_pairs(const Pairs<V> &v, const float2 (&c)[V / 2], const float2 (&s)[V / 2], int lane,
                                           int P, Pairs<V> &o) {
    const auto &a = back ? v.b : v.a, &b = back ? v.a : v.b;
    auto &ta = back ? o.b : o.a, &tb = back ? o.a : o.b;
    [[maybe_unused]] const int left = P - pair_of_lane<V, L>(lane, 0);
    if constexpr (ALL) {
#pragma unroll
        for (int i = 0; i < V / 2; i++) turn(a[i], b[i], c[i], s[i], ta[i], tb[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; i++) {   // halves by pieces: P is a multiple of V
            const bool x = pair_of_lane<V, L>(0, L == kHalf ? 0 : 2 * i) < left;
            const bool y = L == kHalf ? x : pair_of_lane<V, L>(0, 2 * i + 1) < left;
            turn_some(a[i], b[i], c[i], s[i], x, y, ta[i], tb[i]);
        }
    }
}

template <typename T, Layout L, int V>
__device__ __forceinline__ Raw<T, L, V> load_raw(const T *row, int lane, int P, int D, bool half) {
    Raw<T, L, V> r;
    if constexpr (L == kAny) {
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int p = lane + 32 * i;
            r.v[2 * i] = r.v[2 * i + 1] = from_f32<T>(0.f);
            if (p < D / 2) {
                r.v[2 * i] = row[first_of(p, P, half)];
                r.v[2 * i + 1] = row[second_of(p, P, D, half)];
            }
        }
    } else {
        static_assert(V * sizeof(T) == 16 || V * sizeof(T) == 8, "a piece is V values");
        using piece = typename Piece<V * sizeof(T)>::type;
        const int p = V * lane;
        const bool in = p < D / 2;
        const T *x = row + (L == kHalf ? first_of(p, P, true) : 2 * p);
        const T *y = L == kHalf ? row + second_of(p, P, D, true) : x + V;
        r.w[0] = in ? *reinterpret_cast<const piece *>(x) : piece{};
        r.w[1] = in ? *reinterpret_cast<const piece *>(y) : piece{};
    }
    return r;
}

__device__ __forceinline__ float2 floats(unsigned x, unsigned y) {
    return make_float2(__uint_as_float(x), __uint_as_float(y));
}

template <typename T, Layout L, int V> __device__ __forceinline__ Pairs<V> pairs_of(const Raw<T, L, V> &r) {
    Pairs<V> o;
    if constexpr (L == kAny) {
#pragma unroll
        for (int i = 0; i < V / 2; i++) {
            o.a[i] = make_float2(to_f32(r.v[4 * i]), to_f32(r.v[4 * i + 2]));
            o.b[i] = make_float2(to_f32(r.v[4 * i + 1]), to_f32(r.v[4 * i + 3]));
        }
    } else {
        const auto x = r.w[0], y = r.w[1];
        if constexpr (sizeof(T) * V == 8) {
            if constexpr (L == kHalf) {
                o.a[0] = get_pair(x.x), o.a[1] = get_pair(x.y);
                o.b[0] = get_pair(y.x), o.b[1] = get_pair(y.y);
            } else {
                o.a[0] = floats(x.x << 16, x.y << 16), o.b[0] = floats(x.x & 0xffff0000u, x.y & 0xffff0000u);
                o.a[1] = floats(y.x << 16, y.y << 16), o.b[1] = floats(y.x & 0xffff0000u, y.y & 0xffff0000u);
            }
        } else if constexpr (sizeof(T) == 4) {
            if constexpr (L == kHalf) {
                o.a[0] = floats(x.x, x.y), o.a[1] = floats(x.z, x.w);
                o.b[0] = floats(y.x, y.y), o.b[1] = floats(y.z, y.w);
            } else {
                o.a[0] = floats(x.x, x.z), o.b[0] = floats(x.y, x.w);
                o.a[1] = floats(y.x, y.z), o.b[1] = floats(y.y, y.w);
            }
        } else if constexpr (L == kHalf) {
            o.a[0] = get_pair(x.x), o.a[1] = get_pair(x.y), o.a[2] = get_pair(x.z), o.a[3] = get_pair(x.w);
            o.b[0] = get_pair(y.x), o.b[1] = get_pair(y.y), o.b[2] = get_pair(y.z), o.b[3] = get_pair(y.w);
        } else {   // a word holds a pair
            o.a[0] = floats(x.x << 16, x.y << 16), o.b[0] = floats(x.x & 0xffff0000u, x.y & 0xffff0000u);
            o.a[1] = floats(x.z << 16, x.w << 16), o.b[1] = floats(x.z & 0xffff0000u, x.w & 0xffff0000u);
            o.a[2] = floats(y.x << 16, y.y << 16), o.b[2] = floats(y.x & 0xffff0000u, y.y & 0xffff0000u);
            o.a[3] = floats(y.z << 16, y.w << 16), o.b[3] = floats(y.z & 0xffff0000u, y.w & 0xffff0000u);
        }
    }
    return o;
}

template <typename T, Layout L, int V>
__device__ __forceinline__ void store_pairs(T *row, const Pairs<V> &v, int lane, int P, int D, bool half) {
    if constexpr (L == kAny) {
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int p = lane + 32 * i;
            if (p < D / 2) {
                row[first_of(p, P, half)] = from_f32<T>(i % 2 ? v.a[i / 2].y : v.a[i / 2].x);
                row[second_of(p, P, D, half)] = from_f32<T>(i % 2 ? v.b[i / 2].y : v.b[i / 2].x);
            }
        }
    } else {
        const int p = V * lane;
        if (p >= D / 2) return;
        T *x = row + (L == kHalf ? first_of(p, P, true) : 2 * p);
        T *y = L == kHalf ? row + second_of(p, P, D, true) : x + V;
        [[maybe_unused]] auto word = [&](int i) {
            return i % 2 ? put_pair(make_float2(v.a[i / 2].y, v.b[i / 2].y)) : put_pair(make_float2(v.a[i / 2].x, v.b[i / 2].x));
        };
        if constexpr (sizeof(T) * V == 8) {
            if constexpr (L == kHalf) {
                *reinterpret_cast<uint2 *>(x) = make_uint2(put_pair(v.a[0]), put_pair(v.a[1]));
                *reinterpret_cast<uint2 *>(y) = make_uint2(put_pair(v.b[0]), put_pair(v.b[1]));
            } else {
                *reinterpret_cast<uint2 *>(x) = make_uint2(word(0), word(1));
                *reinterpret_cast<uint2 *>(y) = make_uint2(word(2), word(3));
            }
        } else if constexpr (sizeof(T) == 4) {
            if constexpr (L == kHalf) {
                *reinterpret_cast<float4 *>(x) = make_float4(v.a[0].x, v.a[0].y, v.a[1].x, v.a[1].y);
                *reinterpret_cast<float4 *>(y) = make_float4(v.b[0].x, v.b[0].y, v.b[1].x, v.b[1].y);
            } else {
                *reinterpret_cast<float4 *>(x) = make_float4(v.a[0].x, v.b[0].x, v.a[0].y, v.b[0].y);
                *reinterpret_cast<float4 *>(y) = make_float4(v.a[1].x, v.b[1].x, v.a[1].y, v.b[1].y);
            }
        } else if constexpr (L == kHalf) {
            *reinterpret_cast<uint4 *>(x) = make_uint4(put_pair(v.a[0]), put_pair(v.a[1]), put_pair(v.a[2]), put_pair(v.a[3]));
            *reinterpret_cast<uint4 *>(y) = make_uint4(put_pair(v.b[0]), put_pair(v.b[1]), put_pair(v.b[2]), put_pair(v.b[3]));
        } else {
            *reinterpret_cast<uint4 *>(x) = make_uint4(word(0), word(1), word(2), word(3));
            *reinterpret_cast<uint4 *>(y) = make_uint4(word(4), word(5), word(6), word(7));
        }
    }
}

template <int G> __device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int d = G / 2; d > 0; d /= 2) x += __shfl_xor_sync(0xffffffffu, x, d, G);
    return x;
}

// cos and sin of the lane's pairs for the token's positions.  With fp32 data by
// sincospi (2 ulp), with bf16 data by the SFU's, 2^-21 off within a turn.
template <typename T, int V, Layout L>
__device__ __forceinline__ void angles(const RotArgs &a, int lane, long long at, const unsigned long long *turn,
                                       unsigned bad, float2 (&cs)[V / 2], float2 (&sn)[V / 2]) {
    const int p0 = a.P > 0 ? a.pos[at] : 0;
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int p = pair_of_lane<V, L>(lane, i);
        float c = 1.f, s = 0.f;
        if (p < a.P) {
            const int x = a.by_axis ? a.pos[at + a.axes[p] * a.sa] : p0;
            const unsigned long long u = (unsigned long long)(long long)x * turn[p];
            const float half_turns = (float)(int)((u + 0x80000000ull) >> 32) * 0x1p-31f;
            if constexpr (sizeof(T) == 4) {
                sincospif(half_turns, &s, &c);
            } else {
                s = __sinf(half_turns * 3.14159265f);
                c = __cosf(half_turns * 3.14159265f);
            }
            if (bad >> i & 1) s = c = __int_as_float(0x7fffffff);
        }
        (i % 2 ? cs[i / 2].y : cs[i / 2].x) = c;
        (i % 2 ? sn[i / 2].y : sn[i / 2].x) = s;
    }
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// G lanes to a token; BWD: the gradients; NORM: with the norm; ALL: no channels behind the
// rotated ones.  U heads are worked on while the next U are on their way.
template <typename T, int V, int G, Layout L, bool BWD, bool NORM, bool ALL>
__global__ void __launch_bounds__(kThreads, slots_of(L, BWD)) rotate_kernel(const __grid_constant__ RotArgs a) {
    constexpr int U = L == kAny ? (BWD ? 1 : 2) : BWD && sizeof(T) == 4 ? 2 : 4, E = V / 2;
    const int lane = threadIdx.x % G, D = a.D, P = a.P;
    const bool half = L == kHalf || (L == kAny && a.half);
    const unsigned groups = gridDim.x * (kThreads / G), tokens = (unsigned)a.B * a.N, items = tokens * a.splits;
    const float mean = 1.f / (float)D;
    __shared__ unsigned long long turn[kMaxPairs];   // of every pair, a position
    // the weights, by lanes: first and second values of a lane's pairs, two pairs to a piece
    __shared__ float4 weights[NORM ? 2 : 1][NORM ? E : 1][NORM ? G : 1];
    if constexpr (NORM) {
        for (int i = threadIdx.x; i < 2 * E * G; i += kThreads) {
            const int s = i / (E * G), e = i / G % E, ln = i % G;
            const int p = pair_of_lane<V, L>(ln, 2 * e), q = pair_of_lane<V, L>(ln, 2 * e + 1);
            auto at = [&](int c) { return a.w[s] ? a.w[s][c] : 1.f; };
            float4 v = make_float4(1.f, 1.f, 1.f, 1.f);
            if (p < D / 2) v.x = at(first_of(p, P, half)), v.z = at(second_of(p, P, D, half));
            if (q < D / 2) v.y = at(first_of(q, P, half)), v.w = at(second_of(q, P, D, half));
            weights[s][e][ln] = v;
        }
    }
    unsigned bad = 0;
    float2 dwa[BWD && NORM ? E : 1], dwb[BWD && NORM ? E : 1];
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int p = pair_of_lane<V, L>(lane, i);
        const float f = p < P ? a.freq[p] : 0.f;
        bad |= (f - f != 0.f ? 1u : 0u) << i;
    }
#pragma unroll
    for (int i = 0; i < (BWD && NORM ? E : 1); i++) dwa[i] = dwb[i] = both(0.f);
    if (threadIdx.x < P) turn[threadIdx.x] = turns(a.freq[threadIdx.x]);
    __syncthreads();
    // every group of a warp walks the same number of times: the sums' shuffles take whole
    // warps (at most 2^31 items, so nothing below wraps)
    const unsigned first = blockIdx.x * (kThreads / G) + threadIdx.x / G;
    const unsigned warp_first = blockIdx.x * (kThreads / G) + threadIdx.x / 32 * (32 / G);
    for (unsigned it = first, wit = warp_first; wit < items; it += groups, wit += groups) {
        const bool live = it < items;
        const unsigned split = live ? it / tokens : 0u, token = live ? it - split * tokens : 0u;
        const unsigned bu = token / a.N;
        const long long b = bu, n = token - bu * a.N;
        // forward a token's queries and then its keys; backward each by CTAs of its own, whose
        // threads have room for one side's sums
        const int s0 = BWD ? blockIdx.y : 0, H0 = a.H[s0], H = BWD ? H0 : H0 + a.H[1], step = U * a.splits;
        const T *x0 = static_cast<const T *>(a.x[s0]) + b * a.xb[s0] + n * a.xn[s0];
        const T *x1 = BWD ? static_cast<const T *>(a.dy[s0]) + b * a.db[s0] + n * a.dn[s0]
                          : static_cast<const T *>(a.x[1]) + b * a.xb[1] + n * a.xn[1];
        T *y0 = static_cast<T *>(a.y[s0]) + b * a.yb[s0] + n * a.yn[s0];
        T *y1 = BWD ? nullptr : static_cast<T *>(a.y[1]) + b * a.yb[1] + n * a.yn[1];
        Raw<T, L, V> nx[U], nd[U];
        auto fetch = [&](int h0) {
#pragma unroll
            for (int j = 0; j < U; j++) {
                const int h = h0 + j * a.splits + (int)split, hh = live && h < H ? h : 0;   // one that is not there: read, not used
                if constexpr (BWD) {
                    if (NORM) nx[j] = load_raw<T, L, V>(x0 + hh * a.xh[s0], lane, P, D, half);
                    nd[j] = load_raw<T, L, V>(x1 + hh * a.dh[s0], lane, P, D, half);
                } else {
                    nx[j] = load_raw<T, L, V>(hh < H0 ? x0 + hh * a.xh[0] : x1 + (hh - H0) * a.xh[1], lane, P, D, half);
                }
            }
        };
        if (H > 0) fetch(0);
        float2 cs[E], sn[E];
        angles<T, V, L>(a, lane, b * a.sb + n * a.sn, turn, bad, cs, sn);
#pragma unroll 1
        for (int h0 = 0; h0 < H; h0 += step) {
            Raw<T, L, V> rx[U], rd[U];
#pragma unroll
            for (int j = 0; j < U; j++) rx[j] = nx[j], rd[j] = nd[j];
            if (h0 + step < H) fetch(h0 + step);   // the next heads on their way
#pragma unroll
            for (int j = 0; j < U; j++) {
                const int h = h0 + j * a.splits + (int)split;
                const bool on = live && h < H;
                const int s = BWD ? s0 : h >= H0;
                Pairs<V> v, o;
                float rstd = 1.f;
                if (NORM || !BWD) v = pairs_of<T, L, V>(rx[j]);
                if constexpr (NORM) {
                    float2 sum = both(0.f);
#pragma unroll
                    for (int i = 0; i < E; i++)
                        sum = fma_pair(v.a[i], v.a[i], fma_pair(v.b[i], v.b[i], sum));
                    rstd = rsqrtf(fmaf(group_sum<G>(sum.x + sum.y), mean, a.eps));
                }
                if constexpr (!BWD) {
                    if constexpr (NORM) {
#pragma unroll
                        for (int i = 0; i < E; i++) {
                            const float4 w = weights[s][i][lane];
                            v.a[i] = mul_pair(mul_pair(v.a[i], both(rstd)), make_float2(w.x, w.y));
                            v.b[i] = mul_pair(mul_pair(v.b[i], both(rstd)), make_float2(w.z, w.w));
                        }
                    }
                    turn_pairs<V, L, false, ALL>(v, cs, sn, lane, P, o);
                } else {
                    const Pairs<V> d = pairs_of<T, L, V>(rd[j]);
                    Pairs<V> u;
                    turn_pairs<V, L, true, ALL>(d, cs, sn, lane, P, u);
                    if constexpr (!NORM) {
                        o = u;
                    } else {
                        const float2 r = both(rstd);
                        float2 dot2 = both(0.f);
#pragma unroll
                        for (int i = 0; i < E; i++) {
                            v.a[i] = mul_pair(v.a[i], r), v.b[i] = mul_pair(v.b[i], r);
                            if (on) {   // a head that is not there adds nothing
                                dwa[i] = fma_pair(u.a[i], v.a[i], dwa[i]);
                                dwb[i] = fma_pair(u.b[i], v.b[i], dwb[i]);
                            }
                            const float4 w = weights[s][i][lane];
                            u.a[i] = mul_pair(u.a[i], make_float2(w.x, w.y));
                            u.b[i] = mul_pair(u.b[i], make_float2(w.z, w.w));
                            dot2 = fma_pair(u.a[i], v.a[i], fma_pair(u.b[i], v.b[i], dot2));
                        }
                        const float2 dot = both(-group_sum<G>(dot2.x + dot2.y) * mean);
#pragma unroll
                        for (int i = 0; i < E; i++) {
                            o.a[i] = mul_pair(r, fma_pair(v.a[i], dot, u.a[i]));
                            o.b[i] = mul_pair(r, fma_pair(v.b[i], dot, u.b[i]));
                        }
                    }
                }
                if (on) store_pairs<T, L, V>(BWD || s == 0 ? y0 + h * a.yh[s0] : y1 + (h - H0) * a.yh[1], o, lane, P, D, half);
            }
        }
    }
    if constexpr (BWD && NORM) {
        if (a.ws == nullptr) return;
        // the groups' sums of this CTA, added in the groups' order
        extern __shared__ float sums[];   // [groups][D]
        float *mine = sums + (size_t)(threadIdx.x / G) * D;
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int p = pair_of_lane<V, L>(lane, i);
            if (p < D / 2) {
                mine[first_of(p, P, half)] = i % 2 ? dwa[i / 2].y : dwa[i / 2].x;
                mine[second_of(p, P, D, half)] = i % 2 ? dwb[i / 2].y : dwb[i / 2].x;
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += kThreads) {
            float t = 0.f;
            for (int g = 0; g < kThreads / G; g++) t += sums[(size_t)g * D + c];
            a.ws[((size_t)blockIdx.x * 2 + blockIdx.y) * D + c] = t;
        }
    }
}

// Columns of the CTAs' sums [n][2D]: 32 columns to a CTA, rows over its 32 warps, whose
// loads are all on their way at once.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps) weight_sums_kernel(const float *ws, int n, int D, float *dwq, float *dwk) {
    __shared__ float part[kSumWarps][33];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    float t = 0.f;
    if (c < 2 * D)
#pragma unroll 10
        for (int r = warp; r < n; r += kSumWarps) t += ws[(size_t)r * 2 * D + c];
    part[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && c < 2 * D) {
#pragma unroll
        for (int i = 1; i < kSumWarps; i++) t += part[i][lane];
        float *dst = c < D ? dwq : dwk;
        if (dst) dst[c < D ? c : c - D] = t;
    }
}

constexpr int kSms = 152;
constexpr int kBwdCtas = kSms * 2;   // for each of queries and keys; their sums are written: few, that stay

bool on_boundary(const void *p, long long b, long long h, long long n, size_t bytes, size_t piece) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(b * bytes) | (uintptr_t)(h * bytes) |
                             (uintptr_t)(n * bytes)) & (piece - 1)) == 0;
}

template <typename T, int V, int G, Layout L, bool BWD>
cudaError_t launch(const RotArgs &a, int ctas, bool norm, cudaStream_t st) {
    const size_t smem = BWD && norm && a.ws ? (size_t)(kThreads / G) * a.D * sizeof(float) : 0;
    const dim3 grid(ctas, BWD ? 2 : 1);
    auto run = [&](auto with, auto all) {
        rotate_kernel<T, V, G, L, BWD, with.value, all.value><<<grid, kThreads, smem, st>>>(a);
    };
    constexpr std::true_type yes;
    constexpr std::false_type no;
    if (norm) 2 * a.P == a.D ? run(yes, yes) : run(yes, no);
    else 2 * a.P == a.D ? run(no, yes) : run(no, no);
    count_launches(1);
    return cudaGetLastError();
}

// Lanes to a token where rows are taken by pieces of V values: what D takes, rounded up.
int lanes_of(int D, int V) { return (D <= 64 ? 32 : D <= 128 ? 64 : 128) / V; }

template <typename T, int V, Layout L, bool BWD>
cudaError_t pick_lanes(const RotArgs &a, int ctas, bool norm, cudaStream_t st) {
    constexpr int least = 32 / V;   // D = 64
    if (a.D <= 64) return launch<T, V, least, L, BWD>(a, ctas, norm, st);
    return a.D <= 128 ? launch<T, V, 2 * least, L, BWD>(a, ctas, norm, st) : launch<T, V, 4 * least, L, BWD>(a, ctas, norm, st);
}

template <typename T, bool BWD> cudaError_t pick(const RotArgs &a, Layout l, int V, int ctas, bool norm, cudaStream_t st) {
    if (l == kAny) return a.D <= 128 ? launch<T, 2, 32, kAny, BWD>(a, ctas, norm, st) : launch<T, 4, 32, kAny, BWD>(a, ctas, norm, st);
    if constexpr (sizeof(T) == 2 && !BWD)
        if (V == 8) return l == kHalf ? pick_lanes<T, 8, kHalf, BWD>(a, ctas, norm, st) : pick_lanes<T, 8, kAdjacent, BWD>(a, ctas, norm, st);
    return l == kHalf ? pick_lanes<T, 4, kHalf, BWD>(a, ctas, norm, st) : pick_lanes<T, 4, kAdjacent, BWD>(a, ctas, norm, st);
}

cudaError_t rotate(const RotateProblem &p, bool bwd) {
    RotArgs a{};
    const bool half = p.rot.pairs == LA_PAIRS_HALF;
    const la_view x[2] = {p.q, p.k}, y[2] = {p.qo, p.ko}, dy[2] = {p.dqo, p.dko};
    const size_t size = p.s.dtype == LA_DTYPE_F32 ? 4 : 2;
    // pieces of 16 bytes where every row allows them; for bf16 else, and backward, of 8
    bool wide[2];   // pieces of 16 and of 8 bytes
    for (int i = 0; i < 2; i++) {
        const int V = (16 >> i) / (int)size;
        wide[i] = V >= 4 && p.s.D % (2 * V) == 0 && (!half || p.rot.P % V == 0);
    }
    for (int s = 0; s < 2; s++) {
        a.H[s] = s ? p.s.Hk : p.s.Hq;
        a.x[s] = x[s].data, a.y[s] = y[s].data, a.dy[s] = dy[s].data;
        a.xb[s] = x[s].sb, a.xh[s] = x[s].sh, a.xn[s] = x[s].sn;
        a.yb[s] = y[s].sb, a.yh[s] = y[s].sh, a.yn[s] = y[s].sn;
        a.db[s] = dy[s].sb, a.dh[s] = dy[s].sh, a.dn[s] = dy[s].sn;
        a.w[s] = s ? p.wk : p.wq;
        if (a.H[s] == 0) continue;
        for (int i = 0; i < 2; i++)
            wide[i] = wide[i] && on_boundary(x[s].data, x[s].sb, x[s].sh, x[s].sn, size, 16 >> i) &&
                      on_boundary(y[s].data, y[s].sb, y[s].sh, y[s].sn, size, 16 >> i) &&
                      (!bwd || on_boundary(dy[s].data, dy[s].sb, dy[s].sh, dy[s].sn, size, 16 >> i));
    }
    a.pos = p.rot.pos, a.sa = p.rot.sa, a.sb = p.rot.sb, a.sn = p.rot.sn, a.freq = p.rot.freq;
    a.B = p.s.B, a.N = p.s.N, a.D = p.s.D, a.P = p.rot.P, a.eps = p.eps;
    if (p.rot.axes && p.rot.P) {
        memcpy(a.axes, p.rot.axes, p.rot.P);
        for (int i = 0; i < p.rot.P; i++) a.by_axis |= p.rot.axes[i] != 0;
    }
    // else single values, 32 lanes to a token
    const Layout l = !wide[0] && !wide[1] ? kAny : half ? kHalf : kAdjacent;
    const int V = size == 2 && wide[0] && !bwd ? 8 : 4;
    a.half = half;
    const int G = l == kAny ? 32 : lanes_of(p.s.D, V);
    const long long tokens = (long long)p.s.B * p.s.N, per = kThreads / G;
    // a token's heads are shared by as many groups as fill the SMs at once, and no more
    // (4096 tokens of 32 heads of 64: 9.4 and 16.7 us, with twice as many 11.8 and 21.3)
    const int heads = bwd ? std::max(p.s.Hq, p.s.Hk) : p.s.Hq + p.s.Hk;
    long long splits = 1;
    while (splits < heads && tokens * splits * 2 <= (long long)kSms * slots_of(l, bwd) / (bwd ? 2 : 1) * per) splits *= 2;
    a.splits = (int)splits;
    const bool sums = bwd && p.norm && (p.dwq || p.dwk);
    a.ws = sums ? static_cast<float *>(p.ws) : nullptr;
    const long long ctas = std::min((tokens * splits + per - 1) / per, bwd && p.norm ? (long long)kBwdCtas : 1LL << 30);
    const bool f32 = p.s.dtype == LA_DTYPE_F32;
    cudaError_t e = bwd ? (f32 ? pick<float, true>(a, l, V, (int)ctas, p.norm, p.stream)
                               : pick<__nv_bfloat16, true>(a, l, V, (int)ctas, p.norm, p.stream))
                        : (f32 ? pick<float, false>(a, l, V, (int)ctas, p.norm, p.stream)
                               : pick<__nv_bfloat16, false>(a, l, V, (int)ctas, p.norm, p.stream));
    if (e != cudaSuccess || !sums) return e;
    weight_sums_kernel<<<(2 * p.s.D + 31) / 32, 32 * kSumWarps, 0, p.stream>>>(a.ws, (int)ctas, p.s.D, p.dwq, p.dwk);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

size_t rotate_ws_bytes(const la_qk_shape &s) { return (size_t)kBwdCtas * 2 * s.D * sizeof(float); }
cudaError_t rotate_forward(const RotateProblem &p) { return rotate(p, false); }
cudaError_t rotate_backward(const RotateProblem &p) { return rotate(p, true); }

}  // namespace la
