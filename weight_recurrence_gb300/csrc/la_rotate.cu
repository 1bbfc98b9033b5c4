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
// of a warp take neighbouring tokens, whose rows lie side by side.
#include <algorithm>
#include <cstring>

#include "la_layer.h"
#include "la_pair.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = kRotateMaxD / 2;
constexpr int kMaxAxes = 8;

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

// 2^64 / (2 pi): a position's turn of 2^64 parts per radian
constexpr unsigned long long kTurn = 0x28BE60DB9391054Aull;

// f radians in 2^-64 turns, mod a turn: f = m 2^e exactly, so the product with
// kTurn (its error 2^-62 of itself) and a shift give every bit that counts.
__device__ __forceinline__ unsigned long long turns(float f) {
    const unsigned bits = __float_as_uint(f);
    const int field = (bits >> 23) & 255;
    const unsigned m = field ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
    const int e = (field ? field : 1) - 150;
    const unsigned __int128 p = (unsigned __int128)m * kTurn;
    unsigned long long t;
    if (e >= 0) t = e < 64 ? (unsigned long long)p << e : 0ull;
    else t = e > -100 ? (unsigned long long)(p >> -e) : 0ull;
    return bits >> 31 ? 0ull - t : t;
}

// How a lane's four pairs lie in a head's row: kHalf, kAdjacent: four
// neighbouring pairs by 8 or 16 byte accesses; kAny: pairs a warp apart by
// single values.
enum Layout { kHalf, kAdjacent, kAny };

// Channels of pair p: rotated pairs first, the channels behind them as pairs
// that do not turn.
__device__ __forceinline__ int first_of(int p, int P, bool half) { return half ? (p < P ? p : p + P) : 2 * p; }
__device__ __forceinline__ int second_of(int p, int P, int D, bool half) {
    return half ? (p < P ? p + P : p + D / 2) : 2 * p + 1;
}

// A lane's share of a row as it lies in memory: eight values.
template <typename T, Layout L> struct Raw {
    uint4 w[sizeof(T) == 4 ? 2 : 1];
};
template <typename T> struct Raw<T, kAny> {
    T v[8];
};

template <typename T, Layout L>
__device__ __forceinline__ Raw<T, L> load_raw(const T *row, int lane, int P, int D, bool half) {
    Raw<T, L> r;
    if constexpr (L == kAny) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int p = lane + 32 * i;
            r.v[2 * i] = r.v[2 * i + 1] = from_f32<T>(0.f);
            if (p < D / 2) {
                r.v[2 * i] = row[first_of(p, P, half)];
                r.v[2 * i + 1] = row[second_of(p, P, D, half)];
            }
        }
    } else {
        const int p = 4 * lane;
        const bool in = p < D / 2;
        if constexpr (L == kAdjacent) {
            const uint4 *s = reinterpret_cast<const uint4 *>(row + 2 * p);
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; i++) r.w[i] = in ? s[i] : make_uint4(0, 0, 0, 0);
        } else if constexpr (sizeof(T) == 4) {
            r.w[0] = in ? *reinterpret_cast<const uint4 *>(row + first_of(p, P, true)) : make_uint4(0, 0, 0, 0);
            r.w[1] = in ? *reinterpret_cast<const uint4 *>(row + second_of(p, P, D, true)) : make_uint4(0, 0, 0, 0);
        } else {
            const uint2 z = make_uint2(0, 0);
            const uint2 a = in ? *reinterpret_cast<const uint2 *>(row + first_of(p, P, true)) : z;
            const uint2 b = in ? *reinterpret_cast<const uint2 *>(row + second_of(p, P, D, true)) : z;
            r.w[0] = make_uint4(a.x, a.y, b.x, b.y);
        }
    }
    return r;
}

// pair i of the lane's four, in fp32
template <typename T, Layout L> __device__ __forceinline__ float2 pair_of(const Raw<T, L> &r, int i) {
    if constexpr (L == kAny) {
        return make_float2(to_f32(r.v[2 * i]), to_f32(r.v[2 * i + 1]));
    } else if constexpr (sizeof(T) == 4) {
        if constexpr (L == kAdjacent) {
            const uint4 q = r.w[i / 2];
            return i % 2 ? make_float2(__uint_as_float(q.z), __uint_as_float(q.w))
                         : make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
        } else {
            const unsigned a = i == 0 ? r.w[0].x : i == 1 ? r.w[0].y : i == 2 ? r.w[0].z : r.w[0].w;
            const unsigned b = i == 0 ? r.w[1].x : i == 1 ? r.w[1].y : i == 2 ? r.w[1].z : r.w[1].w;
            return make_float2(__uint_as_float(a), __uint_as_float(b));
        }
    } else {
        const uint4 q = r.w[0];
        if constexpr (L == kAdjacent) {
            return get_pair(i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w);
        } else {
            const float2 a = get_pair(i < 2 ? q.x : q.y), b = get_pair(i < 2 ? q.z : q.w);
            return i % 2 ? make_float2(a.y, b.y) : make_float2(a.x, b.x);
        }
    }
}

template <typename T, Layout L>
__device__ __forceinline__ void store_pairs(T *row, const float2 (&v)[4], int lane, int P, int D, bool half) {
    if constexpr (L == kAny) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int p = lane + 32 * i;
            if (p < D / 2) {
                row[first_of(p, P, half)] = from_f32<T>(v[i].x);
                row[second_of(p, P, D, half)] = from_f32<T>(v[i].y);
            }
        }
    } else {
        const int p = 4 * lane;
        if (p >= D / 2) return;
        if constexpr (sizeof(T) == 4) {
            if constexpr (L == kAdjacent) {
                float4 *d = reinterpret_cast<float4 *>(row + 2 * p);
                d[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
                d[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
            } else {
                *reinterpret_cast<float4 *>(row + first_of(p, P, true)) = make_float4(v[0].x, v[1].x, v[2].x, v[3].x);
                *reinterpret_cast<float4 *>(row + second_of(p, P, D, true)) = make_float4(v[0].y, v[1].y, v[2].y, v[3].y);
            }
        } else if constexpr (L == kAdjacent) {
            *reinterpret_cast<uint4 *>(row + 2 * p) =
                make_uint4(put_pair(v[0]), put_pair(v[1]), put_pair(v[2]), put_pair(v[3]));
        } else {
            *reinterpret_cast<uint2 *>(row + first_of(p, P, true)) =
                make_uint2(put_pair(make_float2(v[0].x, v[1].x)), put_pair(make_float2(v[2].x, v[3].x)));
            *reinterpret_cast<uint2 *>(row + second_of(p, P, D, true)) =
                make_uint2(put_pair(make_float2(v[0].y, v[1].y)), put_pair(make_float2(v[2].y, v[3].y)));
        }
    }
}

template <int G> __device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int d = G / 2; d > 0; d /= 2) x += __shfl_xor_sync(0xffffffffu, x, d, G);
    return x;
}

// cos and sin of the lane's four pairs for the token's positions
template <int G, Layout L>
__device__ __forceinline__ void angles(const RotArgs &a, int lane, long long at, const unsigned long long (&turn)[4],
                                       const float (&bad)[4], float2 (&cs)[4]) {
    const int p0 = a.pos[at];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int p = L == kAny ? lane + 32 * i : 4 * lane + i;
        cs[i] = make_float2(1.f, 0.f);
        if (p < a.P) {
            const int x = a.by_axis ? a.pos[at + a.axes[p] * a.sa] : p0;
            const unsigned long long u = (unsigned long long)(long long)x * turn[i];
            const float half_turns = (float)(int)((u + 0x80000000ull) >> 32) * 0x1p-31f;
            float s, c;
            sincospif(half_turns, &s, &c);
            cs[i] = make_float2(c + bad[i], s + bad[i]);
        }
    }
}

__device__ __forceinline__ float2 turned(float2 v, float2 cs) {
    return make_float2(v.x * cs.x - v.y * cs.y, v.y * cs.x + v.x * cs.y);
}
__device__ __forceinline__ float2 turned_back(float2 v, float2 cs) {
    return make_float2(v.x * cs.x + v.y * cs.y, v.y * cs.x - v.x * cs.y);
}

// G lanes to a token; BWD: the gradients; NORM: with the norm.  U heads are on
// their way at a time.
template <typename T, int G, Layout L, bool BWD, bool NORM>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const RotArgs a) {
    constexpr int U = BWD ? 2 : 4;
    const int lane = threadIdx.x % G, D = a.D, P = a.P;
    const bool half = L == kHalf || (L == kAny && a.half);
    const long long groups = (long long)gridDim.x * (kThreads / G);
    const long long tokens = (long long)a.B * a.N, items = tokens * a.splits;
    unsigned long long turn[4];
    float bad[4];
    float2 w[2][4], dw[2][4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int p = L == kAny ? lane + 32 * i : 4 * lane + i;
        const float f = p < P ? a.freq[p] : 0.f;
        turn[i] = turns(f);
        bad[i] = f - f;
#pragma unroll
        for (int s = 0; s < 2; s++) {
            dw[s][i] = make_float2(0.f, 0.f);
            w[s][i] = NORM && a.w[s] && p < D / 2
                          ? make_float2(a.w[s][first_of(p, P, half)], a.w[s][second_of(p, P, D, half)])
                          : make_float2(1.f, 1.f);
        }
    }
    // every group of a warp walks the same number of times: the sums' shuffles take whole warps
    const long long first = (long long)blockIdx.x * (kThreads / G) + threadIdx.x / G;
    const long long warp_first = (long long)blockIdx.x * (kThreads / G) + threadIdx.x / 32 * (32 / G);
    for (long long it = first, wit = warp_first; wit < items; it += groups, wit += groups) {
        const bool live = it < items;
        const long long token = live ? it % tokens : 0;
        const int split = live ? (int)(it / tokens) : 0;
        const long long b = token / a.N, n = token - b * a.N;
        float2 cs[4];
        if (P > 0) {
            angles<G, L>(a, lane, b * a.sb + n * a.sn, turn, bad, cs);
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) cs[i] = make_float2(1.f, 0.f);
        }
#pragma unroll
        for (int s = 0; s < 2; s++) {
            const T *x = static_cast<const T *>(a.x[s]) + b * a.xb[s] + n * a.xn[s];
            const T *dy = BWD ? static_cast<const T *>(a.dy[s]) + b * a.db[s] + n * a.dn[s] : nullptr;
            T *y = static_cast<T *>(a.y[s]) + b * a.yb[s] + n * a.yn[s];
            const int H = a.H[s];
            for (int h0 = 0; h0 < H; h0 += U * a.splits) {
                Raw<T, L> rx[U], rd[U];
#pragma unroll
                for (int j = 0; j < U; j++) {
                    const int h = h0 + j * a.splits + split;
                    const bool on = live && h < H;
                    // a head that is not there: the row's own start, read and not used
                    const int hh = on ? h : 0;
                    if (NORM || !BWD) rx[j] = load_raw<T, L>(x + hh * a.xh[s], lane, P, D, half);
                    if (BWD) rd[j] = load_raw<T, L>(dy + hh * a.dh[s], lane, P, D, half);
                }
#pragma unroll
                for (int j = 0; j < U; j++) {
                    const int h = h0 + j * a.splits + split;
                    const bool on = live && h < H;
                    float2 v[4], o[4];
                    float rstd = 1.f;
                    if (NORM || !BWD) {
                        float sum = 0.f;
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            v[i] = pair_of(rx[j], i);
                            sum = fmaf(v[i].x, v[i].x, fmaf(v[i].y, v[i].y, sum));
                        }
                        if (NORM) rstd = 1.f / sqrtf(group_sum<G>(sum) / (float)D + a.eps);
                    }
                    if constexpr (!BWD) {
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            if (NORM) v[i] = make_float2(v[i].x * rstd * w[s][i].x, v[i].y * rstd * w[s][i].y);
                            o[i] = turned(v[i], cs[i]);
                        }
                    } else if constexpr (!NORM) {
#pragma unroll
                        for (int i = 0; i < 4; i++) o[i] = turned_back(pair_of(rd[j], i), cs[i]);
                    } else {
                        float2 u[4];
                        float dot = 0.f;
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            u[i] = turned_back(pair_of(rd[j], i), cs[i]);
                            v[i].x *= rstd;
                            v[i].y *= rstd;
                            if (on) {
                                dw[s][i].x = fmaf(u[i].x, v[i].x, dw[s][i].x);
                                dw[s][i].y = fmaf(u[i].y, v[i].y, dw[s][i].y);
                            }
                            u[i].x *= w[s][i].x;
                            u[i].y *= w[s][i].y;
                            dot = fmaf(u[i].x, v[i].x, fmaf(u[i].y, v[i].y, dot));
                        }
                        dot = group_sum<G>(dot) / (float)D;
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            o[i] = make_float2(rstd * (u[i].x - v[i].x * dot), rstd * (u[i].y - v[i].y * dot));
                    }
                    if (on) store_pairs<T, L>(y + h * a.yh[s], o, lane, P, D, half);
                }
            }
        }
    }
    if constexpr (BWD && NORM) {
        if (a.ws == nullptr) return;
        // the groups' sums of this CTA, added in the groups' order
        extern __shared__ float sums[];   // [groups][2][D]
        float *mine = sums + (size_t)(threadIdx.x / G) * 2 * D;
#pragma unroll
        for (int s = 0; s < 2; s++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int p = L == kAny ? lane + 32 * i : 4 * lane + i;
                if (p < D / 2) {
                    mine[s * D + first_of(p, P, half)] = dw[s][i].x;
                    mine[s * D + second_of(p, P, D, half)] = dw[s][i].y;
                }
            }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * D; c += kThreads) {
            float t = 0.f;
            for (int g = 0; g < kThreads / G; g++) t += sums[(size_t)g * 2 * D + c];
            a.ws[(size_t)blockIdx.x * 2 * D + c] = t;
        }
    }
}

// Columns of the CTAs' sums [n][2D]: 32 columns to a CTA, rows over its 8 warps.
__global__ void __launch_bounds__(256) weight_sums_kernel(const float *ws, int n, int D, float *dwq, float *dwk) {
    __shared__ float part[8][33];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    float t = 0.f;
    if (c < 2 * D)
#pragma unroll 4
        for (int r = warp; r < n; r += 8) t += ws[(size_t)r * 2 * D + c];
    part[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && c < 2 * D) {
        for (int i = 1; i < 8; i++) t += part[i][lane];
        float *dst = c < D ? dwq : dwk;
        if (dst) dst[c < D ? c : c - D] = t;
    }
}

constexpr int kSms = 152;
constexpr int kBwdCtas = kSms * 4;   // their sums are written: few, that stay

bool on_boundary(const void *p, long long b, long long h, long long n, size_t bytes) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(b * bytes) | (uintptr_t)(h * bytes) |
                             (uintptr_t)(n * bytes)) & 15) == 0;
}

template <typename T, int G, Layout L, bool BWD> cudaError_t launch(const RotArgs &a, int ctas, bool norm, cudaStream_t st) {
    const size_t smem = BWD && norm && a.ws ? (size_t)(kThreads / G) * 2 * a.D * sizeof(float) : 0;
    if (norm) rotate_kernel<T, G, L, BWD, true><<<ctas, kThreads, smem, st>>>(a);
    else rotate_kernel<T, G, L, BWD, false><<<ctas, kThreads, smem, st>>>(a);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T, bool BWD> cudaError_t pick(const RotArgs &a, int G, Layout l, int ctas, bool norm, cudaStream_t st) {
    if (l == kAny) return launch<T, 32, kAny, BWD>(a, ctas, norm, st);
    if (l == kHalf) {
        if (G == 8) return launch<T, 8, kHalf, BWD>(a, ctas, norm, st);
        return G == 16 ? launch<T, 16, kHalf, BWD>(a, ctas, norm, st) : launch<T, 32, kHalf, BWD>(a, ctas, norm, st);
    }
    if (G == 8) return launch<T, 8, kAdjacent, BWD>(a, ctas, norm, st);
    return G == 16 ? launch<T, 16, kAdjacent, BWD>(a, ctas, norm, st) : launch<T, 32, kAdjacent, BWD>(a, ctas, norm, st);
}

cudaError_t rotate(const RotateProblem &p, bool bwd) {
    RotArgs a{};
    const bool half = p.rot.pairs == LA_PAIRS_HALF;
    const la_view x[2] = {p.q, p.k}, y[2] = {p.qo, p.ko}, dy[2] = {p.dqo, p.dko};
    const size_t size = p.s.dtype == LA_DTYPE_F32 ? 4 : 2;
    bool wide = p.s.D % 8 == 0 && (!half || p.rot.P % 4 == 0);
    for (int s = 0; s < 2; s++) {
        a.H[s] = s ? p.s.Hk : p.s.Hq;
        a.x[s] = x[s].data, a.y[s] = y[s].data, a.dy[s] = dy[s].data;
        a.xb[s] = x[s].sb, a.xh[s] = x[s].sh, a.xn[s] = x[s].sn;
        a.yb[s] = y[s].sb, a.yh[s] = y[s].sh, a.yn[s] = y[s].sn;
        a.db[s] = dy[s].sb, a.dh[s] = dy[s].sh, a.dn[s] = dy[s].sn;
        a.w[s] = s ? p.wk : p.wq;
        if (a.H[s] == 0) continue;
        wide = wide && on_boundary(x[s].data, x[s].sb, x[s].sh, x[s].sn, size) &&
               on_boundary(y[s].data, y[s].sb, y[s].sh, y[s].sn, size) &&
               (!bwd || on_boundary(dy[s].data, dy[s].sb, dy[s].sh, dy[s].sn, size));
    }
    a.pos = p.rot.pos, a.sa = p.rot.sa, a.sb = p.rot.sb, a.sn = p.rot.sn, a.freq = p.rot.freq;
    a.B = p.s.B, a.N = p.s.N, a.D = p.s.D, a.P = p.rot.P, a.eps = p.eps;
    if (p.rot.axes && p.rot.P) {
        memcpy(a.axes, p.rot.axes, p.rot.P);
        for (int i = 0; i < p.rot.P; i++) a.by_axis |= p.rot.axes[i] != 0;
    }
    // 16 byte pieces where every row allows them, else single values, 32 lanes to a token
    const Layout l = !wide ? kAny : half ? kHalf : kAdjacent;
    a.half = half;
    const int G = l == kAny || p.s.D > 128 ? 32 : p.s.D > 64 ? 16 : 8;
    const long long tokens = (long long)p.s.B * p.s.N, per = kThreads / G;
    // a token's heads are shared by as many groups as it takes to fill the SMs
    const int heads = std::max(p.s.Hq, p.s.Hk);
    long long splits = 1;
    while (splits < heads && tokens * splits * 2 <= (long long)kSms * 4 * per) splits *= 2;
    a.splits = (int)splits;
    const bool sums = bwd && p.norm && (p.dwq || p.dwk);
    a.ws = sums ? static_cast<float *>(p.ws) : nullptr;
    const long long ctas = std::min((tokens * splits + per - 1) / per, bwd && p.norm ? (long long)kBwdCtas : 1LL << 30);
    const bool f32 = p.s.dtype == LA_DTYPE_F32;
    cudaError_t e = bwd ? (f32 ? pick<float, true>(a, G, l, (int)ctas, p.norm, p.stream)
                               : pick<__nv_bfloat16, true>(a, G, l, (int)ctas, p.norm, p.stream))
                        : (f32 ? pick<float, false>(a, G, l, (int)ctas, p.norm, p.stream)
                               : pick<__nv_bfloat16, false>(a, G, l, (int)ctas, p.norm, p.stream));
    if (e != cudaSuccess || !sums) return e;
    weight_sums_kernel<<<(2 * p.s.D + 31) / 32, 256, 0, p.stream>>>(a.ws, (int)ctas, p.s.D, p.dwq, p.dwk);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

size_t rotate_ws_bytes(const la_qk_shape &s) { return (size_t)kBwdCtas * 2 * s.D * sizeof(float); }
cudaError_t rotate_forward(const RotateProblem &p) { return rotate(p, false); }
cudaError_t rotate_backward(const RotateProblem &p) { return rotate(p, true); }

}  // namespace la
