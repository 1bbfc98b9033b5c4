// la_layernorm.cu - layer norm of rows with the residual sum in front, and
// its backward with the reduction of the weight's and bias' gradients.
//
// Both are bound by HBM.  A group of TPR threads (part of a warp, a warp, or a
// CTA) holds a row in registers, so every value is read once: the mean first,
// then the variance about it (not the mean of the squares, which loses it next
// to a large mean), then the output.  The backward's CTAs stay and walk over
// rows, because each thread keeps its columns' sums of dy xh and dy in fp32
// registers; the sums of all groups are added in a fixed order.
//
//   s = x + res (kept as stored), xh = (s - mean) rstd, y = xh w + b
//   ds = rstd (g - mean(g) - xh mean(g xh)) + dsum with g = dy w
//   dw = sum of dy xh, db = sum of dy over the rows
//
// Measured: 32768 rows of 2048, bf16, with the residual: forward 86 us (6.2 TB/s),
// backward 91 us (5.9 TB/s); 262144 rows of 64: 13.3 and 24.2 us; 16 rows of 2048:
// 2.0 us (latency).  Wide rows keep 5.5 to 6.4 TB/s forward.  Backward, 64 Mi bf16
// values: rows of 8192 4.8 TB/s (83 us), their sums leave room for 8 warps an SM; rows
// of 16384 2.2 TB/s (185 us), their sums live in shared memory with one row on its
// way.  32 Mi fp32 values: rows of 4096 5.8 TB/s (69 us), of 8192, with the sums in shared
// memory, 4.5 (89 us), of 16384, whose rows are loaded when they are due, 3.3 (123 us).
// Wide rows off 16 bytes are taken by single values: 8191 bf16 values 3.4 TB/s forward,
// 1.4 backward.
#include <algorithm>

#include "la_layer.h"
#include "la_pair.cuh"
#include "tc_ptx.cuh"

namespace la {
namespace {

constexpr int kSms = 152;

// A thread's share of a row: K pieces of 16 bytes, TPR pieces apart, or (rows
// not all on 16 bytes) as many single values, TPR values apart.
template <typename T, int TPR, int K, bool WIDE> struct Share {
    static constexpr int VEC = 16 / (int)sizeof(T), E = K * VEC;
    using Bits = std::conditional_t<sizeof(T) == 4, unsigned, unsigned short>;
    uint4 piece[WIDE ? K : 1];
    Bits one[WIDE ? 1 : E];

    // column of element i
    static __device__ __forceinline__ int column(int i, int lane) {
        return WIDE ? ((i / VEC) * TPR + lane) * VEC + i % VEC : i * TPR + lane;
    }
    __device__ __forceinline__ void load(const T *row, int lane, int C) {
        if constexpr (WIDE) {
#pragma unroll
            for (int k = 0; k < K; k++) {
                const int c = (k * TPR + lane) * VEC;
                piece[k] = c < C ? *reinterpret_cast<const uint4 *>(row + c) : make_uint4(0, 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; i++) {
                const int c = i * TPR + lane;
                one[i] = c < C ? reinterpret_cast<const Bits *>(row)[c] : Bits(0);
            }
        }
    }
    __device__ __forceinline__ void store(T *row, int lane, int C) const {
        if constexpr (WIDE) {
#pragma unroll
            for (int k = 0; k < K; k++) {
                const int c = (k * TPR + lane) * VEC;
                if (c < C) *reinterpret_cast<uint4 *>(row + c) = piece[k];
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; i++) {
                const int c = i * TPR + lane;
                if (c < C) reinterpret_cast<Bits *>(row)[c] = one[i];
            }
        }
    }
    // elements 2i and 2i + 1
    __device__ __forceinline__ float2 get(int i) const {
        if constexpr (WIDE && sizeof(T) == 4)
            return i % 2 ? make_float2(__uint_as_float(piece[i / 2].z), __uint_as_float(piece[i / 2].w))
                         : make_float2(__uint_as_float(piece[i / 2].x), __uint_as_float(piece[i / 2].y));
        else if constexpr (WIDE)
            return get_pair((&piece[i / 4].x)[i % 4]);
        else if constexpr (sizeof(T) == 4)
            return make_float2(__uint_as_float(one[2 * i]), __uint_as_float(one[2 * i + 1]));
        else
            return make_float2(__uint_as_float((unsigned)one[2 * i] << 16),
                               __uint_as_float((unsigned)one[2 * i + 1] << 16));
    }
    __device__ __forceinline__ void set(int i, float2 v) {
        if constexpr (WIDE && sizeof(T) == 4) {
            (&piece[i / 2].x)[i % 2 * 2] = __float_as_uint(v.x);
            (&piece[i / 2].x)[i % 2 * 2 + 1] = __float_as_uint(v.y);
        } else if constexpr (WIDE) {
            (&piece[i / 4].x)[i % 4] = put_pair(v);
        } else if constexpr (sizeof(T) == 4) {
            one[2 * i] = __float_as_uint(v.x);
            one[2 * i + 1] = __float_as_uint(v.y);
        } else {
            const unsigned w = put_pair(v);
            one[2 * i] = (unsigned short)w;
            one[2 * i + 1] = (unsigned short)(w >> 16);
        }
    }
};

// A thread's shares of NT tensors on their way, S rows deep: 16-byte pieces
// through its own places in shared memory (no other thread touches them, so no
// barrier), single values through registers, one row ahead.  S = 0: loaded when
// they are taken (the widest rows, a CTA each, whose threads have no room for more).
template <typename T, int TPR, int K, bool WIDE, int NT, int S> struct Feed {
    using Sh = Share<T, TPR, K, WIDE>;
    static constexpr bool kShared = WIDE && S > 0, kHeld = !WIDE && S > 0;
    static constexpr int DEPTH = kShared ? S : 1;
    static constexpr size_t bytes(int threads) { return kShared ? (size_t)S * NT * K * 16 * threads : 0; }
    uint4 *slot;
    int threads, lane, C;
    Sh held[kHeld ? NT : 1];

    __device__ __forceinline__ void fetch(int stage, int k, const T *row) {
        if constexpr (kShared) {
#pragma unroll
            for (int i = 0; i < K; i++) {
                const int c = (i * TPR + lane) * Sh::VEC;
                if (c < C)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                     tc::smem_u32(&slot[((stage * NT + k) * K + i) * threads])),
                                 "l"(row + c)
                                 : "memory");
            }
        } else if constexpr (kHeld) {
            held[k].load(row, lane, C);
        }
    }
    __device__ __forceinline__ void commit() {
        if constexpr (kShared) asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ void wait() {
        if constexpr (kShared) asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
    }
    // columns past C are 0; row: the one that was fetched into the stage
    __device__ __forceinline__ Sh take(int stage, int k, const T *row) {
        Sh r;
        if constexpr (kShared) {
#pragma unroll
            for (int i = 0; i < K; i++)
                r.piece[i] = (i * TPR + lane) * Sh::VEC < C ? slot[((stage * NT + k) * K + i) * threads]
                                                            : make_uint4(0, 0, 0, 0);
        } else if constexpr (kHeld) {
            r = held[k];
        } else {
            r.load(row, lane, C);
        }
        return r;
    }
};

// fp32 parameters of the thread's columns; a null pointer gives `none`.
template <int TPR, int K, int VEC, bool WIDE>
__device__ __forceinline__ void load_columns(float2 (&v)[K * VEC / 2], const float *p, int lane, int C, float none) {
#pragma unroll
    for (int i = 0; i < K * VEC / 2; i++) v[i] = make_float2(none, none);
    if (p == nullptr) return;
    if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < K * VEC; i += 4) {
            const int c = ((i / VEC) * TPR + lane) * VEC + i % VEC;
            if (c < C) {
                const float4 q = *reinterpret_cast<const float4 *>(p + c);
                v[i / 2] = make_float2(q.x, q.y), v[i / 2 + 1] = make_float2(q.z, q.w);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < K * VEC; i++)
            if (i * TPR + lane < C) (i % 2 ? v[i / 2].y : v[i / 2].x) = p[i * TPR + lane];
    }
}

// Sums of N values over a row's threads, given to each of them.  Calls of one
// CTA take the two halves of `sh` in turn, so that one barrier a call is enough.
template <int TPR, int N> struct Sums {
    float (*sh)[N][TPR / 32 > 0 ? TPR / 32 : 1];   // [2]
    int turn = 0;
    __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
        for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o /= 2)
#pragma unroll
            for (int n = 0; n < N; n++) v[n] += __shfl_xor_sync(~0u, v[n], o);
        if constexpr (TPR > 32) {
            constexpr int NW = TPR / 32;
            const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
            if (lane == 0) {
#pragma unroll
                for (int n = 0; n < N; n++) sh[turn][n][warp] = v[n];
            }
            __syncthreads();
#pragma unroll
            for (int n = 0; n < N; n++) {
                // every thread adds the warps' sums in the same order
                if constexpr (NW <= 8) {
                    float s = sh[turn][n][0];
#pragma unroll
                    for (int i = 1; i < NW; i++) s += sh[turn][n][i];
                    v[n] = s;
                } else {
                    float s = lane < NW ? sh[turn][n][lane] : 0.f;
#pragma unroll
                    for (int o = NW / 2; o > 0; o /= 2) s += __shfl_xor_sync(~0u, s, o);
                    v[n] = __shfl_sync(~0u, s, 0);
                }
            }
            turn ^= 1;
        }
    }
};

// A tensor's rows as a group meets them, `step` rows apart.
template <typename T> struct Walk {
    T *row;
    long long to_next;
    __device__ __forceinline__ Walk(const la_rows &v, long long first, long long step)
        : row(static_cast<T *>(v.data) + first * v.stride), to_next(step * v.stride) {}
    __device__ __forceinline__ T *next() {
        T *r = row;
        row += to_next;
        return r;
    }
};

template <int TPR> constexpr int threads_of() { return TPR > 256 ? TPR : TPR > 32 ? TPR : 256; }

// Groups walk over rows gridDim * GROUPS apart.
template <typename T, int TPR, int K, bool WIDE, int S, int CTAS>
__global__ void __launch_bounds__(threads_of<TPR>(), CTAS) ln_forward_kernel(NormProblem p) {
    using F = Feed<T, TPR, K, WIDE, 2, S>;
    using Sh = typename F::Sh;
    constexpr int E2 = Sh::E / 2, GROUPS = threads_of<TPR>() / TPR;
    __shared__ float sh[2][1][TPR / 32 > 0 ? TPR / 32 : 1];
    extern __shared__ __align__(16) uint4 smem[];
    Sums<TPR, 1> sum{sh};
    pdl_wait_cta();
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
    F feed{smem + threadIdx.x, threads_of<TPR>(), lane, p.C};
    const long long step = (long long)gridDim.x * GROUPS, first = (long long)blockIdx.x * GROUPS + group;
    Walk<const T> x_ahead(p.x, first, step), res_ahead(p.res, first, step), x_here = x_ahead, res_here = res_ahead;
    Walk<T> sum_here(p.sum, first, step), y_here(p.y, first, step);
    auto fetch = [&](long long r, int stage) {
        if (r < p.rows) {
            feed.fetch(stage, 0, x_ahead.next());
            if (p.res.data) feed.fetch(stage, 1, res_ahead.next());
        }
        feed.commit();
    };
#pragma unroll
    for (int i = 0; i < F::DEPTH; i++) fetch(first + i * step, i);
    float2 w[E2], b[E2];
    load_columns<TPR, K, Sh::VEC, WIDE>(w, p.w, lane, p.C, 1.f);
    load_columns<TPR, K, Sh::VEC, WIDE>(b, p.b, lane, p.C, 0.f);
    int stage = 0;
    // a CTA's groups run the same number of rounds (their barriers and shuffles meet)
    for (long long base = (long long)blockIdx.x * GROUPS; base < p.rows; base += step) {
        const long long r = base + group;
        feed.wait();
        Sh a = feed.take(stage, 0, x_here.next());
        float2 v[E2];
#pragma unroll
        for (int i = 0; i < E2; i++) v[i] = a.get(i);
        if (p.res.data) {
            const Sh c = feed.take(stage, 1, res_here.next());
#pragma unroll
            for (int i = 0; i < E2; i++) {   // the stream as it is kept, and normalised
                a.set(i, add_pair(v[i], c.get(i)));
                v[i] = a.get(i);
            }
            if (p.sum.data && r < p.rows) a.store(sum_here.next(), lane, p.C);
        }
        fetch(r + F::DEPTH * step, stage);
        stage = stage == F::DEPTH - 1 ? 0 : stage + 1;
        float2 s2 = v[0];
#pragma unroll
        for (int i = 1; i < E2; i++) s2 = add_pair(s2, v[i]);
        float s[1] = {s2.x + s2.y};
        sum(s);
        const float mean = s[0] / p.C;
        s[0] = 0.f;
#pragma unroll
        for (int k = 0; k < K; k++) {
            float2 q = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = k * Sh::VEC / 2; i < (k + 1) * Sh::VEC / 2; i++) {
                v[i] = add_pair(v[i], make_float2(-mean, -mean));
                if (!WIDE) {   // columns past C do not count
                    if (Sh::column(2 * i, lane) >= p.C) v[i].x = 0.f;
                    if (Sh::column(2 * i + 1, lane) >= p.C) v[i].y = 0.f;
                }
                q = fma_pair(v[i], v[i], q);
            }
            if (!WIDE || (k * TPR + lane) * Sh::VEC < p.C) s[0] += q.x + q.y;
        }
        sum(s);
        const float rstd = rsqrtf(s[0] / p.C + p.eps);
        if (r < p.rows) {
            Sh y;
#pragma unroll
            for (int i = 0; i < E2; i++) y.set(i, fma_pair(mul_pair(v[i], make_float2(rstd, rstd)), w[i], b[i]));
            y.store(y_here.next(), lane, p.C);
            if (p.mean && lane == 0) p.mean[r] = mean, p.rstd[r] = rstd;
        }
    }
}

template <typename T, int TPR, int K, bool WIDE, int S, int CTAS>
__global__ void __launch_bounds__(threads_of<TPR>(), CTAS) ln_backward_kernel(NormProblem p) {
    using F = Feed<T, TPR, K, WIDE, 3, S>;
    using Sh = typename F::Sh;
    constexpr int E = Sh::E, E2 = E / 2, GROUPS = threads_of<TPR>() / TPR;
    __shared__ float sh[2][2][TPR / 32 > 0 ? TPR / 32 : 1];
    extern __shared__ __align__(16) uint4 smem[];
    // After the feed, and over it once the walk is done, [GROUPS][2][C] where a
    // CTA has several groups; the sums themselves, [2][E][threads], where a CTA of
    // 1024 threads leaves 64 registers to each.
    constexpr bool kOutside = TPR == 1024;
    float *columns = reinterpret_cast<float *>(smem) + (kOutside ? F::bytes(TPR) / sizeof(float) : 0);
    Sums<TPR, 2> sum{sh};
    pdl_wait_cta();
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
    F feed{smem + threadIdx.x, threads_of<TPR>(), lane, p.C};
    const long long step = (long long)gridDim.x * GROUPS, first = (long long)blockIdx.x * GROUPS + group;
    Walk<const T> dy_ahead(p.y, first, step), s_ahead(p.x, first, step), dsum_ahead(p.res, first, step);
    Walk<const T> dy_here = dy_ahead, s_here = s_ahead, dsum_here = dsum_ahead;
    Walk<T> ds_here(p.ds, first, step);
    float mean = 0.f, rstd = 0.f;
    auto fetch = [&](long long r, int stage) {
        if (r < p.rows) {
            feed.fetch(stage, 0, dy_ahead.next());
            feed.fetch(stage, 1, s_ahead.next());
            if (p.res.data) feed.fetch(stage, 2, dsum_ahead.next());
        }
        feed.commit();
    };
    auto next_stats = [&](long long r) {
        if (r < p.rows) mean = p.mean[r], rstd = p.rstd[r];
    };
#pragma unroll
    for (int i = 0; i < F::DEPTH; i++) fetch(first + i * step, i);
    next_stats(first);
    float2 w[kOutside ? 1 : E2], dw[kOutside ? 1 : E2], db[kOutside ? 1 : E2];
    if constexpr (kOutside) {
#pragma unroll
        for (int i = 0; i < 2 * E; i++) columns[i * TPR + lane] = 0.f;
    } else {
        load_columns<TPR, K, Sh::VEC, WIDE>(w, p.w, lane, p.C, 1.f);
#pragma unroll
        for (int i = 0; i < E2; i++) dw[i] = db[i] = make_float2(0.f, 0.f);
    }
    int stage = 0;
    for (long long base = (long long)blockIdx.x * GROUPS; base < p.rows; base += step) {
        const long long r = base + group;
        feed.wait();
        const Sh dy = feed.take(stage, 0, dy_here.next()), s = feed.take(stage, 1, s_here.next());
        Sh extra;
        if (p.res.data) extra = feed.take(stage, 2, dsum_here.next());
        const float2 m = make_float2(-mean, -mean), rs = make_float2(rstd, rstd);
        fetch(r + F::DEPTH * step, stage);
        next_stats(r + step);
        stage = stage == F::DEPTH - 1 ? 0 : stage + 1;
        float2 g[E2], xh[E2], t1 = make_float2(0.f, 0.f), t2 = t1;
        if (r < p.rows) {
#pragma unroll
            for (int i = 0; i < E2; i++) {   // g is 0 in the columns past C
                g[i] = dy.get(i);
                xh[i] = mul_pair(add_pair(s.get(i), m), rs);
                if constexpr (kOutside) {
                    const int c0 = Sh::column(2 * i, lane), c1 = Sh::column(2 * i + 1, lane);
                    float *at = columns + 2 * i * TPR + lane;
                    at[0] = fmaf(g[i].x, xh[i].x, at[0]), at[TPR] = fmaf(g[i].y, xh[i].y, at[TPR]);
                    at[E * TPR] += g[i].x, at[(E + 1) * TPR] += g[i].y;
                    if (p.w) g[i] = mul_pair(g[i], make_float2(c0 < p.C ? p.w[c0] : 0.f, c1 < p.C ? p.w[c1] : 0.f));
                } else {
                    dw[i] = fma_pair(g[i], xh[i], dw[i]);
                    db[i] = add_pair(db[i], g[i]);
                    g[i] = mul_pair(g[i], w[i]);
                }
                t1 = add_pair(t1, g[i]);
                t2 = fma_pair(g[i], xh[i], t2);
            }
        }
        float t[2] = {t1.x + t1.y, t2.x + t2.y};
        sum(t);
        if (r < p.rows) {
            const float2 a = make_float2(-t[0] / p.C, -t[0] / p.C), b = make_float2(-t[1] / p.C, -t[1] / p.C);
            Sh ds;
#pragma unroll
            for (int i = 0; i < E2; i++) {
                const float2 d = fma_pair(xh[i], b, add_pair(g[i], a));
                ds.set(i, p.res.data ? fma_pair(rs, d, extra.get(i)) : mul_pair(rs, d));
            }
            ds.store(ds_here.next(), lane, p.C);
        }
    }
    if constexpr (GROUPS > 1) __syncthreads();   // every thread has taken its last rows
    if (p.ws == nullptr) return;
    float *part = static_cast<float *>(p.ws) + (long long)blockIdx.x * 2 * p.C;
    if constexpr (GROUPS == 1) {
#pragma unroll
        for (int i = 0; i < E; i++) {
            const int c = Sh::column(i, lane);
            if (c >= p.C) continue;
            if constexpr (kOutside) part[c] = columns[i * TPR + lane], part[p.C + c] = columns[(E + i) * TPR + lane];
            else part[c] = i % 2 ? dw[i / 2].y : dw[i / 2].x, part[p.C + c] = i % 2 ? db[i / 2].y : db[i / 2].x;
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; i++) {
            const int c = Sh::column(i, lane);
            if (c < p.C) {
                columns[group * 2 * p.C + c] = i % 2 ? dw[i / 2].y : dw[i / 2].x;
                columns[group * 2 * p.C + p.C + c] = i % 2 ? db[i / 2].y : db[i / 2].x;
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * p.C; c += threads_of<TPR>()) {
            float a = 0.f;
#pragma unroll
            for (int k = 0; k < GROUPS; k++) a += columns[k * 2 * p.C + c];
            part[c] = a;
        }
    }
}

// Adds the CTAs' column sums: 32 columns a CTA, its warps taking the parts in turn,
// kAhead of them on their way at once (with 4 at once it took 9 us, whatever C).
constexpr int kFinishWarps = 32, kAhead = 10;
__global__ void __launch_bounds__(32 * kFinishWarps) ln_finish_kernel(const float *ws, float *dw, float *db, int C,
                                                                      int parts) {
    __shared__ float sh[kFinishWarps][33];
    pdl_wait_cta();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    float a = 0.f;
    if (c < 2 * C) {
        for (int i0 = warp; i0 < parts; i0 += kAhead * kFinishWarps) {
            float v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; k++) {
                const int i = i0 + k * kFinishWarps;
                v[k] = i < parts ? ws[(long long)i * 2 * C + c] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < kAhead; k++) a += v[k];
        }
    }
    sh[warp][lane] = a;
    __syncthreads();
    static_assert(kFinishWarps == 32, "");   // warp w adds column w
    a = sh[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o /= 2) a += __shfl_xor_sync(~0u, a, o);
    const int column = blockIdx.x * 32 + warp;
    if (lane == 0 && column < 2 * C) {
        if (column < C) {
            if (dw) dw[column] = a;
        } else if (db) {
            db[column - C] = a;
        }
    }
}

// CTAs that walk over the rows: as many as the SMs hold, no more than there are
// rows for.
int ctas_of(long long rows, int groups, int per_sm) {
    return (int)std::min((long long)kSms * per_sm, (rows + groups - 1) / groups);
}

// Rows on their way (S) and CTAs a SM (counted for CTAs of 256 threads), within the
// registers and shared memory that the widths leave.  Measured (bf16, forward |
// backward): 262144 rows of 64, a piece a thread: 13.3 | 24.2 us with 4 CTAs and 4
// rows | 3 and 3 (forward with 5 and 3: 17.0, backward with 4 and 2: 32); 32768 rows
// of 2048 with the residual, 4 pieces a thread: 86 | 91 us with 2 and 2 | 1 and 2
// (forward with 3 CTAs, 80 registers: 114; backward with 1 row on its way: 100).
template <typename T, int TPR, int K, bool WIDE> struct Shape {
    static constexpr int THREADS = threads_of<TPR>();
    static constexpr bool kLean = WIDE || sizeof(T) == 4;   // single bf16 values take more registers
    static constexpr int per_sm(int ctas) { return ctas * 256 / THREADS; }
    static constexpr int FWD_S = THREADS == 1024 && K == 4 ? 1 : K == 1 ? 4 : 2;
    static constexpr int FWD_CTAS = THREADS == 1024  ? 1
                                    : THREADS == 512 ? (kLean ? 2 : 1)
                                                     : per_sm(K == 1 ? (kLean ? 4 : 2) : K == 2 ? (kLean ? 3 : 2) : 2);
    static constexpr int BWD_S = K == 1 ? 3 : THREADS < 1024 ? 2 : K == 2 && WIDE ? 1 : 0;
    static constexpr int BWD_CTAS = THREADS >= 512 ? 1 : per_sm(K == 1 ? (kLean ? 3 : 2) : K == 2 ? (kLean ? 2 : 1) : 1);
};

struct Forward {
    template <typename T, int TPR, int K, bool WIDE> static cudaError_t run(const NormProblem &p) {
        constexpr int THREADS = threads_of<TPR>(), GROUPS = THREADS / TPR;
        using C = Shape<T, TPR, K, WIDE>;
        const auto kernel = ln_forward_kernel<T, TPR, K, WIDE, C::FWD_S, C::FWD_CTAS>;
        const size_t smem = Feed<T, TPR, K, WIDE, 2, C::FWD_S>::bytes(THREADS);
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        e = launch_pdl(kernel, dim3((unsigned)ctas_of(p.rows, GROUPS, C::FWD_CTAS)), dim3(THREADS), smem, p.stream, 0u,
                       p);
        count_launches(1);
        return e;
    }
};

struct Backward {
    template <typename T, int TPR, int K, bool WIDE> static cudaError_t run(NormProblem p) {
        constexpr int THREADS = threads_of<TPR>(), GROUPS = THREADS / TPR;
        using C = Shape<T, TPR, K, WIDE>;
        const auto kernel = ln_backward_kernel<T, TPR, K, WIDE, C::BWD_S, C::BWD_CTAS>;
        const int parts = ctas_of(p.rows, GROUPS, C::BWD_CTAS);
        if (!p.dw && !p.db) p.ws = nullptr;
        size_t smem = Feed<T, TPR, K, WIDE, 3, C::BWD_S>::bytes(THREADS);
        if (GROUPS > 1) smem = std::max(smem, (size_t)GROUPS * 2 * p.C * sizeof(float));
        if (TPR == 1024) smem += 2 * Share<T, TPR, K, WIDE>::E * TPR * sizeof(float);
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        e = launch_pdl(kernel, dim3((unsigned)parts), dim3(THREADS), smem, p.stream, 0u, p);
        count_launches(1);
        if (e != cudaSuccess || !p.ws) return e;
        e = launch_pdl(ln_finish_kernel, dim3((unsigned)((2 * p.C + 31) / 32)), dim3(32 * kFinishWarps), 0, p.stream,
                       0u, (const float *)p.ws, p.dw, p.db, p.C, parts);
        count_launches(1);
        return e;
    }
};

// The narrowest group that holds the row: up to a warp (no barrier) with at most
// 4 pieces a thread, then CTAs with 2.
template <typename Call, typename T, bool WIDE> cudaError_t by_width(const NormProblem &p) {
    const int pieces = (p.C + 16 / (int)sizeof(T) - 1) / (16 / (int)sizeof(T));
    if (pieces <= 8) return Call::template run<T, 8, 1, WIDE>(p);
    if (pieces <= 16) return Call::template run<T, 16, 1, WIDE>(p);
    if (pieces <= 32) return Call::template run<T, 32, 1, WIDE>(p);
    if (pieces <= 64) return Call::template run<T, 32, 2, WIDE>(p);
    if constexpr (WIDE) {   // 4 pieces a thread share the sums' cost (rows of 2048: 87 | 91 us, with 1 piece 89 | 103 us)
        if (pieces <= 128) return Call::template run<T, 32, 4, WIDE>(p);
        if (pieces <= 256) return Call::template run<T, 64, 4, WIDE>(p);
        if (pieces <= 512) return Call::template run<T, 128, 4, WIDE>(p);
        if (pieces <= 1024) return Call::template run<T, 256, 4, WIDE>(p);
    } else {                // whose shares take more registers
        if (pieces <= 128) return Call::template run<T, 64, 2, WIDE>(p);
        if (pieces <= 256) return Call::template run<T, 128, 2, WIDE>(p);
        if (pieces <= 512) return Call::template run<T, 256, 2, WIDE>(p);
        if (pieces <= 1024) return Call::template run<T, 512, 2, WIDE>(p);
    }
    if constexpr (sizeof(T) == 4)
        if (pieces > 2048) return Call::template run<T, 1024, 4, WIDE>(p);
    return Call::template run<T, 1024, 2, WIDE>(p);
}

template <typename Call> cudaError_t by_type(const NormProblem &p) {
    const int size = p.dtype == LA_DTYPE_F32 ? 4 : 2;
    unsigned long long bits = (unsigned long long)p.C * size;
    for (const la_rows &v : {p.x, p.res, p.sum, p.y, p.ds})   // those that a call lacks are 0
        bits |= reinterpret_cast<uintptr_t>(v.data) | (unsigned long long)(p.rows > 1 ? v.stride : 0) * size;
    bits |= reinterpret_cast<uintptr_t>(p.w) | reinterpret_cast<uintptr_t>(p.b);
    const bool wide = bits % 16 == 0;
    if (p.dtype == LA_DTYPE_F32) return wide ? by_width<Call, float, true>(p) : by_width<Call, float, false>(p);
    return wide ? by_width<Call, __nv_bfloat16, true>(p) : by_width<Call, __nv_bfloat16, false>(p);
}

}  // namespace

// A part per CTA of the backward: at most 8 a SM, at most one per row.
size_t layernorm_ws_bytes(long long rows, int C) {
    return (size_t)std::min(rows, 8LL * kSms) * 2 * C * sizeof(float);
}

cudaError_t layernorm_forward(const NormProblem &p) { return by_type<Forward>(p); }
cudaError_t layernorm_backward(const NormProblem &p) { return by_type<Backward>(p); }

}  // namespace la
