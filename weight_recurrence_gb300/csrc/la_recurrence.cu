// la_recurrence.cu - the gated linear recurrence h_t = a_t h_{t-1} + u_t of
// every channel, and its backward l_t = dout_t + a_{t+1} l_{t+1}.
//
// Both are bound by HBM: a few operations a value against 6 bytes (forward,
// bf16) or 12 (backward).  What stands between that and one pass over the
// data is the order of the tokens.  A row's update is an affine map of the
// state, h -> a h + u, and a run of rows is one too, h -> A h + H with A the
// product of its gates and H the run started from 0, so runs are walked side
// by side and joined by their (A, H).
//
// A strip of 32 lanes' channels belongs to one CTA, or to a cluster of CTAs
// where there are few strips.  They walk its tokens in tiles: each warp takes
// R consecutive rows, first forms (A, H) of them, then learns the state before
// them (the warps' maps through shared memory, the CTAs' through distributed
// shared memory) and runs the recurrence proper from it.  Every value is read
// once and written once, without workspace, flags in global memory or atomics,
// and the grouping depends on the sizes alone, so equal calls give equal bits.
#include <initializer_list>
#include <type_traits>

#include "la_gate.cuh"
#include "la_layer.h"
#include "tc_ptx.cuh"

namespace la {
namespace {


struct Dims {
    const int *lens;
    int H, N, D;
    int strips;        // groups of 32 lanes' channels in a sequence
    int *err;          // device error word
};

// V neighbouring channels of one row as they lie in memory.
__device__ __forceinline__ float2 get_pair(unsigned r) {
    return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
}
__device__ __forceinline__ unsigned put_pair(float2 v) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const unsigned *>(&p);
}
template <typename T, int V> struct Raw;
template <> struct Raw<float, 1> {
    using type = float;
    static __device__ __forceinline__ Lanes<1> get(type r) { return {{r}}; }
    static __device__ __forceinline__ type put(const Lanes<1> &v) { return v.p[0]; }
};
template <> struct Raw<float, 2> {
    using type = float2;
    static __device__ __forceinline__ Lanes<2> get(type r) { return {{r}}; }
    static __device__ __forceinline__ type put(const Lanes<2> &v) { return v.p[0]; }
};
template <> struct Raw<__nv_bfloat16, 1> {
    using type = unsigned short;
    static __device__ __forceinline__ Lanes<1> get(type r) { return {{__uint_as_float((unsigned)r << 16)}}; }
    static __device__ __forceinline__ type put(const Lanes<1> &v) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(v.p[0]));
    }
};
template <> struct Raw<__nv_bfloat16, 2> {
    using type = unsigned;
    static __device__ __forceinline__ Lanes<2> get(type r) { return {{get_pair(r)}}; }
    static __device__ __forceinline__ type put(const Lanes<2> &v) { return put_pair(v.p[0]); }
};
template <> struct Raw<__nv_bfloat16, 4> {
    using type = uint2;
    static __device__ __forceinline__ Lanes<4> get(type r) { return {{get_pair(r.x), get_pair(r.y)}}; }
    static __device__ __forceinline__ type put(const Lanes<4> &v) {
        return make_uint2(put_pair(v.p[0]), put_pair(v.p[1]));
    }
};

__device__ __forceinline__ unsigned cluster_ctas() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void st_async_v2(uint32_t raddr, float x, float y, uint32_t rbar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(raddr),
                 "r"(__float_as_uint(x)), "r"(__float_as_uint(y)), "r"(rbar)
                 : "memory");
}

// A product of gates past fp32's range would turn an empty state into NaN
// (inf * 0): it is held at the largest finite value instead.
__device__ __forceinline__ float finite(float A) {
    return fminf(fmaxf(A, -3.402823466e38f), 3.402823466e38f);
}

constexpr uint64_t kWaitNs = 2000000000ull;   // limit of a wait on the other CTAs of a cluster

// The joining of a tile's maps (A, H), one per warp and channel.  For that the
// CTA's threads change sides: G = W / V neighbouring lanes own a channel, each
// of them the maps of V consecutive warps, so that a map is read once and not
// by every warp after it (which cost a third of all instructions).  The owners
// form the CTA's map, carry the channel's state over the tile, and leave the
// state before each warp's rows in place of its H.  Everything is in two sets,
// used in turn, so that a set is not written again before all have read it.
// In a cluster each CTA's map goes to all of its CTAs by st.async, which
// completes their mbarrier: a cluster barrier per tile waited for the tile's
// global stores as well (its release) and took 12000 cycles.
template <int V, int W> struct Joint {
    static constexpr int G = W / V, C = 32 * V;
    static_assert(G * V == W, "");
    float A[2][W][C + 4], H[2][W][C + 4];   // the 4: owners of a warp read distinct banks
    uint64_t bar[2];
};

template <int V, int W> struct Join {
    using J = Joint<V, W>;
    using Vec = std::conditional_t<V == 4, float4, std::conditional_t<V == 2, float2, float>>;
    J &j;
    float2 *cta;             // [2][ctas][C]: the cluster's maps
    unsigned ctas, rank;
    int warp, lane, channel, sub;
    float state;             // of the owned channel
    int it = 0;
    bool alive = true;
    int *err;

    // first: the strip's first channel in the states [B,H,D], of which `left` exist.
    __device__ __forceinline__ Join(J &j_, unsigned ctas_, unsigned rank_, const float *first, int left, int *err_)
        : j(j_), cta(reinterpret_cast<float2 *>(&j_ + 1)), ctas(ctas_), rank(rank_), warp(threadIdx.x >> 5),
          lane(threadIdx.x & 31), channel(threadIdx.x / J::G), sub(threadIdx.x % J::G), err(err_) {
        state = first && channel < left ? first[channel] : 0.f;
        if (ctas > 1) {
            if (threadIdx.x == 0) {
                tc::mbar_init(&j.bar[0], 1);
                tc::mbar_init(&j.bar[1], 1);
                tc::fence_mbar_init();
            }
            tc::cluster_arrive_release();   // the others' barriers are there once they have started
            tc::cluster_wait_acquire();
        }
    }
    // Writes the last state; no CTA leaves while another may still store into it.
    __device__ __forceinline__ void end(float *first, int left) {
        if (first && channel < left && sub == 0 && rank == 0) first[channel] = state;
        if (ctas > 1) {
            tc::cluster_arrive_release();
            tc::cluster_wait_acquire();
        }
    }

    static __device__ __forceinline__ void put(float *to, const Lanes<V> &v) { *reinterpret_cast<Vec *>(to) = *reinterpret_cast<const Vec *>(&v); }
    static __device__ __forceinline__ Lanes<V> get(const float *from) {
        const Vec r = *reinterpret_cast<const Vec *>(from);
        return *reinterpret_cast<const Lanes<V> *>(&r);
    }

    // A, H: this thread's rows; returns the state before them.
    __device__ __forceinline__ Lanes<V> operator()(const Lanes<V> &A, const Lanes<V> &H) {
        const int set = it & 1;
        Lanes<V> bounded;
#pragma unroll
        for (int v = 0; v < V; v++) bounded.set(v, finite(A.get(v)));
        put(&j.A[set][warp][lane * V], bounded);
        put(&j.H[set][warp][lane * V], H);
        __syncthreads();
        float a[V], h[V], ta = 1.f, th = 0.f;
#pragma unroll
        for (int i = 0; i < V; i++) a[i] = j.A[set][sub * V + i][channel], h[i] = j.H[set][sub * V + i][channel];
#pragma unroll
        for (int i = 0; i < V; i++) ta *= a[i], th = fmaf(a[i], th, h[i]);
        ta = finite(ta);
        float ea = 1.f, eh = 0.f;   // map of the owners before this one
        if constexpr (J::G > 1) {
#pragma unroll
            for (int o = 1; o < J::G; o *= 2) {
                const float oa = __shfl_up_sync(~0u, ta, o, J::G), oh = __shfl_up_sync(~0u, th, o, J::G);
                if (sub >= o) th = fmaf(ta, oh, th), ta = finite(ta * oa);
            }
            ea = __shfl_up_sync(~0u, ta, 1, J::G);
            eh = __shfl_up_sync(~0u, th, 1, J::G);
            if (sub == 0) ea = 1.f, eh = 0.f;
            ta = __shfl_sync(~0u, ta, J::G - 1, J::G);
            th = __shfl_sync(~0u, th, J::G - 1, J::G);
        }
        float start = state;
        if (ctas == 1) {
            state = fmaf(ta, state, th);
        } else {
            float2 *maps = cta + (size_t)set * ctas * J::C;
            if (threadIdx.x == 0) tc::mbar_arrive_expect_tx(&j.bar[set], ctas * J::C * (unsigned)sizeof(float2));
            const uint32_t to = tc::smem_u32(&maps[rank * J::C + channel]), bar = tc::smem_u32(&j.bar[set]);
            for (unsigned r = sub; r < ctas; r += J::G)
                st_async_v2(tc::mapa_shared(to, r), ta, th, tc::mapa_shared(bar, r));
            if (alive && !tc::mbar_try_wait(&j.bar[set], (it >> 1) & 1)) {
                alive = tc::mbar_wait_bounded(&j.bar[set], (it >> 1) & 1, globaltimer_ns() + kWaitNs, nullptr);
                if (!alive) record_error(err, kErrTimeout);
            }
            for (unsigned r = 0; r < ctas; r++) {
                if (r == rank) start = state;
                const float2 m = maps[r * J::C + channel];
                state = fmaf(m.x, state, m.y);
            }
        }
        start = fmaf(ea, start, eh);
#pragma unroll
        for (int i = 0; i < V; i++) {
            j.H[set][sub * V + i][channel] = start;
            start = fmaf(a[i], start, h[i]);
        }
        __syncthreads();
        it++;
        return get(&j.H[set][warp][lane * V]);
    }
};

// A thread's place: its channels, its sequence, its CTA's part of the cluster.
template <int V> struct Place {
    unsigned ctas, rank;
    long long b, h, bh;
    int d0, d, len;          // first channel of the strip, of the thread
    bool ok;                 // its channels exist (all V or none: D is a multiple of V)
    __device__ __forceinline__ explicit Place(const Dims &s) {
        ctas = cluster_ctas();
        rank = tc::cluster_ctarank();
        const unsigned strip = blockIdx.x / ctas;
        bh = strip / s.strips;
        b = bh / s.H;
        h = bh % s.H;
        d0 = (int)(strip % s.strips) * 32 * V;
        d = d0 + (threadIdx.x & 31) * V;
        ok = d < s.D;
        len = s.lens ? min(max(s.lens[b], 0), s.N) : s.N;
    }
    template <typename T> __device__ __forceinline__ T *rows(const la_view &v) const {
        return static_cast<T *>(v.data) + b * v.sb + h * v.sh + (ok ? d : 0);
    }
};

// Rows at or past a sequence's length become 0.
template <typename T, int V, int W>
__device__ __forceinline__ void clear_rows(T *p, long long sn, const Place<V> &q, long long N) {
    using RT = typename Raw<T, V>::type;
    if (!q.ok) return;
    for (long long t = q.len + q.rank * W + (threadIdx.x >> 5); t < N; t += q.ctas * W)
        *reinterpret_cast<RT *>(p + t * sn) = RT{};
}

template <typename T, int GATE, int V, int W, int R, int CTAS>
__global__ void __launch_bounds__(32 * W, CTAS) rec_forward_kernel(la_view x, la_view g, la_view out, Dims s,
                                                                  const float *h0, float *hN) {
    using RT = typename Raw<T, V>::type;
    using Io = Raw<T, V>;
    extern __shared__ __align__(16) unsigned char smem[];
    pdl_wait_cta();
    const Place<V> q(s);
    const long long at = q.bh * s.D + q.d0;
    Join<V, W> join(*reinterpret_cast<Joint<V, W> *>(smem), q.ctas, q.rank, h0 ? h0 + at : nullptr, s.D - q.d0, s.err);
    const T *px = q.template rows<T>(x), *pg = q.template rows<T>(g);
    T *po = q.template rows<T>(out);
    const long long step = (long long)q.ctas * W * R;                // rows of a tile
    const long long first = (long long)(q.rank * W + join.warp) * R; // this warp's rows in it
    const int tiles = (int)((q.len + step - 1) / step);
    // rows of this thread in the tile that starts at t0
    auto rows_at = [&](long long t0) { return q.ok ? (int)min((long long)R, max(q.len - t0, 0LL)) : 0; };

    RT rx[R] = {}, rg[R] = {};   // the next tile's rows, on their way while this one's are used
    {
        const int n = rows_at(first);
        const T *ax = px + (n ? first : 0) * x.sn, *ag = pg + (n ? first : 0) * g.sn;
#pragma unroll
        for (int r = 0; r < R; r++, ax += x.sn, ag += g.sn)
            if (r < n) rx[r] = *reinterpret_cast<const RT *>(ax), rg[r] = *reinterpret_cast<const RT *>(ag);
    }
    for (int it = 0; it < tiles; it++) {
        const long long t0 = it * step + first;
        const int n = rows_at(t0), next = rows_at(t0 + step);
        const T *ax = px + (next ? t0 + step : 0) * x.sn, *ag = pg + (next ? t0 + step : 0) * g.sn;
        Lanes<V> a[R], u[R];
#pragma unroll
        for (int r = 0; r < R; r++, ax += x.sn, ag += g.sn) {
            Lanes<V> w;
            const Lanes<V> xv = Io::get(rx[r]), gv = Io::get(rg[r]);
            if (r < next) rx[r] = *reinterpret_cast<const RT *>(ax), rg[r] = *reinterpret_cast<const RT *>(ag);
            gate_of<GATE, V>(gv, a[r], w);
            u[r] = GATE == LA_GATE_SIGMOID ? mul(w, xv) : xv;
        }
        if (n < R) {   // rows past the end leave the state as it is
#pragma unroll
            for (int r = 0; r < R; r++)
                if (r >= n) a[r] = all<V>(1.f), u[r] = all<V>(0.f);
        }
        Lanes<V> A = a[0], H = u[0];
#pragma unroll
        for (int r = 1; r < R; r++) A = mul(A, a[r]), H = fma(a[r], H, u[r]);
        Lanes<V> h = join(A, H);
        T *p = po + (n ? t0 : 0) * out.sn;
#pragma unroll
        for (int r = 0; r < R; r++, p += out.sn) {
            h = fma(a[r], h, u[r]);
            if (r < n) *reinterpret_cast<RT *>(p) = Io::put(h);
        }
    }
    clear_rows<T, V, W>(po, out.sn, q, s.N);
    join.end(hN ? hN + at : nullptr, s.D - q.d0);
}

// Up to kShortRows tokens (a decoded token among them) there is nothing to
// split: a thread takes its channels' few rows in order.
constexpr int kShortRows = 16, kShortThreads = 128;

template <typename T, int GATE, int V>
__global__ void __launch_bounds__(kShortThreads) rec_short_kernel(la_view x, la_view g, la_view out, Dims s,
                                                                  long long groups, const float *h0, float *hN) {
    using RT = typename Raw<T, V>::type;
    constexpr int R = 4;
    pdl_wait_cta();
    const long long i = (long long)blockIdx.x * kShortThreads + threadIdx.x;
    if (i >= groups) return;
    const unsigned per = (unsigned)(s.D / V);
    const long long bh = i / per, b = bh / s.H, h = bh % s.H;
    const int d = (int)(i % per) * V;
    const int len = s.lens ? min(max(s.lens[b], 0), s.N) : s.N;
    const T *px = static_cast<const T *>(x.data) + b * x.sb + h * x.sh + d;
    const T *pg = static_cast<const T *>(g.data) + b * g.sb + h * g.sh + d;
    T *po = static_cast<T *>(out.data) + b * out.sb + h * out.sh + d;
    Lanes<V> c;
#pragma unroll
    for (int v = 0; v < V; v++) c.set(v, h0 ? h0[i * V + v] : 0.f);
    for (int t0 = 0; t0 < len; t0 += R) {
        RT rx[R], rg[R];
#pragma unroll
        for (int r = 0; r < R; r++) {
            rx[r] = rg[r] = RT{};
            if (t0 + r < len) {
                rx[r] = *reinterpret_cast<const RT *>(px + (t0 + r) * x.sn);
                rg[r] = *reinterpret_cast<const RT *>(pg + (t0 + r) * g.sn);
            }
        }
#pragma unroll
        for (int r = 0; r < R; r++) {
            if (t0 + r >= len) break;
            Lanes<V> a, w;
            gate_of<GATE, V>(Raw<T, V>::get(rg[r]), a, w);
            c = fma(a, c, mul(w, Raw<T, V>::get(rx[r])));
            *reinterpret_cast<RT *>(po + (t0 + r) * out.sn) = Raw<T, V>::put(c);
        }
    }
    for (int t = len; t < s.N; t++) *reinterpret_cast<RT *>(po + t * out.sn) = RT{};
    if (hN) {
#pragma unroll
        for (int v = 0; v < V; v++) hN[i * V + v] = c.get(v);
    }
}

// The same walk from the last token to the first: the state is mu_t = a_t l_t,
// which the token before adds to its own gradient.
template <typename T, int GATE, int V, int W, int R, int CTAS>
__global__ void __launch_bounds__(32 * W, CTAS) rec_backward_kernel(la_view x, la_view g, la_view out, la_view dout,
                                                                   la_view dx, la_view dg, Dims s, const float *h0,
                                                                   const float *dhN, float *dh0) {
    using RT = typename Raw<T, V>::type;
    using Io = Raw<T, V>;
    constexpr bool kSigmoid = GATE == LA_GATE_SIGMOID;
    extern __shared__ __align__(16) unsigned char smem[];
    pdl_wait_cta();
    const Place<V> q(s);
    const long long at = q.bh * s.D + q.d0;
    Join<V, W> join(*reinterpret_cast<Joint<V, W> *>(smem), q.ctas, q.rank, dhN ? dhN + at : nullptr, s.D - q.d0,
                    s.err);
    const T *px = kSigmoid ? q.template rows<T>(x) : nullptr, *pg = q.template rows<T>(g);
    const T *po = q.template rows<T>(out), *pd = q.template rows<T>(dout);
    T *pdx = q.template rows<T>(dx), *pdg = q.template rows<T>(dg);
    const long long step = (long long)q.ctas * W * R;
    const long long first = (long long)(q.rank * W + join.warp) * R;
    const int tiles = (int)((q.len + step - 1) / step);
    // rows t, t - 1, ... of this thread in the tile whose row `first` is t
    auto rows_at = [&](long long t) { return q.ok ? (int)min((long long)R, max(t + 1, 0LL)) : 0; };

    // the next tile's rows on their way: g and dout from where this tile's are
    // turned into a, w and d, h_{t-1} and x from where they are used
    RT rg[R] = {}, rd[R] = {}, rb[R] = {}, rx[R] = {};
    {
        const long long t = q.len - 1 - first;
        const int n = rows_at(t);
#pragma unroll
        for (int r = 0; r < R; r++) {
            if (r < n) {
                rg[r] = *reinterpret_cast<const RT *>(pg + (t - r) * g.sn);
                rd[r] = *reinterpret_cast<const RT *>(pd + (t - r) * dout.sn);
                if (t - r > 0) rb[r] = *reinterpret_cast<const RT *>(po + (t - r - 1) * out.sn);
                if constexpr (kSigmoid) rx[r] = *reinterpret_cast<const RT *>(px + (t - r) * x.sn);
            }
        }
    }
    for (int it = 0; it < tiles; it++) {
        const long long t0 = q.len - 1 - (it * step + first), t1 = t0 - step;
        const int n = rows_at(t0), next = rows_at(t1);
        const T *ag = pg + (next ? t1 : 0) * g.sn, *ad = pd + (next ? t1 : 0) * dout.sn;
        Lanes<V> a[R], w[R], d[R];
#pragma unroll
        for (int r = 0; r < R; r++, ag -= g.sn, ad -= dout.sn) {
            const Lanes<V> gv = Io::get(rg[r]);
            d[r] = Io::get(rd[r]);
            if (r < next) rg[r] = *reinterpret_cast<const RT *>(ag), rd[r] = *reinterpret_cast<const RT *>(ad);
            gate_of<GATE, V>(gv, a[r], w[r]);
        }
        if (n < R) {   // rows before the first leave the state as it is
#pragma unroll
            for (int r = 0; r < R; r++)
                if (r >= n) a[r] = all<V>(1.f), d[r] = all<V>(0.f);
        }
        Lanes<V> A = a[0], H = mul(a[0], d[0]);
#pragma unroll
        for (int r = 1; r < R; r++) A = mul(A, a[r]), H = mul(a[r], add(d[r], H));
        Lanes<V> mu = join(A, H);
        T *to_x = pdx + (n ? t0 : 0) * dx.sn, *to_g = pdg + (n ? t0 : 0) * dg.sn;
        const T *ab = po + (next ? t1 - 1 : 0) * out.sn;
        const T *ax = kSigmoid ? px + (next ? t1 : 0) * x.sn : nullptr;
        const int next_b = next && t1 - next < 0 ? next - 1 : next;   // row 0 has no row before it
#pragma unroll
        for (int r = 0; r < R; r++, to_x -= dx.sn, to_g -= dg.sn) {
            Lanes<V> before = Io::get(rb[r]), xv;
            if (r < next_b) rb[r] = *reinterpret_cast<const RT *>(ab);
            ab -= out.sn;
            if constexpr (kSigmoid) {
                xv = Io::get(rx[r]);
                if (r < next) rx[r] = *reinterpret_cast<const RT *>(ax);
                ax -= x.sn;
            }
            if (t0 == r && q.ok) {   // the first token: the state that the forward started from
#pragma unroll
                for (int v = 0; v < V; v++) before.set(v, h0 ? h0[q.bh * s.D + q.d + v] : 0.f);
            }
            const Lanes<V> l = add(d[r], mu);
            mu = mul(a[r], l);
            const Lanes<V> ox = kSigmoid ? mul(l, w[r]) : l;
            const Lanes<V> og = kSigmoid ? mul(mul(mu, w[r]), fma(xv, all<V>(-1.f), before))
                                         : mul(GATE == LA_GATE_LOG ? mu : l, before);
            if (r < n) {
                *reinterpret_cast<RT *>(to_x) = Io::put(ox);
                *reinterpret_cast<RT *>(to_g) = Io::put(og);
            }
        }
    }
    clear_rows<T, V, W>(pdx, dx.sn, q, s.N);
    clear_rows<T, V, W>(pdg, dg.sn, q, s.N);
    join.end(dh0 ? dh0 + at : nullptr, s.D - q.d0);
}

// Tiles: W warps of R rows a CTA, CTAS of them a SM.
#ifndef FWD_CFG
#define FWD_CFG 8, 8, 2
#endif
#ifndef BWD_CFG
#define BWD_CFG 8, 8, 1
#endif
#ifndef MAXK
#define MAXK 8
#endif
#ifndef FILL
#define FILL 2
#endif
template <int W_, int R_, int C_> struct Tile {
    static constexpr int W = W_, R = R_, CTAS = C_;
};
using Fwd = Tile<FWD_CFG>;
using Bwd = Tile<BWD_CFG>;

// CTAs per strip: enough that every SM has as many as it can hold, as far as
// the tokens fill their tiles.
int cluster_of(long long strips, int N, int rows, int ctas, const DeviceInfo &dev) {
    int k = 1;
    while (k < MAXK && strips * k * FILL < (long long)ctas * dev.sm_count * 2 && (long long)N > (long long)k * rows) k *= 2;
    return k;
}

template <int V, typename Tile, typename Kernel, typename... Args>
cudaError_t launch_tiles(Kernel kernel, const RecProblem &p, Dims s, const DeviceInfo &dev, Args... args) {
    const long long strips = (long long)p.B * p.H * s.strips;
    const int k = cluster_of(strips, p.N, Tile::W * Tile::R, Tile::CTAS, dev);
    const size_t smem = sizeof(Joint<V, Tile::W>) + (k > 1 ? 2 * k * 32 * V * sizeof(float2) : 0);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && k > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3((unsigned)(strips * k)), dim3(32 * Tile::W), smem, p.stream, (unsigned)k, args...);
    count_launches(1);
    return e;
}

// Channels a lane takes: 8 bytes of a row, or as many as its alignment and the
// strides allow; half of that where the last strip would be less than half full.
template <typename T> int lane_channels(int D, std::initializer_list<la_view> views) {
    const int most = 8 / (int)sizeof(T);
    unsigned long long bits = (unsigned)D;
    for (const la_view &v : views)
        bits |= (unsigned long long)(reinterpret_cast<uintptr_t>(v.data) / sizeof(T)) | v.sb | v.sh | v.sn;
#ifdef MAXV
    int V = MAXV / (int)(sizeof(T) / 2);
#else
    int V = most;
#endif
    while (V > 1 && (bits & (V - 1))) V /= 2;
    if (V == most && D % (32 * V) != 0 && D % (32 * V) <= 16 * V && D < 256 * V) V /= 2;
    return V;
}

template <typename T, int GATE, int V> cudaError_t forward_v(const RecProblem &p, const DeviceInfo &dev) {
    Dims s{p.lens, p.H, p.N, p.D, (p.D + 32 * V - 1) / (32 * V)};
    if (p.N <= kShortRows) {
        const long long groups = (long long)p.B * p.H * (p.D / V);
        const cudaError_t e = launch_pdl(rec_short_kernel<T, GATE, V>,
                                         dim3((unsigned)((groups + kShortThreads - 1) / kShortThreads)),
                                         dim3(kShortThreads), 0, p.stream, 0u, p.x, p.g, p.out, s, groups, p.h0, p.hN);
        count_launches(1);
        return e;
    }
    s.err = dev.err_word;
    return launch_tiles<V, Fwd>(rec_forward_kernel<T, GATE, V, Fwd::W, Fwd::R, Fwd::CTAS>, p, s, dev, p.x, p.g, p.out,
                                s, p.h0, p.hN);
}

template <typename T, int GATE, int V> cudaError_t backward_v(const RecProblem &p, const DeviceInfo &dev) {
    Dims s{p.lens, p.H, p.N, p.D, (p.D + 32 * V - 1) / (32 * V)};
    s.err = dev.err_word;
    return launch_tiles<V, Bwd>(rec_backward_kernel<T, GATE, V, Bwd::W, Bwd::R, Bwd::CTAS>, p, s, dev, p.x, p.g, p.out,
                                p.dout, p.dx, p.dg, s, p.h0, p.dhN, p.dh0);
}

template <int GATE> cudaError_t forward_g(const RecProblem &p, const DeviceInfo &dev) {
    if (p.dtype == LA_DTYPE_F32)
        return lane_channels<float>(p.D, {p.x, p.g, p.out}) == 2 ? forward_v<float, GATE, 2>(p, dev)
                                                                 : forward_v<float, GATE, 1>(p, dev);
    switch (lane_channels<__nv_bfloat16>(p.D, {p.x, p.g, p.out})) {
        case 4: return forward_v<__nv_bfloat16, GATE, 4>(p, dev);
        case 2: return forward_v<__nv_bfloat16, GATE, 2>(p, dev);
        default: return forward_v<__nv_bfloat16, GATE, 1>(p, dev);
    }
}

template <int GATE> cudaError_t backward_g(const RecProblem &p, const DeviceInfo &dev) {
    if (p.dtype == LA_DTYPE_F32)
        return lane_channels<float>(p.D, {p.x, p.g, p.out, p.dout, p.dx, p.dg}) == 2
                   ? backward_v<float, GATE, 2>(p, dev)
                   : backward_v<float, GATE, 1>(p, dev);
    switch (lane_channels<__nv_bfloat16>(p.D, {p.x, p.g, p.out, p.dout, p.dx, p.dg})) {
        case 4: return backward_v<__nv_bfloat16, GATE, 4>(p, dev);
        case 2: return backward_v<__nv_bfloat16, GATE, 2>(p, dev);
        default: return backward_v<__nv_bfloat16, GATE, 1>(p, dev);
    }
}

}  // namespace

cudaError_t recurrence_forward(const RecProblem &p, const DeviceInfo &dev) {
    switch (p.gate) {
        case LA_GATE_DECAY: return forward_g<LA_GATE_DECAY>(p, dev);
        case LA_GATE_LOG: return forward_g<LA_GATE_LOG>(p, dev);
        case LA_GATE_SIGMOID: return forward_g<LA_GATE_SIGMOID>(p, dev);
    }
    return cudaErrorInvalidValue;
}

cudaError_t recurrence_backward(const RecProblem &p, const DeviceInfo &dev) {
    switch (p.gate) {
        case LA_GATE_DECAY: return backward_g<LA_GATE_DECAY>(p, dev);
        case LA_GATE_LOG: return backward_g<LA_GATE_LOG>(p, dev);
        case LA_GATE_SIGMOID: return backward_g<LA_GATE_SIGMOID>(p, dev);
    }
    return cudaErrorInvalidValue;
}

}  // namespace la
