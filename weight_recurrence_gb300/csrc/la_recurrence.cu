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
#include <algorithm>

#include "la_gate.cuh"
#include "la_layer.h"

namespace la {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCluster = 8;

struct Dims {
    const int *lens;
    int H, N, D;
    int strips;        // groups of 32 lanes' channels in a sequence
};

// V neighbouring channels of one row as they lie in memory.
template <typename T, int V> struct Raw;
template <> struct Raw<float, 1> {
    using type = float;
    static __device__ __forceinline__ void get(type r, float (&v)[1]) { v[0] = r; }
    static __device__ __forceinline__ type put(const float (&v)[1]) { return v[0]; }
};
template <> struct Raw<__nv_bfloat16, 1> {
    using type = unsigned short;
    static __device__ __forceinline__ void get(type r, float (&v)[1]) { v[0] = __uint_as_float((unsigned)r << 16); }
    static __device__ __forceinline__ type put(const float (&v)[1]) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    }
};
template <> struct Raw<__nv_bfloat16, 2> {
    using type = unsigned;
    static __device__ __forceinline__ void get(type r, float (&v)[2]) {
        v[0] = __uint_as_float(r << 16);
        v[1] = __uint_as_float(r & 0xffff0000u);
    }
    static __device__ __forceinline__ type put(const float (&v)[2]) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[0], v[1]);
        return *reinterpret_cast<const unsigned *>(&p);
    }
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// Copies one thread's channels of a row to its own place in shared memory:
// asynchronously where they are 4 bytes (zeros where !ok), else (one bf16) at once.
template <typename RT> __device__ __forceinline__ void copy_row(RT *dst, const void *src, bool ok) {
    if constexpr (sizeof(RT) == 4) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(ok ? 4 : 0)
                     : "memory");
    } else {
        *dst = ok ? *static_cast<const RT *>(src) : RT(0);
    }
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

__device__ __forceinline__ unsigned cluster_ctas() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void store_remote(const void *local, unsigned rank, float v) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(local)), "r"(rank));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

// A map's value; an A past fp32's range leaves an empty state empty.
__device__ __forceinline__ float apply(float A, float c, float H) { return c == 0.f ? H : fmaf(A, c, H); }

// Maps of one tile: two sets, so that one barrier a tile keeps a set whole
// until every thread has read it.
template <int V> struct Maps {
    float warp[2][kWarps][2][32 * V];        // (A, H) of each warp's rows
    float cta[2][kMaxCluster][2][32 * V];    // of each CTA of the cluster, written by it
};

// Joins the tile's maps.  A, H: this thread's rows; state: the state before
// the tile, replaced by the state after it; returns in `before` the state
// before this thread's rows.
template <int V>
__device__ __forceinline__ void join(Maps<V> &m, int set, unsigned ctas, unsigned rank, const float (&A)[V],
                                     const float (&H)[V], float (&state)[V], float (&before)[V]) {
    const int warp = threadIdx.x >> 5, at = (threadIdx.x & 31) * V;
#pragma unroll
    for (int v = 0; v < V; v++) m.warp[set][warp][0][at + v] = A[v], m.warp[set][warp][1][at + v] = H[v];
    __syncthreads();
    float pa[V], ph[V], ta[V], th[V];        // maps of the warps before this one, and of all
#pragma unroll
    for (int v = 0; v < V; v++) pa[v] = ta[v] = 1.f, ph[v] = th[v] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
        if (w == warp) {
#pragma unroll
            for (int v = 0; v < V; v++) pa[v] = ta[v], ph[v] = th[v];
        }
#pragma unroll
        for (int v = 0; v < V; v++) {
            const float a = m.warp[set][w][0][at + v], h = m.warp[set][w][1][at + v];
            ta[v] *= a;
            th[v] = apply(a, th[v], h);
        }
    }
    float start[V];
#pragma unroll
    for (int v = 0; v < V; v++) start[v] = state[v];
    if (ctas == 1) {
#pragma unroll
        for (int v = 0; v < V; v++) state[v] = apply(ta[v], state[v], th[v]);
    } else {
        for (unsigned r = warp; r < ctas; r += kWarps) {
#pragma unroll
            for (int v = 0; v < V; v++) {
                store_remote(&m.cta[set][rank][0][at + v], r, ta[v]);
                store_remote(&m.cta[set][rank][1][at + v], r, th[v]);
            }
        }
        cluster_arrive();
        cluster_wait();
        for (unsigned r = 0; r < ctas; r++) {
            if (r == rank) {
#pragma unroll
                for (int v = 0; v < V; v++) start[v] = state[v];
            }
#pragma unroll
            for (int v = 0; v < V; v++) state[v] = apply(m.cta[set][r][0][at + v], state[v], m.cta[set][r][1][at + v]);
        }
    }
#pragma unroll
    for (int v = 0; v < V; v++) before[v] = apply(pa[v], start[v], ph[v]);
}

// A thread's place: its channels, its sequence, its CTA's part of the cluster.
template <int V> struct Place {
    unsigned ctas, rank;
    long long b, h, state;   // state: index of its first channel in [B,H,D]
    int d, len;
    bool ok;                 // its channels exist (all V or none: D is a multiple of V)
    __device__ __forceinline__ explicit Place(const Dims &s) {
        ctas = cluster_ctas();
        rank = cluster_rank();
        const unsigned strip = blockIdx.x / ctas;
        const long long bh = strip / s.strips;
        b = bh / s.H;
        h = bh % s.H;
        d = (int)(strip % s.strips) * 32 * V + (threadIdx.x & 31) * V;
        ok = d < s.D;
        state = bh * s.D + d;
        len = s.lens ? min(max(s.lens[b], 0), s.N) : s.N;
    }
    template <typename T> __device__ __forceinline__ T *rows(const la_view &v) const {
        return static_cast<T *>(v.data) + b * v.sb + h * v.sh + (ok ? d : 0);
    }
};

// Rows [from, N) of an output become 0.
template <typename T, int V>
__device__ __forceinline__ void clear_rows(T *p, long long sn, const Place<V> &q, long long N) {
    if (!q.ok) return;
    for (long long t = q.len + q.rank * kWarps + (threadIdx.x >> 5); t < N; t += q.ctas * kWarps)
        *reinterpret_cast<typename Raw<T, V>::type *>(p + t * sn) = 0;
}

constexpr int kFwdRows = 16, kFwdStages = 3;

template <typename T, int V> struct FwdShared {
    Maps<V> maps;
    typename Raw<T, V>::type tile[kFwdStages][2][kFwdRows][kThreads];
};

template <typename T, int GATE, int V>
__global__ void __launch_bounds__(kThreads, 2) rec_forward_kernel(la_view x, la_view g, la_view out, Dims s,
                                                                  const float *h0, float *hN) {
    using RT = typename Raw<T, V>::type;
    constexpr int R = kFwdRows, S = kFwdStages;
    extern __shared__ __align__(16) unsigned char smem[];
    FwdShared<T, V> &sh = *reinterpret_cast<FwdShared<T, V> *>(smem);
    pdl_wait_cta();
    const Place<V> q(s);
    const int warp = threadIdx.x >> 5;
    const T *px = q.template rows<T>(x), *pg = q.template rows<T>(g);
    T *po = q.template rows<T>(out);
    const long long step = (long long)q.ctas * kWarps * R;           // rows of a tile
    const long long first = (long long)(q.rank * kWarps + warp) * R; // this warp's rows in it
    const int tiles = (int)((q.len + step - 1) / step);

    auto fetch = [&](int it) {
        if (it < tiles) {
#pragma unroll
            for (int r = 0; r < R; r++) {
                const long long t = it * step + first + r;
                const bool ok = q.ok && t < q.len;
                copy_row<RT>(&sh.tile[it % S][0][r][threadIdx.x], ok ? px + t * x.sn : px, ok);
                copy_row<RT>(&sh.tile[it % S][1][r][threadIdx.x], ok ? pg + t * g.sn : pg, ok);
            }
        }
        copy_commit();
    };

    float state[V];
#pragma unroll
    for (int v = 0; v < V; v++) state[v] = h0 && q.ok ? h0[q.state + v] : 0.f;
    if (q.ctas > 1) {   // the others' shared memory is there once they have started
        cluster_arrive();
        cluster_wait();
    }
    for (int i = 0; i < S - 1; i++) fetch(i);
    for (int it = 0; it < tiles; it++) {
        fetch(it + S - 1);   // into the stage that this thread emptied a tile ago
        copy_wait<S - 1>();
        const long long t0 = it * step + first;
        float a[R][V], u[R][V], A[V], H[V], h[V];
#pragma unroll
        for (int v = 0; v < V; v++) A[v] = 1.f, H[v] = 0.f;
#pragma unroll
        for (int r = 0; r < R; r++) {
            float xv[V], gv[V];
            Raw<T, V>::get(sh.tile[it % S][0][r][threadIdx.x], xv);
            Raw<T, V>::get(sh.tile[it % S][1][r][threadIdx.x], gv);
            const bool in = t0 + r < q.len;
#pragma unroll
            for (int v = 0; v < V; v++) {
                float w;
                gate_of<GATE>(gv[v], a[r][v], w);
                u[r][v] = in ? w * xv[v] : 0.f;
                a[r][v] = in ? a[r][v] : 1.f;
                A[v] *= a[r][v];
                H[v] = fmaf(a[r][v], H[v], u[r][v]);
            }
        }
        join<V>(sh.maps, it & 1, q.ctas, q.rank, A, H, state, h);
#pragma unroll
        for (int r = 0; r < R; r++) {
#pragma unroll
            for (int v = 0; v < V; v++) h[v] = fmaf(a[r][v], h[v], u[r][v]);
            if (q.ok && t0 + r < q.len) *reinterpret_cast<RT *>(po + (t0 + r) * out.sn) = Raw<T, V>::put(h);
        }
    }
    clear_rows<T, V>(po, out.sn, q, s.N);
    if (hN && q.ok && warp == 0 && q.rank == 0) {
#pragma unroll
        for (int v = 0; v < V; v++) hN[q.state + v] = state[v];
    }
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
    float c[V];
#pragma unroll
    for (int v = 0; v < V; v++) c[v] = h0 ? h0[i * V + v] : 0.f;
    for (int t0 = 0; t0 < len; t0 += R) {
        RT rx[R], rg[R];
#pragma unroll
        for (int r = 0; r < R; r++) {
            rx[r] = rg[r] = RT(0);
            if (t0 + r < len) {
                rx[r] = *reinterpret_cast<const RT *>(px + (t0 + r) * x.sn);
                rg[r] = *reinterpret_cast<const RT *>(pg + (t0 + r) * g.sn);
            }
        }
#pragma unroll
        for (int r = 0; r < R; r++) {
            if (t0 + r >= len) break;
            float xv[V], gv[V];
            Raw<T, V>::get(rx[r], xv);
            Raw<T, V>::get(rg[r], gv);
#pragma unroll
            for (int v = 0; v < V; v++) {
                float a, w;
                gate_of<GATE>(gv[v], a, w);
                c[v] = fmaf(a, c[v], w * xv[v]);
            }
            *reinterpret_cast<RT *>(po + (t0 + r) * out.sn) = Raw<T, V>::put(c);
        }
    }
    for (int t = len; t < s.N; t++) *reinterpret_cast<RT *>(po + t * out.sn) = RT(0);
    if (hN) {
#pragma unroll
        for (int v = 0; v < V; v++) hN[i * V + v] = c[v];
    }
}

constexpr int kBwdRows = 8, kBwdStages = 3;

template <typename T, int GATE, int V> struct BwdShared {
    Maps<V> maps;
    typename Raw<T, V>::type tile[kBwdStages][GATE == LA_GATE_SIGMOID ? 4 : 3][kBwdRows][kThreads];
};

// The same walk from the last token to the first: the state is mu_t = a_t l_t,
// which the token before adds to its own gradient.
template <typename T, int GATE, int V>
__global__ void __launch_bounds__(kThreads, 2) rec_backward_kernel(la_view x, la_view g, la_view out, la_view dout,
                                                                   la_view dx, la_view dg, Dims s, const float *h0,
                                                                   const float *dhN, float *dh0) {
    using RT = typename Raw<T, V>::type;
    constexpr int R = kBwdRows, S = kBwdStages;
    constexpr bool kSigmoid = GATE == LA_GATE_SIGMOID;
    extern __shared__ __align__(16) unsigned char smem[];
    BwdShared<T, GATE, V> &sh = *reinterpret_cast<BwdShared<T, GATE, V> *>(smem);
    pdl_wait_cta();
    const Place<V> q(s);
    const int warp = threadIdx.x >> 5;
    const T *px = kSigmoid ? q.template rows<T>(x) : nullptr, *pg = q.template rows<T>(g);
    const T *po = q.template rows<T>(out), *pd = q.template rows<T>(dout);
    T *pdx = q.template rows<T>(dx), *pdg = q.template rows<T>(dg);
    const long long step = (long long)q.ctas * kWarps * R;
    const long long first = (long long)(q.rank * kWarps + warp) * R;
    const int tiles = (int)((q.len + step - 1) / step);

    auto fetch = [&](int it) {   // rows counted from the end
        if (it < tiles) {
#pragma unroll
            for (int r = 0; r < R; r++) {
                const long long t = q.len - 1 - (it * step + first + r);
                const bool ok = q.ok && t >= 0;
                RT(*to)[R][kThreads] = sh.tile[it % S];
                copy_row<RT>(&to[0][r][threadIdx.x], ok ? pg + t * g.sn : pg, ok);
                copy_row<RT>(&to[1][r][threadIdx.x], ok ? pd + t * dout.sn : pd, ok);
                copy_row<RT>(&to[2][r][threadIdx.x], ok && t > 0 ? po + (t - 1) * out.sn : po, ok && t > 0);
                if constexpr (kSigmoid) copy_row<RT>(&to[3][r][threadIdx.x], ok ? px + t * x.sn : px, ok);
            }
        }
        copy_commit();
    };

    float state[V], h_first[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
        state[v] = dhN && q.ok ? dhN[q.state + v] : 0.f;
        h_first[v] = h0 && q.ok ? h0[q.state + v] : 0.f;
    }
    if (q.ctas > 1) {
        cluster_arrive();
        cluster_wait();
    }
    for (int i = 0; i < S - 1; i++) fetch(i);
    for (int it = 0; it < tiles; it++) {
        fetch(it + S - 1);
        copy_wait<S - 1>();
        const long long t0 = q.len - 1 - (it * step + first);
        RT(*tile)[R][kThreads] = sh.tile[it % S];
        float a[R][V], w[R][V], d[R][V], A[V], H[V], mu[V];
#pragma unroll
        for (int v = 0; v < V; v++) A[v] = 1.f, H[v] = 0.f;
#pragma unroll
        for (int r = 0; r < R; r++) {
            float gv[V];
            Raw<T, V>::get(tile[0][r][threadIdx.x], gv);
            Raw<T, V>::get(tile[1][r][threadIdx.x], d[r]);
            const bool in = t0 - r >= 0;
#pragma unroll
            for (int v = 0; v < V; v++) {
                gate_of<GATE>(gv[v], a[r][v], w[r][v]);
                a[r][v] = in ? a[r][v] : 1.f;   // d is 0 there
                A[v] *= a[r][v];
                H[v] = a[r][v] * (d[r][v] + H[v]);
            }
        }
        join<V>(sh.maps, it & 1, q.ctas, q.rank, A, H, state, mu);
#pragma unroll
        for (int r = 0; r < R; r++) {
            const long long t = t0 - r;
            float before[V], xv[V], ox[V], og[V];
            Raw<T, V>::get(tile[2][r][threadIdx.x], before);
            if constexpr (kSigmoid) Raw<T, V>::get(tile[3][r][threadIdx.x], xv);
#pragma unroll
            for (int v = 0; v < V; v++) {
                if (t == 0) before[v] = h_first[v];
                const float l = d[r][v] + mu[v];
                mu[v] = a[r][v] * l;
                ox[v] = kSigmoid ? l * w[r][v] : l;
                og[v] = kSigmoid ? (mu[v] * w[r][v]) * (before[v] - xv[v])
                                 : (GATE == LA_GATE_LOG ? mu[v] : l) * before[v];
            }
            if (q.ok && t >= 0) {
                *reinterpret_cast<RT *>(pdx + t * dx.sn) = Raw<T, V>::put(ox);
                *reinterpret_cast<RT *>(pdg + t * dg.sn) = Raw<T, V>::put(og);
            }
        }
    }
    clear_rows<T, V>(pdx, dx.sn, q, s.N);
    clear_rows<T, V>(pdg, dg.sn, q, s.N);
    if (dh0 && q.ok && warp == 0 && q.rank == 0) {
#pragma unroll
        for (int v = 0; v < V; v++) dh0[q.state + v] = state[v];
    }
}

// CTAs per strip: enough that every SM has its two, as far as the tokens fill
// their tiles.
int cluster_of(long long strips, int N, int rows, const DeviceInfo &dev) {
    int k = 1;
    while (k < kMaxCluster && strips * k < 2LL * dev.sm_count && (long long)N > (long long)k * kWarps * rows) k *= 2;
    return k;
}

bool pairs(const la_view &v) {
    return (reinterpret_cast<uintptr_t>(v.data) & 3) == 0 && ((v.sb | v.sh | v.sn) & 1) == 0;
}

template <typename T, int GATE, int V> cudaError_t forward_v(const RecProblem &p, const DeviceInfo &dev) {
    if (p.N <= kShortRows) {
        const long long groups = (long long)p.B * p.H * (p.D / V);
        const cudaError_t e = launch_pdl(rec_short_kernel<T, GATE, V>,
                                         dim3((unsigned)((groups + kShortThreads - 1) / kShortThreads)),
                                         dim3(kShortThreads), 0, p.stream, 0u, p.x, p.g, p.out,
                                         Dims{p.lens, p.H, p.N, p.D, 0}, groups, p.h0, p.hN);
        count_launches(1);
        return e;
    }
    Dims s{p.lens, p.H, p.N, p.D, (p.D + 32 * V - 1) / (32 * V)};
    const long long strips = (long long)p.B * p.H * s.strips;
    const int k = cluster_of(strips, p.N, kFwdRows, dev);
    const size_t smem = sizeof(FwdShared<T, V>);
    cudaError_t e = cudaFuncSetAttribute(rec_forward_kernel<T, GATE, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(rec_forward_kernel<T, GATE, V>, dim3((unsigned)(strips * k)), dim3(kThreads), smem, p.stream,
                   (unsigned)k, p.x, p.g, p.out, s, p.h0, p.hN);
    count_launches(1);
    return e;
}

template <typename T, int GATE, int V> cudaError_t backward_v(const RecProblem &p, const DeviceInfo &dev) {
    Dims s{p.lens, p.H, p.N, p.D, (p.D + 32 * V - 1) / (32 * V)};
    const long long strips = (long long)p.B * p.H * s.strips;
    const int k = cluster_of(strips, p.N, kBwdRows, dev);
    const size_t smem = sizeof(BwdShared<T, GATE, V>);
    cudaError_t e = cudaFuncSetAttribute(rec_backward_kernel<T, GATE, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(rec_backward_kernel<T, GATE, V>, dim3((unsigned)(strips * k)), dim3(kThreads), smem, p.stream,
                   (unsigned)k, p.x, p.g, p.out, p.dout, p.dx, p.dg, s, p.h0, p.dhN, p.dh0);
    count_launches(1);
    return e;
}

template <int GATE> cudaError_t forward_g(const RecProblem &p, const DeviceInfo &dev) {
    if (p.dtype == LA_DTYPE_F32) return forward_v<float, GATE, 1>(p, dev);
    // two bf16 channels a lane where every row starts on 4 bytes
    if (p.D % 2 == 0 && pairs(p.x) && pairs(p.g) && pairs(p.out)) return forward_v<__nv_bfloat16, GATE, 2>(p, dev);
    return forward_v<__nv_bfloat16, GATE, 1>(p, dev);
}

template <int GATE> cudaError_t backward_g(const RecProblem &p, const DeviceInfo &dev) {
    if (p.dtype == LA_DTYPE_F32) return backward_v<float, GATE, 1>(p, dev);
    if (p.D % 2 == 0 && pairs(p.x) && pairs(p.g) && pairs(p.out) && pairs(p.dout) && pairs(p.dx) && pairs(p.dg))
        return backward_v<__nv_bfloat16, GATE, 2>(p, dev);
    return backward_v<__nv_bfloat16, GATE, 1>(p, dev);
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
