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
// A strip of 32 lanes' channels belongs to one CTA, which walks its tokens in
// tiles: each warp takes R consecutive rows, first forms (A, H) of them, then
// learns the state before them (the warps' maps joined through shared memory)
// and runs the recurrence proper from it.  Every value is read once and written
// once (8 x 4096 tokens of 2048 channels, bf16, sigmoid gate: forward 63 us,
// 6.3 TB/s, backward 117 to 125 us from box to box, 6.4 to 6.9 TB/s with what the L2
// still holds of it; fp32 the same rates).  Where the strips alone would leave SMs empty, a sequence is cut into
// segments, one CTA each, after a first launch that forms each segment's (A, H)
// alone; that reads x and g (g and dout) a second time (65536 tokens of 1024
// channels: forward 106 us, 6.3 TB/s over both readings, of which the maps take
// 42; backward 171 us).  (Sequences cut into 2, 4 or 8 calls, so that the second
// reading meets the L2: 113, 125 and 173 us.  Clusters of CTAs that
// walk one sequence side by side and exchange their maps through distributed
// shared memory read everything once, but wait for one another at every tile:
// 1.1 us for 512 rows, 142 us for N = 65536, D = 64.)  No atomics and no flags,
// and the grouping depends on the sizes alone: equal calls give equal bits.
#include <algorithm>
#include <cfloat>
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
    int segments;      // CTAs of a strip
    long long rows;    // tokens of a segment (a multiple of kSegmentRows)
    long long channels;   // B*H*D
    float2 *maps;      // [segments - 1][B*H*D] (A, H) of the segments but the last
    float *start;      // [B*H*D] the state before the first
};

// V neighbouring channels of one row as they lie in memory.
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

// A strip's row as the lanes share it.  WIDE (every row starts on 16 bytes and D
// fills 16-byte pieces): V neighbouring channels each.  Else V channels 32 apart,
// loaded and stored one by one, the lanes' next to one another.
template <typename T, int V, bool WIDE> struct Row {
    static __device__ __forceinline__ int channel(int lane, int v) { return WIDE ? lane * V + v : v * 32 + lane; }
    // channel of position `at` among the lanes' values in order
    static __device__ __forceinline__ int channel_at(int at) { return WIDE ? at : at % V * 32 + at / V; }
    // p: the row's first channel of the strip, of which `left` exist
    static __device__ __forceinline__ void store(T *p, int lane, int left, const Lanes<V> &x) {
        if constexpr (WIDE) {
            if (lane * V < left) *reinterpret_cast<typename Raw<T, V>::type *>(p + lane * V) = Raw<T, V>::put(x);
        } else {
#pragma unroll
            for (int v = 0; v < V; v++)
                if (channel(lane, v) < left) p[channel(lane, v)] = from_f32<T>(x.get(v));
        }
    }
};

// Joining by products fails where the walk in order does not: a product of gates
// past fp32's range is inf, or NaN (inf * 0) after a gate of 0 or on an empty
// state, and one below it is 0, which an infinite state turns into NaN.  None of
// these ever becomes finite again along a chain of joins, so what is finite is
// right.  What is not is walked again token by token, by one thread a channel: a
// segment whose start it is the end of, or the rows of a CTA after its last tile
// (there only values that are not finite are written, the others keep their bits).
// A state that was NaN before stays NaN either way.  Walking costs up to 0.25 us a token
// (8 x 4096 tokens of 2048 channels, every one with a NaN at its start: forward 0.6 to
// 0.9 ms, backward 1.0 to 1.5); noticing it costs 1 % of a pass or less.
__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) <= FLT_MAX; }

// `n` tokens of one channel in order: load(t) fetches a token's values, several
// tokens ahead; step(t, values, h) returns the state after the token.
template <typename Load, typename Step>
__device__ __forceinline__ float in_order(long long n, float h, Load load, Step step) {
    constexpr int R = 4;
    for (long long t = 0; t < n; t += R) {
        decltype(load(t)) v[R];
#pragma unroll
        for (int r = 0; r < R; r++) v[r] = load(min(t + r, n - 1));
#pragma unroll
        for (int r = 0; r < R; r++)
            if (t + r < n) h = step(t + r, v[r], h);
    }
    return h;
}
// One token: v = x, or BACK: dout.
template <typename T, int GATE, bool BACK> __device__ __forceinline__ float next_state(float h, float g, float v, float *w) {
    Lanes<1> a, u;
    gate_of<T, GATE, 1>(Lanes<1>{{g}}, a, u);
    *w = u.p[0];
    return BACK ? a.p[0] * (v + h) : fmaf(a.p[0], h, GATE == LA_GATE_SIGMOID ? u.p[0] * v : v);
}
// The state after n tokens from g and x (BACK: dout) on, gn and xn apart.
template <typename T, int GATE, bool BACK>
__device__ __noinline__ float state_after(const T *g, long long gn, const T *x, long long xn, long long n, float h) {
    return in_order(
        n, h, [=](long long t) { return make_float2(to_f32<T>(g[t * gn]), to_f32<T>(x[t * xn])); },
        [=](long long, float2 v, float s) {
            float w;
            return next_state<T, GATE, BACK>(s, v.x, v.y, &w);
        });
}
template <typename T> __device__ __forceinline__ void mend(T *p, float was, float v) {
    if (!is_finite(was)) *p = from_f32<T>(v);
}

// The joining of a tile's maps (A, H), one per warp and channel.  For that the
// CTA's threads change sides: G = W / V neighbouring lanes own a channel, each
// of them the maps of V consecutive warps, so that a map is read once and not
// by every warp after it (which cost a third of all instructions).  The owners
// carry the channel's state over the tile and leave the state before each
// warp's rows in place of its H.  Everything is in two sets, used in turn, so
// that a set is not written again before all have read it.
template <int V, int W> struct Joint {
    static constexpr int G = W / V, C = 32 * V;
    static_assert(G * V == W, "");
    float A[2][W][C + 4], H[2][W][C + 4];   // the 4: owners of a warp read distinct banks
    float start[C];                         // the channels' states before the CTA's rows
};

template <int V> using Vec = std::conditional_t<V == 4, float4, std::conditional_t<V == 2, float2, float>>;
template <int V> __device__ __forceinline__ void put_lanes(float *to, const Lanes<V> &v) {
    *reinterpret_cast<Vec<V> *>(to) = *reinterpret_cast<const Vec<V> *>(&v);
}
template <int V> __device__ __forceinline__ Lanes<V> get_lanes(const float *from) {
    const Vec<V> r = *reinterpret_cast<const Vec<V> *>(from);
    return *reinterpret_cast<const Lanes<V> *>(&r);
}

template <typename Row, int V, int W> struct Join {
    using J = Joint<V, W>;
    J &j;
    int warp, lane, at, sub; // at: position of the owned channel, sub: which of its owners
    int channel;
    bool real;               // whether the owned channel exists (else its maps are rubbish)
    float state;             // of the owned channel
    float zero = 0.f;        // NaN once a joined state was not finite
    int set = 0;

    // first: the strip's first channel of the state before the CTA's rows.
    __device__ __forceinline__ Join(J &j_, const float *first, int left)
        : j(j_), warp(threadIdx.x >> 5), lane(threadIdx.x & 31), at(threadIdx.x / J::G), sub(threadIdx.x % J::G),
          channel(Row::channel_at(threadIdx.x / J::G)), real(channel < left) {
        state = first && real ? first[channel] : 0.f;
    }
    // Over the segments before this one; maps: their strip's first channel,
    // `pitch` apart.  The owners of a channel take equal runs of them.  walk(c, i, h):
    // state_after() channel c's tokens of segment i.
    template <typename Walk>
    __device__ __forceinline__ void skip(const float2 *maps, int segments, long long pitch, Walk walk) {
        const float first = state;
        float a = 1.f, h = 0.f;
        if (real) {
            const int to = (sub + 1) * segments / J::G;
#pragma unroll 16
            for (int i = sub * segments / J::G; i < to; i++) {
                const float2 m = maps[i * pitch + channel];
                h = fmaf(m.x, h, m.y);
                a *= m.x;
            }
        }
#pragma unroll
        for (int i = 0; i < J::G; i++)
            state = fmaf(__shfl_sync(~0u, a, i, J::G), state, __shfl_sync(~0u, h, i, J::G));
        if (real && !is_finite(state)) {
            state = first;
            for (int i = 0; i < segments && state == state; i++) {
                const float2 m = maps[i * pitch + channel];
                const float after = fmaf(m.x, state, m.y);
                state = is_finite(after) ? after : walk(channel, i, state);
            }
        }
        if (sub == 0) j.start[at] = state;
    }
    // After the last tile, by all threads.  redo(c, h): walks channel c's rows of the CTA
    // from the state h and mends them.  The state goes to `first`, if there is one.
    template <typename Redo> __device__ __forceinline__ void end(float *first, Redo redo) {
        const bool bad = real && !(zero == 0.f && is_finite(state));
        const unsigned all = __ballot_sync(~0u, bad) >> (lane / J::G * J::G) & ((1u << J::G) - 1);
        if (__syncthreads_or(bad)) {   // and the rows are written
            if (all && sub == 0 && j.start[at] == j.start[at]) state = redo(channel, j.start[at]);
        }
        if (first && real && sub == 0) first[channel] = state;
    }

    // A, H: this thread's rows; returns the state before them.
    __device__ __forceinline__ Lanes<V> operator()(const Lanes<V> &A, const Lanes<V> &H) {
        put_lanes(&j.A[set][warp][lane * V], A);
        put_lanes(&j.H[set][warp][lane * V], H);
        __syncthreads();
        float a[V], h[V], ta = 1.f, th = 0.f;
#pragma unroll
        for (int i = 0; i < V; i++) a[i] = j.A[set][sub * V + i][at], h[i] = j.H[set][sub * V + i][at];
#pragma unroll
        for (int i = 0; i < V; i++) ta *= a[i], th = fmaf(a[i], th, h[i]);
        float ea = 1.f, eh = 0.f;   // map of the owners before this one
        if constexpr (J::G > 1) {
#pragma unroll
            for (int o = 1; o < J::G; o *= 2) {
                const float oa = __shfl_up_sync(~0u, ta, o, J::G), oh = __shfl_up_sync(~0u, th, o, J::G);
                if (sub >= o) th = fmaf(ta, oh, th), ta *= oa;
            }
            ea = __shfl_up_sync(~0u, ta, 1, J::G);
            eh = __shfl_up_sync(~0u, th, 1, J::G);
            if (sub == 0) ea = 1.f, eh = 0.f;
            ta = __shfl_sync(~0u, ta, J::G - 1, J::G);
            th = __shfl_sync(~0u, th, J::G - 1, J::G);
        }
        float before = fmaf(ea, state, eh);
        state = fmaf(ta, state, th);
#pragma unroll
        for (int i = 0; i < V; i++) {
            j.H[set][sub * V + i][at] = before;
            before = fmaf(a[i], before, h[i]);
        }
        // the state after this owner's warps, by other products than the channel's own state
        zero = fmaf(before, 0.f, zero);
        __syncthreads();
        const Lanes<V> r = get_lanes<V>(&j.H[set][warp][lane * V]);
        set ^= 1;
        return r;
    }
};

// A CTA's place (`cta`: its number): its sequence, its channels, its rows
// [from, to) in the order of the walk.
template <int V> struct Place {
    long long b, h, at;      // at: its first channel in [B,H,D]
    int d0, left, len, segment;
    long long from, to;
    __device__ __forceinline__ Place(const Dims &s, int segments, unsigned cta = blockIdx.x) {
        const unsigned strip = cta / segments;
        segment = cta % segments;
        const long long bh = strip / s.strips;
        b = bh / s.H;
        h = bh % s.H;
        d0 = (int)(strip % s.strips) * 32 * V;
        left = s.D - d0;
        at = bh * s.D + d0;
        len = s.lens ? min(max(s.lens[b], 0), s.N) : s.N;
        from = min(segment * s.rows, (long long)len);
        to = min(from + s.rows, (long long)len);
    }
    template <typename T> __device__ __forceinline__ T *strip(const la_view &v) const {
        return static_cast<T *>(v.data) + b * v.sb + h * v.sh + d0;
    }
    // whether the last token is among its rows (no token at all: the first segment)
    __device__ __forceinline__ bool last() const { return to == len && (from < to || segment == 0); }
};

// Rows at or past a sequence's length become 0, the segments taking turns.
template <typename Row, typename T, int V, int W>
__device__ __forceinline__ void clear_rows(T *p, long long sn, const Place<V> &q, const Dims &s) {
    for (long long t = q.len + q.segment * W + (threadIdx.x >> 5); t < s.N; t += s.segments * W)
        Row::store(p + t * sn, threadIdx.x & 31, q.left, all<V>(0.f));
}

// A warp's rows of NT tensors on their way through shared memory, S tiles deep,
// in 16-byte pieces: neighbouring lanes copy neighbouring pieces, two or four rows
// a request.  A row that does not start on 16 bytes is copied from the boundary
// before it (so a copy begins up to 15 bytes before the row, in a piece that holds
// some of it, and never ends past it) and is read from where it starts in the
// first piece; copies of single values held the memory pipe up.
template <typename T, int V, int NT, int R, int S, bool WIDE> struct Ring {
    static constexpr int kRow = 32 * V * (int)sizeof(T), kPieces = kRow / 16, kRows = 32 / kPieces;
    static constexpr int kPitch = kRow + (WIDE ? 0 : 16);
    using Slot = unsigned char (*)[NT][R][kPitch];
    Slot slot;               // [S], this warp's
    int lane;

    static __device__ __forceinline__ void copy16(unsigned char *to, const unsigned char *from, int bytes) {
        if constexpr (WIDE)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(to)), "l"(from) : "memory");
        else
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(to)), "l"(from),
                         "r"(min(bytes, 16))
                         : "memory");
    }
    // Rows 0 .. n - 1 of tensor `k`: row r at p + r * sn (p: the row's first
    // channel of the strip), `left` channels of it exist.
    __device__ __forceinline__ void copy(int stage, int k, const T *p, long long sn, int n, int left) const {
        const int piece = lane % kPieces, row = lane / kPieces, bytes = min(left, 32 * V) * (int)sizeof(T);
        const long long step = sn * (long long)sizeof(T);
        const unsigned char *from = reinterpret_cast<const unsigned char *>(p) + row * step;
        unsigned char *to = slot[stage][k][row] + piece * 16;
        if constexpr (WIDE) {
            if (piece * 16 < bytes) {
                from += piece * 16;
#pragma unroll
                for (int r = 0; r < R; r += kRows, from += kRows * step)
                    if (r + row < n) copy16(to + r * kPitch, from, 16);
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; r += kRows, from += kRows * step) {
                const int shift = (int)(reinterpret_cast<uintptr_t>(from) & 15), have = shift + bytes - piece * 16;
                if (r + row < n && have > 0) copy16(to + r * kPitch, from - shift + piece * 16, have);
            }
            // the piece that a shifted row has more, of every row
            from = reinterpret_cast<const unsigned char *>(p) + lane * step;
            const int shift = (int)(reinterpret_cast<uintptr_t>(from) & 15), have = shift + bytes - kRow;
            if (lane < R && lane < n && have > 0) copy16(slot[stage][k][lane] + kRow, from - shift + kRow, have);
        }
    }
    __device__ __forceinline__ void commit() const { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // All but the LEFT newest commits have landed, for the whole warp.
    template <int LEFT> __device__ __forceinline__ void wait() const {
        asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
        __syncwarp();
    }
    // Row r of tensor k, whose rows were copied from p on (row 0), sn apart.
    __device__ __forceinline__ Lanes<V> get(int stage, int k, int r, const T *p, long long sn) const {
        if constexpr (WIDE) {
            using RT = typename Raw<T, V>::type;
            return Raw<T, V>::get(reinterpret_cast<const RT *>(slot[stage][k][r])[lane]);
        } else {
            const unsigned shift = ((unsigned)reinterpret_cast<uintptr_t>(p) + r * (unsigned)sn * (unsigned)sizeof(T)) & 15u;
            const T *row = reinterpret_cast<const T *>(slot[stage][k][r] + shift);
            Lanes<V> x;
#pragma unroll
            for (int v = 0; v < V; v++) x.set(v, to_f32<T>(row[v * 32 + lane]));
            return x;
        }
    }
};

template <typename Ring, int W, int NT, int R, int S> using Slots = unsigned char[W][S][NT][R][Ring::kPitch];

template <typename T, int V, bool WIDE, int W, int R, int S> struct Tiles {
    using Row = la::Row<T, V, WIDE>;
    using Ring = la::Ring<T, V, 2, R, S, WIDE>;
    __align__(16) Slots<Ring, W, 2, R, S> slot;
    __align__(16) Joint<V, W> joint;
};

// A channel's `n` rows from x, g, out on, for Join::end().
template <typename T, int GATE>
__device__ __noinline__ float redo_forward(const T *x, long long xn, const T *g, long long gn, T *out, long long on,
                                           long long n, float h) {
    struct Row1 { float x, g, out; };
    return in_order(
        n, h, [=](long long t) { return Row1{to_f32<T>(x[t * xn]), to_f32<T>(g[t * gn]), to_f32<T>(out[t * on])}; },
        [=](long long t, const Row1 &v, float s) {
            float w;
            s = next_state<T, GATE, false>(s, v.g, v.x, &w);
            mend(out + t * on, v.out, s);
            return s;
        });
}

template <typename T, int GATE, int V, bool WIDE, int W, int R, int S, int CTAS>
__global__ void __launch_bounds__(32 * W, CTAS) rec_forward_kernel(la_view x, la_view g, la_view out, Dims s,
                                                                  const float *h0, float *hN) {
    using Sh = Tiles<T, V, WIDE, W, R, S>;
    using Row = typename Sh::Row;
    extern __shared__ __align__(16) unsigned char smem[];
    auto &sh = *reinterpret_cast<Sh *>(smem);
    pdl_wait_cta();
    const Place<V> q(s, s.segments);
    Join<Row, V, W> join(sh.joint, s.segments > 1 ? s.start + q.at : h0 ? h0 + q.at : nullptr, q.left);
    const typename Sh::Ring ring{sh.slot[join.warp], join.lane};
    const T *px = q.template strip<T>(x), *pg = q.template strip<T>(g);
    T *po = q.template strip<T>(out);
    const long long first = q.from + join.warp * R;   // this warp's rows in the first tile
    const int tiles = (int)((q.to - q.from + W * R - 1) / (W * R));
    auto fetch = [&](int it, int stage) {
        const long long t = first + (long long)it * (W * R);
        if (t < q.to) {
            const int n = (int)min((long long)R, q.to - t);
            ring.copy(stage, 0, px + t * x.sn, x.sn, n, q.left);
            ring.copy(stage, 1, pg + t * g.sn, g.sn, n, q.left);
        }
        ring.commit();
    };
    for (int i = 0; i < S; i++) fetch(i, i);
    join.skip(s.maps + q.at, q.segment, s.channels, [&](int c, int i, float h) {
        const long long t = min(i * s.rows, (long long)q.len), end = min(t + s.rows, (long long)q.len);
        return state_after<T, GATE, false>(pg + t * g.sn + c, g.sn, px + t * x.sn + c, x.sn, end - t, h);
    });
    int stage = 0;
    for (int it = 0; it < tiles; it++) {
        ring.template wait<S - 1>();
        const long long t0 = first + (long long)it * (W * R);
        const int n = (int)min((long long)R, max(q.to - t0, 0LL));
        const T *rx = px + t0 * x.sn, *rg = pg + t0 * g.sn;
        Lanes<V> a[R], u[R];
#pragma unroll
        for (int r = 0; r < R; r++) {
            Lanes<V> w;
            gate_of<T, GATE, V>(ring.get(stage, 1, r, rg, g.sn), a[r], w);
            u[r] = ring.get(stage, 0, r, rx, x.sn);
            if (GATE == LA_GATE_SIGMOID) u[r] = mul(w, u[r]);
        }
        __syncwarp();   // the stage is free
        fetch(it + S, stage);
        stage = stage == S - 1 ? 0 : stage + 1;
        if (n < R) {    // rows past the end leave the state as it is
#pragma unroll
            for (int r = 0; r < R; r++)
                if (r >= n) a[r] = all<V>(1.f), u[r] = all<V>(0.f);
        }
        Lanes<V> A = a[0], H = u[0];
#pragma unroll
        for (int r = 1; r < R; r++) A = mul(A, a[r]), H = fma(a[r], H, u[r]);
        Lanes<V> h = join(A, H);
        T *p = po + t0 * out.sn;
#pragma unroll
        for (int r = 0; r < R; r++, p += out.sn) {
            h = fma(a[r], h, u[r]);
            if (r < n) Row::store(p, join.lane, q.left, h);
        }
    }
    clear_rows<Row, T, V, W>(po, out.sn, q, s);
    join.end(hN && q.last() ? hN + q.at : nullptr, [&](int c, float h) {
        return redo_forward<T, GATE>(px + q.from * x.sn + c, x.sn, pg + q.from * g.sn + c, g.sn, po + q.from * out.sn + c,
                                     out.sn, q.to - q.from, h);
    });
}

// (A, H) of every segment but the last, and a copy of the state that the walk
// starts from (a caller's hN may be its h0).  Warps take consecutive eighths of
// a segment and meet once at its end.  BACK: the backward's maps, of g and dout.
template <typename T, int V, bool WIDE, int W, int R, int S> struct MapTiles {
    using Row = la::Row<T, V, WIDE>;
    using Ring = la::Ring<T, V, 2, R, S, WIDE>;
    __align__(16) Slots<Ring, W, 2, R, S> slot;
    __align__(16) float A[W][32 * V], H[W][32 * V];
};
template <typename T, int GATE, int V, bool WIDE, bool BACK, int W, int R, int S, int CTAS>
__global__ void __launch_bounds__(32 * W, CTAS) rec_maps_kernel(la_view g, la_view x, Dims s, const float *state) {
    using Sh = MapTiles<T, V, WIDE, W, R, S>;
    extern __shared__ __align__(16) unsigned char smem[];
    auto &sh = *reinterpret_cast<Sh *>(smem);
    pdl_wait_cta();
    const Place<V> q(s, s.segments - 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const typename Sh::Ring ring{sh.slot[warp], lane};
    const T *px = q.template strip<T>(x), *pg = q.template strip<T>(g);
    const long long per = s.rows / W, first = min(q.from + warp * per, q.to), last = min(first + per, q.to);
    const int pieces = (int)((last - first + R - 1) / R);
    const long long nx = BACK ? -x.sn : x.sn, ng = BACK ? -g.sn : g.sn;   // to the next row of the walk
    px += (BACK ? q.len - 1 : 0) * x.sn + first * nx;
    pg += (BACK ? q.len - 1 : 0) * g.sn + first * ng;
    auto fetch = [&](int i, int stage) {
        const long long t = (long long)i * R;
        if (first + t < last) {
            const int n = (int)min((long long)R, last - first - t);
            ring.copy(stage, 0, px + t * nx, nx, n, q.left);
            ring.copy(stage, 1, pg + t * ng, ng, n, q.left);
        }
        ring.commit();
    };
    for (int i = 0; i < S; i++) fetch(i, i);
    Lanes<V> A = all<V>(1.f), H = all<V>(0.f);
    int stage = 0;
    for (int i = 0; i < pieces; i++) {
        ring.template wait<S - 1>();
        const int n = (int)min((long long)R, last - (first + (long long)i * R));
        auto step = [&](int r) {
            Lanes<V> a, w;
            gate_of<T, GATE, V>(ring.get(stage, 1, r, pg + (long long)i * R * ng, ng), a, w);
            const Lanes<V> v = ring.get(stage, 0, r, px + (long long)i * R * nx, nx);
            A = mul(A, a);
            if (BACK) H = mul(a, add(v, H));
            else H = fma(a, H, GATE == LA_GATE_SIGMOID ? mul(w, v) : v);
        };
        if (n >= R) {
#pragma unroll
            for (int r = 0; r < R; r++) step(r);
        } else {
            for (int r = 0; r < n; r++) step(r);
        }
        __syncwarp();
        fetch(i + S, stage);
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    put_lanes(&sh.A[warp][lane * V], A);
    put_lanes(&sh.H[warp][lane * V], H);
    __syncthreads();
    for (int c = threadIdx.x; c < 32 * V; c += 32 * W) {
        const int d = Sh::Row::channel_at(c);
        if (d >= q.left) continue;
        float a = 1.f, h = 0.f;
#pragma unroll
        for (int w = 0; w < W; w++) {
            h = fmaf(sh.A[w][c], h, sh.H[w][c]);
            a *= sh.A[w][c];
        }
        s.maps[q.segment * s.channels + q.at + d] = make_float2(a, h);
        if (q.segment == 0) s.start[q.at + d] = state ? state[q.at + d] : 0.f;
    }
}

// Up to kShortRows tokens (a decoded token among them) there is nothing to
// split: a thread takes its channels' few rows in order, bound by latency.  (64
// sequences of 1024 channels, bf16: 16 tokens 4.1 us, in tiles 5.5; 32 tokens 13.4
// and 6.1.  One token of them 1.8 us, half a megabyte.)
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
            gate_of<T, GATE, V>(Raw<T, V>::get(rg[r]), a, w);
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
// which the token before adds to its own gradient.  The rows of g and dout are
// free once they have become a, w and d, those of h_{t-1} and x only after the
// join, so they go through two rings.  h_{t-1} is the forward's output as it was
// stored: for bf16 data within 2^-8 of its size where the forward itself carries fp32.
// Only dg has it as a factor, and is itself rounded to bf16 (8 x 4096 x 2048, sigmoid: dg
// 1.8e-3 off the exact one in the mean square, 1.7e-3 with fp32 states; dx, dh0 and the
// carried l do not depend on it).  The fp32 states would have to be kept by the caller,
// twice the bytes of out, or formed again from all of x and g, a second walk.
template <typename T, int V, bool WIDE, int W, int NL, int R, int S> struct BackTiles {
    using Row = la::Row<T, V, WIDE>;
    using Early = Ring<T, V, 2, R, S, WIDE>;
    using Late = Ring<T, V, NL, R, S, WIDE>;
    __align__(16) Slots<Early, W, 2, R, S> early;
    __align__(16) Slots<Late, W, NL, R, S> late;
    __align__(16) Joint<V, W> joint;
};

// A channel's `n` rows from x, g, dout, dx, dg down, for Join::end(); out: the row
// before the first of them; whole: the last of them is the sequence's first, which
// has h0 before it.
template <typename T, int GATE>
__device__ __noinline__ float redo_backward(const T *x, long long xn, const T *g, long long gn, const T *out, long long on,
                                            const T *dout, long long dn, T *dx, long long dxn, T *dg, long long dgn,
                                            float h0, bool whole, long long n, float mu) {
    constexpr bool kSigmoid = GATE == LA_GATE_SIGMOID;
    struct Row1 { float x, g, before, dout, dx, dg; };
    return in_order(
        n, mu,
        [=](long long i) {
            const long long above = whole && i == n - 1 ? i - 1 : i;   // (its own row's out is not used)
            return Row1{kSigmoid ? to_f32<T>(x[-i * xn]) : 0.f, to_f32<T>(g[-i * gn]), to_f32<T>(out[-above * on]),
                        to_f32<T>(dout[-i * dn]), to_f32<T>(dx[-i * dxn]), to_f32<T>(dg[-i * dgn])};
        },
        [=](long long i, const Row1 &v, float s) {
            float w;
            const float l = v.dout + s, before = whole && i == n - 1 ? h0 : v.before;
            s = next_state<T, GATE, true>(s, v.g, v.dout, &w);
            mend(dx - i * dxn, v.dx, kSigmoid ? l * w : l);
            mend(dg - i * dgn, v.dg, kSigmoid ? s * w * (before - v.x) : (GATE == LA_GATE_LOG ? s : l) * before);
            return s;
        });
}

template <typename T, int GATE, int V, bool WIDE, int W, int R, int S, int CTAS>
__global__ void __launch_bounds__(32 * W, CTAS) rec_backward_kernel(la_view x, la_view g, la_view out, la_view dout,
                                                                   la_view dx, la_view dg, Dims s, const float *h0,
                                                                   const float *dhN, float *dh0) {
    constexpr bool kSigmoid = GATE == LA_GATE_SIGMOID;
    constexpr int NL = kSigmoid ? 2 : 1;
    using Sh = BackTiles<T, V, WIDE, W, NL, R, S>;
    using Row = typename Sh::Row;
    extern __shared__ __align__(16) unsigned char smem[];
    auto &sh = *reinterpret_cast<Sh *>(smem);
    pdl_wait_cta();
    const Place<V> q(s, s.segments);
    Join<Row, V, W> join(sh.joint, s.segments > 1 ? s.start + q.at : dhN ? dhN + q.at : nullptr, q.left);
    const typename Sh::Early early{sh.early[join.warp], join.lane};
    const typename Sh::Late late{sh.late[join.warp], join.lane};
    const T *px = kSigmoid ? q.template strip<T>(x) : nullptr, *pg = q.template strip<T>(g);
    const T *po = q.template strip<T>(out), *pd = q.template strip<T>(dout);
    T *pdx = q.template strip<T>(dx), *pdg = q.template strip<T>(dg);
    const long long first = q.len - 1 - (q.from + join.warp * R);   // this warp's first row, and the CTA's last
    const long long end = q.len - q.to;
    const int tiles = (int)((q.to - q.from + W * R - 1) / (W * R));
    auto fetch_early = [&](int it, int stage) {   // rows t, t - 1, ...
        const long long t = first - (long long)it * (W * R);
        if (t >= end) {
            const int n = (int)min((long long)R, t - end + 1);
            early.copy(stage, 0, pg + t * g.sn, -g.sn, n, q.left);
            early.copy(stage, 1, pd + t * dout.sn, -dout.sn, n, q.left);
        }
        early.commit();
    };
    auto fetch_late = [&](int it, int stage) {
        const long long t = first - (long long)it * (W * R);
        if (t >= end) {
            const int n = (int)min((long long)R, t - end + 1);
            late.copy(stage, 0, po + (t - 1) * out.sn, -out.sn, (int)min((long long)n, t), q.left);
            if constexpr (kSigmoid) late.copy(stage, 1, px + t * x.sn, -x.sn, n, q.left);
        }
        late.commit();
    };
    for (int i = 0; i < S; i++) fetch_early(i, i), fetch_late(i, i);
    join.skip(s.maps + q.at, q.segment, s.channels, [&](int c, int i, float mu) {
        const long long t = min(i * s.rows, (long long)q.len), end = min(t + s.rows, (long long)q.len);
        const long long row = q.len - 1 - t;
        return state_after<T, GATE, true>(pg + row * g.sn + c, -g.sn, pd + row * dout.sn + c, -dout.sn, end - t, mu);
    });
    int stage = 0;
    for (int it = 0; it < tiles; it++) {
        early.template wait<2 * S - 1>();   // commits in turn: early, late, early, ...
        const long long t0 = first - (long long)it * (W * R);
        const int n = (int)min((long long)R, max(t0 - end + 1, 0LL));
        const T *rg = pg + t0 * g.sn, *rd = pd + t0 * dout.sn, *rb = po + (t0 - 1) * out.sn;
        const T *rx = kSigmoid ? px + t0 * x.sn : nullptr;
        Lanes<V> a[R], w[R], d[R];
#pragma unroll
        for (int r = 0; r < R; r++) {
            d[r] = early.get(stage, 1, r, rd, -dout.sn);
            gate_of<T, GATE, V>(early.get(stage, 0, r, rg, -g.sn), a[r], w[r]);
        }
        __syncwarp();
        fetch_early(it + S, stage);
        if (n < R) {   // rows before the first leave the state as it is
#pragma unroll
            for (int r = 0; r < R; r++)
                if (r >= n) a[r] = all<V>(1.f), d[r] = all<V>(0.f);
        }
        Lanes<V> A = a[0], H = mul(a[0], d[0]);
#pragma unroll
        for (int r = 1; r < R; r++) A = mul(A, a[r]), H = mul(a[r], add(d[r], H));
        Lanes<V> mu = join(A, H);
        late.template wait<2 * S - 1>();
        T *to_x = pdx + t0 * dx.sn, *to_g = pdg + t0 * dg.sn;
#pragma unroll
        for (int r = 0; r < R; r++, to_x -= dx.sn, to_g -= dg.sn) {
            Lanes<V> before = late.get(stage, 0, r, rb, -out.sn);
            if (t0 == r) {   // the first token: the state that the forward started from
#pragma unroll
                for (int v = 0; v < V; v++) {
                    const int c = Row::channel(join.lane, v);
                    before.set(v, h0 && c < q.left ? h0[q.at + c] : 0.f);
                }
            }
            const Lanes<V> l = add(d[r], mu);
            mu = mul(a[r], l);
            Lanes<V> ox = l, og;
            if constexpr (kSigmoid) {
                ox = mul(l, w[r]);
                og = mul(mul(mu, w[r]), fma(late.get(stage, NL - 1, r, rx, -x.sn), all<V>(-1.f), before));
            } else {
                og = mul(GATE == LA_GATE_LOG ? mu : l, before);
            }
            if (r < n) {
                Row::store(to_x, join.lane, q.left, ox);
                Row::store(to_g, join.lane, q.left, og);
            }
        }
        __syncwarp();
        fetch_late(it + S, stage);
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    clear_rows<Row, T, V, W>(pdx, dx.sn, q, s);
    clear_rows<Row, T, V, W>(pdg, dg.sn, q, s);
    join.end(dh0 && q.last() ? dh0 + q.at : nullptr, [&](int c, float mu) {
        // the place anew, from the CTA's number: held in registers through the walk it would
        // cost 1.3 us of 25 (4 x 16 sequences of 2048 tokens, 64 channels)
        unsigned cta;
        asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(cta));
        const Place<V> q(s, s.segments, cta);
        const T *px = kSigmoid ? q.template strip<T>(x) : nullptr, *pg = q.template strip<T>(g);
        const T *po = q.template strip<T>(out), *pd = q.template strip<T>(dout);
        T *pdx = q.template strip<T>(dx), *pdg = q.template strip<T>(dg);
        const long long t = q.len - 1 - q.from;
        return redo_backward<T, GATE>(px + t * x.sn + c, x.sn, pg + t * g.sn + c, g.sn, po + (t - 1) * out.sn + c, out.sn,
                                      pd + t * dout.sn + c, dout.sn, pdx + t * dx.sn + c, dx.sn, pdg + t * dg.sn + c,
                                      dg.sn, h0 ? h0[q.at + c] : 0.f, q.to == q.len, q.to - q.from, mu);
    });
}

// Tiles: W warps of R rows a CTA, S of them on their way, CTAS CTAs a SM.  ROW:
// bytes of a strip's row, 256 or 128; rows of 256 bytes come by ROWS a warp, those of
// 128 by twice as many.
template <int ROW, int ROWS, int S_, int C_> struct Tile {
    static constexpr int W = 8, R = ROW == 256 ? ROWS : ROWS * 2, S = S_, CTAS = C_;
};
// Many CTAs: two a SM hide each other's joins.  No more CTAs than SMs: twice the
// rows a tile for the same number of joins (128 strips of 4096 tokens, bf16:
// forward 63 us, backward 117 us, against 68 and 137 us with the small tiles; 304
// segments of 65536 tokens: 115 and 176 us against 106 and 171 us).
template <int ROW> using Fwd = Tile<ROW, 8, 2, 2>;
template <int ROW> using FwdFew = Tile<ROW, 16, 3, 1>;
template <int ROW> using Bwd = Tile<ROW, 4, 2, 2>;
template <int ROW> using BwdFew = Tile<ROW, 8, 3, 1>;
template <int ROW> using Pre = Tile<ROW, 8, 2, 3>;
constexpr int kSms = 152;
// A multiple of the warps, which share a segment's rows evenly in the maps' launch.  A
// tile has 32 to 256 rows: in segments as short as this one the larger tiles leave
// half to three quarters of their warps without rows.
constexpr int kSegmentRows = 64;

// Segments of a strip: none of it (1) where the strips fill half of the SMs (64
// narrow ones of 2048 tokens, bf16: 18.0 | 24.7 us in segments, 31.7 | 58.5 without;
// 128: 19.9 | 35.7 us without) or the sequence has at most `whole` tokens (8 strips,
// forward | backward: 128 tokens 5.4 | 5.9 us in segments, 3.5 | 5.2 without; 256:
// 5.6 | 6.1 and 5.3 | 8.7; 512: 6.0 | 6.6 and 9.0 | 15.7), else as many as give
// every SM two CTAs, of at least kSegmentRows tokens (512 tokens: 6.0 | 6.6 us with
// 64, 6.3 | 8.4 with 128).
int segments_of(long long strips, int N, int whole, long long *rows) {
    long long n = strips * 2 <= kSms && N > whole ? 2 * kSms / strips : 1;
    n = std::min(n, ((long long)N + kSegmentRows - 1) / kSegmentRows);
    *rows = (((long long)N + n - 1) / n + kSegmentRows - 1) / kSegmentRows * kSegmentRows;
    return (int)(((long long)N + *rows - 1) / *rows);
}

// Groups of C channels in a row.
int strips_of(int D, int C) { return (int)(((long long)D + C - 1) / C); }

template <int V> Dims dims_of(const RecProblem &p, int whole) {
    Dims s{p.lens, p.H, p.N, p.D, strips_of(p.D, 32 * V), 1, 0, (long long)p.B * p.H * p.D, nullptr, nullptr};
    s.segments = segments_of((long long)p.B * p.H * s.strips, p.N, whole, &s.rows);
    s.maps = static_cast<float2 *>(p.ws);
    s.start = reinterpret_cast<float *>(s.maps + (s.segments - 1) * s.channels);
    return s;
}

template <typename Tile, typename Kernel, typename... Args>
cudaError_t launch_tiles(Kernel kernel, size_t smem, const RecProblem &p, const Dims &s, int segments, Args... args) {
    const long long ctas = (long long)p.B * p.H * s.strips * segments;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3((unsigned)ctas), dim3(32 * Tile::W), smem, p.stream, 0u, args...);
    count_launches(1);
    return e;
}

template <typename T, int GATE, int V, bool WIDE, bool BACK>
cudaError_t segment_maps(const RecProblem &p, const Dims &s) {
    if (s.segments == 1) return cudaSuccess;
    using C = Pre<32 * V * (int)sizeof(T)>;
    return launch_tiles<C>(rec_maps_kernel<T, GATE, V, WIDE, BACK, C::W, C::R, C::S, C::CTAS>,
                           sizeof(MapTiles<T, V, WIDE, C::W, C::R, C::S>), p, s, s.segments - 1, p.g, BACK ? p.dout : p.x, s,
                           BACK ? p.dhN : p.h0);
}

template <typename T, int GATE, int V> cudaError_t short_v(const RecProblem &p) {
    const long long groups = (long long)p.B * p.H * (p.D / V);
    const cudaError_t e =
        launch_pdl(rec_short_kernel<T, GATE, V>, dim3((unsigned)((groups + kShortThreads - 1) / kShortThreads)),
                   dim3(kShortThreads), 0, p.stream, 0u, p.x, p.g, p.out, dims_of<V>(p, kShortRows), groups, p.h0, p.hN);
    count_launches(1);
    return e;
}

bool few_ctas(const RecProblem &p, const Dims &s) {
    return (long long)p.B * p.H * s.strips * s.segments <= kSms;
}

struct Forward {
    static constexpr int kUnsplit = kSms / 2 + 1, kWhole = 256;
    template <typename T, int GATE, int V, bool WIDE> static cudaError_t run(const RecProblem &p) {
        if (p.N <= kShortRows) return short_v<T, GATE, WIDE ? V : 1>(p);
        const Dims s = dims_of<V>(p, kWhole);
        const cudaError_t e = segment_maps<T, GATE, V, WIDE, false>(p, s);
        if (e != cudaSuccess) return e;
        constexpr int ROW = 32 * V * (int)sizeof(T);
        return few_ctas(p, s) ? tiles<T, GATE, V, WIDE, FwdFew<ROW>>(p, s) : tiles<T, GATE, V, WIDE, Fwd<ROW>>(p, s);
    }
    template <typename T, int GATE, int V, bool WIDE, typename C>
    static cudaError_t tiles(const RecProblem &p, const Dims &s) {
        return launch_tiles<C>(rec_forward_kernel<T, GATE, V, WIDE, C::W, C::R, C::S, C::CTAS>,
                               sizeof(Tiles<T, V, WIDE, C::W, C::R, C::S>), p, s, s.segments,
                               p.x, p.g, p.out, s, p.h0, p.hN);
    }
};

struct Backward {
    static constexpr int kUnsplit = kSms * 2 / 3 + 1, kWhole = 128;
    template <typename T, int GATE, int V, bool WIDE> static cudaError_t run(const RecProblem &p) {
        const Dims s = dims_of<V>(p, kWhole);
        const cudaError_t e = segment_maps<T, GATE, V, WIDE, true>(p, s);
        if (e != cudaSuccess) return e;
        constexpr int ROW = 32 * V * (int)sizeof(T);
        return few_ctas(p, s) ? tiles<T, GATE, V, WIDE, BwdFew<ROW>>(p, s) : tiles<T, GATE, V, WIDE, Bwd<ROW>>(p, s);
    }
    template <typename T, int GATE, int V, bool WIDE, typename C>
    static cudaError_t tiles(const RecProblem &p, const Dims &s) {
        return launch_tiles<C>(rec_backward_kernel<T, GATE, V, WIDE, C::W, C::R, C::S, C::CTAS>,
                               sizeof(BackTiles<T, V, WIDE, C::W, GATE == LA_GATE_SIGMOID ? 2 : 1, C::R, C::S>), p, s,
                               s.segments, p.x, p.g, p.out, p.dout,
                               p.dx, p.dg, s, p.h0, p.dhN, p.dh0);
    }
};

// Largest power of two that divides every row's first address, in bytes (at most 16).
int row_alignment(const RecProblem &p, int size) {
    unsigned long long bits = 16 | (unsigned long long)p.D * size;
    for (const la_view &v : {p.x, p.g, p.out, p.dout, p.dx, p.dg})   // those that a call lacks are 0
        bits |= reinterpret_cast<uintptr_t>(v.data) | (unsigned long long)(v.sb | v.sh | v.sn) * size;
    return (int)(bits & (~bits + 1));
}

// Channels a lane takes: 8 bytes of a row.  Half of that where the last strip would
// be less than half full, and where it makes enough strips to do without segments:
// from half as many as SMs in the forward, whose segments cost more (64 strips of
// 4096 tokens, bf16: 53 us in segments, 36 us as 128 narrow strips; 40 of 8192: 68
// and 62 us), from two thirds in the backward (the same: 80 and 68 us; 92 and 119 us).
template <typename Call, typename T, int GATE> cudaError_t choose(const RecProblem &p) {
    constexpr int V = 8 / (int)sizeof(T), C = 32 * V;
    const long long heads = (long long)p.B * p.H, strips = heads * strips_of(p.D, C);
    const long long narrow = heads * strips_of(p.D, C / 2);
    const bool half = (p.D % C != 0 && p.D % C <= C / 2 && p.D < 8 * C) ||
                      (strips * 2 <= kSms && narrow >= Call::kUnsplit);
    if (row_alignment(p, sizeof(T)) == 16)
        return half ? Call::template run<T, GATE, V / 2, true>(p) : Call::template run<T, GATE, V, true>(p);
    return half ? Call::template run<T, GATE, V / 2, false>(p) : Call::template run<T, GATE, V, false>(p);
}

template <typename Call, int GATE> cudaError_t choose(const RecProblem &p) {
    return p.dtype == LA_DTYPE_F32 ? choose<Call, float, GATE>(p) : choose<Call, __nv_bfloat16, GATE>(p);
}

template <typename Call> cudaError_t choose_gate(const RecProblem &p) {
    switch (p.gate) {
        case LA_GATE_DECAY: return choose<Call, LA_GATE_DECAY>(p);
        case LA_GATE_LOG: return choose<Call, LA_GATE_LOG>(p);
        case LA_GATE_SIGMOID: return choose<Call, LA_GATE_SIGMOID>(p);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

// Segments times channels is at most 304 strips' worth (of 128 channels) where
// there is more than one segment.
size_t recurrence_ws_bytes(const la_shape &s) {
    const long long channels = (long long)s.B * s.H * s.D;
    if (s.N <= Backward::kWhole || channels == 0) return 0;   // the shorter of the two
    const long long strips = (long long)s.B * s.H * strips_of(s.D, 128);   // the fewest that any lane width gives
    if (strips * 2 > kSms) return 0;
    const long long most = std::min(2LL * kSms / strips, ((long long)s.N + kSegmentRows - 1) / kSegmentRows);
    return (size_t)most * channels * sizeof(float2);
}

cudaError_t recurrence_forward(const RecProblem &p) { return choose_gate<Forward>(p); }
cudaError_t recurrence_backward(const RecProblem &p) { return choose_gate<Backward>(p); }

}  // namespace la
