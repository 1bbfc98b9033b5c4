// la_decay.cu - linear attention with a decay for each head: sweeps in fp32
// arithmetic on CUDA cores (fp32 data, rows off 16 bytes), the scan of the
// segments' states, and the step of one token.
#include <algorithm>

#include "la_common.cuh"
#include "la_decay.h"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 32;      // tokens a chunk
constexpr int kCols = 64;      // columns of z that a CTA takes
constexpr int kSms = 152;

// What a token of a sequence decays to after e more tokens.  e^0 = 1 also where
// g is -infinity.
__device__ __forceinline__ float decayed(float g, int e) { return e == 0 ? 1.f : expf(g * (float)e); }

template <typename T>
__device__ __forceinline__ const T *row_of(const la_view &v, long long b, int h, long long t) {
    return static_cast<const T *>(v.data) + b * v.sb + h * v.sh + t * v.sn;
}

size_t sweep_smem(int D) {
    return sizeof(float) * ((size_t)D * kCols + 2 * kRows * (D + 1) + kRows * kCols + kRows * (kRows + 1) + kRows + 1);
}

// One CTA walks over one segment of one head for up to kCols columns of z, chunk
// by chunk, the state in shared memory.
template <typename T>
__global__ void __launch_bounds__(kThreads) sweep_kernel(const DecayLaunch l) {
    extern __shared__ float sm[];
    int y = blockIdx.y, k = 0;
    for (; k + 1 < l.sweeps; k++) {
        const int blocks = (l.sweep[k].M + kCols - 1) / kCols;
        if (y < blocks) break;
        y -= blocks;
    }
    const DecaySweep &s = l.sweep[k];
    const int D = s.D, M = s.M, m0 = y * kCols, cols = min(kCols, M - m0), ld = D + 1;
    float *S = sm, *X = S + D * kCols, *Y = X + kRows * ld, *Z = Y + kRows * ld, *A = Z + kRows * kCols;
    float *w = A + kRows * (kRows + 1);   // decays by 0..kRows tokens
    const int seg = blockIdx.x % l.segs, bh = blockIdx.x / l.segs, b = bh / l.H, h = bh % l.H, tid = threadIdx.x;
    if (l.sums && seg == (s.backwards ? 0 : l.segs - 1)) return;   // nobody asks for that one
    const float g = l.log_decay[h];
    const int len = l.lens ? max(0, min(l.N, l.lens[b])) : l.N;
    const int first = seg * l.seg_tokens;
    const int n = max(0, min(len - first, l.seg_tokens)), chunks = (n + kRows - 1) / kRows;
    const size_t DM = (size_t)D * M;
    const float *start = l.sums || s.start == nullptr ? nullptr
                                                      : s.start + (l.starts ? (size_t)bh * l.segs + seg : bh) * DM;
    auto at = [&](int d, int m) { return s.transposed ? (size_t)m * D + d : (size_t)d * M + m; };
    for (int i = tid; i < D * kCols; i += kThreads) {
        const int d = i / kCols, m = i % kCols;
        S[i] = start && m < cols ? start[at(d, m0 + m)] : 0.f;
    }
    if (tid <= kRows) w[tid] = decayed(g, tid);
    T *out = static_cast<T *>(s.out.data);
    if (out) out += b * s.out.sb + h * s.out.sh;
    for (int it = 0; it < chunks; it++) {
        const int c = s.backwards ? chunks - 1 - it : it;
        const int t0 = first + c * kRows, rows = min(kRows, n - c * kRows);
        __syncthreads();
        for (int i = tid; i < kRows * D; i += kThreads) {
            const int r = i / D, d = i % D;
            X[r * ld + d] = out && r < rows ? to_f32(row_of<T>(s.x, b, h, t0 + r)[d]) : 0.f;
            Y[r * ld + d] = r < rows ? to_f32(row_of<T>(s.y, b, h, t0 + r)[d]) : 0.f;
        }
        for (int i = tid; i < kRows * kCols; i += kThreads) {
            const int r = i / kCols, m = i % kCols;
            Z[i] = r < rows && m < cols ? to_f32(row_of<T>(s.z, b, h, t0 + r)[m0 + m]) : 0.f;
        }
        __syncthreads();
        if (out) {
            for (int i = tid; i < kRows * kRows; i += kThreads) {
                const int r = i / kRows, j = i % kRows, e = s.backwards ? j - r : r - j;
                float t = 0.f;
                if (e >= 0 && r < rows && j < rows) {
                    for (int d = 0; d < D; d++) t = fmaf(X[r * ld + d], Y[j * ld + d], t);
                    t *= w[e];
                }
                A[r * (kRows + 1) + j] = t;
            }
            __syncthreads();
            for (int i = tid; i < rows * kCols; i += kThreads) {
                const int r = i / kCols, m = i % kCols;
                if (m >= cols) continue;
                float intra = 0.f, inter = 0.f;
                const int j0 = s.backwards ? r : 0, j1 = s.backwards ? rows : r + 1;
                for (int j = j0; j < j1; j++) intra = fmaf(A[r * (kRows + 1) + j], Z[j * kCols + m], intra);
                for (int d = 0; d < D; d++) inter = fmaf(X[r * ld + d], S[d * kCols + m], inter);
                const float by = w[s.backwards ? rows - 1 - r : r + 1];
                out[(long long)(t0 + r) * s.out.sn + m0 + m] =
                    from_f32<T>(fmaf(s.c_intra, intra, s.c_inter * by * inter));
            }
            __syncthreads();
        }
        const float2 a = kept(g, rows);
        for (int i = tid; i < D * kCols; i += kThreads) {
            const int d = i / kCols, m = i % kCols;
            float t = 0.f;
            for (int r = 0; r < rows; r++)
                t = fmaf(Y[r * ld + d] * w[s.backwards ? r + 1 : rows - 1 - r], Z[r * kCols + m], t);
            S[i] = fmaf(s.c_state, t, keep(a, S[i]));
        }
    }
    __syncthreads();
    // the state leaves where the sequence's last segment (backwards: its first) ends
    const int last = max(0, (len + l.seg_tokens - 1) / l.seg_tokens - 1);
    if (s.end && (l.sums || seg == (s.backwards ? 0 : last))) {
        float *end = s.end + (l.sums ? (size_t)bh * l.segs + seg : bh) * DM;
        for (int i = tid; i < D * kCols; i += kThreads) {
            const int d = i / kCols, m = i % kCols;
            if (m < cols) end[at(d, m0 + m)] = S[i];
        }
    }
    if (out)   // rows past the length
        for (int t = first + n; t < min(first + l.seg_tokens, l.N); t++)
            for (int m = tid; m < cols; m += kThreads) out[(long long)t * s.out.sn + m0 + m] = from_f32<T>(0.f);
}

// Sums of the segments [B*H][segs][DM] become the states at their starts (for
// sweeps backwards in time: behind their last tokens).
__global__ void __launch_bounds__(256) scan_kernel(float *ws, const float *start, const float *log_decay,
                                                   const int *lens, int H, int N, int segs, int seg_tokens, int DM,
                                                   int backwards) {
    const int bh = blockIdx.y, e = blockIdx.x * 256 + threadIdx.x;
    const float g = log_decay[bh % H];
    const int len = lens ? max(0, min(N, lens[bh / H])) : N;
    if (e >= DM) return;
    float *p = ws + (size_t)bh * segs * DM + e;
    float s = start ? start[(size_t)bh * DM + e] : 0.f;
    // the segment that ends the sequence, and what the state loses over it and over the whole ones before
    const int last = len > 0 ? (len - 1) / seg_tokens : -1;
    const float2 whole = kept(g, seg_tokens), part = kept(g, len - last * seg_tokens);
#pragma unroll 4
    for (int i = 0; i < segs; i++) {
        const int seg = backwards ? segs - 1 - i : i;
        const float sum = i < segs - 1 ? p[(size_t)seg * DM] : 0.f;   // no state comes after the last one
        p[(size_t)seg * DM] = s;
        if (seg <= last) s = keep(seg == last ? part : whole, s) + sum;
    }
}

// ------------------------------------------------------------- one token

struct StepArgs {
    la_view q, k, v, y;
    const float *log_decay;
    float *S;
    int H, D, M, blocks;
    float scale;
};

// S <- a S + k v^T, y = scale q^T S for L lanes' columns of one head: VEC values
// a lane, the rows over the CTA's threads, all of them on their way at once.
template <typename T, int L, int K, int VEC>
__global__ void __launch_bounds__(128) step_kernel(const StepArgs a) {
    constexpr int R = 128 / L;   // rows a pass
    __shared__ float qs[R * K], ks[R * K], part[4][L * VEC];
    const int bh = blockIdx.x / a.blocks, blk = blockIdx.x % a.blocks, b = bh / a.H, h = bh % a.H, tid = threadIdx.x;
    const int m = (blk * L + tid % L) * VEC, r = tid / L;
    float *S = a.S + (size_t)bh * a.D * a.M + m;
    float s[K][VEC];
    const bool in = m < a.M;
#pragma unroll
    for (int k = 0; k < K; k++) {
        const int d = r + k * R;
#pragma unroll
        for (int i = 0; i < VEC; i++) s[k][i] = 0.f;
        if (in && d < a.D) {
            if constexpr (VEC == 4) {
                const float4 t = *reinterpret_cast<const float4 *>(S + (size_t)d * a.M);
                s[k][0] = t.x, s[k][1] = t.y, s[k][2] = t.z, s[k][3] = t.w;
            } else {
                s[k][0] = S[(size_t)d * a.M];
            }
        }
    }
    const T *q = row_of<T>(a.q, b, h, 0), *kk = row_of<T>(a.k, b, h, 0), *vv = row_of<T>(a.v, b, h, 0);
    for (int d = tid; d < R * K; d += 128) {
        qs[d] = d < a.D ? to_f32(q[d]) : 0.f;
        ks[d] = d < a.D ? to_f32(kk[d]) : 0.f;
    }
    float v[VEC], acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; i++) v[i] = in ? to_f32(vv[m + i]) : 0.f, acc[i] = 0.f;
    const float2 decay = kept(a.log_decay[h], 1);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; k++) {
        const int d = r + k * R;
        if (d >= a.D) continue;
        const float kd = ks[d], qd = qs[d];
#pragma unroll
        for (int i = 0; i < VEC; i++) {
            s[k][i] = fmaf(kd, v[i], keep(decay, s[k][i]));
            acc[i] = fmaf(qd, s[k][i], acc[i]);
        }
        if (in) {
            if constexpr (VEC == 4)
                *reinterpret_cast<float4 *>(S + (size_t)d * a.M) = make_float4(s[k][0], s[k][1], s[k][2], s[k][3]);
            else
                S[(size_t)d * a.M] = s[k][0];
        }
    }
    // rows of the warp, then of the warps
#pragma unroll
    for (int i = 0; i < VEC; i++)
#pragma unroll
        for (int o = L; o < 32; o *= 2) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    if (tid % 32 < L)
#pragma unroll
        for (int i = 0; i < VEC; i++) part[tid / 32][tid % 32 * VEC + i] = acc[i];
    __syncthreads();
    const int c = blk * L * VEC + tid;
    if (tid < L * VEC && c < a.M) {
        T *y = static_cast<T *>(a.y.data) + b * a.y.sb + h * a.y.sh;
        y[c] = from_f32<T>(a.scale * ((part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid])));
    }
}

template <typename T, int L, int VEC> cudaError_t step_of(const StepArgs &a, long long heads, cudaStream_t st) {
    constexpr int R = 128 / L;
    const int ctas = (int)(heads * a.blocks);
    if (a.D <= R * 4) step_kernel<T, L, 4, VEC><<<ctas, 128, 0, st>>>(a);
    else if (a.D <= R * 8) step_kernel<T, L, 8, VEC><<<ctas, 128, 0, st>>>(a);
    else step_kernel<T, L, 16, VEC><<<ctas, 128, 0, st>>>(a);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T> cudaError_t step(const DecayProblem &p) {
    StepArgs a{p.q, p.k, p.v, p.out, p.log_decay, p.SN, p.H, p.D, p.M, 1, p.scale};
    const long long heads = (long long)p.B * p.H;
    if (p.M % 4 == 0 && (reinterpret_cast<uintptr_t>(p.SN) & 15) == 0) {
        a.blocks = (p.M + 63) / 64;
        // few heads: columns over more CTAs (16 of them a CTA, whole 32 byte sectors still)
        if (heads * a.blocks < kSms * 4) {
            a.blocks = (p.M + 31) / 32;
            return step_of<T, 8, 4>(a, heads, p.stream);
        }
        return step_of<T, 16, 4>(a, heads, p.stream);
    }
    a.blocks = (p.M + 15) / 16;
    return step_of<T, 16, 1>(a, heads, p.stream);
}

// ------------------------------------------------------------- segments

struct Cut {
    int segs, tokens;
};

// Segments of a sequence.  `ctas` walk over the whole sequences side by side, one to
// an SM; cut, there are `segs` times as many, which have first to find the states at
// their starts: `sums` CTAs a segment, then a scan that moves `states` bytes a segment.
// In chunks of 128 tokens (about 2.1 us): a CTA's start and end cost six, a chunk's sums
// 0.9, a scan's launch two.  16 heads of 65536 tokens, D = M = 128: 4 segments 519 us,
// 19 566; 16 heads of 16384, backward: 1 segment 278 us, 3 303.
Cut cut_of(long long ctas, long long sums, double states, int N) {
    const long long chunks = ((long long)N + 127) / 128;
    long long best = 1;
    double least = 0;
    for (long long segs = 1; segs <= std::min<long long>(chunks, 4 * kSms) && (segs == 1 || ctas * segs <= 4 * kSms); segs++) {
        const long long per = (chunks + segs - 1) / segs;
        if (segs > 1 && (chunks + per - 1) / per != segs) continue;   // the same as fewer
        auto waves = [&](long long n) { return (n + kSms - 1) / kSms; };
        double cost = waves(ctas * segs) * (per + 6.0);
        if (segs > 1) cost += waves(sums * (segs - 1)) * (0.9 * per + 6) + 2 + segs * states / (6.5e6 * 2.1);
        if (segs == 1 || cost < least) best = segs, least = cost;
    }
    const long long per = (chunks + best - 1) / best;
    return {(int)best, best == 1 ? std::max(N, 1) : (int)(per * 128)};
}
int blocks_of(int w) { return (w + kCols - 1) / kCols; }
Cut cut_of(int B, int H, int N, int D, int M, bool backward) {
    const long long heads = (long long)B * H, d = blocks_of(D), m = blocks_of(M);
    const double states = 16.0 * heads * D * M;   // written, scanned, read
    return backward ? cut_of(heads * (2 * d + m), heads * 2 * m, 2 * states, N) : cut_of(heads * m, heads * m, states, N);
}

template <typename T> cudaError_t simt_decay(const DecayLaunch &l) {
    int blocks = 0, D = 0;
    for (int i = 0; i < l.sweeps; i++) blocks += blocks_of(l.sweep[i].M), D = std::max(D, l.sweep[i].D);
    const size_t smem = sweep_smem(D);
    cudaError_t e = cudaFuncSetAttribute(sweep_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sweep_smem(kDecayMaxD));
    if (e != cudaSuccess) return e;
    sweep_kernel<T><<<dim3((unsigned)((long long)l.B * l.H * l.segs), blocks), kThreads, smem, l.stream>>>(l);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t run(const DecayLaunch &l, la_dtype dtype) {
    if (tc_decay_supported(l, dtype)) return tc_decay(l);
    return dtype == LA_DTYPE_F32 ? simt_decay<float>(l) : simt_decay<__nv_bfloat16>(l);
}

cudaError_t scan(const DecayLaunch &l, float *ws, const float *start, int DM, int backwards) {
    scan_kernel<<<dim3((DM + 255) / 256, l.B * l.H), 256, 0, l.stream>>>(ws, start, l.log_decay, l.lens, l.H, l.N,
                                                                       l.segs, l.seg_tokens, DM, backwards);
    count_launches(1);
    return cudaGetLastError();
}

DecayLaunch launch_of(const DecayProblem &p, const Cut &cut) {
    DecayLaunch l{};
    l.log_decay = p.log_decay, l.lens = p.lens, l.B = p.B, l.H = p.H, l.N = p.N;
    l.segs = cut.segs, l.seg_tokens = cut.tokens, l.stream = p.stream;
    return l;
}

}  // namespace

size_t decay_ws_bytes(const la_shape &s, bool backward) {
    const Cut c = cut_of(s.B, s.H, s.N, s.D, s.M, backward);
    if (c.segs == 1) return 0;
    return (size_t)s.B * s.H * c.segs * s.D * s.M * sizeof(float) * (backward ? 2 : 1);
}

cudaError_t decay_forward(const DecayProblem &p) {
    DecayLaunch l = launch_of(p, cut_of(p.B, p.H, p.N, p.D, p.M, false));
    const la_view none{nullptr, 0, 0, 0};
    l.sweeps = 1;
    DecaySweep &s = l.sweep[0];
    s = {none, p.k, p.v, none, nullptr, nullptr, p.D, p.M, 0, 0, p.scale, p.scale, 1.f};
    float *ws = static_cast<float *>(p.ws);
    if (l.segs > 1) {
        l.sums = 1;
        s.end = ws;
        cudaError_t e = run(l, p.dtype);
        if (e == cudaSuccess) e = scan(l, ws, p.S0, p.D * p.M, 0);
        if (e != cudaSuccess) return e;
        l.sums = 0;
    }
    s.x = p.q, s.out = p.out;
    s.start = l.segs > 1 ? ws : p.S0, s.end = p.SN;
    l.starts = l.segs > 1;
    return run(l, p.dtype);
}

cudaError_t decay_backward(const DecayProblem &p) {
    DecayLaunch l = launch_of(p, cut_of(p.B, p.H, p.N, p.D, p.M, true));
    const la_view none{nullptr, 0, 0, 0};
    const int DM = p.D * p.M;
    const float *S0 = p.S0, *dSN = p.dSN;
    if (l.segs > 1) {
        float *wf = static_cast<float *>(p.ws), *wb = wf + (size_t)p.B * p.H * l.segs * DM;
        l.sums = 1, l.sweeps = 2;
        l.sweep[0] = {none, p.k, p.v, none, nullptr, wf, p.D, p.M, 0, 0, 0.f, 0.f, 1.f};
        l.sweep[1] = {none, p.q, p.dout, none, nullptr, wb, p.D, p.M, 0, 1, 0.f, 0.f, p.scale};
        cudaError_t e = run(l, p.dtype);
        if (e == cudaSuccess) e = scan(l, wf, S0, DM, 0);
        if (e == cudaSuccess) e = scan(l, wb, dSN, DM, 1);
        if (e != cudaSuccess) return e;
        l.sums = 0, l.starts = 1;
        S0 = wf, dSN = wb;
    }
    l.sweeps = 3;
    l.sweep[0] = {p.dout, p.v, p.k, p.dq, S0, nullptr, p.M, p.D, 1, 0, p.scale, p.scale, 1.f};
    l.sweep[1] = {p.k, p.q, p.dout, p.dv, dSN, p.dS0, p.D, p.M, 0, 1, p.scale, 1.f, p.scale};
    l.sweep[2] = {p.v, p.dout, p.q, p.dk, dSN, nullptr, p.M, p.D, 1, 1, p.scale, 1.f, p.scale};
    return run(l, p.dtype);
}

cudaError_t decay_step(const DecayProblem &p) {
    return p.dtype == LA_DTYPE_F32 ? step<float>(p) : step<__nv_bfloat16>(p);
}

}  // namespace la
