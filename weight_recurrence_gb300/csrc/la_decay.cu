// la_decay.cu - linear attention with a decay for each head: sweeps in fp32
// arithmetic on CUDA cores (fp32 data, short bf16 rows off 16 bytes), the scan of
// the segments' states, the packing of long bf16 rows, and steps of one or a few tokens.
#include <algorithm>

#include "la_common.cuh"
#include "la_decay.h"
#include "la_pair.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 64;      // tokens a chunk
constexpr int kCols = 64;      // columns of z that a CTA takes
constexpr int kSms = 152;

// What a token of a sequence decays to after e more tokens.  e^0 = 1 also where
// g is -infinity.
__device__ __forceinline__ float decayed(float g, int e) { return e == 0 ? 1.f : expf(g * (float)e); }

template <typename T>
__device__ __forceinline__ const T *row_of(const la_view &v, long long b, int h, long long t) {
    return static_cast<const T *>(v.data) + b * v.sb + h * v.sh + t * v.sn;
}

// Shared memory of a CTA (floats): x and y [kRows][64 DT], z and the weighted z
// [kRows][kCols], the scores [kRows][kRows + 4], the state [64 DT][kCols], decays.
constexpr int kScores = kRows + 4;
constexpr size_t sweep_smem(int dt) {
    return sizeof(float) * ((size_t)2 * kRows * 64 * dt + 2 * kRows * kCols + kRows * kScores + 64 * dt * kCols + kRows + 4);
}

// Where the 16-byte piece p of row r of x or y lies: threads read rows 4 apart at the
// same time, so each four rows turn the pieces' order by one.
template <int DT> __device__ __forceinline__ int place(int r, int p) { return r * 64 * DT + 4 * (p ^ (r >> 2 & 7)); }

// A thread's share of kRows rows of up to 64 U columns: pieces of four values, 16
// threads to a row.  Zeros behind `rows` rows and `n` columns.
template <typename T, int U>
__device__ __forceinline__ void fetch(float4 (&v)[4 * U], const T *src, long long sn, int rows, int n, bool wide) {
    const int c0 = threadIdx.x % 16 * 4, r0 = threadIdx.x / 16;
#pragma unroll
    for (int i = 0; i < 4 * U; i++) {
        const int r = r0 + 16 * (i % 4), c = c0 + 64 * (i / 4);
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows && c < n) {
            const T *p = src + (long long)r * sn + c;
            if constexpr (sizeof(T) == 4) {
                if (wide) {
                    v[i] = *reinterpret_cast<const float4 *>(p);
                    continue;
                }
            }
            v[i].x = to_f32(p[0]);
            if (c + 1 < n) v[i].y = to_f32(p[1]);
            if (c + 2 < n) v[i].z = to_f32(p[2]);
            if (c + 3 < n) v[i].w = to_f32(p[3]);
        }
    }
}
template <int DT> __device__ __forceinline__ void put_rows(float *dst, const float4 (&v)[4 * DT]) {
    const int p0 = threadIdx.x % 16, r0 = threadIdx.x / 16;
#pragma unroll
    for (int i = 0; i < 4 * DT; i++)
        *reinterpret_cast<float4 *>(dst + place<DT>(r0 + 16 * (i % 4), p0 + 16 * (i / 4))) = v[i];
}

__device__ __forceinline__ float4 piece(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ void axpy(float4 &acc, float a, const float4 &v) {
    acc.x = fmaf(a, v.x, acc.x), acc.y = fmaf(a, v.y, acc.y), acc.z = fmaf(a, v.z, acc.z), acc.w = fmaf(a, v.w, acc.w);
}
__device__ __forceinline__ float dot(const float4 &a, const float4 &b, float t) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, t))));
}

// One CTA walks over one segment of one head for up to kCols columns of z, in chunks
// of kRows tokens.  Every product is taken by tiles of 4 x 4 in registers: threads
// (ti, tj) of 16 x 16.  The state lies in registers too (rows 4 ti.. and, DT = 2,
// 64 + 4 ti.., columns 4 tj..) with a copy in shared memory for x S.  Bound by the
// instructions and the waits between a chunk's five steps: 160 D + 2048 multiply-adds
// for a token and 64 columns keep the FMA pipe 42 % busy, issue 63 %, the shared
// memory 59 % (the backward of 128 heads of 1024 tokens, 64 channels: 384 us).
// Tiles of 8 x 4 on half of the threads were slower (7 ragged sequences of 1537
// tokens, 5 heads: 108 -> 128 us), and so were 512 threads above 64 channels (128
// heads of 1024 tokens, 128 channels: 491 -> 555 us).  Tensor cores would need six
// bf16 products (or three of tf32) in place of each of these to keep fp32's digits.
template <typename T, int DT>
__global__ void __launch_bounds__(kThreads, DT == 1 ? 2 : 1) sweep_kernel(const __grid_constant__ DecayLaunch l) {
    extern __shared__ __align__(16) float sm[];
    int y = blockIdx.y, k = 0;
    for (; k + 1 < l.sweeps; k++) {
        const int blocks = (l.sweep[k].M + kCols - 1) / kCols;
        if (y < blocks) break;
        y -= blocks;
    }
    const DecaySweep &s = l.sweep[k];
    const int D = s.D, M = s.M, m0 = y * kCols, cols = min(kCols, M - m0), Dp = (D + 3) / 4 * 4;
    float *X = sm, *Y = X + kRows * 64 * DT, *Z = Y + kRows * 64 * DT, *Zw = Z + kRows * kCols, *A = Zw + kRows * kCols;
    float *S = A + kRows * kScores, *w = S + 64 * DT * kCols;   // w: decays by 0..kRows tokens
    const int seg = blockIdx.x % l.segs, bh = blockIdx.x / l.segs, b = bh / l.H, h = bh % l.H, tid = threadIdx.x;
    const int ti = tid / 16, tj = tid % 16;
    if (l.sums && seg == (s.backwards ? 0 : l.segs - 1)) return;   // nobody asks for that one
    const float g = l.log_decay[h];
    const int len = l.lens ? max(0, min(l.N, l.lens[b])) : l.N;
    const int first = seg * l.seg_tokens;
    const int n = max(0, min(len - first, l.seg_tokens)), chunks = (n + kRows - 1) / kRows;
    const size_t DM = (size_t)D * M;
    const bool back = s.backwards != 0;
    const float *start = l.sums || s.start == nullptr ? nullptr
                                                      : s.start + (l.starts ? (size_t)bh * l.segs + seg : (size_t)bh) * DM;
    auto at = [&](int d, int m) { return s.transposed ? (size_t)m * D + d : (size_t)d * M + m; };
    float4 sv[DT][4];   // rows 64 u + 4 ti + i, columns 4 tj..
#pragma unroll
    for (int u = 0; u < DT; u++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int d = 64 * u + 4 * ti + i, m = m0 + 4 * tj;
            auto get = [&](int j) { return start && d < D && 4 * tj + j < cols ? start[at(d, m + j)] : 0.f; };
            sv[u][i] = make_float4(get(0), get(1), get(2), get(3));
        }
    auto put_state = [&] {
#pragma unroll
        for (int u = 0; u < DT; u++)
#pragma unroll
            for (int i = 0; i < 4; i++) *reinterpret_cast<float4 *>(S + (64 * u + 4 * ti + i) * kCols + 4 * tj) = sv[u][i];
    };
    put_state();
    if (tid <= kRows) w[tid] = decayed(g, tid);
    __syncthreads();
    T *out = static_cast<T *>(s.out.data);
    if (out) out += b * s.out.sb + h * s.out.sh + m0;
    // rows by 16 bytes where every one lies on them
    auto on16 = [&](const la_view &v, int c) {
        return sizeof(T) == 4 && c % 4 == 0 && ((reinterpret_cast<uintptr_t>(v.data) & 15) | (v.sb & 3) | (v.sh & 3) | (v.sn & 3)) == 0;
    };
    const bool xw = on16(s.x, D), yw = on16(s.y, D), zw = on16(s.z, cols), ow = on16(s.out, cols);
    for (int it = 0; it < chunks; it++) {
        const int c = back ? chunks - 1 - it : it, t0 = first + c * kRows, rows = min(kRows, n - c * kRows);
        {
            // all of the chunk's loads on their way, then into shared memory
            float4 vx[4 * DT], vy[4 * DT], vz[4];
            if (out) fetch<T, DT>(vx, row_of<T>(s.x, b, h, t0), s.x.sn, rows, D, xw);
            fetch<T, DT>(vy, row_of<T>(s.y, b, h, t0), s.y.sn, rows, D, yw);
            fetch<T, 1>(vz, row_of<T>(s.z, b, h, t0) + m0, s.z.sn, rows, cols, zw);
            __syncthreads();   // the last chunk's have been read
            if (out) put_rows<DT>(X, vx);
            put_rows<DT>(Y, vy);
#pragma unroll
            for (int i = 0; i < 4; i++) {   // z, and z weighed for the state
                const int r = ti + 16 * i;
                const float by = r < rows ? w[back ? r + 1 : rows - 1 - r] : 0.f;
                *reinterpret_cast<float4 *>(Z + r * kCols + 4 * tj) = vz[i];
                *reinterpret_cast<float4 *>(Zw + r * kCols + 4 * tj) = make_float4(by * vz[i].x, by * vz[i].y, by * vz[i].z, by * vz[i].w);
            }
            __syncthreads();
        }
        if (out) {
            // scores: the 136 tiles on and below the diagonal (backwards: above), decayed
            if (tid < 136) {
                int pi = (int)((sqrtf(8.f * tid + 1.f) - 1.f) * 0.5f);
                while (pi * (pi + 1) / 2 > tid) pi--;
                while ((pi + 1) * (pi + 2) / 2 <= tid) pi++;
                const int pj = tid - pi * (pi + 1) / 2;
                const int i0 = 4 * (back ? pj : pi), j0 = 4 * (back ? pi : pj);
                if (i0 < rows && j0 < rows) {
                    float p[4][4] = {};
#pragma unroll 2
                    for (int d = 0; d < Dp; d += 4) {
                        float4 x[4];
#pragma unroll
                        for (int i = 0; i < 4; i++) x[i] = piece(X + place<DT>(i0 + i, d / 4));
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const float4 v = piece(Y + place<DT>(j0 + j, d / 4));
#pragma unroll
                            for (int i = 0; i < 4; i++) p[i][j] = dot(x[i], v, p[i][j]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        float q[4];
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const int e = back ? j0 + j - i0 - i : i0 + i - j0 - j;
                            q[j] = e >= 0 ? p[i][j] * w[e] : 0.f;
                        }
                        *reinterpret_cast<float4 *>(A + (i0 + i) * kScores + j0) = make_float4(q[0], q[1], q[2], q[3]);
                    }
                }
            }
            __syncthreads();
            // output rows 4 ti.., columns 4 tj..: x S, then the scores' part
            float4 o[4];
#pragma unroll
            for (int i = 0; i < 4; i++) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int d = 0; d < (4 * ti < rows ? Dp : 0); d += 4) {
                float4 v[4];
#pragma unroll
                for (int j = 0; j < 4; j++) v[j] = piece(S + (d + j) * kCols + 4 * tj);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float4 x = piece(X + place<DT>(4 * ti + i, d / 4));
                    axpy(o[i], x.x, v[0]), axpy(o[i], x.y, v[1]), axpy(o[i], x.z, v[2]), axpy(o[i], x.w, v[3]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int r = 4 * ti + i;
                const float by = r < rows ? s.c_inter * w[back ? rows - 1 - r : r + 1] : 0.f;
                o[i] = make_float4(by * o[i].x, by * o[i].y, by * o[i].z, by * o[i].w);
            }
            float4 q[4];
#pragma unroll
            for (int i = 0; i < 4; i++) q[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            const int j_first = back ? 4 * ti + 4 : 0, j_end = back ? (rows + 3) / 4 * 4 : 4 * ti < rows ? 4 * ti : 0;
#pragma unroll 2
            for (int j = j_first; j < j_end; j += 4) {
                float4 v[4];
#pragma unroll
                for (int e = 0; e < 4; e++) v[e] = piece(Z + (j + e) * kCols + 4 * tj);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float4 a = piece(A + (4 * ti + i) * kScores + j);
                    axpy(q[i], a.x, v[0]), axpy(q[i], a.y, v[1]), axpy(q[i], a.z, v[2]), axpy(q[i], a.w, v[3]);
                }
            }
            // the tile on the diagonal: hidden tokens are left out, whatever they hold
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float4 v = piece(Z + (4 * ti + e) * kCols + 4 * tj);
#pragma unroll
                for (int i = 0; i < 4; i++)
                    if (back ? e >= i : e <= i) axpy(q[i], A[(4 * ti + i) * kScores + 4 * ti + e], v);
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int r = 4 * ti + i;
                if (r >= rows) continue;
                axpy(o[i], s.c_intra, q[i]);
                T *p = out + (long long)(t0 + r) * s.out.sn + 4 * tj;
                if constexpr (sizeof(T) == 4) {
                    if (ow && 4 * tj < cols) {
                        *reinterpret_cast<float4 *>(p) = o[i];
                        continue;
                    }
                }
                if (4 * tj < cols) p[0] = from_f32<T>(o[i].x);
                if (4 * tj + 1 < cols) p[1] = from_f32<T>(o[i].y);
                if (4 * tj + 2 < cols) p[2] = from_f32<T>(o[i].z);
                if (4 * tj + 3 < cols) p[3] = from_f32<T>(o[i].w);
            }
        }
        __syncthreads();   // the weighed z; S has been read
        const float2 a = kept(g, rows);
        float4 inc[DT][4];
#pragma unroll
        for (int u = 0; u < DT; u++)
#pragma unroll
            for (int i = 0; i < 4; i++) inc[u][i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int r0 = 0; r0 < rows; r0 += 4) {   // rows past the end are zeros
            const int turn = r0 >> 2 & 7;
#pragma unroll
            for (int r = r0; r < r0 + 4; r++) {
                const float4 v = piece(Zw + r * kCols + 4 * tj);
#pragma unroll
                for (int u = 0; u < DT; u++) {
                    const float4 d = piece(Y + r * 64 * DT + 4 * ((16 * u + ti) ^ turn));
                    axpy(inc[u][0], d.x, v), axpy(inc[u][1], d.y, v), axpy(inc[u][2], d.z, v), axpy(inc[u][3], d.w, v);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < DT; u++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                float4 &t = sv[u][i];
                const float4 &e = inc[u][i];
                t = make_float4(fmaf(s.c_state, e.x, keep(a, t.x)), fmaf(s.c_state, e.y, keep(a, t.y)),
                                fmaf(s.c_state, e.z, keep(a, t.z)), fmaf(s.c_state, e.w, keep(a, t.w)));
            }
        if (out) put_state();
    }
    // the state leaves where the sequence's last segment (backwards: its first) ends
    if (s.end && (l.sums || seg == (back ? 0 : last_segment(len, l.seg_tokens)))) {
        float *end = s.end + (l.sums ? (size_t)bh * l.segs + seg : (size_t)bh) * DM;
#pragma unroll
        for (int u = 0; u < DT; u++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int d = 64 * u + 4 * ti + i, m = m0 + 4 * tj;
                const float v[4] = {sv[u][i].x, sv[u][i].y, sv[u][i].z, sv[u][i].w};
#pragma unroll
                for (int j = 0; j < 4; j++)
                    if (d < D && 4 * tj + j < cols) end[at(d, m + j)] = v[j];
            }
    }
    if (out)   // rows past the length
        for (int t = first + n + ti / 4; t < min(first + l.seg_tokens, l.N); t += 4)
            if (const int m = tid % kCols; m < cols) out[(long long)t * s.out.sn + m] = from_f32<T>(0.f);
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
    // the segment that ends the sequence (-1: there is none), and what the state loses over it and over the whole ones before
    const int last = len > 0 ? last_segment(len, seg_tokens) : -1;
    const int rest = len - last * seg_tokens;
    const float2 whole = kept(g, seg_tokens), part = kept(g, rest);
    // (a loop of its own for the rare far growth: with a choice in one loop its loads are not
    // on their way together, and 16 heads of 65536 tokens, D = M = 128, take 543 us for 490)
    auto walk = [&](auto grown) {
#pragma unroll 4
        for (int i = 0; i < segs; i++) {
            const int seg = backwards ? segs - 1 - i : i;
            const float sum = i < segs - 1 ? p[(size_t)seg * DM] : 0.f;   // no state comes after the last one
            p[(size_t)seg * DM] = s;
            if (seg <= last) s = grown(seg == last) + sum;
        }
    };
    if (grows_far(g, seg_tokens)) walk([&](bool end) { return keep_far(g, end ? rest : seg_tokens, s); });
    else walk([&](bool end) { return keep(end ? part : whole, s); });
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
// a lane, the rows over the CTA's threads, all of them on their way at once.  Bound by
// HBM, the state read and written (4096 heads of 64 x 64, 134 MB: 23.5 us, 5.8 TB/s);
// a few heads by the launch and the host's call (32 heads 5.6 us).
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
    constexpr int most = kDecayMaxD / R;   // rows of a thread: 16, or 8 where there are 16 a pass
    if (a.D <= R * 4) step_kernel<T, L, 4, VEC><<<ctas, 128, 0, st>>>(a);
    else if (most == 8 || a.D <= R * 8) step_kernel<T, L, 8, VEC><<<ctas, 128, 0, st>>>(a);
    else step_kernel<T, L, most, VEC><<<ctas, 128, 0, st>>>(a);
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

// ------------------------------------------------------------- a few tokens

constexpr int kShort = 16;     // tokens of a sequence up to which the walk goes token by token
constexpr int kGroup = 4;      // tokens whose outputs are joined together

struct ShortArgs {
    la_view q, k, v, out;
    const float *log_decay, *S0;
    const int *lens;
    float *SN;
    int H, N, D, M, blocks;
    float scale;
};

// The same as the step over up to kShort tokens, the state in registers from the first
// to the last: it is read and written once, where chunks of 128 tokens would mostly
// multiply zeros.  4096 heads of 64 x 64, 134 MB of states: one token 28 us, then 3 to 4 us
// a token, four instructions for each two values of the state.
template <typename T, int L, int K, int VEC>
__global__ void __launch_bounds__(128) short_kernel(const ShortArgs a) {
    constexpr int R = 128 / L, W = L * VEC;   // rows a pass, columns a CTA
    __shared__ float2 kq[kShort][R * K];
    __shared__ __align__(16) float vs[kShort][W], part[2][4][kGroup][W];
    const int bh = blockIdx.x / a.blocks, blk = blockIdx.x % a.blocks, b = bh / a.H, h = bh % a.H, tid = threadIdx.x;
    const int m0 = blk * W, col = tid % L * VEC, m = m0 + col, r = tid / L, cols = min(W, a.M - m0);
    const int n = a.lens ? max(0, min(a.N, a.lens[b])) : a.N;
    const size_t at = (size_t)bh * a.D * a.M + m;
    const bool in = m < a.M, out = a.out.data != nullptr;
    float s[K][VEC];
#pragma unroll
    for (int k = 0; k < K; k++) {
        const int d = r + k * R;
#pragma unroll
        for (int i = 0; i < VEC; i++) s[k][i] = 0.f;
        if (a.S0 && in && d < a.D) {
            const float *p = a.S0 + at + (size_t)d * a.M;
            if constexpr (VEC == 4) {
                const float4 t = *reinterpret_cast<const float4 *>(p);
                s[k][0] = t.x, s[k][1] = t.y, s[k][2] = t.z, s[k][3] = t.w;
            } else {
                s[k][0] = *p;
            }
        }
    }
    const T *q = out ? row_of<T>(a.q, b, h, 0) : nullptr, *kk = row_of<T>(a.k, b, h, 0), *vv = row_of<T>(a.v, b, h, 0) + m0;
    // rows behind the last token of a group add nothing (a row that is not there is 0)
    const int groups = (n + kGroup - 1) / kGroup;
    for (int i = tid; i < groups * kGroup * R * K; i += 128) {
        const int t = i / (R * K), d = i % (R * K);
        const bool is = t < n && d < a.D;
        kq[t][d] = make_float2(is ? to_f32(kk[t * a.k.sn + d]) : 0.f, is && out ? to_f32(q[t * a.q.sn + d]) : 0.f);
    }
    for (int i = tid; i < groups * kGroup * W; i += 128) {
        const int t = i / W, c = i % W;
        vs[t][c] = t < n && c < cols ? to_f32(vv[t * a.v.sn + c]) : 0.f;
    }
    const float2 decay = kept(a.log_decay[h], 1);
    T *y = out ? static_cast<T *>(a.out.data) + b * a.out.sb + h * a.out.sh + m0 : nullptr;
    __syncthreads();
    for (int g = 0; g < groups; g++) {
        float acc[kGroup][VEC];
#pragma unroll
        for (int j = 0; j < kGroup; j++) {
            const int t = g * kGroup + j;
            float v[VEC];
#pragma unroll
            for (int i = 0; i < VEC; i++) v[i] = vs[t][col + i], acc[j][i] = 0.f;
            if (t >= n) continue;
#pragma unroll
            for (int k = 0; k < K; k++) {
                if (r + k * R >= a.D) continue;
                const float2 x = kq[t][r + k * R];
                if constexpr (VEC == 4) {
                    const float2 kd = make_float2(x.x, x.x), qd = make_float2(x.y, x.y);
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        float2 t2 = make_float2(s[k][i], s[k][i + 1]);
                        t2 = fma_pair(make_float2(decay.y, decay.y), t2, mul_pair(make_float2(decay.x, decay.x), t2));
                        t2 = fma_pair(kd, make_float2(v[i], v[i + 1]), t2);
                        const float2 o = fma_pair(qd, t2, make_float2(acc[j][i], acc[j][i + 1]));
                        s[k][i] = t2.x, s[k][i + 1] = t2.y, acc[j][i] = o.x, acc[j][i + 1] = o.y;
                    }
                } else {
                    s[k][0] = fmaf(x.x, v[0], keep(decay, s[k][0]));
                    acc[j][0] = fmaf(x.y, s[k][0], acc[j][0]);
                }
            }
        }
        if (!out) continue;
        // rows of the warp, then of the warps
#pragma unroll
        for (int j = 0; j < kGroup; j++)
#pragma unroll
            for (int i = 0; i < VEC; i++) {
#pragma unroll
                for (int o = L; o < 32; o *= 2) acc[j][i] += __shfl_xor_sync(0xffffffffu, acc[j][i], o);
                if (tid % 32 < L) part[g & 1][tid / 32][j][col + i] = acc[j][i];
            }
        __syncthreads();
        for (int i = tid; i < kGroup * W; i += 128) {
            const int j = i / W, c = i % W, t = g * kGroup + j;
            const float(&p)[4][kGroup][W] = part[g & 1];
            if (t < n && c < cols)
                y[t * a.out.sn + c] = from_f32<T>(a.scale * ((p[0][j][c] + p[1][j][c]) + (p[2][j][c] + p[3][j][c])));
        }
    }
    if (a.SN && in)
#pragma unroll
        for (int k = 0; k < K; k++) {
            const int d = r + k * R;
            if (d >= a.D) continue;
            float *p = a.SN + at + (size_t)d * a.M;
            if constexpr (VEC == 4) *reinterpret_cast<float4 *>(p) = make_float4(s[k][0], s[k][1], s[k][2], s[k][3]);
            else *p = s[k][0];
        }
    if (out)   // rows past the length
        for (int i = tid; i < (a.N - n) * W; i += 128) {
            const int t = n + i / W, c = i % W;
            if (c < cols) y[t * a.out.sn + c] = from_f32<T>(0.f);
        }
}

template <typename T, int L, int VEC> cudaError_t short_of(const ShortArgs &a, long long heads, cudaStream_t st) {
    constexpr int R = 128 / L;
    const int ctas = (int)(heads * a.blocks);
    constexpr int most = kDecayMaxD / R;   // rows of a thread: 16, or 8 where there are 16 a pass
    if (a.D <= R * 4) short_kernel<T, L, 4, VEC><<<ctas, 128, 0, st>>>(a);
    else if (most == 8 || a.D <= R * 8) short_kernel<T, L, 8, VEC><<<ctas, 128, 0, st>>>(a);
    else short_kernel<T, L, most, VEC><<<ctas, 128, 0, st>>>(a);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T> cudaError_t short_forward(const DecayProblem &p) {
    ShortArgs a{p.q, p.k, p.v, p.out, p.log_decay, p.S0, p.lens, p.SN, p.H, p.N, p.D, p.M, 1, p.scale};
    const long long heads = (long long)p.B * p.H;
    const bool wide = p.M % 4 == 0 && ((reinterpret_cast<uintptr_t>(p.SN) | reinterpret_cast<uintptr_t>(p.S0)) & 15) == 0;
    a.blocks = (p.M + 63) / 64;
    if (wide && heads * a.blocks >= kSms * 4) return short_of<T, 16, 4>(a, heads, p.stream);
    if (wide) {   // few heads: columns over more CTAs
        a.blocks = (p.M + 31) / 32;
        return short_of<T, 8, 4>(a, heads, p.stream);
    }
    a.blocks = (p.M + 15) / 16;
    return short_of<T, 16, 1>(a, heads, p.stream);
}

// ------------------------------------------------------------- segments

struct Cut {
    int segs, tokens;
};

// What a walk costs, in chunks of 128 tokens: a CTA's start and end, a chunk's sums
// alone, a scan's launch; the chunk's time where the SMs are full (it weighs a scan's
// bytes against the rest); CTAs that an SM holds.
struct Cost {
    double start, sums, scan, us;
    int slots;
};
// tensor cores (bf16) and FMA units
constexpr Cost kTensor = {6.0, 0.9, 2.0, 2.1, 1}, kFma64 = {0.5, 0.4, 0.4, 32.0, 2}, kFma128 = {0.5, 0.4, 0.4, 30.0, 1};

// Segments of a sequence.  `ctas` walk over the whole sequences side by side; cut,
// there are `segs` times as many, which have first to find the states at their
// starts: `sums` CTAs a segment, then a scan that moves `states` bytes a segment.
// Measured, us: tensor cores, 16 heads of 65536 tokens, D = M = 128: 9 segments (taken)
// 490, 4 506, 8 540, 19 554, none 1087; backward of 16 heads of 16384: none (taken)
// 264, 2 383, 3 290; 8 heads of 16384, D = M = 64: 19 (taken) 45, 4 126, none 262.
// FMA units, 35 heads of 1537, D = M = 64: 7 (taken) and 13 107, 4 119, none 236.
Cut cut_of(long long ctas, long long sums, double states, int N, const Cost &cost) {
    const long long chunks = ((long long)N + 127) / 128, slots = (long long)kSms * cost.slots;
    long long best = 1;
    double least = 0;
    for (long long segs = 1; segs <= std::min(chunks, 4 * slots) && (segs == 1 || ctas * segs <= 4 * slots); segs++) {
        const long long per = (chunks + segs - 1) / segs;
        if (segs > 1 && (chunks + per - 1) / per != segs) continue;   // the same as fewer
        auto waves = [&](long long n) { return (n + slots - 1) / slots; };
        double t = waves(ctas * segs) * (per + cost.start);
        if (segs > 1)
            t += waves(sums * (segs - 1)) * (cost.sums * per + cost.start) + cost.scan + segs * states / (6.5e6 * cost.us);
        if (segs == 1 || t < least) best = segs, least = t;
    }
    const long long per = (chunks + best - 1) / best;
    return {(int)best, best == 1 ? std::max(N, 1) : (int)(per * 128)};
}
int blocks_of(int w) { return (w + kCols - 1) / kCols; }
Cut cut_of(int B, int H, int N, int D, int M, la_dtype dtype, bool backward) {
    const long long heads = (long long)B * H, d = blocks_of(D), m = blocks_of(M);
    const double states = 16.0 * heads * D * M;   // written, scanned, read
    const Cost &cost = dtype == LA_DTYPE_BF16 ? kTensor : std::max(D, backward ? M : D) <= 64 ? kFma64 : kFma128;
    return backward ? cut_of(heads * (2 * d + m), heads * 2 * m, 2 * states, N, cost)
                    : cut_of(heads * m, heads * m, states, N, cost);
}

template <typename T, int DT> cudaError_t simt_launch(const DecayLaunch &l, int blocks) {
    cudaError_t e = cudaFuncSetAttribute(sweep_kernel<T, DT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sweep_smem(DT));
    if (e != cudaSuccess) return e;
    sweep_kernel<T, DT><<<dim3((unsigned)((long long)l.B * l.H * l.segs), blocks), kThreads, sweep_smem(DT), l.stream>>>(l);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T> cudaError_t simt_decay(const DecayLaunch &l) {
    int blocks = 0, D = 0;
    for (int i = 0; i < l.sweeps; i++) blocks += blocks_of(l.sweep[i].M), D = std::max(D, l.sweep[i].D);
    return D <= 64 ? simt_launch<T, 1>(l, blocks) : simt_launch<T, 2>(l, blocks);
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

// ------------------------------------------------------------- rows off 16 bytes

struct PackArgs {
    la_view v[4];
    uint4 *to[4];
    int n[4];      // values of a row
    int count, H, N;
    long long rows;
    const int *lens;
};

// Rows of n bf16 values to rows of whole 16-byte pieces, zeros behind; rows past a
// length are left alone.  One tensor to a grid row.
__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ PackArgs a) {
    const la_view &v = a.v[blockIdx.y];
    const int n = a.n[blockIdx.y], pieces = (n + 7) / 8;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < a.rows * pieces; i += (long long)gridDim.x * 256) {
        const long long row = i / pieces;
        const int c = (int)(i - row * pieces) * 8, t = (int)(row % a.N);
        const long long bh = row / a.N;
        const int b = (int)(bh / a.H), h = (int)(bh % a.H);
        if (a.lens && t >= a.lens[b]) continue;
        const uint16_t *p = static_cast<const uint16_t *>(v.data) + b * v.sb + h * v.sh + t * v.sn + c;
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 8; j++) o[j] = c + j < n ? p[j] : 0u;
        a.to[blockIdx.y][i] = make_uint4(o[0] | o[1] << 16, o[2] | o[3] << 16, o[4] | o[5] << 16, o[6] | o[7] << 16);
    }
}

// bf16 rows that are not a multiple of 16 bytes long (contiguous ones then lie off
// those boundaries) are packed first where sequences are long: two passes of memory
// more, and then the tensor cores (2 heads of 2379 tokens, D = 99, M = 118: 43 us with it,
// 87 on FMA units; 8 heads of 32 and of 64 tokens take 10.5 and 14.8 us there, 5.9 on
// tensor cores without the packing).
bool packs(int N, int D, int M, la_dtype dtype) { return dtype == LA_DTYPE_BF16 && N >= 64 && (D % 8 || M % 8); }
size_t packed_bytes(int B, int H, int N, int n) { return ((size_t)B * H * N * ((n + 7) / 8) * 16 + 255) / 256 * 256; }

// The problem's inputs packed at ws, its views turned to them.
cudaError_t pack(DecayProblem &p, char *ws, bool backward) {
    la_view *views[4] = {&p.k, &p.v, backward ? &p.dout : nullptr, backward || p.out.data ? &p.q : nullptr};
    PackArgs a{};
    a.H = p.H, a.N = p.N, a.lens = p.lens, a.rows = (long long)p.B * p.H * p.N;
    long long most = 0;
    for (int i = 0; i < 4; i++) {
        if (views[i] == nullptr) continue;
        const int n = i == 0 || i == 3 ? p.D : p.M, pieces = (n + 7) / 8;
        a.v[a.count] = *views[i], a.to[a.count] = reinterpret_cast<uint4 *>(ws), a.n[a.count++] = n;
        const long long row = pieces * 8;
        *views[i] = {ws, row * p.N * p.H, row * p.N, row};
        ws += packed_bytes(p.B, p.H, p.N, n);
        most = std::max(most, a.rows * pieces);
    }
    const int ctas = (int)std::min<long long>((most + 255) / 256, kSms * 8);
    pack_kernel<<<dim3(ctas, a.count), 256, 0, p.stream>>>(a);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

size_t decay_ws_bytes(const la_shape &s, bool backward) {
    const Cut c = cut_of(s.B, s.H, s.N, s.D, s.M, s.dtype, backward);
    size_t bytes = 0;
    if (c.segs > 1) bytes += (size_t)s.B * s.H * c.segs * s.D * s.M * sizeof(float) * (backward ? 2 : 1);
    if (packs(s.N, s.D, s.M, s.dtype))
        bytes = (bytes + 255) / 256 * 256 + 2 * packed_bytes(s.B, s.H, s.N, s.D) + (backward ? 2 : 1) * packed_bytes(s.B, s.H, s.N, s.M);
    return bytes;
}

cudaError_t decay_forward(const DecayProblem &given) {
    DecayProblem p = given;
    // 4096 heads of 64 x 64, 4 and 16 tokens: 41 and 76 us (bf16), in chunks 177 and 178; 8
    // heads, 8 and 16 tokens: 4.6 and 6.7 us, in chunks 5.9 on tensor cores, 8.8 and 9.1 else
    const bool few = (long long)p.B * p.H * blocks_of(p.M) <= kSms;
    if (p.N <= (few && p.dtype == LA_DTYPE_BF16 ? kShort / 2 : kShort)) return p.dtype == LA_DTYPE_F32 ? short_forward<float>(p) : short_forward<__nv_bfloat16>(p);
    DecayLaunch l = launch_of(p, cut_of(p.B, p.H, p.N, p.D, p.M, p.dtype, false));
    const la_view none{nullptr, 0, 0, 0};
    float *ws = static_cast<float *>(p.ws);
    if (p.out.data == nullptr) p.q = none;
    if (packs(p.N, p.D, p.M, p.dtype)) {
        const size_t states = l.segs > 1 ? (size_t)p.B * p.H * l.segs * p.D * p.M * sizeof(float) : 0;
        const cudaError_t e = pack(p, static_cast<char *>(p.ws) + (states + 255) / 256 * 256, false);
        if (e != cudaSuccess) return e;
    }
    l.sweeps = 1;
    DecaySweep &s = l.sweep[0];
    s = {none, p.k, p.v, none, nullptr, nullptr, p.D, p.M, 0, 0, p.scale, p.scale, 1.f};
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

cudaError_t decay_backward(const DecayProblem &given) {
    DecayProblem p = given;
    DecayLaunch l = launch_of(p, cut_of(p.B, p.H, p.N, p.D, p.M, p.dtype, true));
    const la_view none{nullptr, 0, 0, 0};
    const int DM = p.D * p.M;
    const float *S0 = p.S0, *dSN = p.dSN;
    const size_t states = l.segs > 1 ? (size_t)p.B * p.H * l.segs * DM : 0;   // of one direction
    if (packs(p.N, p.D, p.M, p.dtype)) {
        const cudaError_t e = pack(p, static_cast<char *>(p.ws) + (2 * states * sizeof(float) + 255) / 256 * 256, true);
        if (e != cudaSuccess) return e;
    }
    if (l.segs > 1) {
        float *wf = static_cast<float *>(p.ws), *wb = wf + states;
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
