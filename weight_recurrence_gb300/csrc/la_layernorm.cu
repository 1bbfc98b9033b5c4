// la_layernorm.cu - layer norm of rows with the residual sum in front, and
// its backward with the reduction of the weight's and bias' gradients.
//
// Both are bound by HBM.  A group of TPR threads (part of a warp, a warp, or a
// CTA) holds a row in registers, so every value is read once: the mean first,
// then the variance about it (not the mean of the squares, which loses it next
// to a large mean), then the output.  The backward's CTAs stay and walk over
// rows, because each thread keeps its columns' sums of dy xh and dy in fp32
// registers; the sums of all groups are added in a fixed order.
#include <algorithm>

#include "la_common.cuh"
#include "la_layer.h"

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
    __device__ __forceinline__ float get(int i) const {
        if constexpr (WIDE) {
            const unsigned w = (&piece[i / VEC].x)[(i % VEC) * sizeof(T) / 4];
            if constexpr (sizeof(T) == 4) return __uint_as_float(w);
            else return __uint_as_float(i % 2 ? w & 0xffff0000u : w << 16);
        } else {
            if constexpr (sizeof(T) == 4) return __uint_as_float(one[i]);
            else return __uint_as_float((unsigned)one[i] << 16);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[E]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < E; i++) {
                if constexpr (WIDE) (&piece[i / VEC].x)[i % VEC] = __float_as_uint(v[i]);
                else one[i] = __float_as_uint(v[i]);
            }
        } else if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                const __nv_bfloat162 p = __floats2bfloat162_rn(v[i], v[i + 1]);
                (&piece[i / VEC].x)[(i % VEC) / 2] = *reinterpret_cast<const unsigned *>(&p);
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; i++) one[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
        }
    }
};

// fp32 parameters of the thread's columns; a null pointer gives `none`.
template <int TPR, int K, int VEC, bool WIDE>
__device__ __forceinline__ void load_columns(float (&v)[K * VEC], const float *p, int lane, int C, float none) {
#pragma unroll
    for (int i = 0; i < K * VEC; i++) v[i] = none;
    if (p == nullptr) return;
    if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < K * VEC; i += 4) {
            const int c = ((i / VEC) * TPR + lane) * VEC + i % VEC;
            if (c < C) {
                const float4 q = *reinterpret_cast<const float4 *>(p + c);
                v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < K * VEC; i++)
            if (i * TPR + lane < C) v[i] = p[i * TPR + lane];
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
            const int warp = threadIdx.x / 32;
            if (threadIdx.x % 32 == 0) {
#pragma unroll
                for (int n = 0; n < N; n++) sh[turn][n][warp] = v[n];
            }
            __syncthreads();
#pragma unroll
            for (int n = 0; n < N; n++) {
                // every warp adds the warps' sums in the same tree
                float s = threadIdx.x % 32 < TPR / 32 ? sh[turn][n][threadIdx.x % 32] : 0.f;
#pragma unroll
                for (int o = TPR / 64; o > 0; o /= 2) s += __shfl_xor_sync(~0u, s, o);
                v[n] = __shfl_sync(~0u, s, 0);
            }
            turn ^= 1;
        }
    }
};

template <typename T> __device__ __forceinline__ T *row_at(const la_rows &v, long long r) {
    return static_cast<T *>(v.data) + r * v.stride;
}

template <int TPR> constexpr int threads_of() { return TPR > 256 ? TPR : TPR > 32 ? TPR : 256; }

// ROWS rows of a group are on their way together where a row is short.
template <typename T, int TPR, int K, bool WIDE, int ROWS>
__global__ void __launch_bounds__(threads_of<TPR>()) ln_forward_kernel(NormProblem p) {
    using S = Share<T, TPR, K, WIDE>;
    constexpr int E = S::E, GROUPS = threads_of<TPR>() / TPR;
    __shared__ float sh[2][1][TPR / 32 > 0 ? TPR / 32 : 1];
    Sums<TPR, 1> sum{sh};
    pdl_wait_cta();
    const int lane = threadIdx.x % TPR;
    const long long r0 = ((long long)blockIdx.x * GROUPS + threadIdx.x / TPR) * ROWS;
    float v[ROWS][E];
    {
        S a[ROWS], b[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; j++)
            if (r0 + j < p.rows) {
                a[j].load(row_at<T>(p.x, r0 + j), lane, p.C);
                if (p.res.data) b[j].load(row_at<T>(p.res, r0 + j), lane, p.C);
            }
#pragma unroll
        for (int j = 0; j < ROWS; j++) {
#pragma unroll
            for (int i = 0; i < E; i++) v[j][i] = a[j].get(i);
            if (p.res.data) {
#pragma unroll
                for (int i = 0; i < E; i++) v[j][i] += b[j].get(i);
                a[j].set(v[j]);   // the stream as it is kept, and normalised
                if (p.sum.data && r0 + j < p.rows) a[j].store(row_at<T>(p.sum, r0 + j), lane, p.C);
#pragma unroll
                for (int i = 0; i < E; i++) v[j][i] = a[j].get(i);
            }
        }
    }
    float w[E], b[E];
    load_columns<TPR, K, S::VEC, WIDE>(w, p.w, lane, p.C, 1.f);
    load_columns<TPR, K, S::VEC, WIDE>(b, p.b, lane, p.C, 0.f);
#pragma unroll
    for (int j = 0; j < ROWS; j++) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < E; i++) s[0] += v[j][i];   // columns past C are 0
        sum(s);
        const float mean = s[0] / p.C;
        s[0] = 0.f;
#pragma unroll
        for (int i = 0; i < E; i++) {
            v[j][i] -= mean;
            if (S::column(i, lane) < p.C) s[0] = fmaf(v[j][i], v[j][i], s[0]);
        }
        sum(s);
        const float rstd = 1.f / sqrtf(s[0] / p.C + p.eps);
        if (r0 + j < p.rows) {
            S y;
            float out[E];
#pragma unroll
            for (int i = 0; i < E; i++) out[i] = fmaf(v[j][i] * rstd, w[i], b[i]);
            y.set(out);
            y.store(row_at<T>(p.y, r0 + j), lane, p.C);
            if (p.mean && lane == 0) p.mean[r0 + j] = mean, p.rstd[r0 + j] = rstd;
        }
    }
}

// Groups walk over rows gridDim * GROUPS apart; the next row is on its way
// while one is worked on.
template <typename T, int TPR, int K, bool WIDE>
__global__ void __launch_bounds__(threads_of<TPR>()) ln_backward_kernel(NormProblem p) {
    using S = Share<T, TPR, K, WIDE>;
    constexpr int E = S::E, GROUPS = threads_of<TPR>() / TPR;
    __shared__ float sh[2][2][TPR / 32 > 0 ? TPR / 32 : 1];
    // [GROUPS][2][C] where a CTA has several groups; the sums themselves, [2][E]
    // [threads], where a CTA of 1024 threads leaves 64 registers to each
    constexpr bool kOutside = TPR == 1024;
    extern __shared__ float columns[];
    Sums<TPR, 2> sum{sh};
    pdl_wait_cta();
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const long long step = (long long)gridDim.x * GROUPS;
    float w[kOutside ? 1 : E], dw[kOutside ? 1 : E], db[kOutside ? 1 : E];
    if constexpr (kOutside) {
#pragma unroll
        for (int i = 0; i < 2 * E; i++) columns[i * TPR + lane] = 0.f;
    } else {
        load_columns<TPR, K, S::VEC, WIDE>(w, p.w, lane, p.C, 1.f);
#pragma unroll
        for (int i = 0; i < E; i++) dw[i] = db[i] = 0.f;
    }
    S dy, s, extra;
    float mean = 0.f, rstd = 0.f;
    auto fetch = [&](long long r) {
        if (r < p.rows) {
            dy.load(row_at<T>(p.y, r), lane, p.C);
            s.load(row_at<T>(p.x, r), lane, p.C);
            if (p.res.data) extra.load(row_at<T>(p.res, r), lane, p.C);
            mean = p.mean[r], rstd = p.rstd[r];
        }
    };
    if constexpr (!kOutside) fetch((long long)blockIdx.x * GROUPS + group);
    // a CTA's groups run the same number of rounds (their barriers and shuffles meet)
    for (long long base = (long long)blockIdx.x * GROUPS; base < p.rows; base += step) {
        const long long r = base + group;
        float g[E], xh[E], t[2] = {0.f, 0.f};
        if constexpr (kOutside) fetch(r);
        const float rs = rstd;
#pragma unroll
        for (int i = 0; i < E; i++) {
            g[i] = dy.get(i);
            xh[i] = (s.get(i) - mean) * rs;
        }
        const S here = extra;
        if constexpr (!kOutside) fetch(r + step);
        if (r < p.rows) {
#pragma unroll
            for (int i = 0; i < E; i++) {   // g is 0 in the columns past C
                if constexpr (kOutside) {
                    const int c = S::column(i, lane);
                    columns[i * TPR + lane] = fmaf(g[i], xh[i], columns[i * TPR + lane]);
                    columns[(E + i) * TPR + lane] += g[i];
                    g[i] *= p.w && c < p.C ? p.w[c] : 1.f;
                } else {
                    dw[i] = fmaf(g[i], xh[i], dw[i]);
                    db[i] += g[i];
                    g[i] *= w[i];
                }
                t[0] += g[i];
                t[1] = fmaf(g[i], xh[i], t[1]);
            }
        }
        sum(t);
        if (r < p.rows) {
            const float a = t[0] / p.C, b = t[1] / p.C;
            float out[E];
#pragma unroll
            for (int i = 0; i < E; i++)
                out[i] = fmaf(rs, g[i] - a - xh[i] * b, p.res.data ? here.get(i) : 0.f);
            S ds;
            ds.set(out);
            ds.store(row_at<T>(p.ds, r), lane, p.C);
        }
    }
    if (p.ws == nullptr) return;
    float *part = static_cast<float *>(p.ws) + (long long)blockIdx.x * 2 * p.C;
    if constexpr (GROUPS == 1) {
#pragma unroll
        for (int i = 0; i < E; i++) {
            const int c = S::column(i, lane);
            if (c >= p.C) continue;
            if constexpr (kOutside) part[c] = columns[i * TPR + lane], part[p.C + c] = columns[(E + i) * TPR + lane];
            else part[c] = dw[i], part[p.C + c] = db[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; i++) {
            const int c = S::column(i, lane);
            if (c < p.C) columns[group * 2 * p.C + c] = dw[i], columns[group * 2 * p.C + p.C + c] = db[i];
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

// Adds the CTAs' column sums: 32 columns a CTA, its warps taking the parts in turn.
constexpr int kFinishWarps = 16;
__global__ void __launch_bounds__(32 * kFinishWarps) ln_finish_kernel(const float *ws, float *dw, float *db, int C,
                                                                      int parts) {
    __shared__ float sh[kFinishWarps][33];
    pdl_wait_cta();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    float a = 0.f;
    if (c < 2 * C) {
#pragma unroll 4
        for (int i = warp; i < parts; i += kFinishWarps) a += ws[(long long)i * 2 * C + c];
    }
    sh[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && c < 2 * C) {
        a = 0.f;
#pragma unroll
        for (int w = 0; w < kFinishWarps; w++) a += sh[w][lane];
        if (c < C) {
            if (dw) dw[c] = a;
        } else if (db) {
            db[c - C] = a;
        }
    }
}

// CTAs of the backward: enough to fill the SMs twice over (four times with
// CTAs of 256 threads and less), no more than there are rows for.
int parts_of(long long rows, int groups, int threads) {
    const long long most = kSms * (threads > 512 ? 2 : threads > 256 ? 3 : 4), need = (rows + groups - 1) / groups;
    return (int)std::min(most, need);
}

struct Forward {
    template <typename T, int TPR, int K, bool WIDE> static cudaError_t run(const NormProblem &p) {
        constexpr int E = Share<T, TPR, K, WIDE>::E, ROWS = TPR > 32 ? 1 : E <= 8 ? 4 : E <= 16 ? 2 : 1;
        constexpr int per = threads_of<TPR>() / TPR * ROWS;
        const long long ctas = (p.rows + per - 1) / per;
        if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
        const cudaError_t e = launch_pdl(ln_forward_kernel<T, TPR, K, WIDE, ROWS>, dim3((unsigned)ctas),
                                         dim3(threads_of<TPR>()), 0, p.stream, 0u, p);
        count_launches(1);
        return e;
    }
};

struct Backward {
    template <typename T, int TPR, int K, bool WIDE> static cudaError_t run(NormProblem p) {
        constexpr int THREADS = threads_of<TPR>(), GROUPS = THREADS / TPR;
        const int parts = parts_of(p.rows, GROUPS, THREADS);
        if (!p.dw && !p.db) p.ws = nullptr;
        size_t smem = GROUPS > 1 ? (size_t)GROUPS * 2 * p.C * sizeof(float) : 0;
        if (TPR == 1024) smem = 2 * Share<T, TPR, K, WIDE>::E * TPR * sizeof(float);
        cudaError_t e = cudaFuncSetAttribute(ln_backward_kernel<T, TPR, K, WIDE>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        e = launch_pdl(ln_backward_kernel<T, TPR, K, WIDE>, dim3((unsigned)parts), dim3(THREADS), smem, p.stream, 0u,
                       p);
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
    if (pieces <= 128) return Call::template run<T, 128, 1, WIDE>(p);
    if (pieces <= 256) return Call::template run<T, 256, 1, WIDE>(p);
    if (pieces <= 512) return Call::template run<T, 256, 2, WIDE>(p);
    if (pieces <= 1024) return Call::template run<T, 512, 2, WIDE>(p);
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

// A part per CTA of the backward: at most 4 a SM, at most one per row.
size_t layernorm_ws_bytes(long long rows, int C) {
    return (size_t)std::min(rows, 4LL * kSms) * 2 * C * sizeof(float);
}

cudaError_t layernorm_forward(const NormProblem &p) { return by_type<Forward>(p); }
cudaError_t layernorm_backward(const NormProblem &p) { return by_type<Backward>(p); }

}  // namespace la
