// la_layernorm.cu - layer norm of rows with the residual sum in front, and
// its backward with the reduction of the weight's and bias' gradients.
#include "la_common.cuh"
#include "la_layer.h"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxParts = 512;   // CTAs that walk the rows of the backward, each with its column sums

template <typename T> __device__ __forceinline__ T *row(const la_rows &v, long long r) {
    return (T *)v.data + r * v.stride;
}

// Sum over the CTA, given to every thread.
__device__ __forceinline__ float cta_sum(float v, float *sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; i++) s += sh[i];
    return s;
}

// One CTA per row; s is kept in shared memory between the three passes over
// it (mean, variance about the mean, output).
template <typename T>
__global__ void __launch_bounds__(kThreads) ln_forward_kernel(NormProblem p) {
    extern __shared__ float buf[];
    __shared__ float sh[kThreads / 32];
    const long long r = blockIdx.x;
    float acc = 0.f;
    for (int c = threadIdx.x; c < p.C; c += kThreads) {
        float v = to_f32<T>(row<T>(p.x, r)[c]);
        if (p.res.data) {
            const T s = from_f32<T>(v + to_f32<T>(row<T>(p.res, r)[c]));
            if (p.sum.data) row<T>(p.sum, r)[c] = s;
            v = to_f32<T>(s);
        }
        buf[c] = v;
        acc += v;
    }
    const float mu = cta_sum(acc, sh) / p.C;
    acc = 0.f;
    for (int c = threadIdx.x; c < p.C; c += kThreads) acc += (buf[c] - mu) * (buf[c] - mu);
    const float rstd = 1.f / sqrtf(cta_sum(acc, sh) / p.C + p.eps);
    for (int c = threadIdx.x; c < p.C; c += kThreads)
        row<T>(p.y, r)[c] = from_f32<T>((buf[c] - mu) * rstd * (p.w ? p.w[c] : 1.f) + (p.b ? p.b[c] : 0.f));
    if (p.mean && threadIdx.x == 0) p.mean[r] = mu, p.rstd[r] = rstd;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) ln_backward_kernel(NormProblem p) {
    __shared__ float sh[kThreads / 32];
    const long long r = blockIdx.x;
    const float mu = p.mean[r], rstd = p.rstd[r];
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < p.C; c += kThreads) {
        const float v = to_f32<T>(row<T>(p.y, r)[c]) * (p.w ? p.w[c] : 1.f);
        s1 += v;
        s2 += v * ((to_f32<T>(row<T>(p.x, r)[c]) - mu) * rstd);
    }
    s1 = cta_sum(s1, sh) / p.C;
    s2 = cta_sum(s2, sh) / p.C;
    for (int c = threadIdx.x; c < p.C; c += kThreads) {
        const float v = to_f32<T>(row<T>(p.y, r)[c]) * (p.w ? p.w[c] : 1.f);
        const float xh = (to_f32<T>(row<T>(p.x, r)[c]) - mu) * rstd;
        float d = rstd * (v - s1 - xh * s2);
        if (p.res.data) d += to_f32<T>(row<T>(p.res, r)[c]);
        row<T>(p.ds, r)[c] = from_f32<T>(d);
    }
}

// Column sums of dy xh and dy over every `parts`-th row.
template <typename T>
__global__ void __launch_bounds__(kThreads) ln_columns_kernel(NormProblem p, int parts) {
    const int c = blockIdx.y * kThreads + threadIdx.x;
    if (c >= p.C) return;
    float dw = 0.f, db = 0.f;
    for (long long r = blockIdx.x; r < p.rows; r += parts) {
        const float d = to_f32<T>(row<T>(p.y, r)[c]);
        dw += d * ((to_f32<T>(row<T>(p.x, r)[c]) - p.mean[r]) * p.rstd[r]);
        db += d;
    }
    float *ws = (float *)p.ws + (long long)blockIdx.x * 2 * p.C;
    ws[c] = dw;
    ws[p.C + c] = db;
}

__global__ void __launch_bounds__(kThreads) ln_finish_kernel(const float *ws, float *dw, float *db, int C, int parts) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= C) return;
    float a = 0.f, b = 0.f;
    for (int i = 0; i < parts; i++) a += ws[(long long)i * 2 * C + c], b += ws[(long long)i * 2 * C + C + c];
    if (dw) dw[c] = a;
    if (db) db[c] = b;
}

int parts_of(long long rows) { return (int)(rows < kMaxParts ? rows : kMaxParts); }

template <typename T> cudaError_t forward_t(const NormProblem &p) {
    cudaError_t e = cudaFuncSetAttribute(ln_forward_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kNormMaxC * (int)sizeof(float));
    if (e != cudaSuccess) return e;
    ln_forward_kernel<T><<<(unsigned)p.rows, kThreads, p.C * sizeof(float), p.stream>>>(p);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T> cudaError_t backward_t(const NormProblem &p) {
    ln_backward_kernel<T><<<(unsigned)p.rows, kThreads, 0, p.stream>>>(p);
    count_launches(1);
    if (p.dw || p.db) {
        const int parts = parts_of(p.rows);
        const unsigned cols = (unsigned)((p.C + kThreads - 1) / kThreads);
        ln_columns_kernel<T><<<dim3((unsigned)parts, cols), kThreads, 0, p.stream>>>(p, parts);
        ln_finish_kernel<<<cols, kThreads, 0, p.stream>>>((const float *)p.ws, p.dw, p.db, p.C, parts);
        count_launches(2);
    }
    return cudaGetLastError();
}

}  // namespace

size_t layernorm_ws_bytes(long long rows, int C) { return (size_t)parts_of(rows) * 2 * C * sizeof(float); }

cudaError_t layernorm_forward(const NormProblem &p, const DeviceInfo &) {
    if (p.rows > 0x7fffffff) return cudaErrorInvalidValue;
    return p.dtype == LA_DTYPE_F32 ? forward_t<float>(p) : forward_t<__nv_bfloat16>(p);
}

cudaError_t layernorm_backward(const NormProblem &p, const DeviceInfo &) {
    if (p.rows > 0x7fffffff) return cudaErrorInvalidValue;
    return p.dtype == LA_DTYPE_F32 ? backward_t<float>(p) : backward_t<__nv_bfloat16>(p);
}

}  // namespace la
