// la_grad.cu - the global norm of a list of tensors and clipping by it.
//
// The norm reads every value once and the clipping a second time (its factor
// needs all of them), so HBM bounds both.  (Walking backwards in the second pass,
// from the values that the first left in L2, gained 1 us of 135 for 266 MB.)  The
// list travels in the kernels'
// parameters: no copy to the device, nothing kept between calls, and a call
// can be captured into a graph.  The tensors are cut into chunks of one size,
// dealt out to the CTAs in turn, so that thousands of small tensors and one
// large one load the SMs alike.  A CTA's sum has a fixed order and so has the
// sum of the CTAs' sums: equal calls give equal bits.
#include <algorithm>

#include "la_layer.h"
#include "la_pair.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kSms = 152;
constexpr int kCtas = 8 * kSms;      // at most, per launch, each with a partial sum
constexpr int kFew = 32, kMany = 512;   // tensors of one launch

struct Item {
    const void *src;
    void *dst;
    long long n;
    unsigned first;      // index of its first chunk
    la_dtype dtype;
};
template <int CAP> struct Batch {
    Item item[CAP];
    int count;
    unsigned chunks;
    long long chunk;     // values of a chunk
};

// A chunk: its tensor's values [from, to).
struct Chunk {
    const Item *t;
    long long from, to;
};
template <int CAP> __device__ __forceinline__ Chunk find(const Batch<CAP> &b, unsigned c) {
    int lo = 0, hi = b.count - 1;
    while (lo < hi) {   // the last tensor that starts at or before it
        const int mid = (lo + hi + 1) / 2;
        if (b.item[mid].first <= c) lo = mid;
        else hi = mid - 1;
    }
    const Item &t = b.item[lo];
    const long long from = (long long)(c - t.first) * b.chunk;
    return {&t, from, min(from + b.chunk, t.n)};
}

__device__ __forceinline__ float sum_cta(float v, float *sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; i++) s += sh[i];
    return s;
}

template <typename T> __device__ __forceinline__ float2 pair_of(uint4 v, int i) {
    if constexpr (sizeof(T) == 4) return i ? make_float2(__uint_as_float(v.z), __uint_as_float(v.w))
                                           : make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    else return get_pair((&v.x)[i]);
}

// f(v, p) for every value v of [p, end), 16 bytes at a time where `wide` (the
// values before the first and after the last 16-byte boundary one by one), with
// the loads of kAhead pieces a thread on their way: whole(piece, address) and
// single(value, address).
constexpr int kAhead = 8;
template <typename T, typename Whole, typename Single>
__device__ __forceinline__ void walk(const T *p, const T *end, bool wide, Whole whole, Single single) {
    constexpr int VEC = 16 / (int)sizeof(T);
    const T *body = end, *tail = end;
    if (wide) {
        body = p + ((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T);
        if (body > end) body = end;
        tail = body + (end - body) / VEC * VEC;
    }
    for (const T *q = p + threadIdx.x; q < body; q += kThreads) single(to_f32<T>(*q), q);
    const T *q = body + threadIdx.x * VEC;
    for (; q + (kAhead - 1) * kThreads * VEC < tail; q += kAhead * kThreads * VEC) {
        uint4 v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; i++) v[i] = *reinterpret_cast<const uint4 *>(q + i * kThreads * VEC);
#pragma unroll
        for (int i = 0; i < kAhead; i++) whole(v[i], q + i * kThreads * VEC);
    }
    for (; q < tail; q += kThreads * VEC) whole(*reinterpret_cast<const uint4 *>(q), q);
    for (const T *r = tail + threadIdx.x; r < end; r += kThreads) single(to_f32<T>(*r), r);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) grad_squares_kernel(const __grid_constant__ Batch<CAP> b, float *part) {
    __shared__ float sh[kThreads / 32];
    pdl_wait_cta();
    float2 s = make_float2(0.f, 0.f);
    auto add = [&](auto type, const Chunk &k) {
        using T = decltype(type);
        const T *p = static_cast<const T *>(k.t->src);
        walk<T>(
            p + k.from, p + k.to, true,
            [&](uint4 v, const T *) {
#pragma unroll
                for (int i = 0; i < 8 / (int)sizeof(T); i++) s = fma_pair(pair_of<T>(v, i), pair_of<T>(v, i), s);
            },
            [&](float v, const T *) { s.x = fmaf(v, v, s.x); });
    };
    for (unsigned c = blockIdx.x; c < b.chunks; c += gridDim.x) {
        const Chunk k = find(b, c);
        if (k.t->dtype == LA_DTYPE_F32) add(float(), k);
        else add(__nv_bfloat16(), k);
    }
    const float t = sum_cta(s.x + s.y, sh);
    if (threadIdx.x == 0) part[blockIdx.x] = t;
}

// The norm from the `n` partial sums, the same bits in every CTA.
__device__ __forceinline__ float norm_of(const float *part, int n, double *sh) {
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) s += part[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; i++) s += sh[i];
    return (float)sqrt(s);
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const float *part, int n, float *norm) {
    __shared__ double sh[kThreads / 32];
    pdl_wait_cta();
    const float r = norm_of(part, n, sh);
    if (threadIdx.x == 0) *norm = r;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const __grid_constant__ Batch<CAP> b, const float *part,
                                                              int n, float max_norm, float *norm) {
    __shared__ double sh[kThreads / 32];
    pdl_wait_cta();
    const float r = norm_of(part, n, sh), f = max_norm / (r + 1e-6f);
    const float factor = f > 1.f ? 1.f : f;   // NaN stays
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = r;
    auto scale = [&](auto type, const Chunk &k) {
        using T = decltype(type);
        const T *p = static_cast<const T *>(k.t->src);
        T *to = static_cast<T *>(k.t->dst);
        const bool wide = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(to)) & 15) == 0;
        walk<T>(
            p + k.from, p + k.to, wide,
            [&](uint4 v, const T *at) {
#pragma unroll
                for (int i = 0; i < 8 / (int)sizeof(T); i++) {
                    const float2 y = mul_pair(pair_of<T>(v, i), make_float2(factor, factor));
                    if constexpr (sizeof(T) == 4) {
                        (&v.x)[2 * i] = __float_as_uint(y.x);
                        (&v.x)[2 * i + 1] = __float_as_uint(y.y);
                    } else {
                        (&v.x)[i] = put_pair(y);
                    }
                }
                *reinterpret_cast<uint4 *>(to + (at - p)) = v;
            },
            [&](float v, const T *at) { to[at - p] = from_f32<T>(v * factor); });
    };
    for (unsigned c = blockIdx.x; c < b.chunks; c += gridDim.x) {
        const Chunk k = find(b, c);
        if (k.t->dtype == LA_DTYPE_F32) scale(float(), k);
        else scale(__nv_bfloat16(), k);
    }
}

int batch_size(int count) { return count <= kFew ? kFew : kMany; }
int batches(int count) { return (count + kMany - 1) / kMany; }

// Tensors [from, from + CAP) in chunks: about four a CTA, of 2048 values at least
// (a CTA's threads with 16 bytes of bf16 each), and no more than fit 32 bits.
template <int CAP> void fill(Batch<CAP> &b, const la_tensor *t, int count) {
    long long total = 0;
    for (int i = 0; i < count; i++) total += t[i].n;
    b.chunk = 2048;
    while (b.chunk * kCtas * 4 < total) b.chunk *= 2;
    b.count = 0;
    unsigned chunks = 0;
    for (int i = 0; i < count; i++) {
        if (t[i].n == 0) continue;
        b.item[b.count++] = {t[i].src, t[i].dst, t[i].n, chunks, t[i].dtype};
        chunks += (unsigned)((t[i].n + b.chunk - 1) / b.chunk);
    }
    b.chunks = chunks;
}

template <int CAP>
cudaError_t run(const la_tensor *t, int count, float max_norm, float *norm, float *part, cudaStream_t stream) {
    Batch<CAP> b;
    int parts = 0;
    const int steps = std::max(1, (count + CAP - 1) / CAP);
    for (int i = 0; i < steps; i++) {
        fill(b, t + i * CAP, std::min(CAP, count - i * CAP));
        const int ctas = std::max(1, (int)std::min<unsigned>(b.chunks, kCtas));
        const cudaError_t e =
            launch_pdl(grad_squares_kernel<CAP>, dim3(ctas), dim3(kThreads), 0, stream, 0u, b, part + parts);
        count_launches(1);
        if (e != cudaSuccess) return e;
        parts += ctas;
    }
    if (max_norm < 0.f) {
        const cudaError_t e = launch_pdl(grad_norm_kernel, dim3(1), dim3(kThreads), 0, stream, 0u, (const float *)part,
                                         parts, norm);
        count_launches(1);
        return e;
    }
    for (int i = 0; i < steps; i++) {
        if (steps > 1) fill(b, t + i * CAP, std::min(CAP, count - i * CAP));
        const int ctas = std::max(1, (int)std::min<unsigned>(b.chunks, kCtas));
        const cudaError_t e = launch_pdl(grad_scale_kernel<CAP>, dim3(ctas), dim3(kThreads), 0, stream, 0u, b,
                                         (const float *)part, parts, max_norm, norm);
        count_launches(1);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

size_t grad_ws_bytes(int count) { return sizeof(float) * (size_t)kCtas * std::max(1, batches(count)); }

cudaError_t grad_norm_clip(const la_tensor *t, int count, float max_norm, float *norm, void *ws, cudaStream_t stream) {
    float *part = static_cast<float *>(ws);
    return batch_size(count) == kFew ? run<kFew>(t, count, max_norm, norm, part, stream)
                                     : run<kMany>(t, count, max_norm, norm, part, stream);
}

}  // namespace la
