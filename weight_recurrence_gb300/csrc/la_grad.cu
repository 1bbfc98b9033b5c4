// la_grad.cu - the global norm of a list of tensors and clipping by it.
//
// norm = sqrt(sum of the squares of all values); clipped = value * min(1,
// max_norm / (norm + 1e-6)).  The norm reads every value once and the clipping
// a second time (its factor needs all of them), so HBM bounds both of a long
// list, latency those of a short one.  Measured: the norm of 133 M bf16 values
// 43 us (6.2 TB/s), clipping them 128 us (6.2 TB/s over its three passes, the
// second reading included); clipping 4 Mi fp32 values 10.6 us, 32 Ki 3.5 us.
//
// The list travels in the kernels' parameters: no copy to the device, nothing
// kept between calls, and a call can be captured into a graph.  The tensors are
// cut into chunks of one size that start on 16-byte boundaries, dealt out to the
// CTAs in turn, so that thousands of small tensors and one large one load the SMs
// alike.  A CTA's sum has a fixed order and so has the sum of the CTAs' sums:
// equal calls give equal bits, the norm alone and with clipping.  All sums are
// fp32, over positive terms.  (fp64 is so slow on this machine that joining the
// 1216 sums in it, in every CTA, took 12 us of a call of 23 us.)
//
// Tried and left out: one cluster of eight CTAs that does a short list in one
// launch (6.1 us for 32 Ki values, two launches then 4.7 us); walking backwards in
// the second pass, from the values that the first left in L2 (1 us of 133).
#include <algorithm>

#include "la_layer.h"
#include "la_pair.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kSms = 152;
constexpr int kCtas = 8 * kSms;      // at most, per launch, each with a partial sum
constexpr int kFew = 32, kMany = 512;   // tensors of one launch (a long table costs: 4 Mi values 10.5 | 11.0 us)

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

// Values between the 16-byte boundary at or below a tensor's start and its start.
template <typename T> __host__ __device__ __forceinline__ int lead_of(const void *p) {
    return (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
}
__host__ __device__ __forceinline__ int lead(const Item &t) {
    return t.dtype == LA_DTYPE_F32 ? lead_of<float>(t.src) : lead_of<__nv_bfloat16>(t.src);
}

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
    const long long from = (long long)(c - t.first) * b.chunk - lead(t);
    return {&t, max(from, 0LL), min(from + b.chunk, t.n)};
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

// Every value of the chunk [p, end), taken by `threads` threads of which this is
// `tid`: 16 bytes at a time where `wide` (the few values before the first and
// after the last 16-byte boundary, at a tensor's ends, one by one), one by one
// otherwise, with kAhead loads a thread on their way: whole(piece, address) and
// single(value, address).
constexpr int kAhead = 8;
template <typename T, typename Whole, typename Single>
__device__ __forceinline__ void walk(const T *p, const T *end, bool wide, int tid, int threads, Whole whole,
                                     Single single) {
    constexpr int VEC = 16 / (int)sizeof(T);
    if (!wide) {
        const int n = (int)(end - p);
        for (int j = tid; j < n; j += kAhead * threads) {
            float v[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; i++) v[i] = j + i * threads < n ? to_f32<T>(p[j + i * threads]) : 0.f;
#pragma unroll
            for (int i = 0; i < kAhead; i++)
                if (j + i * threads < n) single(v[i], p + j + i * threads);
        }
        return;
    }
    const int head = min((VEC - lead_of<T>(p)) % VEC, (int)(end - p));
    const T *body = p + head;
    const int n = (int)(end - body) / VEC, rest = (int)(end - body) % VEC;
    if (tid < head) single(to_f32<T>(p[tid]), p + tid);
    if (tid < rest) single(to_f32<T>(body[n * VEC + tid]), body + n * VEC + tid);
    const uint4 *q = reinterpret_cast<const uint4 *>(body);
    for (int j = tid; j < n; j += kAhead * threads) {
        uint4 v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; i++) v[i] = j + i * threads < n ? q[j + i * threads] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kAhead; i++)
            if (j + i * threads < n) whole(v[i], reinterpret_cast<const T *>(q + j + i * threads));
    }
}

// The squares of a chunk's values, added to s.
__device__ __forceinline__ void add_squares(const Chunk &k, int tid, int threads, float2 &s) {
    auto add = [&](auto type) {
        using T = decltype(type);
        const T *p = static_cast<const T *>(k.t->src);
        walk<T>(
            p + k.from, p + k.to, true, tid, threads,
            [&](uint4 v, const T *) {
#pragma unroll
                for (int i = 0; i < 8 / (int)sizeof(T); i++) s = fma_pair(pair_of<T>(v, i), pair_of<T>(v, i), s);
            },
            [&](float v, const T *) { s.x = fmaf(v, v, s.x); });
    };
    if (k.t->dtype == LA_DTYPE_F32) add(float());
    else add(__nv_bfloat16());
}

// A chunk's values times the factor, to the tensor's dst.
__device__ __forceinline__ void scale(const Chunk &k, int tid, int threads, float factor) {
    auto run = [&](auto type) {
        using T = decltype(type);
        const T *p = static_cast<const T *>(k.t->src);
        T *to = static_cast<T *>(k.t->dst);
        walk<T>(
            p + k.from, p + k.to, lead_of<T>(p) == lead_of<T>(to), tid, threads,
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
    if (k.t->dtype == LA_DTYPE_F32) run(float());
    else run(__nv_bfloat16());
}

__device__ __forceinline__ float factor_of(float max_norm, float norm) {
    const float f = max_norm / (norm + 1e-6f);
    return f > 1.f ? 1.f : f;   // NaN stays
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) grad_squares_kernel(const __grid_constant__ Batch<CAP> b, float *part) {
    __shared__ float sh[kThreads / 32];
    pdl_wait_cta();
    float2 s = make_float2(0.f, 0.f);
    for (unsigned c = blockIdx.x; c < b.chunks; c += gridDim.x) add_squares(find(b, c), threadIdx.x, kThreads, s);
    const float t = sum_cta(s.x + s.y, sh);
    if (threadIdx.x == 0) part[blockIdx.x] = t;
}

// The norm from the `n` partial sums, the same bits in every CTA and launch.
__device__ __forceinline__ float norm_of(const float *part, int n, float *sh) {
    float s = 0.f;
    for (int i = threadIdx.x; i < n; i += kThreads) s += part[i];
    return sqrtf(sum_cta(s, sh));
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const float *part, int n, float *norm) {
    __shared__ float sh[kThreads / 32];
    pdl_wait_cta();
    const float r = norm_of(part, n, sh);
    if (threadIdx.x == 0) *norm = r;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const __grid_constant__ Batch<CAP> b, const float *part,
                                                              int n, float max_norm, float *norm) {
    __shared__ float sh[kThreads / 32];
    pdl_wait_cta();
    const float r = norm_of(part, n, sh), factor = factor_of(max_norm, r);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = r;
    for (unsigned c = blockIdx.x; c < b.chunks; c += gridDim.x) scale(find(b, c), threadIdx.x, kThreads, factor);
}

int batch_size(int count) { return count <= kFew ? kFew : kMany; }
int batches(int count) { return (count + kMany - 1) / kMany; }

// The tensors that have values, cut into chunks of `chunk` values.
template <int CAP> void fill(Batch<CAP> &b, const la_tensor *t, int count, long long chunk) {
    b.chunk = chunk;
    b.count = 0;
    unsigned chunks = 0;
    for (int i = 0; i < count; i++) {
        if (t[i].n == 0) continue;
        Item &k = b.item[b.count++] = {t[i].src, t[i].dst, t[i].n, chunks, t[i].dtype};
        chunks += (unsigned)((t[i].n + lead(k) + chunk - 1) / chunk);
    }
    b.chunks = chunks;
}

long long values_of(const la_tensor *t, int count) {
    long long n = 0;
    for (int i = 0; i < count; i++) n += t[i].n;
    return n;
}
// Values of a chunk, in multiples of kUnit: one chunk a CTA while its threads
// load those at once, about four beyond that.  (Clipping 2 Mi fp32 values with
// units of 2048: 7.9 us, of 4096: 6.3; 28 Mi bf16 values with four chunks a CTA:
// 27.7 us, with eight: 35.8; the gradients of 133 M values with four CTAs an SM
// instead of eight: 133.5 us instead of 129.)
constexpr long long kUnit = 4096;
long long chunk_of(const la_tensor *t, int count) {
    const long long k = kCtas * kUnit, units = (values_of(t, count) + k - 1) / k;
    return std::min(1LL << 30, kUnit * std::max(1LL, units * kUnit <= 32 * kThreads ? units : (units + 3) / 4));
}

template <int CAP>
cudaError_t run(const la_tensor *t, int count, float max_norm, float *norm, float *part, cudaStream_t stream) {
    Batch<CAP> b;
    int parts = 0;
    const int steps = std::max(1, (count + CAP - 1) / CAP);
    for (int i = 0; i < steps; i++) {
        const int n = std::min(CAP, count - i * CAP);
        fill(b, t + i * CAP, n, chunk_of(t + i * CAP, n));
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
        const int n = std::min(CAP, count - i * CAP);
        if (steps > 1) fill(b, t + i * CAP, n, chunk_of(t + i * CAP, n));
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
