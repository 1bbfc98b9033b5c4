// la_grad.cu - the global norm of a list of tensors and clipping by it.
#include "la_common.cuh"
#include "la_layer.h"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 128;      // tensors of one launch, in its parameters
constexpr int kParts = 512;      // CTAs of one launch, each with a partial sum

struct Batch {
    la_tensor t[kBatch];
    int count;
};

__device__ __forceinline__ float load(const la_tensor &t, long long i) {
    return t.dtype == LA_DTYPE_F32 ? ((const float *)t.src)[i] : to_f32<__nv_bfloat16>(((const __nv_bfloat16 *)t.src)[i]);
}

__device__ __forceinline__ float cta_sum(float v, float *sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; i++) s += sh[i];
    return s;
}

__global__ void __launch_bounds__(kThreads) grad_squares_kernel(__grid_constant__ const Batch b, float *part) {
    __shared__ float sh[kThreads / 32];
    float s = 0.f;
    for (int k = 0; k < b.count; k++)
        for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < b.t[k].n; i += (long long)kParts * kThreads) {
            const float v = load(b.t[k], i);
            s = fmaf(v, v, s);
        }
    s = cta_sum(s, sh);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ void grad_norm_kernel(const float *part, int n, float *norm) {
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += 32) s += part[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

__global__ void __launch_bounds__(kThreads) grad_scale_kernel(__grid_constant__ const Batch b, const float *norm,
                                                              float max_norm) {
    const float q = max_norm / (*norm + 1e-6f);
    const float c = q > 1.f ? 1.f : q;   // NaN stays
    for (int k = 0; k < b.count; k++)
        for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < b.t[k].n; i += (long long)kParts * kThreads) {
            const float v = load(b.t[k], i) * c;
            if (b.t[k].dtype == LA_DTYPE_F32) ((float *)b.t[k].dst)[i] = v;
            else ((__nv_bfloat16 *)b.t[k].dst)[i] = from_f32<__nv_bfloat16>(v);
        }
}

int batches(int count) { return (count + kBatch - 1) / kBatch; }

}  // namespace

size_t grad_ws_bytes(int count) { return sizeof(float) * (size_t)kParts * (batches(count) + 1); }

cudaError_t grad_norm_clip(const la_tensor *t, int count, float max_norm, float *norm, void *ws,
                           cudaStream_t stream, const DeviceInfo &) {
    float *part = (float *)ws;
    Batch b;
    for (int i = 0; i < batches(count); i++) {
        b.count = 0;
        for (int k = i * kBatch; k < count && k < (i + 1) * kBatch; k++) b.t[b.count++] = t[k];
        grad_squares_kernel<<<kParts, kThreads, 0, stream>>>(b, part + (size_t)i * kParts);
        count_launches(1);
    }
    grad_norm_kernel<<<1, 32, 0, stream>>>(part, batches(count) * kParts, norm);
    count_launches(1);
    for (int i = 0; max_norm >= 0.f && i < batches(count); i++) {
        b.count = 0;
        for (int k = i * kBatch; k < count && k < (i + 1) * kBatch; k++) b.t[b.count++] = t[k];
        grad_scale_kernel<<<kParts, kThreads, 0, stream>>>(b, norm, max_norm);
        count_launches(1);
    }
    return cudaGetLastError();
}

}  // namespace la
