// la_recurrence.cu - the gated linear recurrence h_t = a_t h_{t-1} + u_t of
// every channel, and its backward l_t = dout_t + a_{t+1} l_{t+1}.
#include "la_gate.cuh"
#include "la_layer.h"

namespace la {
namespace {

constexpr int kThreads = 128;

struct Where {
    const int *lens;
    int H, N, D;
    long long BHD;
};

// One thread per channel of a sequence walks its tokens in order.
template <typename T, int GATE>
__global__ void __launch_bounds__(kThreads) rec_forward_kernel(la_view x, la_view g, la_view out, Where s,
                                                               const float *h0, float *hN) {
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i >= s.BHD) return;
    const int d = (int)(i % s.D);
    const long long bh = i / s.D, b = bh / s.H, hd = bh % s.H;
    const int len = s.lens ? min(max(s.lens[b], 0), s.N) : s.N;
    const T *px = (const T *)x.data + b * x.sb + hd * x.sh + d;
    const T *pg = (const T *)g.data + b * g.sb + hd * g.sh + d;
    T *po = (T *)out.data + b * out.sb + hd * out.sh + d;
    float h = h0 ? h0[i] : 0.f;
#pragma unroll 4
    for (long long t = 0; t < len; t++) {
        float a, w;
        gate_of<GATE>(to_f32<T>(pg[t * g.sn]), a, w);
        h = fmaf(a, h, w * to_f32<T>(px[t * x.sn]));
        po[t * out.sn] = from_f32<T>(h);
    }
    for (long long t = len; t < s.N; t++) po[t * out.sn] = from_f32<T>(0.f);
    if (hN) hN[i] = h;
}

template <typename T, int GATE>
__global__ void __launch_bounds__(kThreads) rec_backward_kernel(la_view x, la_view g, la_view out, la_view dout,
                                                                la_view dx, la_view dg, Where s, const float *h0,
                                                                const float *dhN, float *dh0) {
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i >= s.BHD) return;
    const int d = (int)(i % s.D);
    const long long bh = i / s.D, b = bh / s.H, hd = bh % s.H;
    const int len = s.lens ? min(max(s.lens[b], 0), s.N) : s.N;
    const T *px = (const T *)x.data + b * x.sb + hd * x.sh + d;
    const T *pg = (const T *)g.data + b * g.sb + hd * g.sh + d;
    const T *po = (const T *)out.data + b * out.sb + hd * out.sh + d;
    const T *pd = (const T *)dout.data + b * dout.sb + hd * dout.sh + d;
    T *px_ = (T *)dx.data + b * dx.sb + hd * dx.sh + d;
    T *pg_ = (T *)dg.data + b * dg.sb + hd * dg.sh + d;
    for (long long t = len; t < s.N; t++) px_[t * dx.sn] = pg_[t * dg.sn] = from_f32<T>(0.f);
    float mu = dhN ? dhN[i] : 0.f;   // a_{t+1} l_{t+1}
#pragma unroll 4
    for (long long t = len - 1; t >= 0; t--) {
        float a, w;
        gate_of<GATE>(to_f32<T>(pg[t * g.sn]), a, w);
        const float before = t > 0 ? to_f32<T>(po[(t - 1) * out.sn]) : h0 ? h0[i] : 0.f;
        const float l = to_f32<T>(pd[t * dout.sn]) + mu;
        mu = a * l;
        float da = l * before;
        if (GATE == 1) da = mu * before;
        if (GATE == 2) da = (mu * w) * (before - to_f32<T>(px[t * x.sn]));
        px_[t * dx.sn] = from_f32<T>(GATE == 2 ? l * w : l);
        pg_[t * dg.sn] = from_f32<T>(da);
    }
    if (dh0) dh0[i] = mu;
}

template <typename T, int GATE> cudaError_t forward_t(const RecProblem &p) {
    const Where s{p.lens, p.H, p.N, p.D, (long long)p.B * p.H * p.D};
    const unsigned grid = (unsigned)((s.BHD + kThreads - 1) / kThreads);
    rec_forward_kernel<T, GATE><<<grid, kThreads, 0, p.stream>>>(p.x, p.g, p.out, s, p.h0, p.hN);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T, int GATE> cudaError_t backward_t(const RecProblem &p) {
    const Where s{p.lens, p.H, p.N, p.D, (long long)p.B * p.H * p.D};
    const unsigned grid = (unsigned)((s.BHD + kThreads - 1) / kThreads);
    rec_backward_kernel<T, GATE><<<grid, kThreads, 0, p.stream>>>(p.x, p.g, p.out, p.dout, p.dx, p.dg, s, p.h0,
                                                                  p.dhN, p.dh0);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t recurrence_forward(const RecProblem &p, const DeviceInfo &) {
    const bool f32 = p.dtype == LA_DTYPE_F32;
    switch (p.gate) {
        case LA_GATE_DECAY: return f32 ? forward_t<float, 0>(p) : forward_t<__nv_bfloat16, 0>(p);
        case LA_GATE_LOG: return f32 ? forward_t<float, 1>(p) : forward_t<__nv_bfloat16, 1>(p);
        case LA_GATE_SIGMOID: return f32 ? forward_t<float, 2>(p) : forward_t<__nv_bfloat16, 2>(p);
    }
    return cudaErrorInvalidValue;
}

cudaError_t recurrence_backward(const RecProblem &p, const DeviceInfo &) {
    const bool f32 = p.dtype == LA_DTYPE_F32;
    switch (p.gate) {
        case LA_GATE_DECAY: return f32 ? backward_t<float, 0>(p) : backward_t<__nv_bfloat16, 0>(p);
        case LA_GATE_LOG: return f32 ? backward_t<float, 1>(p) : backward_t<__nv_bfloat16, 1>(p);
        case LA_GATE_SIGMOID: return f32 ? backward_t<float, 2>(p) : backward_t<__nv_bfloat16, 2>(p);
    }
    return cudaErrorInvalidValue;
}

}  // namespace la
