// la_layer.h - problems of the operators around the attention (gated linear
// recurrence, layer norm, gradient clipping, attention with decays, norm and
// rotation of queries and keys), as la_layer.cu hands them to their launchers
// with every argument already checked.
#pragma once

#include "la_internal.h"

namespace la {

struct RecProblem {
    la_view x, g, out;         // backward: out is read
    la_view dout, dx, dg;      // backward only
    const int *lens;           // device, [B], or null
    const float *h0;           // or null
    float *hN;                 // or null
    const float *dhN;          // backward: or null
    float *dh0;                // backward: or null
    int B, H, N, D;
    la_dtype dtype;
    la_gate gate;
    void *ws;
    cudaStream_t stream;
};

size_t recurrence_ws_bytes(const la_shape &s);   // s valid
cudaError_t recurrence_forward(const RecProblem &p);
cudaError_t recurrence_backward(const RecProblem &p);

struct NormProblem {
    la_rows x, res, sum, y;    // backward: x is s, res is dsum, sum unused, y is dy
    la_rows ds;                // backward only
    const float *w, *b;
    float *mean, *rstd;        // backward: read
    float *dw, *db;            // backward: or null
    long long rows;
    int C;
    la_dtype dtype;
    float eps;
    void *ws;
    cudaStream_t stream;
};

constexpr int kNormMaxC = 16384;
size_t layernorm_ws_bytes(long long rows, int C);
cudaError_t layernorm_forward(const NormProblem &p);
cudaError_t layernorm_backward(const NormProblem &p);

size_t grad_ws_bytes(int count);
// max_norm < 0: the norm alone
cudaError_t grad_norm_clip(const la_tensor *t, int count, float max_norm, float *norm, void *ws, cudaStream_t stream);

constexpr int kDecayMaxD = 128;

struct DecayProblem {
    la_view q, k, v, out;      // step: out is y
    la_view dout, dq, dk, dv;  // backward only
    const float *log_decay;
    const int *lens;           // device, [B], or null
    const float *S0;           // or null
    float *SN;                 // step: S; or null
    const float *dSN;          // backward: or null
    float *dS0;                // backward: or null
    int B, H, N, D, M;
    la_dtype dtype;
    float scale;
    void *ws;
    cudaStream_t stream;
};

size_t decay_ws_bytes(const la_shape &s, bool backward);   // s valid
cudaError_t decay_forward(const DecayProblem &p);
cudaError_t decay_backward(const DecayProblem &p);
cudaError_t decay_step(const DecayProblem &p);

constexpr int kRotateMaxD = 256;

struct RotateProblem {
    la_view q, k, qo, ko;      // backward: qo is dq, ko is dk
    la_view dqo, dko;          // backward only
    const float *wq, *wk;
    la_rotation rot;
    la_qk_shape s;
    bool norm;
    float eps;
    float *dwq, *dwk;          // backward: or null
    void *ws;
    cudaStream_t stream;
};

size_t rotate_ws_bytes(const la_qk_shape &s);
cudaError_t rotate_forward(const RotateProblem &p);
cudaError_t rotate_backward(const RotateProblem &p);

}  // namespace la
