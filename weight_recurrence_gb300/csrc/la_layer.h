// la_layer.h - problems of the operators around the attention (gated linear
// recurrence, layer norm, gradient clipping), as la_layer.cu hands them to
// their launchers with every argument already checked.
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

}  // namespace la
