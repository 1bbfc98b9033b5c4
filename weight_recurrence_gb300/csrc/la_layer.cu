// la_layer.cu - entry points of the operators around the attention: argument
// checks on the host, then the launchers of la_recurrence.cu, la_layernorm.cu
// and la_grad.cu.
#include <memory>
#include <new>

#include "la_layer.h"

namespace la {
namespace {

size_t elem_bytes(la_dtype t) { return t == LA_DTYPE_F32 ? 4 : 2; }
bool dtype_ok(la_dtype t) { return t == LA_DTYPE_F32 || t == LA_DTYPE_BF16; }
bool aligned(const void *p, size_t a) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
la_status from_cuda(cudaError_t e) { return e == cudaSuccess ? LA_OK : LA_ERR_CUDA; }

// Strides stay below 2^40 elements, so that no sum of offsets that lies in
// memory at all can wrap.
constexpr long long kMaxStride = 1LL << 40;
bool stride_ok(long long s) { return s >= 0 && s <= kMaxStride; }

bool view_ok(const la_view &v, la_dtype t) {
    return aligned(v.data, elem_bytes(t)) && stride_ok(v.sb) && stride_ok(v.sh) && stride_ok(v.sn);
}

// Whether the rows of an output are disjoint: taken from the smallest stride
// up, each dimension's stride is at least the extent of those below it.
bool nested(const la_view &v, int B, int H, int N, int D) {
    long long st[3] = {v.sb, v.sh, v.sn}, n[3] = {B, H, N};
    for (int i = 0; i < 2; i++)
        for (int j = i + 1; j < 3; j++)
            if (n[j] > 1 && (n[i] <= 1 || st[j] < st[i])) {
                const long long a = st[i], b = n[i];
                st[i] = st[j], n[i] = n[j], st[j] = a, n[j] = b;
            }
    __int128 extent = D;
    for (int i = 0; i < 3; i++) {
        if (n[i] <= 1) continue;
        if (st[i] < extent) return false;
        extent += (__int128)st[i] * (n[i] - 1);
    }
    return true;
}

la_status check_rec_shape(const la_shape &s, la_gate gate) {
    if (s.B < 0 || s.H < 0 || s.N < 0 || s.D < 1 || !dtype_ok(s.dtype)) return LA_ERR_INVALID_ARG;
    if (gate != LA_GATE_DECAY && gate != LA_GATE_LOG && gate != LA_GATE_SIGMOID) return LA_ERR_INVALID_ARG;
    if (s.D > 0x7fffffff - 63) return LA_ERR_UNSUPPORTED;
    const __int128 groups = (__int128)s.B * s.H * ((s.D + 31) / 32);
    if (groups > 0x7fffffff) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

// dst (a state) receives src or 0: a call without tokens.
cudaError_t pass_state(float *dst, const float *src, const la_shape &s, cudaStream_t stream) {
    if (dst == nullptr || dst == src) return cudaSuccess;
    const size_t bytes = (size_t)s.B * s.H * s.D * sizeof(float);
    return src ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, stream)
               : cudaMemsetAsync(dst, 0, bytes, stream);
}

bool rows_ok(const la_rows &v, la_dtype t) { return aligned(v.data, elem_bytes(t)) && stride_ok(v.stride); }
bool out_rows_ok(const la_rows &v, la_dtype t, long long rows, int C) {
    return rows_ok(v, t) && (rows <= 1 || v.stride >= C);
}
bool same(const void *a, const void *b) { return a != nullptr && a == b; }

bool workspace_ok(size_t need, const void *ws, size_t bytes) {
    return need == 0 || (bytes >= need && aligned(ws, 16));
}

la_status check_norm(long long rows, int C, la_dtype t) {
    if (rows < 0 || C < 1 || !dtype_ok(t)) return LA_ERR_INVALID_ARG;
    if (C > kNormMaxC || rows > (1LL << 40)) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

// Whether no destination of the list starts where another destination or another
// tensor's source does.  Addresses in an open table, half empty at least: 168 tensors
// 0.7 us of the host.  On the stack for what one launch takes.
la_status check_distinct(const la_tensor *t, int count) {
    struct Slot {
        const void *dst;
        int i;
    };
    constexpr int kOnStack = 1024;
    size_t slots = 16;
    while (slots < (size_t)count * 2) slots *= 2;
    Slot few[kOnStack];
    std::unique_ptr<Slot[]> many;
    if (slots > kOnStack) {
        many.reset(new (std::nothrow) Slot[slots]);
        if (!many) return LA_ERR_UNSUPPORTED;
    }
    Slot *table = many ? many.get() : few;
    for (size_t i = 0; i < slots; i++) table[i].dst = nullptr;
    auto find = [&](const void *p) {   // its slot, or the one it goes to
        size_t at = (reinterpret_cast<uintptr_t>(p) >> 1) * 0x9E3779B97F4A7C15ull >> 20 & (slots - 1);
        while (table[at].dst && table[at].dst != p) at = (at + 1) & (slots - 1);
        return &table[at];
    };
    for (int i = 0; i < count; i++) {
        if (t[i].n == 0) continue;
        Slot *s = find(t[i].dst);
        if (s->dst) return LA_ERR_INVALID_ARG;
        *s = {t[i].dst, i};
    }
    for (int i = 0; i < count; i++) {
        if (t[i].n == 0 || t[i].src == t[i].dst) continue;
        if (find(t[i].src)->dst) return LA_ERR_INVALID_ARG;
    }
    return LA_OK;
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

size_t la_recurrence_workspace_bytes(la_shape s) {
    return check_rec_shape(s, LA_GATE_DECAY) == LA_OK ? recurrence_ws_bytes(s) : (size_t)-1;
}

la_status la_recurrence_forward(la_view x, la_view g, la_view out, const int *lens, la_shape s, la_gate gate,
                                const float *h0, float *hN, void *workspace, size_t ws_bytes, la_stream_t stream) {
    la_status st = check_rec_shape(s, gate);
    if (st != LA_OK) return st;
    if (s.B == 0 || s.H == 0) return LA_OK;
    if ((h0 && !aligned(h0, 4)) || (hN && !aligned(hN, 4)) || (lens && !aligned(lens, 4))) return LA_ERR_INVALID_ARG;
    if (s.N == 0) return from_cuda(pass_state(hN, h0, s, (cudaStream_t)stream));
    if (!view_ok(x, s.dtype) || !view_ok(g, s.dtype) || !view_ok(out, s.dtype)) return LA_ERR_INVALID_ARG;
    if (!nested(out, s.B, s.H, s.N, s.D)) return LA_ERR_INVALID_ARG;
    for (const void *i : {(const void *)x.data, (const void *)g.data, (const void *)lens, (const void *)h0})
        if (same(out.data, i)) return LA_ERR_INVALID_ARG;
    if (hN && (same(hN, out.data) || same(hN, x.data) || same(hN, g.data) || same(hN, lens))) return LA_ERR_INVALID_ARG;
    if (!workspace_ok(recurrence_ws_bytes(s), workspace, ws_bytes)) return LA_ERR_INVALID_ARG;
    RecProblem p{};
    p.x = x, p.g = g, p.out = out, p.lens = lens, p.h0 = h0, p.hN = hN, p.ws = workspace;
    p.B = s.B, p.H = s.H, p.N = s.N, p.D = s.D, p.dtype = s.dtype, p.gate = gate, p.stream = (cudaStream_t)stream;
    return from_cuda(recurrence_forward(p));
}

la_status la_recurrence_step(la_view x, la_view g, la_view y, la_shape s, la_gate gate, float *h,
                             la_stream_t stream) {
    s.N = 1;
    x.sn = g.sn = y.sn = 0;
    if (s.B > 0 && s.H > 0 && h == nullptr) return LA_ERR_INVALID_ARG;
    return la_recurrence_forward(x, g, y, nullptr, s, gate, h, h, nullptr, 0, stream);
}

la_status la_recurrence_backward(la_view x, la_view g, la_view out, la_view dout, la_view dx, la_view dg,
                                 const int *lens, la_shape s, la_gate gate, const float *h0, const float *dhN,
                                 float *dh0, void *workspace, size_t ws_bytes, la_stream_t stream) {
    la_status st = check_rec_shape(s, gate);
    if (st != LA_OK) return st;
    if (s.B == 0 || s.H == 0) return LA_OK;
    if ((h0 && !aligned(h0, 4)) || (dhN && !aligned(dhN, 4)) || (dh0 && !aligned(dh0, 4)) ||
        (lens && !aligned(lens, 4)))
        return LA_ERR_INVALID_ARG;
    if (s.N == 0) return from_cuda(pass_state(dh0, dhN, s, (cudaStream_t)stream));
    if (gate != LA_GATE_SIGMOID) x = la_view{nullptr, 0, 0, 0};
    if ((gate == LA_GATE_SIGMOID && !view_ok(x, s.dtype)) || !view_ok(g, s.dtype) || !view_ok(out, s.dtype) ||
        !view_ok(dout, s.dtype) || !view_ok(dx, s.dtype) || !view_ok(dg, s.dtype))
        return LA_ERR_INVALID_ARG;
    if (!nested(dx, s.B, s.H, s.N, s.D) || !nested(dg, s.B, s.H, s.N, s.D)) return LA_ERR_INVALID_ARG;
    const void *ins[] = {x.data, g.data, out.data, dout.data, lens, h0};
    for (const void *i : ins)
        if (same(dx.data, i) || same(dg.data, i) || same(dh0, i)) return LA_ERR_INVALID_ARG;
    if (dx.data == dg.data || same(dh0, dx.data) || same(dh0, dg.data) || same(dhN, dx.data) || same(dhN, dg.data))
        return LA_ERR_INVALID_ARG;
    if (!workspace_ok(recurrence_ws_bytes(s), workspace, ws_bytes)) return LA_ERR_INVALID_ARG;
    RecProblem p{};
    p.x = x, p.g = g, p.out = out, p.dout = dout, p.dx = dx, p.dg = dg, p.lens = lens, p.h0 = h0, p.dhN = dhN;
    p.dh0 = dh0, p.ws = workspace;
    p.B = s.B, p.H = s.H, p.N = s.N, p.D = s.D, p.dtype = s.dtype, p.gate = gate, p.stream = (cudaStream_t)stream;
    return from_cuda(recurrence_backward(p));
}

la_status la_layernorm_forward(la_rows x, la_rows res, la_rows sum, la_rows y, const float *w, const float *b,
                               float *mean, float *rstd, long long rows, int C, la_dtype dtype, float eps,
                               la_stream_t stream) {
    la_status st = check_norm(rows, C, dtype);
    if (st != LA_OK) return st;
    if (!(eps >= 0.f) || (mean == nullptr) != (rstd == nullptr)) return LA_ERR_INVALID_ARG;
    if (res.data == nullptr && sum.data != nullptr) return LA_ERR_INVALID_ARG;
    if (rows == 0) return LA_OK;
    if (!rows_ok(x, dtype) || !out_rows_ok(y, dtype, rows, C)) return LA_ERR_INVALID_ARG;
    if ((res.data && !rows_ok(res, dtype)) || (sum.data && !out_rows_ok(sum, dtype, rows, C))) return LA_ERR_INVALID_ARG;
    for (const void *p : {(const void *)w, (const void *)b, (const void *)mean, (const void *)rstd})
        if (p && !aligned(p, 4)) return LA_ERR_INVALID_ARG;
    for (const void *i : {(const void *)x.data, (const void *)res.data, (const void *)sum.data, (const void *)w,
                          (const void *)b, (const void *)mean, (const void *)rstd})
        if (same(y.data, i)) return LA_ERR_INVALID_ARG;
    if ((same(sum.data, x.data) && sum.stride != x.stride) || (same(sum.data, res.data) && sum.stride != res.stride))
        return LA_ERR_INVALID_ARG;
    if (same(mean, rstd)) return LA_ERR_INVALID_ARG;
    for (const void *i : {(const void *)w, (const void *)b, (const void *)mean, (const void *)rstd})
        if (same(sum.data, i)) return LA_ERR_INVALID_ARG;
    for (const void *i : {(const void *)x.data, (const void *)res.data, (const void *)w, (const void *)b})
        if (same(mean, i) || same(rstd, i)) return LA_ERR_INVALID_ARG;
    NormProblem p{};
    p.x = x, p.res = res, p.sum = sum, p.y = y, p.w = w, p.b = b, p.mean = mean, p.rstd = rstd;
    p.rows = rows, p.C = C, p.dtype = dtype, p.eps = eps, p.stream = (cudaStream_t)stream;
    return from_cuda(layernorm_forward(p));
}

size_t la_layernorm_workspace_bytes(long long rows, int C, la_dtype dtype) {
    if (check_norm(rows, C, dtype) != LA_OK) return (size_t)-1;
    return layernorm_ws_bytes(rows, C);
}

la_status la_layernorm_backward(la_rows dy, la_rows s, la_rows dsum, la_rows ds, const float *w, const float *mean,
                                const float *rstd, float *dw, float *db, long long rows, int C, la_dtype dtype,
                                void *workspace, size_t ws_bytes, la_stream_t stream) {
    la_status st = check_norm(rows, C, dtype);
    if (st != LA_OK) return st;
    for (const void *p : {(const void *)w, (const void *)dw, (const void *)db})
        if (p && !aligned(p, 4)) return LA_ERR_INVALID_ARG;
    if (same(dw, db) || same(dw, w) || same(db, w)) return LA_ERR_INVALID_ARG;
    if (rows == 0) {   // sums over no rows
        cudaError_t e = cudaSuccess;
        if (dw) e = cudaMemsetAsync(dw, 0, (size_t)C * sizeof(float), (cudaStream_t)stream);
        if (db && e == cudaSuccess) e = cudaMemsetAsync(db, 0, (size_t)C * sizeof(float), (cudaStream_t)stream);
        return from_cuda(e);
    }
    if (!rows_ok(dy, dtype) || !rows_ok(s, dtype) || (dsum.data && !rows_ok(dsum, dtype)) ||
        !out_rows_ok(ds, dtype, rows, C) || !aligned(mean, 4) || !aligned(rstd, 4))
        return LA_ERR_INVALID_ARG;
    for (const void *i : {(const void *)dy.data, (const void *)s.data, (const void *)dsum.data, (const void *)w,
                          (const void *)mean, (const void *)rstd, (const void *)dw, (const void *)db})
        if (same(ds.data, i)) return LA_ERR_INVALID_ARG;
    for (const void *i : {(const void *)dy.data, (const void *)s.data, (const void *)dsum.data, (const void *)mean,
                          (const void *)rstd})
        if (same(dw, i) || same(db, i)) return LA_ERR_INVALID_ARG;
    const size_t need = layernorm_ws_bytes(rows, C);
    if ((dw || db) && (ws_bytes < need || !aligned(workspace, 16))) return LA_ERR_INVALID_ARG;
    NormProblem p{};
    p.x = s, p.res = dsum, p.y = dy, p.ds = ds, p.w = w, p.mean = const_cast<float *>(mean);
    p.rstd = const_cast<float *>(rstd), p.dw = dw, p.db = db;
    p.rows = rows, p.C = C, p.dtype = dtype, p.ws = workspace, p.stream = (cudaStream_t)stream;
    return from_cuda(layernorm_backward(p));
}

size_t la_grad_workspace_bytes(int count) { return count < 0 ? (size_t)-1 : grad_ws_bytes(count); }

static la_status check_grads(const la_tensor *t, int count, const float *norm, void *ws, size_t ws_bytes, bool clip) {
    if (count < 0 || (count > 0 && t == nullptr) || !aligned(norm, 4)) return LA_ERR_INVALID_ARG;
    for (int i = 0; i < count; i++) {
        if (t[i].n < 0 || t[i].n > (1LL << 40) || !dtype_ok(t[i].dtype)) return LA_ERR_INVALID_ARG;
        if (t[i].n == 0) continue;
        if (!aligned(t[i].src, elem_bytes(t[i].dtype)) || (clip && !aligned(t[i].dst, elem_bytes(t[i].dtype))))
            return LA_ERR_INVALID_ARG;
        if (same(norm, t[i].src) || (clip && same(norm, t[i].dst))) return LA_ERR_INVALID_ARG;
    }
    if (ws_bytes < grad_ws_bytes(count) || !aligned(ws, 16)) return LA_ERR_INVALID_ARG;
    return clip ? check_distinct(t, count) : LA_OK;
}

la_status la_grad_norm(const la_tensor *tensors, int count, float *norm, void *workspace, size_t ws_bytes,
                       la_stream_t stream) {
    const la_status st = check_grads(tensors, count, norm, workspace, ws_bytes, false);
    if (st != LA_OK) return st;
    return from_cuda(grad_norm_clip(tensors, count, -1.f, norm, workspace, (cudaStream_t)stream));
}

la_status la_grad_clip(const la_tensor *tensors, int count, float max_norm, float *norm, void *workspace,
                       size_t ws_bytes, la_stream_t stream) {
    if (!(max_norm >= 0.f)) return LA_ERR_INVALID_ARG;
    const la_status st = check_grads(tensors, count, norm, workspace, ws_bytes, true);
    if (st != LA_OK) return st;
    return from_cuda(grad_norm_clip(tensors, count, max_norm, norm, workspace, (cudaStream_t)stream));
}

}  // extern "C"
