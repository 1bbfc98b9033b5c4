// la_layer.cu - entry points of the operators around the attention: argument
// checks on the host, then the launchers of la_recurrence.cu, la_layernorm.cu,
// la_grad.cu, la_decay.cu and la_rotate.cu.
#include <initializer_list>
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

// Sizes of the attention with decays: every head is a CTA's (times its segments
// and blocks of columns) and its state's offset stays in 64 bits.
la_status check_decay(const la_shape &s) {
    if (s.B < 0 || s.H < 0 || s.N < 0 || s.D < 1 || s.M < 1 || !dtype_ok(s.dtype)) return LA_ERR_INVALID_ARG;
    if (s.D > kDecayMaxD || s.M > kDecayMaxD) return LA_ERR_UNSUPPORTED;
    if ((__int128)s.B * s.H * 8 > 0x7fffffff) return LA_ERR_UNSUPPORTED;
    if (s.N > 0x7fffffff - (1 << 20)) return LA_ERR_UNSUPPORTED;   // so that segments end below 2^31
    return LA_OK;
}

// A state buffer: given ones are fp32 arrays.
bool states_ok(std::initializer_list<const void *> states) {
    for (const void *p : states)
        if (p && !aligned(p, 4)) return false;
    return true;
}
bool any_same(const void *a, std::initializer_list<const void *> others) {
    for (const void *p : others)
        if (same(a, p)) return true;
    return false;
}

la_status check_qk(const la_qk_shape &s) {
    if (s.B < 0 || s.N < 0 || s.Hq < 0 || s.Hk < 0 || s.D < 1 || !dtype_ok(s.dtype)) return LA_ERR_INVALID_ARG;
    if (s.D > kRotateMaxD || s.D % 2) return LA_ERR_UNSUPPORTED;
    if ((long long)s.B * s.N > 0x7fffffff - (1 << 20)) return LA_ERR_UNSUPPORTED;   // tokens are counted in 32 bits
    return LA_OK;
}

la_status check_rotation(const la_rotation &r, const la_qk_shape &s) {
    if (r.A < 1 || r.A > 8 || r.P < 0 || r.P > s.D / 2) return LA_ERR_INVALID_ARG;
    if (r.pairs != LA_PAIRS_HALF && r.pairs != LA_PAIRS_ADJACENT) return LA_ERR_INVALID_ARG;
    if (r.P == 0) return LA_OK;
    if (r.axes)
        for (int i = 0; i < r.P; i++)
            if (r.axes[i] >= r.A) return LA_ERR_INVALID_ARG;
    if (s.B == 0 || s.N == 0) return LA_OK;   // no positions
    if (!aligned(r.pos, 4) || !aligned(r.freq, 4)) return LA_ERR_INVALID_ARG;
    if (!stride_ok(r.sa) || !stride_ok(r.sb) || !stride_ok(r.sn)) return LA_ERR_INVALID_ARG;
    return LA_OK;
}

// An output that may be the input it comes from, row for row.
bool in_place_ok(const la_view &out, const la_view &in) {
    return out.data != in.data || (out.sb == in.sb && out.sh == in.sh && out.sn == in.sn);
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

size_t la_decay_workspace_bytes(la_shape s, int backward) {
    return check_decay(s) == LA_OK ? decay_ws_bytes(s, backward != 0) : (size_t)-1;
}

la_status la_decay_forward(la_view q, la_view k, la_view v, la_view out, const float *log_decay, const int *lens,
                           la_shape s, float scale, const float *S0, float *SN, void *workspace, size_t ws_bytes,
                           la_stream_t stream) {
    la_status st = check_decay(s);
    if (st != LA_OK) return st;
    if (s.B == 0 || s.H == 0) return LA_OK;
    if (!states_ok({S0, SN, lens}) || !aligned(log_decay, 4)) return LA_ERR_INVALID_ARG;
    if (out.data == nullptr && SN == nullptr) return LA_ERR_INVALID_ARG;
    if (any_same(SN, {log_decay, lens})) return LA_ERR_INVALID_ARG;
    if (s.N == 0) {
        s.D *= s.M;   // a state of D M values
        return from_cuda(pass_state(SN, S0, s, (cudaStream_t)stream));
    }
    if (!view_ok(k, s.dtype) || !view_ok(v, s.dtype)) return LA_ERR_INVALID_ARG;
    if (out.data) {
        if (!view_ok(q, s.dtype) || !view_ok(out, s.dtype) || !nested(out, s.B, s.H, s.N, s.M)) return LA_ERR_INVALID_ARG;
        if (any_same(out.data, {q.data, k.data, v.data, log_decay, lens, S0, SN})) return LA_ERR_INVALID_ARG;
    }
    if (any_same(SN, {out.data ? q.data : nullptr, k.data, v.data})) return LA_ERR_INVALID_ARG;
    if (!workspace_ok(decay_ws_bytes(s, false), workspace, ws_bytes)) return LA_ERR_INVALID_ARG;
    DecayProblem p{};
    p.q = q, p.k = k, p.v = v, p.out = out, p.log_decay = log_decay, p.lens = lens, p.S0 = S0, p.SN = SN;
    p.B = s.B, p.H = s.H, p.N = s.N, p.D = s.D, p.M = s.M, p.dtype = s.dtype, p.scale = scale;
    p.ws = workspace, p.stream = (cudaStream_t)stream;
    return from_cuda(decay_forward(p));
}

la_status la_decay_step(la_view q, la_view k, la_view v, la_view y, const float *log_decay, la_shape s, float scale,
                        float *S, la_stream_t stream) {
    s.N = 1;
    q.sn = k.sn = v.sn = y.sn = 0;
    const la_status st = check_decay(s);
    if (st != LA_OK) return st;
    if (s.B == 0 || s.H == 0) return LA_OK;
    if (!aligned(S, 4) || !aligned(log_decay, 4)) return LA_ERR_INVALID_ARG;
    if (!view_ok(q, s.dtype) || !view_ok(k, s.dtype) || !view_ok(v, s.dtype) || !view_ok(y, s.dtype) ||
        !nested(y, s.B, s.H, 1, s.M))
        return LA_ERR_INVALID_ARG;
    if (any_same(y.data, {q.data, k.data, v.data, log_decay, S}) || any_same(S, {q.data, k.data, v.data, log_decay}))
        return LA_ERR_INVALID_ARG;
    DecayProblem p{};
    p.q = q, p.k = k, p.v = v, p.out = y, p.log_decay = log_decay, p.SN = S;
    p.B = s.B, p.H = s.H, p.N = 1, p.D = s.D, p.M = s.M, p.dtype = s.dtype, p.scale = scale;
    p.stream = (cudaStream_t)stream;
    return from_cuda(decay_step(p));
}

la_status la_decay_backward(la_view q, la_view k, la_view v, la_view dout, la_view dq, la_view dk, la_view dv,
                            const float *log_decay, const int *lens, la_shape s, float scale, const float *S0,
                            const float *dSN, float *dS0, void *workspace, size_t ws_bytes, la_stream_t stream) {
    la_status st = check_decay(s);
    if (st != LA_OK) return st;
    if (s.B == 0 || s.H == 0) return LA_OK;
    if (!states_ok({S0, dSN, dS0, lens}) || !aligned(log_decay, 4)) return LA_ERR_INVALID_ARG;
    if (any_same(dS0, {S0, dSN, log_decay, lens})) return LA_ERR_INVALID_ARG;
    if (s.N == 0) {
        s.D *= s.M;
        return from_cuda(pass_state(dS0, dSN, s, (cudaStream_t)stream));
    }
    for (const la_view *w : {&q, &k, &v, &dout, &dq, &dk, &dv})
        if (!view_ok(*w, s.dtype)) return LA_ERR_INVALID_ARG;
    if (!nested(dq, s.B, s.H, s.N, s.D) || !nested(dk, s.B, s.H, s.N, s.D) || !nested(dv, s.B, s.H, s.N, s.M))
        return LA_ERR_INVALID_ARG;
    const void *outs[] = {dq.data, dk.data, dv.data, dS0};
    for (const void *o : outs)
        if (any_same(o, {q.data, k.data, v.data, dout.data, S0, dSN, log_decay, lens})) return LA_ERR_INVALID_ARG;
    for (int i = 0; i < 4; i++)
        for (int j = 0; j < i; j++)
            if (same(outs[i], outs[j])) return LA_ERR_INVALID_ARG;
    if (!workspace_ok(decay_ws_bytes(s, true), workspace, ws_bytes)) return LA_ERR_INVALID_ARG;
    DecayProblem p{};
    p.q = q, p.k = k, p.v = v, p.dout = dout, p.dq = dq, p.dk = dk, p.dv = dv, p.log_decay = log_decay, p.lens = lens;
    p.S0 = S0, p.dSN = dSN, p.dS0 = dS0;
    p.B = s.B, p.H = s.H, p.N = s.N, p.D = s.D, p.M = s.M, p.dtype = s.dtype, p.scale = scale;
    p.ws = workspace, p.stream = (cudaStream_t)stream;
    return from_cuda(decay_backward(p));
}

size_t la_qk_rotate_workspace_bytes(la_qk_shape s) {
    return check_qk(s) == LA_OK ? rotate_ws_bytes(s) : (size_t)-1;
}

// The checks that both directions share; y: qo, ko or dq, dk; dy: null data forward.
static la_status check_rotate(const la_view *x, const la_view *y, const la_view *dy, const float *const *w,
                              const la_rotation &rot, const la_qk_shape &s, int norm, float eps) {
    la_status st = check_qk(s);
    if (st != LA_OK) return st;
    st = check_rotation(rot, s);
    if (st != LA_OK) return st;
    if (norm ? !(eps >= 0.f) : w[0] != nullptr || w[1] != nullptr) return LA_ERR_INVALID_ARG;
    if (!states_ok({w[0], w[1]})) return LA_ERR_INVALID_ARG;
    if (s.B == 0 || s.N == 0) return LA_OK;
    const int H[2] = {s.Hq, s.Hk};
    for (int i = 0; i < 2; i++) {
        if (H[i] == 0) continue;
        if (!view_ok(x[i], s.dtype) || !view_ok(y[i], s.dtype) || (dy && !view_ok(dy[i], s.dtype))) return LA_ERR_INVALID_ARG;
        if (!nested(y[i], s.B, H[i], s.N, s.D)) return LA_ERR_INVALID_ARG;
        if (any_same(y[i].data, {w[0], w[1], rot.P ? rot.pos : nullptr, rot.P ? rot.freq : nullptr})) return LA_ERR_INVALID_ARG;
        // in place only on the rows that the output comes from
        if (!in_place_ok(y[i], dy ? dy[i] : x[i]) || (dy && y[i].data == x[i].data)) return LA_ERR_INVALID_ARG;
        const int o = 1 - i;
        if (H[o] == 0) continue;
        if (any_same(y[i].data, {x[o].data, y[o].data, dy ? dy[o].data : nullptr})) return LA_ERR_INVALID_ARG;
    }
    return LA_OK;
}

la_status la_qk_rotate_forward(la_view q, la_view k, la_view qo, la_view ko, const float *wq, const float *wk,
                               la_rotation rot, la_qk_shape s, int norm, float eps, la_stream_t stream) {
    const la_view x[2] = {q, k}, y[2] = {qo, ko};
    const float *const w[2] = {wq, wk};
    const la_status st = check_rotate(x, y, nullptr, w, rot, s, norm, eps);
    if (st != LA_OK || s.B == 0 || s.N == 0 || s.Hq + s.Hk == 0) return st;
    RotateProblem p{};
    p.q = q, p.k = k, p.qo = qo, p.ko = ko, p.wq = wq, p.wk = wk, p.rot = rot, p.s = s, p.norm = norm != 0, p.eps = eps;
    p.stream = (cudaStream_t)stream;
    return from_cuda(rotate_forward(p));
}

la_status la_qk_rotate_backward(la_view dqo, la_view dko, la_view q, la_view k, la_view dq, la_view dk,
                                const float *wq, const float *wk, la_rotation rot, la_qk_shape s, int norm, float eps,
                                float *dwq, float *dwk, void *workspace, size_t ws_bytes, la_stream_t stream) {
    const la_view x[2] = {q, k}, y[2] = {dq, dk}, dy[2] = {dqo, dko};
    const float *const w[2] = {wq, wk};
    const la_status st = check_rotate(x, y, dy, w, rot, s, norm, eps);
    if (st != LA_OK) return st;
    if (!states_ok({dwq, dwk}) || (!norm && (dwq || dwk)) || same(dwq, dwk)) return LA_ERR_INVALID_ARG;
    const bool empty = s.B == 0 || s.N == 0;
    for (const float *d : {dwq, dwk})
        if (any_same(d, {wq, wk, rot.P ? rot.pos : nullptr, rot.P ? rot.freq : nullptr}) ||
            (!empty && s.Hq && any_same(d, {q.data, dq.data, dqo.data})) ||
            (!empty && s.Hk && any_same(d, {k.data, dk.data, dko.data})))
            return LA_ERR_INVALID_ARG;
    if (empty || s.Hq + s.Hk == 0) {   // sums over nothing
        cudaError_t e = cudaSuccess;
        for (float *d : {dwq, dwk})
            if (d && e == cudaSuccess) e = cudaMemsetAsync(d, 0, (size_t)s.D * sizeof(float), (cudaStream_t)stream);
        return from_cuda(e);
    }
    if ((dwq || dwk) && (ws_bytes < rotate_ws_bytes(s) || !aligned(workspace, 16))) return LA_ERR_INVALID_ARG;
    RotateProblem p{};
    p.q = q, p.k = k, p.qo = dq, p.ko = dk, p.dqo = dqo, p.dko = dko, p.wq = wq, p.wk = wk, p.rot = rot, p.s = s;
    p.norm = norm != 0, p.eps = eps, p.dwq = dwq, p.dwk = dwk, p.ws = workspace, p.stream = (cudaStream_t)stream;
    return from_cuda(rotate_backward(p));
}

}  // extern "C"
