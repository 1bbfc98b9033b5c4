"""fp64 numpy oracle of the operators around the attention: the gated linear
recurrence and its backward, layer norm and its backward, and the global
norm.  Written from the formulas token by token and row by row; shares no
code with the CUDA library."""
import numpy as np


def _f64(x):
    if hasattr(x, "detach"):
        x = x.detach().float().cpu().numpy()
    return np.asarray(x, dtype=np.float64)


def gate_factors(gate, g):
    """a, w = du/dx of h_t = a h_{t-1} + w x_t."""
    if gate == "decay":
        return g, np.ones_like(g)
    with np.errstate(over="ignore"):
        if gate == "log":
            return np.exp(g), np.ones_like(g)
        return 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g))


def recurrence(x, g, gate, h0=None, lens=None):
    """x, g [B,H,N,D] -> (out, hN); rows past lens[b] are 0."""
    x, g = _f64(x), _f64(g)
    B, H, N, D = x.shape
    a, w = gate_factors(gate, g)
    out = np.zeros_like(x)
    hN = np.zeros((B, H, D)) if h0 is None else _f64(h0).copy()
    for b in range(B):
        for t in range(N if lens is None else min(max(int(lens[b]), 0), N)):
            hN[b] = a[b, :, t] * hN[b] + w[b, :, t] * x[b, :, t]
            out[b, :, t] = hN[b]
    return out, hN


def recurrence_backward(x, g, gate, dout, h0=None, dhN=None, lens=None, out=None):
    """(dx, dg, dh0); out: where given, h_{t-1} is read from it (the stored,
    rounded output) instead of being computed."""
    x, g, dout = _f64(x), _f64(g), _f64(dout)
    B, H, N, D = x.shape
    h = recurrence(x, g, gate, h0, lens)[0] if out is None else _f64(out)
    start = np.zeros((B, H, D)) if h0 is None else _f64(h0)
    a, w = gate_factors(gate, g)
    dx, dg = np.zeros_like(x), np.zeros_like(x)
    carry = np.zeros((B, H, D)) if dhN is None else _f64(dhN).copy()
    for b in range(B):
        for t in range((N if lens is None else min(max(int(lens[b]), 0), N)) - 1, -1, -1):
            lam = dout[b, :, t] + carry[b]
            before = h[b, :, t - 1] if t > 0 else start[b]
            dx[b, :, t] = lam * w[b, :, t]
            if gate == "decay":
                dg[b, :, t] = lam * before
            elif gate == "log":
                dg[b, :, t] = lam * before * a[b, :, t]
            else:
                dg[b, :, t] = lam * (before - x[b, :, t]) * a[b, :, t] * w[b, :, t]
            carry[b] = a[b, :, t] * lam
    return dx, dg, carry


def layernorm(s, w=None, b=None, eps=1e-5):
    """Rows of s [R,C] -> (y, mean, rstd)."""
    s = _f64(s)
    mean = s.mean(axis=1)
    rstd = 1.0 / np.sqrt(((s - mean[:, None]) ** 2).mean(axis=1) + eps)
    y = (s - mean[:, None]) * rstd[:, None]
    if w is not None:
        y = y * _f64(w)
    if b is not None:
        y = y + _f64(b)
    return y, mean, rstd


def layernorm_backward(dy, s, w=None, eps=1e-5, dsum=None):
    """(ds, dw, db) of rows s [R,C]."""
    dy = _f64(dy)
    xh, _, rstd = layernorm(s, eps=eps)
    v = dy if w is None else dy * _f64(w)
    ds = rstd[:, None] * (v - v.mean(axis=1)[:, None] - xh * (v * xh).mean(axis=1)[:, None])
    if dsum is not None:
        ds = ds + _f64(dsum)
    return ds, (dy * xh).sum(axis=0), dy.sum(axis=0)


def global_norm(tensors):
    return float(np.sqrt(sum((_f64(t) ** 2).sum() for t in tensors)))
