"""fp64 numpy oracle of the linear attention with a decay for each head and of
the norm and rotation of queries and keys, with their backward passes.  Written
from the formulas token by token; shares no code with the CUDA library."""
import numpy as np

from oracle.layer import _f64


def _lengths(lens, B, N):
    return [N] * B if lens is None else [min(max(int(n), 0), N) for n in lens]


def _factor(log_decay):
    with np.errstate(over="ignore"):
        return np.exp(_f64(log_decay))[:, None, None]


def forward(q, k, v, log_decay, scale=1.0, S0=None, lens=None):
    """q, k [B,H,N,D], v [B,H,N,M] -> (out, SN); rows past lens[b] are 0."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, H, N, D = k.shape
    M = v.shape[-1]
    a = _factor(log_decay)
    out = np.zeros((B, H, N, M))
    S = np.zeros((B, H, D, M)) if S0 is None else _f64(S0).copy()
    for b, n in enumerate(_lengths(lens, B, N)):
        for t in range(n):
            S[b] = a * S[b] + k[b, :, t, :, None] * v[b, :, t, None, :]
            out[b, :, t] = scale * np.einsum("hd,hdm->hm", q[b, :, t], S[b])
    return out, S


def backward(q, k, v, dout, log_decay, scale=1.0, S0=None, dSN=None, lens=None):
    """(dq, dk, dv, dS0)."""
    q, k, v, dout = _f64(q), _f64(k), _f64(v), _f64(dout)
    B, H, N, D = k.shape
    M = v.shape[-1]
    a = _factor(log_decay)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    S = np.zeros((B, H, D, M)) if S0 is None else _f64(S0).copy()
    G = np.zeros((B, H, D, M)) if dSN is None else _f64(dSN).copy()
    for b, n in enumerate(_lengths(lens, B, N)):
        for t in range(n):
            S[b] = a * S[b] + k[b, :, t, :, None] * v[b, :, t, None, :]
            dq[b, :, t] = scale * np.einsum("hdm,hm->hd", S[b], dout[b, :, t])
        for t in range(n - 1, -1, -1):
            here = scale * q[b, :, t, :, None] * dout[b, :, t, None, :] + G[b]
            dk[b, :, t] = np.einsum("hdm,hm->hd", here, v[b, :, t])
            dv[b, :, t] = np.einsum("hdm,hd->hm", here, k[b, :, t])
            G[b] = a * here
    return dq, dk, dv, G


def _channels(P, pairs):
    i = np.arange(P)
    return (i, i + P) if pairs == "half" else (2 * i, 2 * i + 1)


def angles(pos, freq, axes=None):
    """[B,N,P] from pos [A,B,N], freq [P]; the products in extended precision where numpy has it."""
    pos = np.asarray(pos).astype(np.longdouble)
    freq = np.asarray(freq, dtype=np.float32).astype(np.longdouble)
    axes = [0] * len(freq) if axes is None else list(axes)
    turn = 2 * np.pi * np.longdouble(1)
    if len(freq) == 0:
        return np.zeros(pos.shape[1:] + (0,))
    return np.stack([np.fmod(pos[a] * f, turn) for a, f in zip(axes, freq)], axis=-1).astype(np.float64)


def turn(x, angle, pairs):
    """Rows x [B,H,N,D] turned by angle [B,N,P]."""
    i, j = _channels(angle.shape[-1], pairs)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    y = x.copy()
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    return y


def rotate(x, angle, w=None, eps=1e-6, norm=True, pairs="half"):
    x = _f64(x)
    if norm:
        x = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
        x = x if w is None else x * _f64(w)
    return turn(x, angle, pairs)


def rotate_backward(dy, x, angle, w=None, eps=1e-6, norm=True, pairs="half"):
    """(dx, dw)."""
    x, u = _f64(x), turn(_f64(dy), -angle, pairs)
    if not norm:
        return u, None
    r = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    xh = x * r
    uw = u if w is None else u * _f64(w)
    return r * (uw - xh * (uw * xh).mean(axis=-1, keepdims=True)), (u * xh).sum(axis=(0, 1, 2))
