"""GPU parity of layer norm (forward with the residual sum, backward with the
weight's and bias' gradients) against the fp64 oracle (oracle/layer.py).

Tolerances, element by element, with u = 2^-24.  A sum of n fp32 values added
in any order by threads and trees has at most k = n/32 + 16 roundings on any
path here (32 values side by side at least), so the mean is within k u avg|s|
and rstd within (k + 4) u of itself; y = (s - mean) rstd w + b then adds a few
roundings.  ds is three such terms, dw and db sums over rows (no path longer
than rows/64 + 600 additions).  An output's own rounding adds half a step.
"""
import numpy as np
import pytest
import torch

from oracle import layer
from weight_recurrence_gb300 import la

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
DTYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.lib()


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _half(dtype, ref):
    return torch.finfo(dtype).eps / 2 * np.abs(ref) + 1e-38


def _close(name, got, ref, tol):
    got = _np(got).reshape(ref.shape)
    assert np.isfinite(got).all(), name
    worst = np.abs(got - ref) / tol
    assert worst.max(initial=0.0) <= 1.0, (name, float(worst.max()), np.unravel_index(worst.argmax(), worst.shape))


def _inputs(shape, dtype, seed, mean=0.5):
    rng = torch.Generator().manual_seed(seed)
    x, res, dy, dsum = torch.randn((4,) + shape, generator=rng)
    w, b = torch.randn((2, shape[-1]), generator=rng)
    return [t.to(dtype).to(DEV) for t in (x + mean, res, dy, dsum)] + [(1 + 0.3 * w).to(DEV), b.to(DEV)]


def check_forward(s, w, b, eps, y, mean, rstd):
    C = s.shape[-1]
    sn = _np(s).reshape(-1, C)
    ref, rm, rr = layer.layernorm(sn, None if w is None else _np(w), None if b is None else _np(b), eps)
    wn, bn = np.ones(C) if w is None else np.abs(_np(w)), np.zeros(C) if b is None else np.abs(_np(b))
    k = C / 32 + 16
    avg = np.abs(sn).mean(axis=1)
    xh = np.abs(sn - rm[:, None]) * rr[:, None]
    tol = U * (wn * ((k + 4) * xh + (k + 2) * (avg * rr)[:, None]) + bn + 2 * np.abs(ref))
    _close("y", y, ref, _half(s.dtype, ref) + 2 * tol)
    if mean is not None:
        _close("mean", mean, rm, (k + 2) * U * avg + 1e-38)
        # the variance moves by 2 avg|s - mean| of the mean's error, and by its square
        _close("rstd", rstd, rr, (k + 8) * U * rr * (2 + 2 * avg * rr))


def check_backward(dy, s, w, eps, dsum, ds, dw, db):
    C = s.shape[-1]
    dn, sn = _np(dy).reshape(-1, C), _np(s).reshape(-1, C)
    extra = None if dsum is None else _np(dsum).reshape(-1, C)
    ref, rw, rb = layer.layernorm_backward(dn, sn, None if w is None else _np(w), eps, extra)
    xh, _, rr = layer.layernorm(sn, eps=eps)
    k = C / 32 + 16
    off = (k + 4) * U * (np.abs(xh) + (np.abs(sn).mean(axis=1) * rr)[:, None])    # error of xh
    v = np.abs(dn if w is None else dn * _np(w))
    big = np.abs(xh) + off
    tol = (k + 12) * U * rr[:, None] * (v + v.mean(axis=1)[:, None] + big * (v * big).mean(axis=1)[:, None])
    tol += rr[:, None] * (off * (v * big).mean(axis=1)[:, None] + big * (v * off).mean(axis=1)[:, None])
    tol += 0.0 if extra is None else 2 * U * (np.abs(extra) + np.abs(ref))
    _close("ds", ds, ref, _half(dy.dtype, ref) + 2 * tol)
    kr = len(dn) / 64 + 600
    _close("dw", dw, rw, kr * U * np.abs(dn * xh).sum(axis=0) + np.abs(dn * off).sum(axis=0) + 1e-30)
    _close("db", db, rb, kr * U * np.abs(dn).sum(axis=0) + 1e-30)


SIZES = [(1, 1), (3, 2), (5, 31), (7, 64), (1000, 64), (33, 65), (130, 96), (40, 128), (9, 200), (513, 256), (6, 777),
         (300, 1024), (17, 1001), (4, 2048), (700, 2050), (5, 4096), (3, 8192), (2, 10007), (2, 16384)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,C", SIZES)
def test_parity(R, C, dtype):
    x, res, dy, dsum, w, b = _inputs((R, C), dtype, R + C)
    for r, d in ((None, None), (res, dsum)):
        y, s, mean, rstd = la.la_layernorm_forward(x, w, b, res=r)
        ds, dw, db = la.la_layernorm_backward(dy, s, w, mean, rstd, dsum=d)
        torch.cuda.synchronize()
        if r is not None:
            assert torch.equal(s, (x.float() + r.float()).to(dtype))
        else:
            assert s is x
        check_forward(s, w, b, 1e-5, y, mean, rstd)
        check_backward(dy, s, w, 1e-5, d, ds, dw, db)


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_rows(dtype):
    x, res, dy, dsum, w, b = _inputs((70001, 48), dtype, 2)
    y, s, mean, rstd = la.la_layernorm_forward(x, w, b, res=res)
    ds, dw, db = la.la_layernorm_backward(dy, s, w, mean, rstd, dsum=dsum)
    check_forward(s, w, b, 1e-5, y, mean, rstd)
    check_backward(dy, s, w, 1e-5, dsum, ds, dw, db)


def test_optional_arguments():
    x, res, dy, _, w, b = _inputs((20, 100), torch.float32, 3)
    for ww, bb in ((None, None), (w, None), (None, b)):
        y, s, mean, rstd = la.la_layernorm_forward(x, ww, bb, eps=1e-3)
        check_forward(x, ww, bb, 1e-3, y, mean, rstd)
        check_backward(dy, s, ww, 1e-3, None, *la.la_layernorm_backward(dy, s, ww, mean, rstd))
    y2, s, mean, rstd = la.la_layernorm_forward(x, w, b, res=res, stats=False)
    assert mean is None and rstd is None
    assert torch.equal(y2, la.la_layernorm_forward(x, w, b, res=res)[0])


def test_a_large_mean_keeps_the_variance():
    """The variance is taken about the mean: values around 1000 with deviation 1."""
    x, _, dy, _, w, b = _inputs((50, 512), torch.float32, 4, mean=1000.0)
    y, s, mean, rstd = la.la_layernorm_forward(x, w, b)
    check_forward(s, w, b, 1e-5, y, mean, rstd)
    ref = layer.layernorm(_np(x))[2]
    # the mean is within 2^-20 of itself here, which moves a variance of 1 by its square
    assert np.abs(_np(rstd) / ref - 1).max() < 1e-5


def test_constant_rows():
    x = torch.full((4, 130), 3.0, device=DEV)
    y, s, mean, rstd = la.la_layernorm_forward(x, eps=1e-5)
    assert not y.any() and (mean == 3.0).all()
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)
    ds, dw, db = la.la_layernorm_backward(torch.ones_like(x), s, None, mean, rstd)
    assert ds.abs().max() <= 1e-5 ** -0.5 * 8 * U and not dw.any() and (db == 4.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_residual_in_place_and_views(dtype):
    x, res, dy, dsum, w, b = _inputs((3, 11, 72), dtype, 5)
    wide = torch.full((3, 11, 150), 7.0, dtype=dtype, device=DEV)
    wide[..., 1:73] = x                                     # odd offset, rows 150 apart
    stream = res.clone()
    y, s, mean, rstd = la.la_layernorm_forward(wide[..., 1:73], w, b, res=stream, sum=stream)
    assert s is stream and torch.equal(s, (x.float() + res.float()).to(dtype))
    check_forward(s, w, b, 1e-5, y, mean, rstd)
    into = wide[..., 75:147]
    ds, dw, db = la.la_layernorm_backward(dy, s, w, mean, rstd, dsum=dsum, ds=into)
    assert ds is into
    check_backward(dy, s, w, 1e-5, dsum, ds, dw, db)
    assert (wide[..., 0] == 7.0).all() and (wide[..., 73:75] == 7.0).all() and (wide[..., 147:] == 7.0).all()


def test_no_rows():
    x = torch.empty(0, 40, device=DEV)
    y, s, mean, rstd = la.la_layernorm_forward(x)
    ds, dw, db = la.la_layernorm_backward(x, s, None, mean, rstd)
    assert y.shape == ds.shape == x.shape and not dw.any() and not db.any()


def test_nan_and_infinite_rows_stay_their_own():
    x, _, dy, _, w, b = _inputs((9, 300), torch.float32, 6)
    clean = la.la_layernorm_forward(x, w, b)[0]
    x[4, 17], x[6, 250] = float("nan"), float("inf")
    y = la.la_layernorm_forward(x, w, b)[0]
    assert torch.isnan(y[4]).all() and torch.isnan(y[6]).any()
    keep = [i for i in range(9) if i not in (4, 6)]
    assert torch.equal(y[keep], clean[keep])


def test_equal_calls_give_equal_bits():
    x, _, dy, _, w, b = _inputs((5000, 320), torch.bfloat16, 7)
    _, s, mean, rstd = la.la_layernorm_forward(x, w, b)
    first = la.la_layernorm_backward(dy, s, w, mean, rstd)
    for _ in range(3):
        assert all(torch.equal(a, c) for a, c in zip(la.la_layernorm_backward(dy, s, w, mean, rstd), first))


def test_offsets_past_32_bits():
    R, C, stride = 33000, 64, 70000
    buf = torch.empty(R * stride, dtype=torch.bfloat16, device=DEV)
    x, y, dy, ds = (buf.as_strided((R, C), (stride, 1), i * C) for i in range(4))
    rng = torch.Generator(device=DEV).manual_seed(1)
    xr, dr = (torch.randn((R, C), generator=rng, device=DEV).to(torch.bfloat16) for _ in range(2))
    x.copy_(xr)
    dy.copy_(dr)
    _, _, mean, rstd = la.la_layernorm_forward(x, y=y)
    ref = la.la_layernorm_forward(xr)
    assert torch.equal(y, ref[0]) and torch.equal(mean, ref[2])
    got = la.la_layernorm_backward(dy, x, None, mean, rstd, ds=ds)
    want = la.la_layernorm_backward(dr, xr, None, mean, rstd)
    assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_stream_and_graph():
    x, res, dy, dsum, w, b = _inputs((700, 512), torch.bfloat16, 8)

    def step(**k):
        y, s, mean, rstd = la.la_layernorm_forward(x, w, b, res=res, **k)
        return (y, s) + la.la_layernorm_backward(dy, s, w, mean, rstd, dsum=dsum, **k)
    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(stream=side)
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x.add_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, step()))
