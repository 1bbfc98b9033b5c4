"""Refusals of the operators around the attention, on the CPU: the C entry
points check their arguments before any CUDA call, the binding checks shapes,
types and devices before that."""
import ctypes

import pytest
import torch

from weight_recurrence_gb300 import build as labuild
from weight_recurrence_gb300 import la

OK, INVALID, UNSUPPORTED = la.LA_OK, la.LA_ERR_INVALID_ARG, la.LA_ERR_UNSUPPORTED
F32, BF16 = la.LA_DTYPE_F32, la.LA_DTYPE_BF16


@pytest.fixture(scope="module")
def lib():
    labuild.build()
    return la.lib()


def _p(i, off=0):
    return ctypes.c_void_p(0x100000 * (i + 1) + off)   # never dereferenced: checks fail first


def _v(i, sb=512, sh=128, sn=16, off=0):
    return la.la_view(0x100000 * (i + 1) + off if i is not None else None, sb, sh, sn)


def _r(i, stride=16, off=0):
    return la.la_rows(0x100000 * (i + 1) + off if i is not None else None, stride)


def _shape(B=2, H=4, N=8, D=16, dt=F32):
    return la.la_shape(B, H, N, D, 0, dt)


def test_recurrence_forward_refusals(lib):
    f, s = lib.la_recurrence_forward, _shape()

    def call(x=_v(0), g=_v(1), out=_v(2), lens=None, s=s, gate=2, h0=None, hN=None, ws=None, n=0):
        return f(x, g, out, lens, s, gate, h0, hN, ws, n, None)
    assert call(s=_shape(B=-1)) == INVALID
    assert call(s=_shape(N=-1)) == INVALID
    assert call(s=_shape(D=0)) == INVALID
    assert call(s=_shape(dt=2)) == INVALID
    assert call(gate=3) == INVALID
    assert call(gate=-1) == INVALID
    for bad in (_v(None), _v(0, off=2), _v(0, sb=-1), _v(0, sn=1 << 41)):
        assert call(x=bad) == INVALID
        assert call(g=bad) == INVALID
        assert call(out=bad) == INVALID
    assert call(lens=_p(5, 2)) == INVALID
    assert call(h0=_p(5, 2)) == INVALID
    assert call(hN=_p(5, 1)) == INVALID
    # outputs on an input or over their own rows
    assert call(out=_v(0)) == INVALID
    assert call(h0=_p(2)) == INVALID
    assert call(hN=_p(2)) == INVALID
    assert call(hN=_p(0)) == INVALID
    for over in (_v(2, sn=0), _v(2, sn=15), _v(2, sh=127), _v(2, sb=511), _v(2, sh=16), _v(2, sb=0)):
        assert call(out=over) == INVALID
    # more channel groups than a grid has CTAs
    assert call(s=_shape(B=1 << 20, H=1 << 12, D=64)) == UNSUPPORTED
    assert call(s=_shape(D=0x7fffffff)) == UNSUPPORTED
    # a few long sequences need workspace
    long = _shape(B=1, H=1, N=65536)
    need = lib.la_recurrence_workspace_bytes(long)
    assert 0 < need < (1 << 22) and lib.la_recurrence_workspace_bytes(_shape(N=64)) == 0
    assert lib.la_recurrence_workspace_bytes(_shape(N=-1)) == la._SIZE_MAX
    assert call(s=long) == INVALID
    assert call(s=long, ws=_p(7), n=need - 1) == INVALID
    assert call(s=long, ws=_p(7, 8), n=need) == INVALID
    # nothing to do
    assert call(x=_v(None), g=_v(None), out=_v(None), s=_shape(B=0)) == OK
    assert call(x=_v(None), g=_v(None), out=_v(None), s=_shape(N=0)) == OK
    assert call(x=_v(None), g=_v(None), out=_v(None), s=_shape(N=0), h0=_p(5), hN=_p(5)) == OK


def test_recurrence_step_refusals(lib):
    f = lib.la_recurrence_step
    assert f(_v(0), _v(1), _v(2), _shape(), 2, None, None) == INVALID
    assert f(_v(0), _v(1), _v(2), _shape(), 2, _p(2), None) == INVALID
    assert f(_v(0), _v(1), _v(2), _shape(), 2, _p(3, 2), None) == INVALID
    assert f(_v(0), _v(1), _v(2, sh=15), _shape(), 2, _p(3), None) == INVALID
    assert f(_v(0), _v(1), _v(2), _shape(), 9, _p(3), None) == INVALID
    assert f(_v(None), _v(None), _v(None), _shape(H=0), 2, None, None) == OK


def test_recurrence_backward_refusals(lib):
    f = lib.la_recurrence_backward

    def call(x=_v(0), g=_v(1), out=_v(2), dout=_v(3), dx=_v(4), dg=_v(5), lens=None, s=_shape(), gate=2, h0=None,
             dhN=None, dh0=None, ws=None, n=0):
        return f(x, g, out, dout, dx, dg, lens, s, gate, h0, dhN, dh0, ws, n, None)
    bad = _v(7, off=1)
    for name in ("x", "g", "out", "dout", "dx", "dg"):
        assert call(**{name: bad}) == INVALID
        assert call(**{name: _v(None)}) == INVALID
    for name in ("lens", "h0", "dhN", "dh0"):
        assert call(**{name: _p(7, 2)}) == INVALID
    for i in range(4):
        assert call(dx=_v(i)) == INVALID
        assert call(dg=_v(i)) == INVALID
        assert call(dh0=_p(i)) == INVALID
    assert call(dx=_v(5)) == INVALID
    assert call(dh0=_p(4)) == INVALID
    assert call(h0=_p(6), dh0=_p(6)) == INVALID
    assert call(dx=_v(4, sn=8)) == INVALID
    assert call(dg=_v(5, sb=0)) == INVALID
    assert call(s=_shape(B=0)) == OK
    assert call(s=_shape(N=0), dhN=_p(6), dh0=_p(6)) == OK


def test_layernorm_refusals(lib):
    f = lib.la_layernorm_forward

    def call(x=_r(0), res=_r(None), sum=_r(None), y=_r(1), w=None, b=None, mean=None, rstd=None, rows=4, C=16, dt=F32,
             eps=1e-5):
        return f(x, res, sum, y, w, b, mean, rstd, rows, C, dt, eps, None)
    assert call(rows=-1) == INVALID
    assert call(C=0) == INVALID
    assert call(C=16385) == UNSUPPORTED
    assert call(dt=5) == INVALID
    assert call(eps=-1.0) == INVALID
    assert call(eps=float("nan")) == INVALID
    assert call(mean=_p(5)) == INVALID                      # one of mean, rstd
    assert call(mean=_p(5), rstd=_p(5)) == INVALID
    assert call(sum=_r(5)) == INVALID                       # sum without res
    assert call(x=_r(None)) == INVALID
    assert call(y=_r(0)) == INVALID
    assert call(y=_r(1, stride=15)) == INVALID
    assert call(x=_r(0, stride=-16)) == INVALID
    assert call(res=_r(2, off=2)) == INVALID
    assert call(res=_r(2), sum=_r(2, stride=32)) == INVALID  # in place with another stride
    assert call(res=_r(1)) == INVALID
    assert call(w=_p(4, 2)) == INVALID
    assert call(rows=0, x=_r(None), y=_r(None)) == OK


def test_layernorm_backward_refusals(lib):
    f = lib.la_layernorm_backward
    need = lib.la_layernorm_workspace_bytes(4, 16, F32)

    def call(dy=_r(0), s=_r(1), dsum=_r(None), ds=_r(2), w=None, mean=_p(3), rstd=_p(4), dw=_p(5), db=_p(6), rows=4,
             C=16, dt=F32, ws=_p(7), n=need):
        return f(dy, s, dsum, ds, w, mean, rstd, dw, db, rows, C, dt, ws, n, None)
    assert 0 < need < (1 << 30)
    assert lib.la_layernorm_workspace_bytes(-1, 16, F32) == la._SIZE_MAX
    assert lib.la_layernorm_workspace_bytes(4, 0, F32) == la._SIZE_MAX
    assert lib.la_layernorm_workspace_bytes(4, 16385, F32) == la._SIZE_MAX
    assert call(n=need - 1) == INVALID
    assert call(ws=None) == INVALID
    assert call(ws=_p(7, 4)) == INVALID
    assert call(mean=None) == INVALID
    assert call(rstd=_p(4, 1)) == INVALID
    assert call(ds=_r(0)) == INVALID
    assert call(ds=_r(1)) == INVALID
    assert call(dsum=_r(2)) == INVALID
    assert call(ds=_r(2, stride=8)) == INVALID
    assert call(dw=_p(6)) == INVALID
    assert call(w=_p(5)) == INVALID
    assert call(dw=_p(5, 2)) == INVALID
    assert call(C=20000) == UNSUPPORTED
    assert call(rows=0, dw=None, db=None, dy=_r(None), s=_r(None), ds=_r(None)) == OK


def test_grad_refusals(lib):
    need = lib.la_grad_workspace_bytes(2)
    assert need > 0 and lib.la_grad_workspace_bytes(-1) == la._SIZE_MAX

    def call(src=0x10000, dst=0x20000, n=8, dt=F32, count=2, norm=_p(3), ws=_p(4), nb=need, mx=1.0, table=True):
        t = (la.la_tensor * 2)(la.la_tensor(0x30000, 0x40000, 4, BF16), la.la_tensor(src, dst, n, dt))
        return lib.la_grad_clip(t if table else None, count, mx, norm, ws, nb, None)
    assert call(src=None) == INVALID
    assert call(src=0x10002) == INVALID
    assert call(dst=0x20001) == INVALID
    assert call(dst=None) == INVALID
    assert call(n=-1) == INVALID
    assert call(dt=3) == INVALID
    assert call(count=-1) == INVALID
    assert call(table=False) == INVALID
    assert call(norm=None) == INVALID
    assert call(norm=_p(3, 2)) == INVALID
    assert call(src=0x10000, norm=ctypes.c_void_p(0x10000)) == INVALID
    assert call(nb=need - 1) == INVALID
    assert call(ws=None) == INVALID
    assert call(mx=-1.0) == INVALID
    assert call(mx=float("nan")) == INVALID


def test_binding_refusals(lib):
    x = torch.zeros(2, 5, 8)
    g = torch.zeros(2, 5, 8)
    with pytest.raises(ValueError, match="CUDA"):
        la.la_recurrence_forward(x, g)
    with pytest.raises(ValueError, match="gate"):
        la.la_recurrence_forward(x, g, "tanh")
    with pytest.raises(ValueError, match="g must have shape"):
        la.la_recurrence_forward(x, g[:, :4])
    with pytest.raises(TypeError):
        la.la_recurrence_forward(x, g.bfloat16())
    with pytest.raises(TypeError):
        la.la_recurrence_forward(x.half(), g.half())
    with pytest.raises(ValueError, match="x must be"):
        la.la_recurrence_forward(x[0], g[0])
    with pytest.raises(ValueError, match="h0 must have shape"):
        la.la_recurrence_forward(x, g, h0=torch.zeros(2, 5))
    with pytest.raises(TypeError, match="h0"):
        la.la_recurrence_forward(x, g, h0=torch.zeros(2, 8, dtype=torch.float64))
    with pytest.raises(TypeError, match="lens"):
        la.la_recurrence_forward(x, g, lens=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="lens"):
        la.la_recurrence_forward(x, g, lens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="sigmoid"):
        la.la_recurrence_backward(None, g, x, x, "sigmoid")
    with pytest.raises(ValueError, match="dout"):
        la.la_recurrence_backward(x, g, x, x[:1])
    with pytest.raises(ValueError, match="h must have shape"):
        la.la_recurrence_step(x[:, 0], g[:, 0], torch.zeros(2, 9))
    w = torch.ones(8)
    with pytest.raises(ValueError, match="CUDA"):
        la.la_layernorm_forward(x, w)
    with pytest.raises(ValueError, match="w must have shape"):
        la.la_layernorm_forward(x, torch.ones(9))
    with pytest.raises(TypeError, match="w must be"):
        la.la_layernorm_forward(x, w.bfloat16())
    with pytest.raises(ValueError, match="res must have shape"):
        la.la_layernorm_forward(x, w, res=x[:1])
    with pytest.raises(ValueError, match="sum needs res"):
        la.la_layernorm_forward(x, w, sum=torch.zeros_like(x))
    with pytest.raises(ValueError, match="mean"):
        la.la_layernorm_backward(x, x, w, None, None)
    with pytest.raises(ValueError, match="no tensors"):
        la.la_grad_norm([])
    with pytest.raises(TypeError):
        la.la_grad_norm([x.half()])
    with pytest.raises(ValueError, match="contiguous"):
        la.la_grad_norm([x.transpose(0, 1)])
    with pytest.raises(ValueError, match="one tensor per gradient"):
        la.la_grad_clip([x, g], 1.0, out=[x])
    with pytest.raises(ValueError, match="CUDA"):
        la.la_grad_clip([x], 1.0)
    for call in (lambda: la.la_recurrence_forward(None, g), lambda: la.la_layernorm_forward(None),
                 lambda: la.la_recurrence_step(x[:, 0], g[:, 0], None), lambda: la.la_grad_norm([None])):
        with pytest.raises(ValueError, match="required"):
            call()
    with pytest.raises(TypeError, match="tensor"):
        la.la_recurrence_forward(x, [g])
    with pytest.raises(TypeError):
        la.la_grad_clip(3, 1.0)
    with pytest.raises(TypeError):
        la.la_layernorm_forward(x, w, eps="small")


def test_strided_views_reach_the_library_as_they_are(lib):
    b = la._bound()
    t = torch.zeros(2, 6, 3, 16)                    # [B, N, H, 2D]
    assert b.view(t[..., 8:].transpose(1, 2), False) == (t.data_ptr() + 8 * 4, 6 * 3 * 16, 16, 48)   # [B, H, N, D]
    assert b.view(torch.zeros(1, 5, 8).expand(4, 5, 8), False)[1:] == (0, 0, 8)
    assert b.view(t[:, 2, :, :8], True)[1:] == (6 * 3 * 16, 16, 0)
    with pytest.raises(ValueError, match="contiguous"):
        b.view(torch.zeros(2, 8, 5).transpose(1, 2), False)
    assert b.rows(t[:, :, 1, :8]) == (t.data_ptr() + 16 * 4, 48)
    assert b.rows(t[0, 0, 0])[1] == 16
    with pytest.raises(ValueError, match="one stride"):
        b.rows(t[:, :4, 1])
    with pytest.raises(TypeError, match="tensor"):
        b.rows([1.0])
    with pytest.raises(TypeError, match="arguments"):
        b.rows(t, t)
