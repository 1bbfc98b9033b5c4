"""Refusals of the attention with decays and of the norm and rotation, on the
CPU: the C entry points check their arguments before any CUDA call, the binding
checks shapes, types and devices before that."""
import ctypes

import pytest
import torch

from weight_recurrence_gb300 import build as labuild
from weight_recurrence_gb300 import la

OK, INVALID, UNSUPPORTED = la.LA_OK, la.LA_ERR_INVALID_ARG, la.LA_ERR_UNSUPPORTED
F32, BF16 = la.LA_DTYPE_F32, la.LA_DTYPE_BF16


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where nothing could be launched")
    labuild.build()
    return la.lib()


def _p(i, off=0):
    return ctypes.c_void_p(0x100000 * (i + 1) + off)   # never dereferenced: checks fail first


def _v(i, sb=512, sh=128, sn=16, off=0):
    return la.la_view(0x100000 * (i + 1) + off if i is not None else None, sb, sh, sn)


def _shape(B=2, H=4, N=8, D=16, M=16, dt=F32):
    return la.la_shape(B, H, N, D, M, dt)


BAD_SHAPES = [(dict(B=-1), INVALID), (dict(H=-1), INVALID), (dict(N=-1), INVALID), (dict(D=0), INVALID),
              (dict(M=0), INVALID), (dict(dt=2), INVALID), (dict(D=129), UNSUPPORTED), (dict(M=256), UNSUPPORTED),
              (dict(B=1 << 16, H=1 << 13), UNSUPPORTED), (dict(N=0x7fffffff), UNSUPPORTED),
              (dict(N=0x7fffffff - (1 << 20) + 1), UNSUPPORTED)]
BAD_VIEWS = [_v(None), _v(0, off=2), _v(0, sb=-1), _v(0, sn=1 << 41)]


def test_decay_forward_refusals(lib):
    def call(q=_v(0), k=_v(1), v=_v(2), out=_v(3), g=_p(4), lens=None, s=_shape(), scale=1.0, S0=None, SN=None, ws=None,
             n=0):
        return lib.la_decay_forward(q, k, v, out, g, lens, s, scale, S0, SN, ws, n, None)
    for change, status in BAD_SHAPES:
        assert call(s=_shape(**change)) == status, change
        assert lib.la_decay_workspace_bytes(_shape(**change), 0) == la._SIZE_MAX
    for bad in BAD_VIEWS:
        for name in ("q", "k", "v"):
            assert call(**{name: bad}) == INVALID
    for bad in (_v(3, off=2), _v(3, sn=0), _v(3, sn=15), _v(3, sh=127), _v(3, sb=511), _v(3, sb=0)):
        assert call(out=bad) == INVALID
    assert call(g=None) == INVALID and call(g=_p(4, 2)) == INVALID
    for name in ("lens", "S0", "SN"):
        assert call(**{name: _p(7, 2)}) == INVALID
    assert call(out=_v(None)) == INVALID                     # nothing wanted
    for i in (0, 1, 2, 4):                                   # an output on an input
        assert call(out=_v(i)) == INVALID
        assert call(SN=_p(i)) == INVALID
    assert call(SN=_p(3)) == INVALID and call(S0=_p(3)) == INVALID and call(lens=_p(3)) == INVALID
    assert call(SN=_p(6), lens=_p(6)) == INVALID
    # a few long sequences need workspace
    long = _shape(B=1, H=2, N=65536)
    need = lib.la_decay_workspace_bytes(long, 0)
    assert need > 0 and lib.la_decay_workspace_bytes(_shape(N=128), 0) == 0
    wide = dict(sb=1 << 30, sh=1 << 22)
    views = dict(q=_v(0, **wide), k=_v(1, **wide), v=_v(2, **wide), out=_v(3, **wide))
    assert call(s=long, **views) == INVALID
    assert call(s=long, ws=_p(8), n=need - 1, **views) == INVALID
    assert call(s=long, ws=_p(8, 8), n=need, **views) == INVALID
    # and bf16 rows that are not whole 16-byte pieces, for their packed copies
    odd = _shape(N=100, D=33, dt=BF16)
    need = lib.la_decay_workspace_bytes(odd, 0)
    assert need >= 2 * 4 * 100 * (2 * 40 + 16) * 2 and lib.la_decay_workspace_bytes(odd, 1) >= need + 2 * 4 * 100 * 16 * 2
    views = dict(q=_v(0, 1 << 20, 1 << 14, 40), k=_v(1, 1 << 20, 1 << 14, 40), v=_v(2, 1 << 20, 1 << 14, 40),
                 out=_v(3, 1 << 20, 1 << 14, 40))
    assert call(s=odd, **views) == INVALID
    assert call(s=odd, ws=_p(8), n=need - 1, **views) == INVALID
    assert call(s=odd, ws=_p(8, 8), n=need, **views) == INVALID
    none = _v(None)
    assert call(q=none, k=none, v=none, out=none, g=None, s=_shape(B=0)) == OK
    assert call(q=none, k=none, v=none, out=none, s=_shape(N=0), S0=_p(6), SN=_p(6)) == OK


def test_decay_step_refusals(lib):
    def call(q=_v(0), k=_v(1), v=_v(2), y=_v(3), g=_p(4), s=_shape(), S=_p(5)):
        return lib.la_decay_step(q, k, v, y, g, s, 1.0, S, None)
    for change, status in BAD_SHAPES:
        if "N" not in change:
            assert call(s=_shape(**change)) == status, change
    for bad in BAD_VIEWS[:3]:
        for name in "qkv":
            assert call(**{name: bad}) == INVALID
    assert call(y=_v(3, sh=15)) == INVALID and call(y=_v(None)) == INVALID
    assert call(S=None) == INVALID and call(S=_p(5, 2)) == INVALID and call(g=None) == INVALID
    for i in (0, 1, 2, 4, 5):
        assert call(y=_v(i)) == INVALID
        if i != 5:
            assert call(S=_p(i)) == INVALID
    assert call(s=_shape(H=0)) == OK


def test_decay_backward_refusals(lib):
    def call(q=_v(0), k=_v(1), v=_v(2), dout=_v(3), dq=_v(4), dk=_v(5), dv=_v(6), g=_p(7), lens=None, s=_shape(), S0=None,
             dSN=None, dS0=None, ws=None, n=0):
        return lib.la_decay_backward(q, k, v, dout, dq, dk, dv, g, lens, s, 1.0, S0, dSN, dS0, ws, n, None)
    for change, status in BAD_SHAPES:
        assert call(s=_shape(**change)) == status, change
        assert lib.la_decay_workspace_bytes(_shape(**change), 1) == la._SIZE_MAX
    for bad in BAD_VIEWS:
        for name in ("q", "k", "v", "dout", "dq", "dk", "dv"):
            assert call(**{name: bad}) == INVALID
    for i, name in ((4, "dq"), (5, "dk"), (6, "dv")):
        assert call(**{name: _v(i, sn=15)}) == INVALID and call(**{name: _v(i, sb=0)}) == INVALID
        for j in (0, 1, 2, 3, 7) + tuple(x for x in (4, 5, 6) if x != i):
            assert call(**{name: _v(j)}) == INVALID
    for name in ("lens", "S0", "dSN", "dS0"):
        assert call(**{name: _p(8, 2)}) == INVALID
    for j in range(8):
        assert call(dS0=_p(j)) == INVALID
    assert call(dS0=_p(8), dSN=_p(8)) == INVALID and call(dS0=_p(8), S0=_p(8)) == INVALID
    assert call(g=None) == INVALID
    long = _shape(B=1, H=1, N=65536)
    need = lib.la_decay_workspace_bytes(long, 1)
    wide = dict(sb=1 << 30, sh=1 << 22)
    views = {n: _v(i, **wide) for i, n in enumerate(("q", "k", "v", "dout", "dq", "dk", "dv"))}
    assert need > 0 and call(s=long, **views) == INVALID
    assert call(s=_shape(B=0)) == OK


def _qk(B=2, N=8, Hq=4, Hk=4, D=16, dt=F32):
    return la.la_qk_shape(B, N, Hq, Hk, D, dt)


def _rot(pos=0x900000, freq=0xA00000, axes=None, A=1, P=8, pairs=0, sa=16, sb=8, sn=1):
    return la.la_rotation(pos, sa, sb, sn, freq, axes, A, P, pairs)


BAD_QK = [(dict(B=-1), INVALID), (dict(N=-1), INVALID), (dict(Hq=-1), INVALID), (dict(Hk=-1), INVALID),
          (dict(D=0), INVALID), (dict(dt=2), INVALID), (dict(D=258), UNSUPPORTED), (dict(D=15), UNSUPPORTED),
          (dict(B=1 << 20, N=1 << 20), UNSUPPORTED)]
BAD_ROT = [dict(A=0), dict(A=9), dict(P=-1), dict(P=9), dict(pairs=2), dict(pos=None), dict(pos=0x900002), dict(freq=None),
           dict(freq=0xA00001), dict(sa=-1), dict(sb=-1), dict(sn=1 << 41), dict(A=2, axes=b"\0\1\2\0\0\0\0\0")]


def test_rotate_forward_refusals(lib):
    def call(q=_v(0), k=_v(1), qo=_v(2), ko=_v(3), wq=None, wk=None, r=_rot(), s=_qk(), norm=1, eps=1e-6):
        return lib.la_qk_rotate_forward(q, k, qo, ko, wq, wk, r, s, norm, eps, None)
    for change, status in BAD_QK:
        assert call(s=_qk(**change)) == status, change
    for change in BAD_ROT:
        assert call(r=_rot(**change)) == INVALID, change
    for bad in BAD_VIEWS:
        for name in ("q", "k", "qo", "ko"):
            assert call(**{name: bad}) == INVALID
    assert call(eps=-1.0) == INVALID and call(eps=float("nan")) == INVALID
    assert call(wq=_p(5, 2)) == INVALID and call(norm=0, wq=_p(5)) == INVALID and call(norm=0, wk=_p(5)) == INVALID
    assert call(qo=_v(2, sn=15)) == INVALID and call(ko=_v(3, sh=0)) == INVALID
    assert call(qo=_v(0, sb=1024)) == INVALID and call(ko=_v(1, sn=32, sh=256, sb=1024)) == INVALID   # in place, other rows
    assert call(qo=_v(1)) == INVALID and call(ko=_v(0)) == INVALID and call(ko=_v(2)) == INVALID
    assert call(qo=_v(8)) == INVALID and call(qo=_v(9)) == INVALID and call(wq=_p(2)) == INVALID
    none = _v(None)
    assert call(q=none, k=none, qo=none, ko=none, s=_qk(N=0)) == OK
    assert call(q=none, k=none, qo=none, ko=none, s=_qk(Hq=0, Hk=0)) == OK


def test_rotate_backward_refusals(lib):
    need = lib.la_qk_rotate_workspace_bytes(_qk())
    assert 0 < need < (1 << 21)
    for change, _ in BAD_QK:
        assert lib.la_qk_rotate_workspace_bytes(_qk(**change)) == la._SIZE_MAX

    def call(dqo=_v(0), dko=_v(1), q=_v(2), k=_v(3), dq=_v(4), dk=_v(5), wq=None, wk=None, r=_rot(), s=_qk(), norm=1,
             eps=1e-6, dwq=None, dwk=None, ws=_p(12), n=need):
        return lib.la_qk_rotate_backward(dqo, dko, q, k, dq, dk, wq, wk, r, s, norm, eps, dwq, dwk, ws, n, None)
    for change, status in BAD_QK:
        assert call(s=_qk(**change)) == status, change
    for change in BAD_ROT:
        assert call(r=_rot(**change)) == INVALID, change
    for bad in BAD_VIEWS:
        for name in ("dqo", "dko", "q", "k", "dq", "dk"):
            assert call(**{name: bad}) == INVALID
    assert call(dq=_v(2)) == INVALID and call(dk=_v(3)) == INVALID          # the forward's input is still read
    assert call(dq=_v(0, sb=1024)) == INVALID and call(dq=_v(1)) == INVALID and call(dk=_v(4)) == INVALID
    assert call(dwq=_p(6, 2)) == INVALID and call(dwq=_p(6), dwk=_p(6)) == INVALID
    assert call(norm=0, dwq=_p(6)) == INVALID
    for i in (0, 2, 4, 8, 9):
        assert call(dwq=_p(i)) == INVALID
    assert call(dwq=_p(6), n=need - 1) == INVALID and call(dwq=_p(6), ws=None) == INVALID
    none = _v(None)
    assert call(none, none, none, none, none, none, s=_qk(B=0)) == OK


# ------------------------------------------------------------- the binding

def _decay_tensors(B=2, H=3, N=5, D=16, M=8):
    return torch.zeros(B, H, N, D), torch.zeros(B, H, N, D), torch.zeros(B, H, N, M), torch.zeros(H)


def test_binding_refuses_decay_arguments(lib):
    q, k, v, g = _decay_tensors()
    f = la.la_decay_forward
    S = torch.zeros(2, 3, 16, 8)
    for bad in [dict(q=None), dict(q=q[:, :, :4]), dict(v=v[:, :2]), dict(q=q[0]), dict(out=q), dict(S0=S[:, :, :8]),
                dict(SN=S.transpose(2, 3)), dict(lens=torch.zeros(3, dtype=torch.int32)), dict(log_decay=torch.zeros(2)),
                dict(k=k.transpose(2, 3)), dict(want_out=False), dict(want_out=False, out=v, SN=S), dict()]:
        a = dict(dict(q=q, k=k, v=v, log_decay=g), **bad)
        with pytest.raises(ValueError):   # the last: not on a CUDA device
            f(**a)
    for bad in [dict(q=q.double(), k=k.double()), dict(v=v.bfloat16()), dict(log_decay=g.double()), dict(S0=S.double()),
                dict(lens=torch.zeros(2, dtype=torch.int64)), dict(q=1), dict(scale="x")]:
        a = dict(dict(q=q, k=k, v=v, log_decay=g), **bad)
        with pytest.raises(TypeError):
            f(**a)
    b = la.la_decay_backward
    with pytest.raises(RuntimeError):       # no truth value
        f(q, k, v, g, want_out=torch.zeros(2))
    for bad in [dict(dout=q), dict(dq=v), dict(dv=q), dict(dSN=S[:1]), dict(dS0=S[..., :4])]:
        with pytest.raises(ValueError):
            b(**dict(dict(q=q, k=k, v=v, dout=v, log_decay=g), **bad))
    st = la.la_decay_step
    for bad in [dict(q=q), dict(S=S[:1]), dict(y=q[:, :, 0]), dict(S=S.transpose(2, 3)), dict()]:
        with pytest.raises(ValueError):
            st(**dict(dict(q=q[:, :, 0], k=k[:, :, 0], v=v[:, :, 0], S=S, log_decay=g), **bad))


def test_binding_refuses_rotation_arguments(lib):
    q, k = torch.zeros(2, 4, 5, 16), torch.zeros(2, 1, 5, 16)
    pos, freq, w = torch.zeros(2, 5, dtype=torch.int32), torch.zeros(8), torch.zeros(16)
    f = la.la_qk_rotate_forward
    base = dict(q=q, k=k, pos=pos, freq=freq)
    for bad in [dict(q=q[0]), dict(k=k[:1]), dict(k=k[..., :8]), dict(pos=pos[:, :4]), dict(pos=pos[:1]), dict(pos=pos[0, 0]),
                dict(freq=torch.zeros(9)), dict(freq=freq[None]), dict(wq=w[:8]), dict(norm=False, wq=w), dict(qo=k),
                dict(axes=(0, 0)), dict(axes=(300,) * 8), dict(pairs="both"), dict(k=None, wk=w), dict(k=None, ko=k),
                dict(q=q.transpose(2, 3)), dict()]:
        with pytest.raises(ValueError):
            f(**dict(base, **bad))
    for bad in [dict(pos=pos.long()), dict(freq=freq.double()), dict(wq=w.bfloat16()), dict(k=k.bfloat16()),
                dict(q=q.half(), k=k.half()), dict(eps="x"), dict(axes=8)]:
        with pytest.raises(TypeError):
            f(**dict(base, **bad))
    b = la.la_qk_rotate_backward
    base = dict(dqo=q, dko=k, q=q, k=k, pos=pos, freq=freq)
    for bad in [dict(dqo=k), dict(dko=None), dict(norm=False, dwq=w), dict(dwq=w[:8]), dict(dq=k), dict(dk=q),
                dict(k=None, dko=None, dwk=w)]:
        with pytest.raises(ValueError):
            b(**dict(base, **bad))


def test_axes_are_numbers_whatever_holds_them():
    want = bytes((0, 1, 2, 1))
    for axes in ((0, 1, 2, 1), [0, 1, 2, 1], want, bytearray(want), torch.tensor([0, 1, 2, 1]),
                 torch.tensor([0, 1, 2, 1]).numpy()):
        assert la._axes_bytes(axes) == want
    assert la._axes_bytes(None) is None


def test_views_reach_the_library_as_they_are(lib):
    x = torch.zeros(2, 5, 3, 16).transpose(1, 2)          # [B,H,N,D] of a token-major projection
    assert la._bound().view(x, False)[1:] == (240, 16, 48)
