"""Outputs that coincide with one another or with an input of the operators
around the attention are refused (CPU: the checks come before any CUDA call)."""
import ctypes

import pytest
import torch

from weight_recurrence_gb300 import build as labuild
from weight_recurrence_gb300 import la

INVALID = la.LA_ERR_INVALID_ARG
F32 = la.LA_DTYPE_F32


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where nothing could be launched")
    labuild.build()
    return la.lib()


def _p(i, off=0):
    return ctypes.c_void_p(0x100000 * (i + 1) + off)   # never dereferenced: checks fail first


@pytest.mark.parametrize("count", [2, 5, 40, 600])
@pytest.mark.parametrize("a,b", [(0, 1), (0, -1), (-2, -1)])
def test_clip_refuses_tensors_that_coincide(lib, count, a, b):
    """A destination may be its own source and nothing else of the list."""
    need = lib.la_grad_workspace_bytes(count)

    def call(change, n=16):
        t = (la.la_tensor * count)(*[la.la_tensor(0x100000 + 0x1000 * i, 0x9000000 + 0x1000 * i, n, F32)
                                     for i in range(count)])
        change(t)
        return lib.la_grad_clip(t, count, 1.0, _p(0x1000), _p(0x1001), need, None)

    def same_tensor(t):            # listed twice, in place
        for i in (a, b):
            t[i].src = t[i].dst = 0x5000000

    def same_dst(t):
        t[b].dst = t[a].dst

    def crossed(t):                # into another's source, read before or after it was written
        t[b].dst = t[a].src

    def swapped(t):
        t[a].dst, t[b].dst = t[b].src, t[a].src

    for change in (same_tensor, same_dst, crossed, swapped):
        assert call(change) == INVALID, change.__name__


def _r(i, stride=16):
    return la.la_rows(0x100000 * (i + 1) if i is not None else None, stride)


def test_layernorm_forward_refuses_outputs_that_coincide(lib):
    f = lib.la_layernorm_forward
    x, res, sum_, y, w, b, mean, rstd = range(8)

    def call(**same):              # name=i: the pointer of argument i
        at = {n: same.get(n, i) for n, i in zip(("x", "res", "sum", "y", "w", "b", "mean", "rstd"), range(8))}
        return f(_r(at["x"]), _r(at["res"]), _r(at["sum"]), _r(at["y"]), _p(at["w"]), _p(at["b"]), _p(at["mean"]),
                 _p(at["rstd"]), 4, 16, F32, 1e-5, None)
    for name in ("sum", "mean", "rstd"):
        for other in {"w": w, "b": b, "y": y, "sum": sum_, "mean": mean, "rstd": rstd}.items():
            if other[0] != name:
                assert call(**{name: other[1]}) == INVALID, (name, other[0])
    for name in ("mean", "rstd", "y"):
        assert call(**{name: x}) == INVALID
        assert call(**{name: res}) == INVALID


def test_layernorm_backward_refuses_outputs_that_coincide(lib):
    f = lib.la_layernorm_backward
    need = lib.la_layernorm_workspace_bytes(4, 16, F32)
    names = ("dy", "s", "dsum", "ds", "w", "mean", "rstd", "dw", "db")

    def call(**same):
        at = {n: same.get(n, i) for i, n in enumerate(names)}
        return f(_r(at["dy"]), _r(at["s"]), _r(at["dsum"]), _r(at["ds"]), _p(at["w"]), _p(at["mean"]), _p(at["rstd"]),
                 _p(at["dw"]), _p(at["db"]), 4, 16, F32, _p(20), need, None)
    for name in ("ds", "dw", "db"):
        for i, other in enumerate(names):
            if other != name:
                assert call(**{name: i}) == INVALID, (name, other)
