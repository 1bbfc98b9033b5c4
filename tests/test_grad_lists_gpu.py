"""Norm and clipping of lists of more than 512 tensors (several tables, their
partial sums side by side), and what the clipping refuses.

Tolerances as in test_grad_gpu.py: the sum of squares is within (n/32768 + 70)
u of itself, u = 2^-24; a clipped value adds the factor's two roundings and its
own half step."""
import numpy as np
import pytest
import torch

from oracle import layer
from weight_recurrence_gb300 import la

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
F, B = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.lib()


def _list(sizes, dtypes, seed):
    g = torch.Generator().manual_seed(seed)
    # each table's tensors larger than the ones before, so that no table's sum can stand for another's
    return [((1 + i // 512) * torch.randn(n, generator=g)).to(dtypes[i % len(dtypes)]).to(DEV)
            for i, n in enumerate(sizes)]


SETS = [[5] * 512, [5] * 513, [37] * 1100, [0] * 512 + [9], [3] * 512 + [0] * 600 + [200001], [4096, 1, 0, 777] * 400]


@pytest.mark.parametrize("dtypes", [[F], [B], [B, F, F]])
@pytest.mark.parametrize("which", range(len(SETS)))
def test_many_tensors(which, dtypes):
    ts = _list(SETS[which], dtypes, which)
    ref = layer.global_norm(ts)
    tol = (sum(t.numel() for t in ts) / 32768 + 70) * U
    norm = la.la_grad_norm(ts).item()
    assert abs(norm - ref) <= tol * ref
    before = [t.clone() for t in ts]
    out = [torch.full_like(t, 7.0) for t in ts]
    assert la.la_grad_clip(ts, 0.25, out=out).item() == norm
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    c = 0.25 / (ref + 1e-6)
    for i, (t, o) in enumerate(zip(before, out)):
        r = t.double().cpu().numpy() * c
        tl = np.abs(r) * (torch.finfo(t.dtype).eps / 2 + tol + 4 * U) + 1e-38
        assert np.all(np.abs(o.double().cpu().numpy() - r) <= tl), i
    assert la.la_grad_clip(ts, 0.25).item() == norm
    assert all(torch.equal(a, b) for a, b in zip(ts, out))


@pytest.mark.parametrize("count", [1, 2, 32, 33, 512, 513, 1025])
def test_one_large_value_anywhere(count):
    """The largest value of a list decides its norm, whichever tensor holds it."""
    ts = [torch.zeros(3, device=DEV) for _ in range(count)]
    for at in {0, count // 2, count - 1}:
        ts[at][1] = 3.0
        assert la.la_grad_norm(ts).item() == 3.0
        out = [torch.full_like(t, 7.0) for t in ts]
        assert la.la_grad_clip(ts, 100.0, out=out).item() == 3.0
        assert all(torch.equal(a, b) for a, b in zip(ts, out))
        ts[at][1] = 0.0


def test_coinciding_tensors_are_refused():
    """And nothing is written."""
    a, b = torch.ones(10, device=DEV), torch.ones(10, device=DEV)
    for grads, out in (([a, b, a], None), ([a, b], [b, a]), ([a, b], [torch.empty_like(a)] * 2)):
        with pytest.raises(la.LAError):
            la.la_grad_clip(grads, 1.0, out=out)
    assert (a == 1.0).all() and (b == 1.0).all()
    assert la.la_grad_norm([a, b, a]).item() == pytest.approx(30 ** 0.5, rel=1e-6)     # reading twice is fine
    assert la.la_grad_clip([a, b], 1.0, out=[a, torch.empty_like(b)]).item() == pytest.approx(20 ** 0.5, rel=1e-6)
    none = torch.empty(0, device=DEV)
    la.la_grad_clip([none, a, none], 1e9)
