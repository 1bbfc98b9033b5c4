"""GPU parity of the global gradient norm and of clipping by it.

Tolerance: every square and sum is fp32 over positive terms, so the sum of
squares is within k u of itself with k the longest path of additions (n/32768
+ 64 is more than any here), u = 2^-24; the root halves that.  A clipped value
adds the factor's two roundings and its own half step."""
import math

import numpy as np
import pytest
import torch

from oracle import layer
from weight_recurrence_gb300 import la

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.lib()


def _grads(sizes, dtypes, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(scale * torch.randn(n, generator=g)).to(dtypes[i % len(dtypes)]).to(DEV) for i, n in enumerate(sizes)]


def _tol(ts):
    return (sum(t.numel() for t in ts) / 32768 + 70) * U


SETS = [[1], [7], [1024], [1025, 3, 0, 8191], [100000], [5] * 300, [65537, 1, 2, 1000003], [0, 0], list(range(1, 400)),
        [4096 * 1024 + 5] * 3]


@pytest.mark.parametrize("dtypes", [[torch.float32], [torch.bfloat16], [torch.bfloat16, torch.float32]])
@pytest.mark.parametrize("which", range(len(SETS)))
def test_norm_and_clip(which, dtypes):
    ts = _grads(SETS[which], dtypes, which)
    ref, tol = layer.global_norm(ts), _tol(ts)
    norm = la.la_grad_norm(ts)
    assert norm.shape == () and abs(norm.item() - ref) <= tol * ref
    before = [t.clone() for t in ts]
    out = [torch.full_like(t, 7.0) for t in ts]
    assert la.la_grad_clip(ts, 0.25, out=out).item() == norm.item()
    assert all(torch.equal(a, b) for a, b in zip(ts, before))       # out of place leaves the gradients
    c = min(1.0, 0.25 / (ref + 1e-6))
    for t, o in zip(before, out):
        r = t.double().cpu().numpy() * c
        assert np.all(np.abs(o.double().cpu().numpy() - r) <= np.abs(r) * (torch.finfo(t.dtype).eps / 2 + tol + 4 * U) + 1e-38)
    assert la.la_grad_clip(ts, 0.25).item() == norm.item()          # in place
    assert all(torch.equal(a, b) for a, b in zip(ts, out))


def test_small_norms_are_left_alone():
    ts = _grads([100, 2000], [torch.float32], 3)
    before = [t.clone() for t in ts]
    la.la_grad_clip(ts, 1e6)
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    la.la_grad_clip(ts, float("inf"))
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    la.la_grad_clip(ts, 0.0)
    assert not any(t.any() for t in ts)


def test_zeros():
    ts = [torch.zeros(50, device=DEV), torch.zeros(3, dtype=torch.bfloat16, device=DEV)]
    assert la.la_grad_clip(ts, 1.0).item() == 0.0
    assert not any(t.any() for t in ts)


def test_nan_and_infinity():
    ts = _grads([300, 40], [torch.float32], 4)
    ts[1][7] = float("inf")
    out = [torch.empty_like(t) for t in ts]
    assert math.isinf(la.la_grad_clip(ts, 1.0, out=out).item())
    assert not out[0].any() and math.isnan(out[1][7].item()) and not out[1][:7].any()
    ts[0][0] = float("nan")
    assert math.isnan(la.la_grad_clip(ts, 1.0, out=out).item())
    assert all(torch.isnan(t).all() for t in out)


@pytest.mark.parametrize("off", [1, 2, 3, 5])
def test_unaligned_views(off):
    """Slices of one buffer at odd offsets, source and destination not alike."""
    for dtype in (torch.float32, torch.bfloat16):
        buf = _grads([9000], [dtype], off)[0]
        dst = torch.full_like(buf, 7.0)
        cuts = [(off, 1000 + off), (1000 + off, 1001 + off), (1001 + off, 8000)]
        ts = [buf[a:b] for a, b in cuts]
        norm = la.la_grad_clip(ts, 0.5, out=[dst[a + 1:b + 1] for a, b in cuts])
        ref = layer.global_norm(ts)
        assert abs(norm.item() - ref) <= _tol(ts) * ref
        want = [torch.empty_like(t) for t in ts]
        la.la_grad_clip(ts, 0.5, out=want)
        assert torch.equal(dst[off + 1:8001], torch.cat(want))
        assert (dst[:off + 1] == 7.0).all() and (dst[8001:] == 7.0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("off", [0, 1, 3, 7])
def test_long_tensors_at_odd_offsets(off, dtype):
    """Many chunks of a tensor that starts between 16-byte boundaries, to a
    destination that starts alike and to one that does not."""
    n = 300007
    buf = _grads([n + 16], [dtype], 10 + off)[0]
    ts = [buf[off:off + n]]
    ref, tol = layer.global_norm(ts), _tol(ts)
    assert abs(la.la_grad_norm(ts).item() - ref) <= tol * ref
    r = ts[0].double().cpu().numpy() * (0.5 / (ref + 1e-6))
    for to in (off, off + 2):
        dst = torch.full_like(buf, 7.0)
        la.la_grad_clip(ts, 0.5, out=[dst[to:to + n]])
        err = np.abs(dst[to:to + n].double().cpu().numpy() - r)
        assert np.all(err <= np.abs(r) * (torch.finfo(dtype).eps / 2 + tol + 4 * U) + 1e-38)
        assert (dst[:to] == 7.0).all() and (dst[to + n:] == 7.0).all()


def test_past_32_bits():
    """One tensor of more than 2^31 values."""
    n = (1 << 31) + 4099
    t = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    t[-1], t[0], t[1 << 31] = 3.0, 4.0, 12.0
    assert la.la_grad_clip([t], 6.5).item() == 13.0
    assert (t[-1].item(), t[0].item(), t[1 << 31].item()) == (1.5, 2.0, 6.0)
    assert torch.count_nonzero(t).item() == 3


def test_equal_calls_give_equal_bits_and_streams_and_graphs():
    ts = _grads([70001, 33, 512 * 512], [torch.bfloat16, torch.float32], 6)
    out = [torch.empty_like(t) for t in ts]
    norms = {la.la_grad_clip(ts, 1.0, out=out).item() for _ in range(5)}
    assert len(norms) == 1
    want = [o.clone() for o in out]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    assert la.la_grad_clip(ts, 1.0, out=out, stream=side).item() in norms
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = la.la_grad_clip(ts, 1.0, out=out)
    for o in out:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert norm.item() in norms and all(torch.equal(a, b) for a, b in zip(out, want))
