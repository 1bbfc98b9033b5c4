"""The recurrence where gates or values are not finite, or gates exceed 1: the
kernels group tokens and join the groups by products of gates, and what a
token-by-token walk gives has to come out all the same.

References are oracle/layer.py's walk in 64 bits.  Which values are NaN and
which infinite follows from the formula alone.  The growing cases are built
from powers of two (gates, inputs and states, all within fp32's and bf16's
normal range and never a sum of two), so every product is exact, and equality
is asked for."""
import numpy as np
import pytest
import torch

from oracle import layer
from weight_recurrence_gb300 import la

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DTYPES = [torch.float32, torch.bfloat16]
# (B, H, N, D): whole sequences, several tiles, sequences cut into segments, more strips than SMs
SIZES = [(1, 1, 17, 20), (2, 1, 100, 100), (1, 1, 100, 64), (1, 1, 400, 400), (2, 3, 1500, 72), (1, 1, 2500, 33),
         (1, 160, 300, 48)]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.lib()


def _to(a, dtype):
    return torch.from_numpy(np.array(a, order="C")).to(dtype).to(DEV)


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _places(N, D):
    """A token for each channel, spread over all positions of tiles and segments."""
    return (np.arange(D) * max(1, N // D) + np.arange(D) // max(1, D // 7)) % N


def _same_kind(name, got, ref):
    """NaN where the reference is, infinities of its sign where it has them, finite elsewhere."""
    got = _np(got)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref), err_msg=name)
    np.testing.assert_array_equal(np.where(np.isinf(got), np.sign(got), 0), np.where(np.isinf(ref), np.sign(ref), 0),
                                  err_msg=name)


def _run(x, g, gate, dout, h0, dhN):
    hN, dh0 = torch.empty(x.shape[:2] + x.shape[3:], device=DEV), torch.empty(x.shape[:2] + x.shape[3:], device=DEV)
    out = la.la_recurrence_forward(x, g, gate, h0=h0, hN=hN)
    dx, dg = la.la_recurrence_backward(x, g, out, dout, gate, h0=h0, dhN=dhN, dh0=dh0)
    torch.cuda.synchronize()
    return out, hN, dx, dg, dh0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("with_state", [True, False])
@pytest.mark.parametrize("which,gate,value", [("g", "decay", np.nan), ("g", "log", np.nan), ("g", "sigmoid", np.nan),
                                              ("x", "decay", np.nan), ("g", "decay", np.inf), ("g", "decay", -np.inf),
                                              ("g", "log", np.inf), ("x", "decay", np.inf), ("x", "log", -np.inf)])
@pytest.mark.parametrize("B,H,N,D", SIZES)
def test_one_value_that_is_not_finite(B, H, N, D, which, gate, value, with_state, dtype):
    """One in every channel, at another token in each: everything after it shows it
    and nothing before it or beside it does."""
    rng = np.random.default_rng(N + D)
    x, dout = rng.standard_normal((2, B, H, N, D))
    g = rng.uniform(0.05, 0.3, (B, H, N, D))       # short memories: products of gates fall below fp32
    if gate == "log":
        g = np.log(g)
    elif gate == "sigmoid":
        g = np.log(g / (1 - g))
    (g if which == "g" else x)[:, :, _places(N, D), np.arange(D)] = value
    x, g, dout = (_to(t, dtype) for t in (x, g, dout))
    h0 = dhN = None
    if with_state:
        h0, dhN = (_to(t, torch.float32) for t in rng.standard_normal((2, B, H, D)))
    got = _run(x, g, gate, dout, h0, dhN)
    with np.errstate(invalid="ignore"):
        out, hN = layer.recurrence(x, g, gate, h0)
        dx, dg, dh0 = layer.recurrence_backward(x, g, gate, dout, h0, dhN, out=_np(got[0]))
    for name, a, r in zip(("out", "hN", "dx", "dg", "dh0"), got, (out, hN, dx, dg, dh0)):
        _same_kind(name, a, r)


def _growing(B, H, N, D, period=50):
    """Gates of 2^8 for 25 tokens after a gate of 0, then of 1; each channel starts
    elsewhere in the period.  A product over 16 tokens is past fp32's range, over
    the gate of 0 too."""
    at = (np.arange(N)[:, None] + 3 * np.arange(D)[None, :]) % period
    g = np.where(at == 0, 0.0, np.where(at <= 25, 256.0, 1.0))
    return [np.broadcast_to(v, (B, H, N, D)) for v in (g, np.where(at == 0, 2.0 ** -100, 0.0))]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,H,N,D", SIZES)
def test_growing_gates_with_resets(B, H, N, D, dtype):
    g, x = _growing(B, H, N, D)
    h0 = np.where(np.arange(D) % 2, 2.0 ** -120, -2.0 ** -110) * np.ones((B, H, D))
    ref, hN = layer.recurrence(x, g, "decay", h0)
    # the backward's carry starts again before a gate of 0
    dout, dhN = np.zeros_like(x), np.full((B, H, D), 2.0 ** -100)
    dout[:, :, :-1] = np.where(g[:, :, 1:] == 0.0, 2.0 ** -100, 0.0)
    ones, one = np.ones_like(x), np.ones((B, H, D))     # h_{t-1}, as the backward is given it: dg = l
    rx, rg, rh = layer.recurrence_backward(x, g, "decay", dout, one, dhN, out=ones)
    assert np.abs(ref).max() < 2.0 ** 120 and np.abs(rx).max() < 2.0 ** 120
    got_h, got_l = torch.empty(B, H, D, device=DEV), torch.empty(B, H, D, device=DEV)
    gates = _to(g, dtype)
    out = la.la_recurrence_forward(_to(x, dtype), gates, "decay", h0=_to(h0, torch.float32), hN=got_h)
    dx, dg = la.la_recurrence_backward(None, gates, _to(ones, dtype), _to(dout, dtype), "decay",
                                       h0=_to(one, torch.float32), dhN=_to(dhN, torch.float32), dh0=got_l)
    torch.cuda.synchronize()
    for name, a, r in (("out", out, ref), ("hN", got_h, hN), ("dx", dx, rx), ("dg", dg, rg), ("dh0", got_l, rh)):
        np.testing.assert_array_equal(_np(a), r, err_msg=name)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [64, 100, 1500])
def test_a_small_state_that_grows(N, dtype):
    """h0 = 2^-100 and gates of 4 for 100 tokens: 2^100, past which gates are 1."""
    x = torch.zeros(1, 1, N, 64, dtype=dtype, device=DEV)
    g = torch.full_like(x, 4.0)
    g[:, :, 100:] = 1.0
    h0, hN = torch.full((1, 1, 64), 2.0 ** -100, device=DEV), torch.empty(1, 1, 64, device=DEV)
    out = la.la_recurrence_forward(x, g, "decay", h0=h0, hN=hN)
    ref = 2.0 ** (2.0 * np.minimum(np.arange(1, N + 1), 100) - 100)
    np.testing.assert_array_equal(_np(out)[0, 0], np.broadcast_to(ref[:, None], (N, 64)))
    np.testing.assert_array_equal(_np(hN)[0, 0], np.full(64, ref[-1]))
