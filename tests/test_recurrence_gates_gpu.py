"""Gates of fp32 calls over their whole range, and what the backward's reading of
a rounded output costs bf16 calls.

u = 2^-24.  A gate of fp32 data is e^g or 1/(1 + e^g) by the hardware's 2^x (off by
2^-22, 4 u) and 1/x (2^-23, 2 u), with the argument's rounding made good to below
u; the sum 1 + e^g, the product with x or h, its own sum and the store round once
each (u/2 of fp32's 2 u spacing counts as u here): 12 u in all, beside values
under fp32's normal range, which count as 0."""
import numpy as np
import pytest
import torch

from oracle import layer
from weight_recurrence_gb300 import la

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
TINY = 2.0 ** -126


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.lib()


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _near(got, ref, steps, name):
    off = np.abs(_np(got) - ref) / (steps * U * np.abs(ref) + TINY)
    assert off.max() <= 1.0, (name, off.max(), np.unravel_index(off.argmax(), off.shape))


@pytest.mark.parametrize("N", [1, 40])
@pytest.mark.parametrize("D", [512, 511])
@pytest.mark.parametrize("gate", ["sigmoid", "log"])
def test_fp32_gates_over_their_range(gate, D, N):
    """Tokens that see nothing before them: out = (1 - a) x, or a h0 with x = 0; and
    the backward's dx = (1 - a) dout."""
    g = torch.linspace(-85.0, 85.0 if gate == "sigmoid" else 0.0, D, device=DEV).repeat(1, 1, N, 1)
    rng = torch.Generator().manual_seed(D)
    x, h0 = (0.5 + torch.rand((1, 1, n, D), generator=rng).to(DEV) for n in (N, 1))
    a, w = layer.gate_factors(gate, _np(g))
    first = torch.zeros_like(x)
    first[:, :, 0] = 1.0                                   # only the first token has a value
    h0 = h0[:, :, 0].contiguous()
    out = la.la_recurrence_forward(torch.zeros_like(x), g, gate, h0=h0)
    _near(out[:, :, 0], a[:, :, 0] * _np(h0), 12, "a h0")
    out = la.la_recurrence_forward(x * first, g, gate)
    _near(out[:, :, 0], (w * _np(x))[:, :, 0], 12, "(1 - a) x")
    last = first.flip(2)
    dx, dg = la.la_recurrence_backward(x, g, torch.zeros_like(x), x * last, gate)
    _near(dx[:, :, -1], (w * _np(x))[:, :, -1], 12, "dx")


@pytest.mark.parametrize("gate", ["decay", "log", "sigmoid"])
def test_bf16_gradient_of_the_gate_against_the_unrounded_state(gate):
    """The backward has h_{t-1} as the forward stored it, within half a step (2^-8
    of its size).  Beside that dg rounds once itself, and the fp32 sums are off by
    what test_recurrence_gpu.py derives for them."""
    B, H, N, D = 2, 2, 700, 72
    rng = torch.Generator().manual_seed(5)
    x, g, dout = torch.randn((3, B, H, N, D), generator=rng)
    g = {"decay": torch.sigmoid(2 + g), "log": -torch.exp(-2 + g), "sigmoid": 2 + 2 * g}[gate]
    x, g, dout = (t.bfloat16().to(DEV) for t in (x, g, dout))
    h0 = torch.randn((B, H, D), generator=rng).to(DEV)
    out = la.la_recurrence_forward(x, g, gate, h0=h0)
    dx, dg = la.la_recurrence_backward(x, g, out, dout, gate, h0=h0)
    xs, ds = _np(x), _np(dout)
    a, w = layer.gate_factors(gate, _np(g))
    h, _ = layer.recurrence(x, g, gate, h0)
    _, rg, _ = layer.recurrence_backward(x, g, gate, dout, h0)        # of the exact states
    before = np.concatenate([_np(h0)[:, :, None], h[:, :, :-1]], axis=2)
    # |lambda| with all terms added, and the error's majorants of lambda and of h
    lam, ml, mh = np.zeros_like(xs), np.zeros_like(xs), np.zeros_like(xs)
    cl, cm = np.zeros((B, H, D)), np.zeros((B, H, D))
    for t in range(N - 1, -1, -1):
        cl = np.abs(ds[:, :, t]) + cl
        cm = cm + cl
        lam[:, :, t], ml[:, :, t] = cl, cm
        cl = a[:, :, t] * cl
        cm = a[:, :, t] * cm + cl
    ch, cm = np.abs(_np(h0)), np.abs(_np(h0))
    for t in range(N):
        mh[:, :, t] = cm                                              # of h_{t-1}
        ch = a[:, :, t] * ch + np.abs(w[:, :, t] * xs[:, :, t])
        cm = a[:, :, t] * cm + ch
    slope = {"decay": np.ones_like(a), "log": a, "sigmoid": a * w}[gate]
    half = torch.finfo(torch.bfloat16).eps / 2
    size = np.abs(before) + (np.abs(xs) if gate == "sigmoid" else 0.0)
    fp32 = 2 * 16 * U * slope * ((ml + lam) * size + lam * mh)
    tol = half * np.abs(rg) + (1 + half) * (half * lam * slope * np.abs(before) + fp32) + 1e-30
    off = np.abs(_np(dg) - rg) / tol
    assert off.max() <= 1.0, off.max()
