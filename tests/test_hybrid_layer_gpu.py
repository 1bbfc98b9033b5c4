"""The example layer (examples/hybrid_layer.py): its hand-written gradients
against autograd in 64 bits on the CPU, a training run, and decoding."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import hybrid_layer  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _reference(p, x, heads):
    """The layer's formulas in torch fp64."""
    def ln(s, w, b):
        m = s - s.mean(-1, keepdim=True)
        return m / (m.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w + b
    y1 = ln(x, p["w1"], p["b1"])
    u, a = y1 @ p["Wx"], torch.sigmoid(y1 @ p["Wg"])
    h, hs = torch.zeros_like(x[:, 0]), []
    for t in range(x.shape[1]):
        h = a[:, t] * h + (1 - a[:, t]) * u[:, t]
        hs.append(h)
    s2 = x + torch.stack(hs, 1) @ p["Wh"]
    y2 = ln(s2, p["w2"], p["b2"])
    B, N, C = x.shape
    q, k, v = ((y2 @ p[n]).view(B, N, heads, -1).transpose(1, 2) for n in ("Wq", "Wk", "Wv"))
    A = torch.tril((torch.nn.functional.elu(q) + 1) @ (torch.nn.functional.elu(k) + 1).transpose(2, 3))
    o = (A @ v / A.sum(-1, keepdim=True)).transpose(1, 2).reshape(B, N, C)
    return ln(s2 + o @ p["Wo"], p["w3"], p["b3"])


def test_gradients_against_autograd():
    B, N, C, heads = 2, 40, 32, 2
    layer = hybrid_layer.HybridLayer(C, heads, seed=5)
    x, dy = (torch.randn(B, N, C, generator=torch.Generator().manual_seed(i)).cuda() for i in (1, 2))
    y = layer.forward(x)
    d, dx = layer.backward(dy)
    p = {n: w.double().cpu().requires_grad_() for n, w in layer.p.items()}
    x64 = x.double().cpu().requires_grad_()
    y64 = _reference(p, x64, heads)
    (y64 * dy.double().cpu()).sum().backward()
    # fp32 kernels and products: a few hundred roundings of 2^-24 between x and any of these
    assert (y.double().cpu() - y64).norm() <= 1e-4 * y64.norm()
    assert (dx.double().cpu() - x64.grad).norm() <= 1e-4 * x64.grad.norm()
    for n, w in p.items():
        assert (d[n].double().cpu() - w.grad).norm() <= 1e-4 * w.grad.norm(), n


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-3), (torch.bfloat16, 0.3)])
def test_trains_and_decodes(dtype, tol):
    losses, off = hybrid_layer.train(steps=30, dtype=dtype)
    assert sum(losses[-5:]) < 0.8 * sum(losses[:5]), losses
    assert off <= tol
