"""The calls of a layer of decaying linear attention run together, as
examples/decay_layer.py has them: outputs and gradients against a plain fp64
program of the same layer, prompts then tokens against whole sequences."""
import importlib.util
import os

import pytest
import torch

from weight_recurrence_gb300 import la

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.lib()
    spec = importlib.util.spec_from_file_location("decay_layer", os.path.join(ROOT, "examples", "decay_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _plain(p, x, pos, log_decay, freq, scale, H, lens):
    """The layer in fp64 on the CPU, differentiable; the recurrence token by token."""
    B, N, C = x.shape
    D = C // H
    q, k, v = (x @ p["W"]).unflatten(-1, (3, H, D)).permute(2, 0, 3, 1, 4)

    def turn(t, w):
        t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w
        ang = (pos.double()[..., None] * freq)[:, None]
        a, b = t[..., :D // 2], t[..., D // 2:]
        return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)
    q, k = turn(q, p["wq"]), turn(k, p["wk"])
    a = log_decay.exp()[:, None, None]
    S, out = torch.zeros(B, H, D, D, dtype=torch.float64), []
    for t in range(N):
        live = (t < lens)[:, None, None, None]
        S = torch.where(live, a * S + k[:, :, t, :, None] * v[:, :, t, None, :], S)
        out.append(torch.where(live[..., 0], scale * torch.einsum("bhd,bhdm->bhm", q[:, :, t], S), 0.0))
    o = torch.stack(out, 2)
    mid = o - o.mean(-1, keepdim=True)
    n = mid / torch.sqrt((mid * mid).mean(-1, keepdim=True) + 1e-5) * p["wn"] + p["bn"]
    return n.transpose(1, 2).flatten(2) @ p["Wo"], S


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 2e-4), (torch.bfloat16, 6e-2)])
def test_outputs_and_gradients(example, dtype, tol):
    """Weights and inputs that bf16 holds exactly, so that only the layer's own roundings differ.  The tolerance: a
    handful of roundings of the type (2^-8) on the way, or fp32's sums and torch's fp32 products, relative to the
    largest value."""
    B, N, C, H = 2, 150, 128, 2
    layer = example.DecayLayer(C, H, dtype)
    g = torch.Generator().manual_seed(5)
    for n in layer.p:
        layer.p[n] = (layer.p[n] + 0.1 * torch.randn(layer.p[n].shape, generator=g).cuda()).bfloat16().float()
    x, dy = (torch.randn(B, N, C, generator=g).bfloat16() for _ in range(2))
    pos = torch.randint(0, 5000, (B, N), generator=g, dtype=torch.int32)
    lens = torch.tensor([N, 97], dtype=torch.int32)
    state = torch.zeros(B, H, C // H, C // H, device="cuda")
    y = layer.forward(x.to(dtype).cuda(), pos.cuda(), lens.cuda(), state)
    # rows past a length: their layer norm is of zeros, which is the bias alone
    d, dx = layer.backward(dy.to(dtype).cuda())

    p = {n: t.detach().double().cpu().requires_grad_() for n, t in layer.p.items()}
    xd = x.double().requires_grad_()
    ref, S = _plain(p, xd, pos, layer.log_decay.double().cpu(), layer.freq.double().cpu(), layer.scale, H, lens)
    (ref * dy.double()).sum().backward()

    def close(name, got, want, tol):
        want = want.detach()
        off = float((got.double().cpu() - want).abs().max() / want.abs().max())
        assert off < tol, (name, off)
    close("y", y, ref, tol)
    close("state", state, S, tol)
    for b, n in enumerate(lens.tolist()):
        close("dx", dx[b, :n], xd.grad[b, :n], 3 * tol)
    for n in d:
        close("d" + n, d[n], p[n].grad, 3 * tol)


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 6e-2)])
def test_prompts_then_tokens(example, dtype, tol):
    off, size = example.prompts_then_tokens(dtype=dtype)
    assert off < tol * size, (off, size)
