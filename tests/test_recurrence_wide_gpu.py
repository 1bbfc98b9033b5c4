"""The recurrence over rows of 2^29 channels and more, whose bytes pass 32 bits.

Every value is exact (small whole numbers, gates of 1/2, one product), so
equality is asked for."""
import pytest
import torch

from weight_recurrence_gb300 import la

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.lib()
    yield
    torch.cuda.empty_cache()


def _whole_numbers(shape, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-3, 4, shape, generator=g, device=DEV, dtype=torch.int8).to(dtype)


@pytest.mark.parametrize("dtype,D", [(torch.float32, (1 << 29) + 40), (torch.float32, (1 << 29) + 41),
                                     (torch.bfloat16, (1 << 30) + 72)])
def test_backward(D, dtype):
    dout = _whole_numbers((1, 1, D), dtype, 1)
    h0 = _whole_numbers((1, D), torch.float32, 2)
    g = torch.full_like(dout, 0.5)
    dh0 = torch.empty_like(h0)
    dx, dg = la.la_recurrence_backward(None, g, dout, dout, "decay", h0=h0, dh0=dh0)
    assert torch.equal(dx, dout)
    assert torch.equal(dg, (dout * h0).to(dtype))
    assert torch.equal(dh0, 0.5 * dout[:, 0].float())


def test_forward_in_tiles():
    D, N = (1 << 29) + 40, 17
    x = _whole_numbers((1, 1, D), torch.float32, 3)
    g = torch.full_like(x, 0.5)
    hN = torch.empty(1, D, device=DEV)
    out = la.la_recurrence_forward(x.expand(1, N, D), g.expand(1, N, D), "decay", hN=hN)
    h = torch.zeros(1, D, device=DEV)
    for t in range(N):
        h.mul_(0.5).add_(x[:, 0])
        assert torch.equal(out[:, t], h), t
    assert torch.equal(hN, h)
