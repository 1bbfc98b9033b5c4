"""GPU parity of the gated linear recurrence (forward, single step, backward)
against the fp64 oracle (oracle/layer.py).

Tolerances, element by element.  With u = 2^-24 and Habs the recurrence run on
absolute values (Habs_t = |a_t| Habs_{t-1} + |u_t|), every rounding at token s
(of a_s, of u_s, of a product of gates that contains a_s, of a sum) is at most
a few u times Habs_s and reaches token t through the gates between: the error
is at most k u M_t with M_t = |a_t| M_{t-1} + Habs_t, whatever the grouping.
k = 16 covers a and w from the exponential (3 ulp = 6 u each), the product
w x, a product of gates and the sums of a scan level by level.  The output's
own rounding adds half a step.  The backward runs the same recurrence on dout;
its h_{t-1} is read from the forward's stored output, so the reference is
given that output too.
"""
import numpy as np
import pytest
import torch

from oracle import layer
from weight_recurrence_gb300 import la

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
K = 16
GATES = ["decay", "log", "sigmoid"]
DTYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.lib()


def _inputs(B, H, N, D, dtype, gate, seed, mean=2.0):
    rng = torch.Generator().manual_seed(seed)
    n = torch.randn((B, H, N, D), generator=rng)
    if gate == "sigmoid":
        g = mean + 2.0 * n
    elif gate == "log":
        g = -torch.exp(-mean + n)
    else:
        g = torch.where(n > 2.2, 0.0, 1.0 - torch.exp(-mean - n.abs())) * torch.where(n < -2.0, -1.0, 1.0)
    x, dout = torch.randn((2, B, H, N, D), generator=rng)
    h0, dhN = torch.randn((2, B, H, D), generator=rng)
    return [t.to(dtype).to(DEV) for t in (x, g, dout)] + [h0.to(DEV), dhN.to(DEV)]


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _majorants(x, g, gate, h0, lens=None):
    """Habs and M of the module's docstring, [B,H,N,D], and their last values."""
    a, w = layer.gate_factors(gate, g)
    B, H, N, D = x.shape
    hab, m = np.zeros_like(x), np.zeros_like(x)
    ch, cm = np.abs(h0).copy(), np.abs(h0).copy()
    for b in range(B):
        for t in range(N if lens is None else min(max(int(lens[b]), 0), N)):
            ch[b] = np.abs(a[b, :, t]) * ch[b] + np.abs(w[b, :, t] * x[b, :, t])
            cm[b] = np.abs(a[b, :, t]) * cm[b] + ch[b]
            hab[b, :, t], m[b, :, t] = ch[b], cm[b]
    return hab, m, ch, cm


def _half(dtype, ref):
    return torch.finfo(dtype).eps / 2 * np.abs(ref) + 1e-38


def _close(name, got, ref, tol):
    got = _np(got)
    assert got.shape == ref.shape, name
    assert np.isfinite(got).all(), name
    worst = np.abs(got - ref) / tol
    assert worst.max(initial=0.0) <= 1.0, (name, float(worst.max()), np.unravel_index(worst.argmax(), worst.shape))


def check_forward(x, g, gate, h0, lens, out, hN):
    xs, gs, hs = _np(x), _np(g), np.zeros(x.shape[:2] + x.shape[3:]) if h0 is None else _np(h0)
    ref, hr = layer.recurrence(xs, gs, gate, hs, lens)
    _, m, _, cm = _majorants(xs, gs, gate, hs, lens)
    _close("out", out, ref, _half(x.dtype, ref) + 2 * K * U * m)
    if hN is not None:
        _close("hN", hN, hr, _half(torch.float32, hr) + K * U * cm)


def check_backward(x, g, gate, dout, h0, dhN, lens, out, dx, dg, dh0):
    xs, gs, ds, os_ = _np(x), _np(g), _np(dout), _np(out)
    z = np.zeros(x.shape[:2] + x.shape[3:])
    hs, dh = z if h0 is None else _np(h0), z if dhN is None else _np(dhN)
    rx, rg, rh = layer.recurrence_backward(xs, gs, gate, ds, hs, dh, lens, out=os_)
    a, w = layer.gate_factors(gate, gs)
    B, H, N, D = xs.shape
    lab, ml, cl, cml = np.zeros_like(xs), np.zeros_like(xs), np.abs(dh).copy(), np.abs(dh).copy()
    for b in range(B):
        for t in range((N if lens is None else min(max(int(lens[b]), 0), N)) - 1, -1, -1):
            cl[b] = np.abs(ds[b, :, t]) + cl[b]
            cml[b] = cml[b] + cl[b]
            lab[b, :, t], ml[b, :, t] = cl[b], cml[b]
            cl[b] = np.abs(a[b, :, t]) * cl[b]
            cml[b] = np.abs(a[b, :, t]) * cml[b] + cl[b]
    _close("dx", dx, rx, _half(x.dtype, rx) + 2 * K * U * ml * w)
    before = np.concatenate([hs[:, :, None], os_[:, :, :-1]], axis=2)
    size = np.abs(before) + (np.abs(xs) if gate == "sigmoid" else 0.0)
    slope = {"decay": np.ones_like(a), "log": a, "sigmoid": a * w}[gate]
    _close("dg", dg, rg, _half(x.dtype, rg) + 2 * K * U * (ml + lab) * size * np.abs(slope))
    if dh0 is not None:
        _close("dh0", dh0, rh, _half(torch.float32, rh) + K * U * cml)


def _both(x, g, dout, gate, h0=None, dhN=None, lens=None, want_states=True):
    hN = torch.empty(x.shape[:2] + x.shape[3:], device=DEV) if want_states else None
    dh0 = torch.empty_like(hN) if want_states else None
    dl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = la.la_recurrence_forward(x, g, gate, h0=h0, hN=hN, lens=dl)
    dx, dg = la.la_recurrence_backward(x, g, out, dout, gate, h0=h0, dhN=dhN, dh0=dh0, lens=dl)
    torch.cuda.synchronize()
    check_forward(x, g, gate, h0, lens, out, hN)
    check_backward(x, g, gate, dout, h0, dhN, lens, out, dx, dg, dh0)
    return out, hN, dx, dg, dh0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("B,H,N,D", [(1, 1, 1, 1), (2, 3, 1, 16), (1, 1, 2, 33), (2, 1, 7, 5), (3, 2, 64, 64),
                                     (1, 2, 65, 128), (2, 1, 129, 200), (1, 1, 1000, 130), (5, 1, 300, 257),
                                     (2, 1, 16, 40), (2, 1, 17, 40), (1, 1, 128, 70), (1, 1, 256, 70), (1, 1, 257, 70),
                                     (3, 1, 513, 333)])
def test_parity(B, H, N, D, gate, dtype):
    x, g, dout, h0, dhN = _inputs(B, H, N, D, dtype, gate, B * 1000 + N + D)
    _both(x, g, dout, gate, h0, dhN)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,H,N,D", [(1, 1, 5000, 64), (1, 1, 4097, 1000), (2, 2, 3333, 32), (40, 4, 600, 128)])
def test_parity_long_memories(B, H, N, D, dtype):
    """Gates next to 1: the state at the end holds thousands of tokens."""
    x, g, dout, h0, dhN = _inputs(B, H, N, D, dtype, "sigmoid", N + D, mean=6.0)
    _both(x, g, dout, "sigmoid", h0, dhN)


def test_without_states():
    x, g, dout, _, _ = _inputs(2, 2, 150, 48, torch.bfloat16, "sigmoid", 3)
    _both(x, g, dout, "sigmoid", want_states=False)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,D", [(37, 16), (300, 40), (2100, 64)])
def test_lengths(N, D, dtype):
    """Rows past a length are 0 in every output and never read, NaN or not."""
    lens = [0, 1, N, N // 2, N + 9, -3]
    x, g, dout, h0, dhN = _inputs(6, 2, N, D, dtype, "sigmoid", N)
    for b, n in enumerate(lens):
        for t in (x, g, dout):
            t[b, :, min(max(n, 0), N):] = float("nan")
    hN, dh0 = torch.empty_like(h0), torch.empty_like(h0)
    dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = la.la_recurrence_forward(x, g, h0=h0, hN=hN, lens=dl)
    dx, dg = la.la_recurrence_backward(x, g, out, dout, h0=h0, dhN=dhN, dh0=dh0, lens=dl)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        n = min(max(n, 0), N)
        for t in (out, dx, dg):
            assert not t[b, :, n:].float().abs().sum().item()
        x[b, :, n:] = g[b, :, n:] = dout[b, :, n:] = 0.0
        if n == 0:
            assert torch.equal(hN[b], h0[b]) and torch.equal(dh0[b], dhN[b])
    check_forward(x, g, "sigmoid", h0, lens, out, hN)
    check_backward(x, g, "sigmoid", dout, h0, dhN, lens, out, dx, dg, dh0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [131, 700])
@pytest.mark.parametrize("D,off", [(64, 0), (64, 1), (40, 3), (33, 0)])
def test_views(D, off, N, dtype):
    """Token-major projections, odd offsets, a repeated input, outputs as views."""
    B, H = 2, 3
    x, g, dout, h0, dhN = _inputs(B, H, N, D, dtype, "sigmoid", 77 + off)
    both = torch.zeros(B, N, H, 2 * D + 5, dtype=dtype, device=DEV)
    both[..., off:off + D] = x.transpose(1, 2)
    both[..., off + D:off + 2 * D] = g.transpose(1, 2)
    xv, gv = (both[..., off + i * D:off + (i + 1) * D].transpose(1, 2) for i in (0, 1))
    grads = torch.full_like(both, 7.0)
    dxv, dgv = (grads[..., off + i * D:off + (i + 1) * D].transpose(1, 2) for i in (0, 1))
    dv = dout[:1].expand(B, H, N, D)          # one gradient for every batch entry
    ov = torch.full((B, H, N, D + 3), 7.0, dtype=dtype, device=DEV)[..., 1:1 + D]
    hN, dh0 = torch.empty_like(h0), torch.empty_like(h0)
    la.la_recurrence_forward(xv, gv, out=ov, h0=h0, hN=hN)
    la.la_recurrence_backward(xv, gv, ov, dv, h0=h0, dhN=dhN, dh0=dh0, dx=dxv, dg=dgv)
    torch.cuda.synchronize()
    check_forward(xv, gv, "sigmoid", h0, None, ov, hN)
    check_backward(xv, gv, "sigmoid", dv, h0, dhN, None, ov, dxv, dgv, dh0)
    for n in (off, 5 - off):                  # what lies around the views is left alone
        edge = grads[..., :off] if n is off else grads[..., off + 2 * D:]
        assert (edge == 7.0).all()


def test_three_dimensions_equal_one_head():
    x, g, dout, h0, _ = _inputs(3, 1, 70, 24, torch.float32, "log", 5)
    a = la.la_recurrence_forward(x, g, "log", h0=h0)
    b = la.la_recurrence_forward(x[:, 0], g[:, 0], "log", h0=h0[:, 0].contiguous())
    assert torch.equal(a[:, 0], b)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("shape", [(1, 1), (64, 1024), (3, 5, 33), (2, 4, 64)])
def test_step_equals_one_token(shape, gate, dtype):
    B, D = shape[0], shape[-1]
    H = shape[1] if len(shape) == 3 else 1
    x, g, _, h0, _ = _inputs(B, H, 1, D, dtype, gate, 9)
    h = h0.clone().reshape(shape)
    y = la.la_recurrence_step(x.reshape(shape), g.reshape(shape), h, gate)
    torch.cuda.synchronize()
    check_forward(x, g, gate, h0, None, y.reshape(x.shape), h.reshape(h0.shape))


def test_steps_continue_a_prefill():
    B, D, N, T = 4, 96, 200, 12
    x, g, _, h0, _ = _inputs(B, 1, N + T, D, torch.bfloat16, "sigmoid", 21)
    h = h0.clone()
    first = la.la_recurrence_forward(x[:, :, :N], g[:, :, :N], h0=h, hN=h)
    rest = [la.la_recurrence_step(x[:, 0, t], g[:, 0, t], h[:, 0]) for t in range(N, N + T)]
    out = torch.cat([first] + [y[:, None, None] for y in rest], dim=2)
    torch.cuda.synchronize()
    check_forward(x, g, "sigmoid", h0, None, out, h)


def test_segments_chain():
    """Two segments joined by the state and its gradient are the whole sequence."""
    x, g, dout, h0, dhN = _inputs(2, 1, 500, 72, torch.float32, "log", 31)
    cut = 211
    mid, last = torch.empty_like(h0), torch.empty_like(h0)
    parts = [(slice(0, cut), h0, mid), (slice(cut, 500), mid, last)]
    outs = [la.la_recurrence_forward(x[:, :, s], g[:, :, s], "log", h0=a, hN=b) for s, a, b in parts]
    carry = dhN.clone()
    grads = []
    for (s, a, _), o in reversed(list(zip(parts, outs))):
        grads.insert(0, la.la_recurrence_backward(x[:, :, s], g[:, :, s], o, dout[:, :, s], "log", h0=a, dhN=carry,
                                                  dh0=carry))
    torch.cuda.synchronize()
    out = torch.cat(outs, dim=2)
    check_forward(x, g, "log", h0, None, out, last)
    dx, dg = (torch.cat(p, dim=2) for p in zip(*grads))
    check_backward(x, g, "log", dout, h0, dhN, None, out, dx, dg, carry)


@pytest.mark.parametrize("N", [1, 70, 1200])
@pytest.mark.parametrize("D", [3, 64])
def test_closed_and_open_gates(N, D):
    """a = 0 forgets everything before it exactly, a = 1 keeps everything."""
    x, _, _, h0, _ = _inputs(1, 1, N, D, torch.float32, "log", 41)
    big = 1e30 * torch.ones_like(h0)
    for gate, v in (("decay", 0.0), ("log", float("-inf")), ("sigmoid", float("-inf")), ("sigmoid", -200.0)):
        out = la.la_recurrence_forward(x, torch.full_like(x, v), gate, h0=big)
        assert torch.equal(out, x), (gate, v)
    for gate, v in (("decay", 1.0), ("log", 0.0)):
        out = la.la_recurrence_forward(torch.zeros_like(x), torch.full_like(x, v), gate, h0=h0)
        assert torch.equal(out, h0[:, :, None].expand_as(x)), gate
    for v in (float("inf"), 200.0):
        out = la.la_recurrence_forward(x, torch.full_like(x, v), "sigmoid", h0=h0)
        assert torch.equal(out, h0[:, :, None].expand_as(x)), v


def test_growing_gates_over_zeros_stay_zero():
    """Products of gates past fp32's range do not turn an empty state into NaN."""
    x = torch.zeros(1, 1, 900, 40, device=DEV)
    g = torch.full_like(x, 1e6)
    hN = torch.empty(1, 1, 40, device=DEV)
    out = la.la_recurrence_forward(x, g, "decay", hN=hN)
    dx, dg = la.la_recurrence_backward(None, g, out, x, "decay")
    for t in (out, hN, dx, dg):
        assert not t.any() and not torch.isnan(t).any()


def test_nan_spreads_forward_only():
    x, g, dout, h0, _ = _inputs(1, 1, 400, 36, torch.float32, "sigmoid", 51)
    clean = la.la_recurrence_forward(x, g, h0=h0)
    x[0, 0, 250, 7] = float("nan")
    out = la.la_recurrence_forward(x, g, h0=h0)
    assert torch.isnan(out[0, 0, 250:, 7]).all()
    out[0, 0, 250:, 7] = clean[0, 0, 250:, 7]
    assert torch.equal(out, clean)
    g[0, 0, 100, 3] = float("nan")
    out = la.la_recurrence_forward(x, g, h0=h0)
    assert torch.isnan(out[0, 0, 100:, 3]).all() and not torch.isnan(out[0, 0, :100, 3]).any()


def test_empty_calls():
    h0 = torch.randn(2, 8, device=DEV)
    hN = torch.empty_like(h0)
    x = torch.empty(2, 0, 8, device=DEV)
    assert la.la_recurrence_forward(x, x, h0=h0, hN=hN).shape == x.shape
    assert torch.equal(hN, h0)
    la.la_recurrence_forward(x, x, hN=hN)
    assert not hN.any()
    la.la_recurrence_backward(x, x, x, x, dhN=h0, dh0=hN)
    assert torch.equal(hN, h0)
    none = torch.empty(0, 5, 8, device=DEV)
    assert la.la_recurrence_forward(none, none).shape == none.shape


def test_offsets_past_32_bits():
    """Token strides that put the last rows past 2^31 elements."""
    N, D, stride = 33000, 16, 70000
    buf = torch.empty(N * stride, dtype=torch.bfloat16, device=DEV)   # 4.6 GB
    views = [buf.as_strided((1, 1, N, D), (0, 0, stride, 1), i * D) for i in range(5)]
    rng = torch.Generator(device=DEV).manual_seed(1)
    ref = [torch.randn((1, 1, N, D), generator=rng, device=DEV).to(torch.bfloat16) + (2.0 if i == 1 else 0.0)
           for i in range(3)]
    for v, r in zip(views, ref):
        v.copy_(r)
    out = la.la_recurrence_forward(views[0], views[1])
    assert torch.equal(out, la.la_recurrence_forward(ref[0], ref[1]))
    la.la_recurrence_backward(views[0], views[1], out, views[2], dx=views[3], dg=views[4])
    dx, dg = la.la_recurrence_backward(ref[0], ref[1], out, ref[2])
    assert torch.equal(views[3], dx) and torch.equal(views[4], dg)


def test_equal_calls_give_equal_bits():
    x, g, dout, h0, dhN = _inputs(2, 1, 3001, 136, torch.bfloat16, "sigmoid", 61)
    runs = []
    for _ in range(3):
        out = la.la_recurrence_forward(x, g, h0=h0)
        runs.append((out,) + la.la_recurrence_backward(x, g, out, dout, h0=h0, dhN=dhN))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_on_a_side_stream():
    x, g, dout, h0, dhN = _inputs(2, 2, 700, 64, torch.bfloat16, "sigmoid", 71)
    want = la.la_recurrence_forward(x, g, h0=h0)
    wdx, wdg = la.la_recurrence_backward(x, g, want, dout, h0=h0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = la.la_recurrence_forward(x, g, h0=h0, stream=side)
    dx, dg = la.la_recurrence_backward(x, g, out, dout, h0=h0, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(dx, wdx) and torch.equal(dg, wdg)


def test_inputs_freed_right_after_a_call_on_another_stream():
    """The allocator keeps memory that a given stream still reads."""
    x, g, _, h0, _ = _inputs(1, 1, 20000, 256, torch.bfloat16, "sigmoid", 72)
    want = la.la_recurrence_forward(x, g, h0=h0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)          # about 10 ms: the call waits behind it
    xs, gs = x.clone(), g.clone()
    torch.cuda.current_stream().synchronize()
    out = la.la_recurrence_forward(xs, gs, h0=h0, stream=side)
    size = xs.shape
    del xs, gs
    rubbish = [torch.full(size, float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    side.synchronize()
    assert torch.equal(out, want) and len(rubbish) == 2


def test_in_a_graph():
    x, g, dout, h0, dhN = _inputs(2, 1, 600, 128, torch.bfloat16, "sigmoid", 81)
    hN, dh0 = torch.empty_like(h0), torch.empty_like(h0)

    def step():
        out = la.la_recurrence_forward(x, g, h0=h0, hN=hN)
        return (out,) + la.la_recurrence_backward(x, g, out, dout, h0=h0, dhN=dhN, dh0=dh0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    other = _inputs(2, 1, 600, 128, torch.bfloat16, "sigmoid", 82)
    for t, o in zip((x, g, dout, h0, dhN), other):
        t.copy_(o)
    graph.replay()
    torch.cuda.synchronize()
    state = hN.clone(), dh0.clone()
    want = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got + state, want + (hN, dh0)))
    check_forward(x, g, "sigmoid", h0, None, got[0], hN)


def test_gradient_matches_differences_of_the_kernel():
    """Directional derivative of the forward kernel against its backward, fp32."""
    x, g, dout, h0, dhN = _inputs(1, 2, 90, 20, torch.float32, "sigmoid", 91)
    hN, dh0 = torch.empty_like(h0), torch.empty_like(h0)
    out = la.la_recurrence_forward(x, g, h0=h0, hN=hN)
    dx, dg = la.la_recurrence_backward(x, g, out, dout, h0=h0, dhN=dhN, dh0=dh0)
    rng = torch.Generator(device=DEV).manual_seed(3)
    for v, d in ((x, dx), (g, dg), (h0, dh0)):
        way = torch.randn(v.shape, generator=rng, device=DEV)
        loss = []
        for e in (1e-2, -1e-2):
            args = [v + e * way if t is v else t for t in (x, g, h0)]
            o = la.la_recurrence_forward(args[0], args[1], h0=args[2], hN=hN)
            loss.append(float((o.double() * dout).sum() + (hN.double() * dhN).sum()))
        slope, want = (loss[0] - loss[1]) / 2e-2, float((d.double() * way).sum())
        # second differences of order e^2 and the forward's rounding over 2 e
        assert abs(slope - want) <= 2e-3 * float(d.double().norm() * way.double().norm())
