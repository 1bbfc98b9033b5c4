"""GPU parity of the norm and rotation of queries and keys against the fp64
oracle (oracle/decay.py).

Tolerances, element by element, with u = 2^-24.  A sum over a head's D squares
takes at most 8 + 5 additions on a lane's and the lanes' way and D products,
so rstd is within 16 u of itself.  The turn is rounded to fp32 in half turns
(an error of u / 2 of at most one half turn, so pi u / 2 in radians), its sine
and cosine add 2 u each: an output n_i c - n_j s is within (16 + 8) u (|n_i| +
|n_j|).  The gradient's average over D adds the same sums.  Sums over heads
and tokens run on one thread's way over at most rows/32 + 700 additions.  An
output's own rounding adds half a step.
"""
import numpy as np
import pytest
import torch

from oracle import decay
from weight_recurrence_gb300 import la

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
DTYPES = [torch.float32, torch.bfloat16]
PAIRS = ["half", "adjacent"]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.lib()


def _np(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def _close(name, got, ref, tol):
    got = _np(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.isfinite(got).all(), name
    worst = np.abs(got - ref) / (tol + 1e-30)
    assert worst.max(initial=0.0) <= 1.0, (name, float(worst.max()), np.unravel_index(worst.argmax(), worst.shape))


def inputs(B, N, Hq, Hk, D, P, A, dtype, seed, layout="heads", far=100000):
    rng = torch.Generator().manual_seed(seed)
    mk = lambda H: torch.randn((B, H, N, D), generator=rng).to(dtype).to(DEV)  # noqa: E731
    q, dq, k, dk = mk(Hq), mk(Hq), mk(Hk), mk(Hk)
    if layout == "tokens":
        both = torch.cat([t.transpose(1, 2).flatten(2) for t in (q, k)], dim=-1)
        q = both[..., :Hq * D].unflatten(-1, (Hq, D)).transpose(1, 2)
        k = both[..., Hq * D:].unflatten(-1, (Hk, D)).transpose(1, 2)
    elif layout == "odd":
        q, k, dq, dk = (torch.cat([t, t[..., :1]], dim=-1)[..., :-1] for t in (q, k, dq, dk))
    pos = torch.randint(-far, far, (A, B, N), generator=rng, dtype=torch.int32).to(DEV)
    freq = (10000.0 ** (-torch.arange(P, dtype=torch.float64) / max(P, 1))).float().to(DEV)
    axes = tuple(int(x) for x in torch.randint(0, A, (P,), generator=rng))
    wq, wk = (1 + 0.3 * torch.randn((2, D), generator=rng)).to(DEV)
    return q, k, dq, dk, pos, freq, axes, wq, wk


def _turned_abs(x, P, pairs):
    """|x_i| + |x_j| of every channel's pair."""
    i, j = decay._channels(P, pairs)
    s = np.abs(x)
    t = s.copy()
    t[..., i] = t[..., j] = s[..., i] + s[..., j]
    return t


def check_one(name, x, dy, w, y, dx, dw, angle, eps, norm, pairs, dtype):
    P, D = angle.shape[-1], x.shape[-1]
    half = torch.finfo(dtype).eps / 2
    xn, wn = _np(x), _np(w)
    ref = decay.rotate(xn, angle, wn, eps, norm, pairs)
    n = xn / np.sqrt((xn * xn).mean(-1, keepdims=True) + eps) if norm else xn
    n = n if wn is None else n * wn
    _close(name, y, ref, 24 * U * _turned_abs(n, P, pairs) + half * np.abs(ref))
    if dx is None:
        return
    dyn = _np(dy)
    rx, rw = decay.rotate_backward(dyn, xn, angle, wn, eps, norm, pairs)
    ua = _turned_abs(dyn, P, pairs)
    if norm:
        r = 1 / np.sqrt((xn * xn).mean(-1, keepdims=True) + eps)
        xh, wa = np.abs(xn) * r, np.ones(D) if wn is None else np.abs(wn)
        size = r * (ua * wa + xh * (ua * wa * xh).mean(-1, keepdims=True))
        _close("d" + name, dx, rx, 90 * U * size + half * np.abs(rx))
        rows = xn.size // D
        _close("dw" + name, dw, rw, (rows / 32 + 700 + 50) * U * (ua * xh).sum((0, 1, 2)))
    else:
        _close("d" + name, dx, rx, 24 * U * ua + half * np.abs(rx))
        assert dw is None


def check(B, N, Hq, Hk, D, P, A=1, dtype=torch.float32, seed=0, layout="heads", norm=True, pairs="half", weights=True,
          eps=1e-6, far=100000):
    q, k, dqo, dko, pos, freq, axes, wq, wk = inputs(B, N, Hq, Hk, D, P, A, dtype, seed, layout, far)
    if not (norm and weights):
        wq = wk = None
    if Hk == 0:
        k = dko = wk = None
    how = dict(wq=wq, wk=wk, eps=eps, norm=norm, pairs=pairs, axes=axes)
    qo, ko = la.la_qk_rotate_forward(q, k, pos, freq, **how)
    dq, dk, dwq, dwk = la.la_qk_rotate_backward(dqo, dko, q, k, pos, freq, **how)
    angle = decay.angles(pos.cpu().numpy(), freq.cpu().numpy(), axes)
    check_one("q", q, dqo, wq, qo, dq, dwq, angle, eps, norm, pairs, dtype)
    if Hk:
        check_one("k", k, dko, wk, ko, dk, dwk, angle, eps, norm, pairs, dtype)
    else:
        assert ko is None and dk is None and dwk is None


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pairs", PAIRS)
@pytest.mark.parametrize("D,P", [(64, 32), (128, 64), (256, 128), (32, 16), (16, 8), (64, 16), (128, 20), (80, 40), (80, 20),
                                 (96, 31), (6, 3), (2, 1), (2, 0), (64, 0), (130, 65), (254, 3), (8, 4), (8, 1)])
def test_widths(D, P, pairs, dtype):
    check(2, 9, 3, 2, D, P, dtype=dtype, pairs=pairs, seed=D + P)


@pytest.mark.parametrize("pairs", PAIRS)
@pytest.mark.parametrize("N", [1, 70])
@pytest.mark.parametrize("D,P", [(8, 4), (24, 8), (24, 12), (40, 20), (72, 36), (72, 4), (104, 0), (136, 68), (248, 100), (48, 20)])
def test_pieces_of_8_bytes(D, P, N, pairs):
    """bf16 heads that are a multiple of 8 channels wide, not of 16."""
    check(2, N, 5, 3, D, P, dtype=torch.bfloat16, pairs=pairs, seed=D + P, layout="tokens")


@pytest.mark.parametrize("pairs", PAIRS)
def test_rows_on_8_bytes(pairs):
    """bf16 rows whose strides are a multiple of 8 bytes, not of 16."""
    q, k, dqo, dko, pos, freq, axes, wq, wk = inputs(2, 21, 3, 2, 64, 32, 1, torch.bfloat16, 12)
    want = la.la_qk_rotate_forward(q, k, pos, freq, wq, wk, pairs=pairs)
    grads = la.la_qk_rotate_backward(dqo, dko, q, k, pos, freq, wq, wk, pairs=pairs)

    def on8(t):
        return torch.cat([t, t[..., :4]], dim=-1)[..., :-4]
    q, k, dqo, dko = (on8(t) for t in (q, k, dqo, dko))
    assert q.stride(-2) == 68
    got = la.la_qk_rotate_forward(q, k, pos, freq, wq, wk, pairs=pairs)
    for a, b in zip((*got, *la.la_qk_rotate_backward(dqo, dko, q, k, pos, freq, wq, wk, pairs=pairs)), (*want, *grads)):
        tol = 2 * torch.finfo(a.dtype).eps if a.dtype == torch.bfloat16 else 1e-5   # sums in another order: a rounding apart
        assert (a.double() - b.double()).abs().max() <= tol * b.double().abs().max()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("norm,weights", [(True, True), (True, False), (False, False)])
@pytest.mark.parametrize("layout", ["heads", "tokens", "odd"])
@pytest.mark.parametrize("pairs", PAIRS)
def test_layouts(pairs, layout, norm, weights, dtype):
    check(2, 37, 5, 3, 64, 24, A=3, dtype=dtype, pairs=pairs, layout=layout, norm=norm, weights=weights)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,N,Hq,Hk", [(1, 1, 1, 0), (1, 1, 1, 1), (64, 1, 16, 4), (1, 1, 40, 8), (3, 1000, 4, 1), (1, 5000, 9, 9),
                                       (5000, 1, 3, 2), (7, 701, 2, 0)])
def test_counts(B, N, Hq, Hk, dtype):
    check(B, N, Hq, Hk, 64, 32, dtype=dtype, seed=N)
    check(B, N, Hq, Hk, 48, 11, A=2, dtype=dtype, seed=N, pairs="adjacent")


def test_more_tokens_than_the_backward_keeps_groups():
    check(3, 9000, 2, 1, 64, 32, dtype=torch.bfloat16)
    check(1, 9000, 1, 2, 34, 17, dtype=torch.float32)


@pytest.mark.parametrize("far", [1 << 24, (1 << 31) - 1])
@pytest.mark.parametrize("pairs", PAIRS)
def test_far_positions(far, pairs):
    check(2, 50, 2, 2, 64, 32, A=2, pairs=pairs, far=far)


def test_frequencies_over_their_range():
    """Radians a position from far above a turn to next to nothing, of both signs; not finite: NaN for that pair alone."""
    q, k, _, _, pos, _, _, wq, wk = inputs(2, 40, 2, 2, 64, 32, 1, torch.float32, 3, far=1 << 20)
    freq = torch.tensor([(-1.0) ** i * 2.0 ** (12 - 3 * i) * 1.3 for i in range(32)], device=DEV)
    freq[30], freq[31] = 0.0, 1e-44
    qo, _ = la.la_qk_rotate_forward(q, k, pos, freq, wq, wk)
    angle = decay.angles(pos.cpu().numpy(), freq.cpu().numpy())
    check_one("q", q, None, wq, qo, None, None, angle, 1e-6, True, "half", torch.float32)
    freq[5], freq[7] = float("nan"), float("inf")
    got, _ = la.la_qk_rotate_forward(q, k, pos, freq, wq, wk)
    hit = [5, 7, 37, 39]
    rest = [c for c in range(64) if c not in hit]
    assert torch.isnan(got[..., hit]).all() and torch.equal(got[..., rest], qo[..., rest])


@pytest.mark.parametrize("dtype", DTYPES)
def test_position_forms(dtype):
    """[N], [B,N] and [A,B,N], and views of them, give the same."""
    q, k, _, _, pos, freq, _, wq, wk = inputs(2, 30, 2, 2, 64, 32, 1, dtype, 4)
    pos = pos[:, :1].expand(1, 2, 30)
    want = la.la_qk_rotate_forward(q, k, pos.contiguous(), freq, wq, wk)
    wide = torch.zeros(2, 60, dtype=torch.int32, device=DEV)
    wide[:, ::2] = pos[0]
    for p in (pos[0, 0], pos[0], pos, wide[:, ::2]):
        got = la.la_qk_rotate_forward(q, k, p, freq, wq, wk, axes=(0,) * 32)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pairs", PAIRS)
@pytest.mark.parametrize("D,P", [(64, 32), (50, 13)])
def test_in_place(D, P, pairs, dtype):
    q, k, dqo, dko, pos, freq, axes, wq, wk = inputs(2, 33, 4, 2, D, P, 2, dtype, 5, "tokens")
    how = dict(wq=wq, wk=wk, pairs=pairs, axes=axes)
    want = la.la_qk_rotate_forward(q, k, pos, freq, **how)
    grads = la.la_qk_rotate_backward(dqo, dko, q, k, pos, freq, **how)
    got = la.la_qk_rotate_backward(dqo, dko, q, k, pos, freq, dq=dqo, dk=dko, **how)
    assert got[0] is not None and all(torch.equal(a, b) for a, b in zip(got, grads))
    got = la.la_qk_rotate_forward(q, k, pos, freq, qo=q, ko=k, **how)
    assert got[0].data_ptr() == q.data_ptr() and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,N,Hq,Hk,D,P", [(1, 1, 37, 5, 64, 32), (2, 700, 24, 24, 64, 32), (3, 5, 1, 30, 128, 64), (4, 900, 9, 2, 66, 30)])
def test_in_place_with_many_heads(B, N, Hq, Hk, D, P, dtype):
    """Rows that are read ahead of the ones that are written over."""
    q, k, dqo, dko, pos, freq, axes, wq, wk = inputs(B, N, Hq, Hk, D, P, 1, dtype, 8, "tokens")
    how = dict(wq=wq, wk=wk)
    want = la.la_qk_rotate_forward(q, k, pos, freq, **how)
    grads = la.la_qk_rotate_backward(dqo, dko, q, k, pos, freq, **how)
    got = la.la_qk_rotate_backward(dqo, dko, q, k, pos, freq, dq=dqo, dk=dko, **how)
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    got = la.la_qk_rotate_forward(q, k, pos, freq, qo=q, ko=k, **how)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("pairs", PAIRS)
@pytest.mark.parametrize("D,P", [(64, 32), (50, 13)])
def test_gradients_against_differences(D, P, pairs):
    """fp32, central differences along random directions.  With e = 2^-6 of a direction the cut third order term is of
    the relative size e^2 (2.4e-4 of the product of norms); the roundings of outputs of size 1 are u / e of it (4e-6)."""
    q, k, dqo, dko, pos, freq, axes, wq, wk = inputs(2, 20, 3, 2, D, P, 1, torch.float32, 11)
    wq, wk = (torch.ones(D, device=DEV) if w is None else w for w in (wq, wk))
    grads = la.la_qk_rotate_backward(dqo, dko, q, k, pos, freq, wq, wk, pairs=pairs)
    args, e = [q, k, wq, wk], 2.0 ** -6
    rng = torch.Generator().manual_seed(3)
    for i, grad in enumerate(grads):
        d = torch.randn(args[i].shape, generator=rng).to(DEV)
        sides = []
        for sign in (e, -e):
            a = [t + sign * d if j == i else t for j, t in enumerate(args)]
            qo, ko = la.la_qk_rotate_forward(a[0], a[1], pos, freq, a[2], a[3], pairs=pairs)
            sides.append(float((dqo.double() * qo.double()).sum() + (dko.double() * ko.double()).sum()))
        want = float((grad.double() * d.double()).sum())
        size = float((dqo if i % 2 == 0 else dko).double().norm()) * float(d.double().norm() if i < 2 else (d.double().norm() * (args[i - 2].numel() / D) ** 0.5))
        assert abs((sides[0] - sides[1]) / (2 * e) - want) <= 1e-3 * size, (i, sides, want, size)


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_query_heads(dtype):
    q, k, dqo, dko, pos, freq, axes, wq, wk = inputs(2, 33, 4, 3, 64, 32, 1, dtype, 9)
    none = q[:, :0]
    want = la.la_qk_rotate_forward(q, k, pos, freq, wq, wk)
    qo, ko = la.la_qk_rotate_forward(none, k, pos, freq, wq, wk)
    assert qo.numel() == 0 and torch.equal(ko, want[1])
    want = la.la_qk_rotate_backward(dqo, dko, q, k, pos, freq, wq, wk)
    dq, dk, dwq, dwk = la.la_qk_rotate_backward(none, dko, none, k, pos, freq, wq, wk)
    assert dq.numel() == 0 and torch.equal(dk, want[1]) and not dwq.any()
    assert (dwk - want[3]).abs().max() <= 1e-5 * want[3].abs().max()


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_of_zeros_and_extremes(dtype):
    q, k, dqo, dko, pos, freq, _, wq, wk = inputs(1, 8, 2, 2, 64, 32, 1, dtype, 6)
    q[:, :, 3] = 0.0
    q[:, :, 4, 5] = float("nan")
    qo, _ = la.la_qk_rotate_forward(q, k, pos, freq, wq, wk)
    assert not qo[:, :, 3].any() and torch.isnan(qo[:, :, 4]).all()
    assert torch.isfinite(qo[:, :, [0, 1, 2, 3, 5, 6, 7]]).all()
    q[:, :, 4] = 1.0
    dq = la.la_qk_rotate_backward(dqo, dko, q, k, pos, freq, wq, wk)[0]
    assert torch.isfinite(dq).all()       # a row of zeros: 1/sqrt(eps) times the rest
    angle = decay.angles(pos[None].cpu().numpy()[0], freq.cpu().numpy())
    check_one("q", q, dqo, wq, la.la_qk_rotate_forward(q, k, pos, freq, wq, wk)[0], dq,
              la.la_qk_rotate_backward(dqo, dko, q, k, pos, freq, wq, wk)[2], angle, 1e-6, True, "half", dtype)


def test_empty_batches():
    for shape in ((0, 2, 5, 16), (2, 2, 0, 16), (2, 0, 5, 16)):
        q = torch.zeros(shape, device=DEV)
        pos, freq = torch.zeros(shape[0], shape[2], dtype=torch.int32, device=DEV), torch.ones(8, device=DEV)
        assert la.la_qk_rotate_forward(q, q.clone(), pos, freq)[1].shape == shape
        dq, dk, dwq, dwk = la.la_qk_rotate_backward(q, q.clone(), q, q.clone(), pos, freq)
        assert dq.shape == shape and not dwq.any() and not dwk.any()


def test_offsets_past_32_bits():
    q, k, _, _, pos, freq, _, wq, wk = inputs(2, 20, 2, 1, 64, 32, 1, torch.bfloat16, 7)
    far = (1 << 31) + 64
    room = torch.empty(far + 20 * 512, dtype=torch.bfloat16, device=DEV)
    at = lambda i, H: room.as_strided((2, H, 20, 64), (far, 64, 512, 1), 128 * i)  # noqa: E731
    at(0, 2).copy_(q)
    at(1, 1).copy_(k)
    got = la.la_qk_rotate_forward(at(0, 2), at(1, 1), pos, freq, wq, wk, qo=at(2, 2), ko=at(3, 1))
    want = la.la_qk_rotate_forward(q, k, pos, freq, wq, wk)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_streams_and_graphs():
    def run(t):
        q, k, dqo, dko, pos, freq, axes, wq, wk = t
        how = dict(wq=wq, wk=wk, axes=axes)
        return [*la.la_qk_rotate_forward(q, k, pos, freq, **how),
                *la.la_qk_rotate_backward(dqo, dko, q, k, pos, freq, **how)]
    sets = [list(inputs(2, 3000, 4, 2, 64, 32, 2, torch.bfloat16, s)) for s in range(3)]
    for t in sets:
        t[6] = sets[0][6]
    want = [run(t) for t in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s, t in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(run(t))
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(outs, want[i % 2]))
    held = [t.clone() if isinstance(t, torch.Tensor) else t for t in sets[0]]
    with torch.cuda.stream(streams[0]):
        run(held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(held)
    for i in (1, 2, 0):
        for h, t in zip(held, sets[i]):
            if isinstance(h, torch.Tensor):
                h.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pairs", PAIRS)
@pytest.mark.parametrize("D,P", [(64, 16), (64, 0), (72, 20), (66, 13), (128, 3), (256, 100)])
def test_channels_behind_the_rotated_ones_stay_apart(D, P, pairs, dtype, bad):
    """A value that is not finite in a channel behind the rotated ones is seen by that channel alone: bit for bit what
    the other channels are without it, rows by pieces (16 and 8 bytes) and by single values."""
    q, k, dqo, dko, pos, freq, axes, wq, wk = inputs(1, 9, 2, 3, D, P, 1, dtype, D + P)
    for c in {2 * P, 2 * P + 1, P + D // 2, D - 1} - set(range(2 * P)):
        rest = [i for i in range(D) if i != c]
        how = dict(norm=False, pairs=pairs)
        hit = [t.clone() for t in (q, k, dqo, dko)]
        for t in hit:
            t[:, :, ::2, c] = bad
        a, b = (la.la_qk_rotate_forward(x, y, pos, freq, **how) for x, y in ((q, k), hit[:2]))
        a += la.la_qk_rotate_backward(dqo, dko, q, k, pos, freq, **how)[:2]
        b += la.la_qk_rotate_backward(hit[2], hit[3], q, k, pos, freq, **how)[:2]
        for clean, got, x in zip(a, b, hit):
            assert torch.equal(got[..., rest], clean[..., rest])
            assert torch.equal(torch.nan_to_num(got[..., c], 1, 2, 3), torch.nan_to_num(x[..., c], 1, 2, 3))
        # with the norm: 1/sqrt(infinity) is 0, so the finite channels are 0; the sums of the weights stay apart
        if bad == float("inf"):
            qo, _ = la.la_qk_rotate_forward(hit[0], k, pos, freq, wq, wk, pairs=pairs)
            assert not qo[:, :, ::2][..., rest].any() and torch.isnan(qo[:, :, ::2, c]).all()
        clean = la.la_qk_rotate_backward(dqo, dko, q, k, pos, freq, wq, wk, pairs=pairs)[2:]
        got = la.la_qk_rotate_backward(hit[2], hit[3], q, k, pos, freq, wq, wk, pairs=pairs)[2:]
        for x, y in zip(got, clean):
            assert torch.equal(x[rest], y[rest]) and not torch.isfinite(x[c])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pairs", PAIRS)
@pytest.mark.parametrize("D,P", [(64, 16), (64, 0), (72, 20), (66, 13)])
def test_channels_behind_the_rotated_ones_are_copied(D, P, pairs, dtype):
    """Without the norm they leave as they came, the signs of zeros among them."""
    q, k, dqo, dko, pos, freq, axes, _, _ = inputs(2, 11, 3, 2, D, P, 1, dtype, D)
    for t in (q, k, dqo, dko):
        t[..., ::3] = 0.0
        t[..., ::2] *= -1.0
    got = la.la_qk_rotate_forward(q, k, pos, freq, norm=False, pairs=pairs)
    got += la.la_qk_rotate_backward(dqo, dko, q, k, pos, freq, norm=False, pairs=pairs)[:2]
    words = torch.int16 if dtype == torch.bfloat16 else torch.int32
    for y, x in zip(got, (q, k, dqo, dko)):
        assert torch.equal(y[..., 2 * P:].contiguous().view(words), x[..., 2 * P:].contiguous().view(words))


def _exact_angles(pos, freq):
    """[B,N,P] from pos [B,N], freq [P], mod a turn in whole numbers: no rounding before the last."""
    one = 1 << 300

    def arctan(x):     # of 1 / x
        t, s, n = one // x, 0, 0
        while t:
            s += (-1) ** n * (t // (2 * n + 1))
            t, n = t // (x * x), n + 1
        return s
    turn = 2 * (4 * (4 * arctan(5) - arctan(239)))
    out = np.zeros(pos.shape + freq.shape)
    for i, f in enumerate(freq.tolist()):
        num, den = f.as_integer_ratio()
        for at in np.ndindex(pos.shape):
            a = int(pos[at]) * num * one // den % turn
            out[at + (i,)] = float(a if 2 * a < turn else a - turn) / float(one)
    return out


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_frequencies_at_far_positions(dtype):
    """Up to 2^60 radians a position, to the last positions of 32 bits: the turn's fraction is what is left of it."""
    q, k, dqo, dko, _, _, _, wq, wk = inputs(2, 12, 2, 2, 64, 32, 1, dtype, 13)
    pos = torch.tensor([-(1 << 31), (1 << 31) - 1, (1 << 31) - 2, -(1 << 31) + 1, 1 << 30, 0, 1, -1, 12345, -987654321,
                        2000000011, 77777777], dtype=torch.int32, device=DEV).expand(2, 12)
    freq = torch.tensor([(-1.0) ** i * 2.0 ** (2 * i - 2) * (1 + i / 64) for i in range(32)], device=DEV)
    qo, ko = la.la_qk_rotate_forward(q, k, pos, freq, wq, wk)
    dq, dk, dwq, dwk = la.la_qk_rotate_backward(dqo, dko, q, k, pos, freq, wq, wk)
    angle = _exact_angles(pos.cpu().numpy(), freq.cpu().numpy().astype(np.float64))
    check_one("q", q, dqo, wq, qo, dq, dwq, angle, 1e-6, True, "half", dtype)
    check_one("k", k, dko, wk, ko, dk, dwk, angle, 1e-6, True, "half", dtype)


def test_most_tokens():
    """The largest token count that is taken: its first, middle and last rows are what they are by themselves, forward
    and backward in place."""
    N = (1 << 31) - 1 - (1 << 20)
    q = torch.ones(1, 1, N, 2, device=DEV, dtype=torch.bfloat16)
    pos = torch.arange(N, device=DEV, dtype=torch.int32)
    freq = torch.tensor([0.7], device=DEV)
    at = [slice(0, 70), slice((1 << 30) - 40, (1 << 30) + 40), slice(N - 100000, N)]
    for s in at:
        q[:, :, s].normal_(generator=torch.Generator(DEV).manual_seed(1))
    out = la.la_qk_rotate_forward(q, None, pos, freq)[0]
    alone = [la.la_qk_rotate_forward(q[:, :, s], None, pos[s], freq)[0] for s in at]
    assert all(torch.equal(out[:, :, s], a) for s, a in zip(at, alone))
    la.la_qk_rotate_backward(out, None, q, None, pos, freq, dq=out)
    grads = [la.la_qk_rotate_backward(a, None, q[:, :, s], None, pos[s], freq)[0] for s, a in zip(at, alone)]
    same = all(torch.equal(out[:, :, s], a) for s, a in zip(at, grads))
    del q, pos, out
    torch.cuda.empty_cache()
    assert same
