"""GPU parity of the linear attention with decays (forward, single step, backward)
against the fp64 oracle (oracle/decay.py).

Tolerances, element by element.  Every output is a sum of products; the same
sum over absolute values is its majorant H (the oracle run on absolute values).
With u = 2^-24 each fp32 rounding is at most u of its term: a product of rows
of D values takes D of them, a decay (exponent, exponential, product) 4 and
the exponent's own rounding u |g e| <= 104 u wherever the decay is not 0, a
chunk's sum over at most 128 tokens and the state's over D, the state's carry
3 for each chunk of 32 at least and 3 a segment.  Tensor cores may truncate
where they add: two u a rounding.  K below counts all of them twice.  With bf16
data the masked scores or the state are rounded once on each term's way:
half a step of H; the output's own rounding adds half a step.
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


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.lib()


def _np(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def _k(N, D):
    return 2 * (2 * D + 2 * 128 + 6 * (N // 32 + 1) + 110)


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def _close(name, got, ref, tol):
    got = _np(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.isfinite(got).all(), name
    worst = np.abs(got - ref) / (tol + 1e-30)
    assert worst.max(initial=0.0) <= 1.0, (name, float(worst.max()), np.unravel_index(worst.argmax(), worst.shape))


def _rows(name, got, ref, H, K, dtype):
    scores = 0.0 if dtype == torch.float32 else 1.02 * _half(dtype)
    _close(name, got, ref, scores * H + K * U * H + _half(dtype) * np.abs(ref))


def inputs(B, H, N, D, M, dtype, seed, layout="heads", decays=None):
    rng = torch.Generator().manual_seed(seed)
    q, k = torch.randn((2, B, H, N, D), generator=rng)
    v, dout = torch.randn((2, B, H, N, M), generator=rng)
    S0, dSN = torch.randn((2, B, H, D, M), generator=rng)
    ts = [t.to(dtype).to(DEV) for t in (q, k, v, dout)]
    if layout == "tokens":      # one projection [B, N, H, .], side by side
        both = torch.cat([t.transpose(1, 2) for t in ts], dim=-1).contiguous()
        ts = [t.transpose(1, 2) for t in both.split([D, D, M, M], dim=-1)]
    elif layout == "odd":       # rows off every boundary
        ts = [torch.cat([t, t[..., :1]], dim=-1).flatten()[: t.numel() + B * H * N].view(B, H, N, -1)[..., :-1] for t in ts]
    if decays is None:
        g = torch.log1p(-torch.exp2(-torch.linspace(0.7, 9.0, H)))
        if H > 2:
            g[-1] = 0.0
    else:
        g = torch.tensor(decays)
    return ts + [S0.to(DEV), dSN.to(DEV), g.float().to(DEV)]


def check(B, H, N, D, M, dtype, seed=0, layout="heads", decays=None, lens=None, scale=None, states=True):
    q, k, v, dout, S0, dSN, g = inputs(B, H, N, D, M, dtype, seed, layout, decays)
    scale = D ** -0.5 if scale is None else scale
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    SN, dS0 = torch.full_like(S0, 9.0), torch.full_like(S0, 9.0)
    if not states:
        S0 = dSN = None
    out = la.la_decay_forward(q, k, v, g, scale, S0=S0, SN=SN, lens=ln)
    dq, dk, dv = la.la_decay_backward(q, k, v, dout, g, scale, S0=S0, dSN=dSN, dS0=dS0, lens=ln)
    qn, kn, vn, dn, Sn, En, gn = (_np(t) for t in (q, k, v, dout, S0, dSN, g))
    ab = [None if t is None else np.abs(t) for t in (qn, kn, vn, dn, Sn, En)]
    K = _k(N, max(D, M))
    ref, refS = decay.forward(qn, kn, vn, gn, scale, Sn, lens)
    H_, HS = decay.forward(ab[0], ab[1], ab[2], gn, abs(scale), ab[4], lens)
    _rows("out", out, ref, H_, K, dtype)
    _close("SN", SN, refS, K * U * HS)
    refs = decay.backward(qn, kn, vn, dn, gn, scale, Sn, En, lens)
    hs = decay.backward(*ab[:4], gn, abs(scale), ab[4], ab[5], lens)
    for name, got, r, h in zip(("dq", "dk", "dv"), (dq, dk, dv), refs, hs):
        _rows(name, got, r, h, K, dtype)
    _close("dS0", dS0, refs[3], K * U * hs[3])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 300])
def test_lengths(N, dtype):
    check(1, 2, N, 64, 64, dtype, seed=N)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,M", [(16, 16), (32, 64), (64, 32), (64, 128), (128, 64), (128, 128), (16, 128), (8, 8), (40, 72),
                                 (120, 24), (1, 1), (3, 5), (65, 63), (127, 128), (128, 1)])
def test_widths(D, M, dtype):
    check(2, 2, 150, D, M, dtype, seed=D * 131 + M)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", ["tokens", "odd"])
@pytest.mark.parametrize("D,M", [(64, 64), (128, 64), (24, 40)])
def test_layouts(layout, D, M, dtype):
    check(2, 3, 170, D, M, dtype, seed=5, layout=layout)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [700, 1409])
def test_segments(N, dtype):
    """Few heads: the sequence is cut."""
    check(1, 1, N, 64, 64, dtype, seed=N)
    check(1, 3, N, 128, 96, dtype, seed=N + 1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[0, 1, 130, 300], [300, 0, 127, 128], [400, -3, 129, 256]])
def test_lens(lens, dtype):
    check(4, 2, 300, 64, 64, dtype, lens=lens)
    check(4, 1, 300, 128, 128, dtype, lens=lens, states=False)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[0], [1], [640], [641], [900]])
def test_lens_in_segments(lens, dtype):
    check(1, 1, 900, 64, 64, dtype, lens=lens)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("decays", [[0.0, 0.0], [-1e-6, -1e-3], [-float("inf"), -50.0], [-0.7, -5.0], [-float("inf"), 0.0],
                                    [0.004, 0.02]])
def test_decays(decays, dtype):
    check(1, 2, 333, 64, 64, dtype, decays=decays)
    check(1, 2, 333, 64, 64, dtype, decays=decays, lens=[200], states=False)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [1.0, 0.0, -2.5])
def test_scale(scale, dtype):
    check(1, 2, 200, 64, 32, dtype, scale=scale)


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(seed):
    r = np.random.default_rng(seed)
    dtype = DTYPES[seed % 2]
    D, M = (int(x) for x in (r.choice([16, 32, 64, 128], 2) if seed % 3 else r.integers(1, 129, 2)))
    B, H, N = int(r.integers(1, 4)), int(r.integers(1, 5)), int(r.integers(1, 600))
    lens = [int(x) for x in r.integers(0, N + 1, B)] if seed % 4 == 0 else None
    check(B, H, N, D, M, dtype, seed, ["heads", "tokens", "odd"][int(r.integers(3))], None, lens)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,M", [(64, 64), (128, 128), (16, 32), (8, 4), (33, 7), (128, 66), (1, 1)])
@pytest.mark.parametrize("B,H", [(1, 1), (3, 2), (90, 8)])
def test_step(B, H, D, M, dtype):
    q, k, v, _, S0, _, g = inputs(B, H, 2, D, M, dtype, seed=D + M)
    S = S0.clone()
    y = la.la_decay_step(q[:, :, 1], k[:, :, 1], v[:, :, 1], S, g, 0.3)
    qn, kn, vn, Sn, gn = (_np(t) for t in (q[:, :, 1:], k[:, :, 1:], v[:, :, 1:], S0, g))
    ref, refS = decay.forward(qn, kn, vn, gn, 0.3, Sn)
    H_, HS = decay.forward(np.abs(qn), np.abs(kn), np.abs(vn), gn, 0.3, np.abs(Sn))
    _close("y", y, ref[:, :, 0], (D + 8) * U * H_[:, :, 0] + _half(dtype) * np.abs(ref[:, :, 0]))
    _close("S", S, refS, 8 * U * HS)


@pytest.mark.parametrize("dtype", DTYPES)
def test_prefill_then_steps_are_the_whole(dtype):
    """A prompt (state alone), then tokens one by one."""
    q, k, v, _, _, _, g = inputs(2, 3, 140, 64, 64, dtype, seed=3)
    S = torch.zeros(2, 3, 64, 64, device=DEV)
    assert la.la_decay_forward(None, k[:, :, :130], v[:, :, :130], g, SN=S, want_out=False) is None
    ys = [la.la_decay_step(q[:, :, t], k[:, :, t], v[:, :, t], S, g, 0.125) for t in range(130, 140)]
    ref, refS = decay.forward(_np(q), _np(k), _np(v), _np(g), 0.125)
    H_, HS = decay.forward(*(np.abs(_np(t)) for t in (q, k, v)), _np(g), 0.125)
    K = _k(140, 64)
    _rows("y", torch.stack(ys, 2), ref[:, :, 130:], H_[:, :, 130:], K, dtype)
    _close("S", S, refS, K * U * HS)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,at", [(300, 140), (900, 384), (900, 517)])
def test_chained_calls_are_the_whole(N, at, dtype):
    """State in place from one call to the next; gradients back the same way."""
    q, k, v, dout, S0, dSN, g = inputs(1, 2, N, 64, 64, dtype, seed=N + at)
    S = S0.clone()
    a = la.la_decay_forward(q[:, :, :at], k[:, :, :at], v[:, :, :at], g, S0=S, SN=S)
    mid = S.clone()
    b = la.la_decay_forward(q[:, :, at:], k[:, :, at:], v[:, :, at:], g, S0=S, SN=S)
    ref, refS = decay.forward(*(_np(t) for t in (q, k, v, g)), 1.0, _np(S0))
    H_, HS = decay.forward(*(np.abs(_np(t)) for t in (q, k, v)), _np(g), 1.0, np.abs(_np(S0)))
    K = _k(N, 64)
    _rows("out", torch.cat([a, b], 2), ref, H_, K, dtype)
    _close("SN", S, refS, K * U * HS)
    d1, d0 = torch.empty_like(S0), torch.empty_like(S0)
    late = la.la_decay_backward(*(t[:, :, at:] for t in (q, k, v, dout)), g, S0=mid, dSN=dSN, dS0=d1)
    early = la.la_decay_backward(*(t[:, :, :at] for t in (q, k, v, dout)), g, S0=S0, dSN=d1, dS0=d0)
    refs = decay.backward(*(_np(t) for t in (q, k, v, dout, g)), 1.0, _np(S0), _np(dSN))
    hs = decay.backward(*(np.abs(_np(t)) for t in (q, k, v, dout)), _np(g), 1.0, np.abs(_np(S0)), np.abs(_np(dSN)))
    for name, e, l, r, h in zip(("dq", "dk", "dv"), early, late, refs, hs):
        _rows(name, torch.cat([e, l], 2), r, h, 2 * K, dtype)
    _close("dS0", d0, refs[3], 2 * K * U * hs[3])


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_tokens(dtype):
    q, k, v, dout, S0, dSN, g = inputs(2, 2, 4, 16, 24, dtype, seed=1)
    none = [t[:, :, :0] for t in (q, k, v, dout)]
    SN, dS0 = torch.empty_like(S0), torch.empty_like(S0)
    assert la.la_decay_forward(*none[:3], g, S0=S0, SN=SN).shape == (2, 2, 0, 24)
    la.la_decay_backward(*none, g, S0=S0, dSN=dSN, dS0=dS0)
    assert torch.equal(SN, S0) and torch.equal(dS0, dSN)
    la.la_decay_forward(*none[:3], g, SN=SN)
    assert not SN.any()
    empty = [t[:0] for t in (q, k, v)]
    assert la.la_decay_forward(*empty, g).shape == (0, 2, 4, 24)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,at", [(300, 130), (300, 0), (900, 600)])
def test_a_token_that_is_not_finite(N, at, dtype, bad):
    """What does not see it is what it is without it; what does is finite where token by token is."""
    q, k, v, dout, _, _, g = inputs(1, 2, N, 64, 64, dtype, seed=at, decays=[-0.1, -0.01])
    K, gn = _k(N, 64), _np(g)
    keep = [c for c in range(64) if c != 3]

    def same(name, got, ref, H, part):
        _rows(name, got[part], ref[part], H[part], K, dtype)
    clean = [_np(t) for t in (q, k, v, dout)]
    ref, _ = decay.forward(*clean[:3], gn)
    H_, _ = decay.forward(*(np.abs(t) for t in clean[:3]), gn)
    for name in ("v", "k"):
        t = dict(q=q, k=k, v=v)
        t[name] = t[name].clone()
        t[name][:, :, at, 3] = bad
        S = torch.empty(1, 2, 64, 64, device=DEV)
        out = la.la_decay_forward(t["q"], t["k"], t["v"], g, SN=S)
        same(name, out, ref, H_, np.s_[:, :, :at])
        if name == "v":     # one column
            same(name, out, ref, H_, np.s_[..., keep])
        with np.errstate(invalid="ignore"):
            hit, hitS = decay.forward(*(_np(x) for x in (t["q"], t["k"], t["v"])), gn)
        assert torch.equal(torch.isfinite(out).cpu(), torch.from_numpy(np.isfinite(hit))), name
        assert torch.equal(torch.isfinite(S).cpu(), torch.from_numpy(np.isfinite(hitS))), name
    # backwards in time, the rows behind it do not see it
    refs = decay.backward(*clean, gn)
    hs = decay.backward(*(np.abs(t) for t in clean), gn)
    for name in ("q", "dout"):
        t = dict(q=q, dout=dout)
        t[name] = t[name].clone()
        t[name][:, :, at, 3] = bad
        _, dk, dv = la.la_decay_backward(t["q"], k, v, t["dout"], g)
        same(name, dk, refs[1], hs[1], np.s_[:, :, at + 1:])
        same(name, dv, refs[2], hs[2], np.s_[:, :, at + 1:])
        with np.errstate(invalid="ignore"):
            hit = decay.backward(*(_np(x) for x in (t["q"], k, v, t["dout"])), gn)
        for got, r in ((dk, hit[1]), (dv, hit[2])):
            assert torch.equal(torch.isfinite(got).cpu(), torch.from_numpy(np.isfinite(r))), name


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_past_a_length_are_not_read(dtype):
    q, k, v, dout, S0, dSN, g = inputs(3, 2, 400, 64, 64, dtype, seed=2)
    lens = torch.tensor([130, 0, 257], dtype=torch.int32, device=DEV)
    what = [torch.empty_like(S0), torch.empty_like(S0)]
    clean = [la.la_decay_forward(q, k, v, g, S0=S0, SN=what[0], lens=lens),
             *la.la_decay_backward(q, k, v, dout, g, S0=S0, dSN=dSN, dS0=what[1], lens=lens)]
    for b, n in enumerate([130, 0, 257]):
        for i, t in enumerate((q, k, v, dout)):
            t[b, :, n:] = [float("nan"), float("inf")][i % 2]
    again = [torch.empty_like(S0), torch.empty_like(S0)]
    got = [la.la_decay_forward(q, k, v, g, S0=S0, SN=again[0], lens=lens),
           *la.la_decay_backward(q, k, v, dout, g, S0=S0, dSN=dSN, dS0=again[1], lens=lens)]
    for a, b in zip(clean + what, got + again):
        assert torch.equal(a, b)
    for t in got:
        assert not t[0, :, 130:].any() and not t[1].any() and not t[2, :, 257:].any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_outputs_into_views_leave_the_rest(dtype):
    q, k, v, dout, _, _, g = inputs(2, 3, 150, 64, 64, dtype, seed=6)
    want = [la.la_decay_forward(q, k, v, g), *la.la_decay_backward(q, k, v, dout, g)]
    room = [torch.full((2, 152, 3, 80), 7.0, dtype=dtype, device=DEV) for _ in range(4)]
    views = [r[:, 1:151, :, 8:72].transpose(1, 2) for r in room]
    la.la_decay_forward(q, k, v, g, out=views[0])
    la.la_decay_backward(q, k, v, dout, g, dq=views[1], dk=views[2], dv=views[3])
    for w, r, view in zip(want, room, views):
        assert torch.equal(w, view)
        view.fill_(7.0)
        assert (r == 7.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_repeated_inputs(dtype):
    """Keys and values shared by the heads, as views that repeat them."""
    q, k, v, dout, _, _, g = inputs(2, 4, 200, 64, 64, dtype, seed=7)
    ks, vs = k[:, :1].expand(-1, 4, -1, -1), v[:, :1].expand(-1, 4, -1, -1)
    a = la.la_decay_forward(q, ks, vs, g)
    b = la.la_decay_forward(q, ks.contiguous(), vs.contiguous(), g)
    ref, _ = decay.forward(*(_np(t) for t in (q, ks, vs, g)))
    H_, _ = decay.forward(*(np.abs(_np(t)) for t in (q, ks, vs)), _np(g))
    for got in (a, b):
        _rows("out", got, ref, H_, _k(200, 64), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [1, 3, 4, 5, 8, 9, 16])
@pytest.mark.parametrize("B,H,D,M", [(2, 2, 64, 64), (3, 60, 64, 64), (160, 4, 128, 128), (2, 160, 40, 72), (90, 2, 33, 7), (2, 3, 128, 66)])
def test_a_few_tokens(B, H, D, M, N, dtype):
    """Few tokens of few and of many heads, lengths from none to all of them, with the state in place, and the state
    alone."""
    lens = [(0, N, N // 2, 1)[b % 4] for b in range(B)]
    q, k, v, _, S0, _, g = inputs(B, H, N, D, M, dtype, seed=N, layout="tokens")
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    S, alone = S0.clone(), torch.empty_like(S0)
    out = la.la_decay_forward(q, k, v, g, 0.3, S0=S, SN=S, lens=ln)
    assert la.la_decay_forward(None, k, v, g, 0.3, S0=S0, SN=alone, lens=ln, want_out=False) is None
    qn, kn, vn, Sn, gn = (_np(t) for t in (q, k, v, S0, g))
    ref, refS = decay.forward(qn, kn, vn, gn, 0.3, Sn, lens)
    H_, HS = decay.forward(np.abs(qn), np.abs(kn), np.abs(vn), gn, 0.3, np.abs(Sn), lens)
    _rows("out", out, ref, H_, _k(N, max(D, M)), dtype)
    _close("SN", S, refS, _k(N, max(D, M)) * U * HS)
    assert torch.equal(S, alone)


@pytest.mark.parametrize("N,lens", [(1, None), (9, [9, 4]), (70, None), (300, [300, 131]), (900, None)])
@pytest.mark.parametrize("D,M", [(64, 64), (24, 72)])
def test_gradients_against_differences(N, lens, D, M):
    """fp32.  The outputs and the last state are linear in each of q, k, v and S0: half the difference at x + d and
    x - d, weighed with dout and dSN, is the gradient's product with d, but for the roundings of both sides (K u of the
    majorants)."""
    q, k, v, dout, S0, dSN, g = inputs(2, 2, N, D, M, torch.float32, seed=N)
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    dS0 = torch.empty_like(S0)
    grads = la.la_decay_backward(q, k, v, dout, g, 0.3, S0=S0, dSN=dSN, dS0=dS0, lens=ln)
    rng = torch.Generator().manual_seed(N + 1)
    K = _k(N, max(D, M))
    args = [q, k, v, S0]
    for i, grad in enumerate((*grads, dS0)):
        d = torch.randn(args[i].shape, generator=rng).to(DEV)
        sides, bound = [], 0.0
        for sign in (1.0, -1.0):
            a = [t + sign * d if j == i else t for j, t in enumerate(args)]
            SN = torch.empty_like(S0)
            out = la.la_decay_forward(a[0], a[1], a[2], g, 0.3, S0=a[3], SN=SN, lens=ln)
            sides.append((_np(dout) * _np(out)).sum() + (_np(dSN) * _np(SN)).sum())
            H_, HS = decay.forward(*(np.abs(_np(t)) for t in a[:3]), _np(g), 0.3, np.abs(_np(a[3])), lens)
            bound += (np.abs(_np(dout)) * H_).sum() + (np.abs(_np(dSN)) * HS).sum()
        ab = [np.abs(_np(t)) for t in (q, k, v, dout, S0, dSN)]
        h = decay.backward(*ab[:4], _np(g), 0.3, ab[4], ab[5], lens)[i]
        bound += (np.abs(_np(d)) * h).sum()
        off = abs((sides[0] - sides[1]) / 2 - (_np(grad) * _np(d)).sum())
        # x + d is rounded too: once more u of every term
        assert off <= (K + 2) * U * bound, (i, off, K * U * bound)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [1, 5, 20, 200, 1100])
def test_states_off_16_bytes(N, dtype):
    """States that start on 4 bytes only, against states on 16: the same sums, at most in another order (fp32: below
    1e-5 of the largest at these lengths)."""
    q, k, v, dout, S0, dSN, g = inputs(1, 2, N, 64, 64, dtype, seed=N)

    def off(t):
        return torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape)

    def run(f):
        a, b, SN, dS0 = f(S0), f(dSN), f(torch.zeros_like(S0)), f(torch.zeros_like(S0))
        out = la.la_decay_forward(q, k, v, g, 0.2, S0=a, SN=SN)
        grads = la.la_decay_backward(q, k, v, dout, g, 0.2, S0=a, dSN=b, dS0=dS0)
        y = la.la_decay_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], a, g, 0.2)
        return [out, SN, *grads, dS0, y, a]
    assert off(S0).data_ptr() % 16 == 4
    for x, y in zip(run(off), run(torch.clone)):
        assert (x - y).abs().max() <= 2 * _half(x.dtype) * y.abs().max() + 1e-5 * y.abs().max()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [1, 3, 20])
def test_many_sequences(N, dtype):
    """More heads than a grid's second dimension holds."""
    B = 70000
    q, k, v, dout, S0, _, g = inputs(B, 1, N, 8, 8, dtype, seed=N)
    SN = torch.empty_like(S0)
    out = la.la_decay_forward(q, k, v, g, 0.5, S0=S0, SN=SN)
    grads = la.la_decay_backward(q, k, v, dout, g, 0.5, S0=S0)
    at = [0, 1, 303, 65535, 65536, B - 1]
    qn, kn, vn, dn, Sn = (_np(t[at]) for t in (q, k, v, dout, S0))
    ab = [np.abs(t) for t in (qn, kn, vn, dn, Sn)]
    gn, K = _np(g), _k(N, 8)
    ref, refS = decay.forward(qn, kn, vn, gn, 0.5, Sn)
    H_, HS = decay.forward(*ab[:3], gn, 0.5, ab[4])
    _rows("out", out[at], ref, H_, K, dtype)
    _close("SN", SN[at], refS, K * U * HS)
    for got, r, h in zip(grads, decay.backward(qn, kn, vn, dn, gn, 0.5, Sn), decay.backward(*ab[:4], gn, 0.5, ab[4])):
        _rows("gradient", got[at], r, h, K, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dims", [(0,), (1,), (0, 1)])
@pytest.mark.parametrize("N", [1, 200, 900])
def test_shared_inputs_are_their_copies(N, dims, dtype):
    """q, k, v and dout repeated by views over the sequences, the heads or both, each by itself and all together: what
    copies of them give, bit for bit, gradients of every head's own."""
    ts = inputs(3, 2, N, 64, 64, dtype, seed=N)
    rows, (S0, dSN, g) = ts[:4], ts[4:]

    def shared(t):
        for d in dims:
            t = t[:1] if d == 0 else t[:, :1]
        return t.expand(3, 2, -1, -1)
    for which in ((0,), (1,), (2,), (3,), (0, 1), (0, 1, 2, 3)):
        views = [shared(t) if i in which else t for i, t in enumerate(rows)]
        q, k, v, dout = views
        a = [la.la_decay_forward(q, k, v, g, S0=S0), *la.la_decay_backward(q, k, v, dout, g, S0=S0, dSN=dSN)]
        q, k, v, dout = (t.contiguous() for t in views)
        b = [la.la_decay_forward(q, k, v, g, S0=S0), *la.la_decay_backward(q, k, v, dout, g, S0=S0, dSN=dSN)]
        assert all(torch.equal(x, y) for x, y in zip(a, b)), which


@pytest.mark.parametrize("D,M", [(33, 64), (64, 33), (99, 118), (1, 1), (127, 128)])
@pytest.mark.parametrize("N,lens", [(64, [64, 0]), (130, [129, 1]), (1500, [1500, 700])])
def test_packed_rows(N, lens, D, M):
    """bf16 rows that are not whole 16-byte pieces, from long sequences on; rows past a length hold NaN and are not
    read."""
    check(2, 1, N, D, M, torch.bfloat16, seed=D, lens=lens)
    q, k, v, dout, S0, dSN, g = inputs(2, 1, N, D, M, torch.bfloat16, D)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)

    def run():
        SN, dS0 = torch.empty_like(S0), torch.empty_like(S0)
        out = la.la_decay_forward(q, k, v, g, S0=S0, SN=SN, lens=ln)
        return [out, SN, *la.la_decay_backward(q, k, v, dout, g, S0=S0, dSN=dSN, dS0=dS0, lens=ln), dS0]
    want = run()
    for b, n in enumerate(lens):
        for t in (q, k, v, dout):
            t[b, :, n:] = float("nan")
    assert all(torch.equal(x, y) for x, y in zip(run(), want))


@pytest.mark.parametrize("dtype", DTYPES)
def test_offsets_past_32_bits(dtype):
    """Sequences more than 2^31 values apart."""
    q, k, v, _, S0, _, g = inputs(2, 1, 140, 64, 64, dtype, seed=8)
    far = (1 << 31) + 64
    room = torch.empty(far + 140 * 256, dtype=dtype, device=DEV)
    at = lambda i, n: room.as_strided((2, 1, 140, n), (far, 140 * 256, 256, 1), 64 * i)  # noqa: E731
    for i, t in enumerate((q, k, v)):
        at(i, 64).copy_(t)
    SN, want_S = torch.empty_like(S0), torch.empty_like(S0)
    out = la.la_decay_forward(at(0, 64), at(1, 64), at(2, 64), g, S0=S0, SN=SN, out=at(3, 64))
    want = la.la_decay_forward(q, k, v, g, S0=S0, SN=want_S)
    assert torch.equal(out, want) and torch.equal(SN, want_S)


def test_streams_and_graphs():
    """Two streams at once, and a captured forward, backward and step replayed on new inputs."""
    def one(seed):
        q, k, v, dout, S0, dSN, g = inputs(1, 2, 1500, 64, 64, torch.bfloat16, seed)
        return [q, k, v, dout, S0, dSN, g]

    def run(t):
        q, k, v, dout, S0, dSN, g = t
        SN, dS0 = torch.empty_like(S0), torch.empty_like(S0)
        out = la.la_decay_forward(q, k, v, g, S0=S0, SN=SN)
        grads = la.la_decay_backward(q, k, v, dout, g, S0=S0, dSN=dSN, dS0=dS0)
        y = la.la_decay_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], SN, g)
        return [out, SN, dS0, *grads, y]
    sets = [one(s) for s in range(3)]
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
    held = [t.clone() for t in sets[0]]
    with torch.cuda.stream(streams[0]):
        run(held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(held)
    for i in (1, 2, 0):
        for h, t in zip(held, sets[i]):
            h.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))


def test_a_given_stream():
    q, k, v, _, S0, _, g = inputs(1, 1, 600, 64, 64, torch.bfloat16, 4)
    want = la.la_decay_forward(q, k, v, g, S0=S0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = la.la_decay_forward(q, k, v, g, S0=S0, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_equal_calls_give_equal_bits():
    for dtype in DTYPES:
        q, k, v, dout, S0, dSN, g = inputs(1, 3, 1300, 128, 64, dtype, 9)
        runs = [[la.la_decay_forward(q, k, v, g, S0=S0), *la.la_decay_backward(q, k, v, dout, g, S0=S0, dSN=dSN)]
                for _ in range(3)]
        for r in runs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("short_of", [0, 1000])
def test_state_of_the_longest_sequence(short_of, dtype):
    """The largest token count that is taken, ones without a decay: every element of the state is the count.  A state
    below 2^31 is off by at most 64 for each chunk that is added to it, of which a segment has less than 2^17 and no
    rounding comes from the sums of whole segments before it; a segment's tokens alone are 0.7 % at most."""
    N = (1 << 31) - 1 - (1 << 20)
    if dtype == torch.float32:      # one row, repeated
        k = torch.ones(1, 1, 1, 8, device=DEV).expand(1, 1, N, 8)
    else:                           # rows 16 bytes apart, as the tensor cores' path takes them
        k = torch.ones(1, 1, N, 8, dtype=dtype, device=DEV)
    S = torch.zeros(1, 1, 8, 8, device=DEV)
    lens = torch.tensor([N - short_of], dtype=torch.int32, device=DEV) if short_of else None
    la.la_decay_forward(None, k, k, torch.zeros(1, device=DEV), SN=S, lens=lens, want_out=False)
    off = (S.double() - (N - short_of)).abs().max()
    del k
    torch.cuda.empty_cache()
    assert off <= 64 * (1 << 17) < N // 200, float(off)


def _growing(dtype, seed):
    """Sequences that are cut into segments of some hundred tokens."""
    H, N = (40, 2000) if dtype == torch.float32 else (8, 5000)
    return H, N, inputs(1, H, N, 16, 16, dtype, seed, decays=[0.3] * H)


@pytest.mark.parametrize("dtype", DTYPES)
def test_growing_states_that_are_zero_stay_zero(dtype):
    """a^n over a segment is past fp32's range, but nothing is there yet to grow."""
    H, N, (q, k, v, dout, _, _, g) = _growing(dtype, 3)
    k[:, :, :N - 100] = 0.0
    SN = torch.empty(1, H, 16, 16, device=DEV)
    out = la.la_decay_forward(q, k, v, g, 0.25, SN=SN)
    qn, kn, vn, gn = (_np(t) for t in (q, k, v, g))
    ref, refS = decay.forward(qn, kn, vn, gn, 0.25)
    H_, HS = decay.forward(np.abs(qn), np.abs(kn), np.abs(vn), gn, 0.25)
    K = _k(N, 16)
    _rows("out", out, ref, H_, K, dtype)
    _close("SN", SN, refS, K * U * HS)
    # backwards in time: gradients of the first tokens' outputs alone
    q, k, v, dout = _growing(dtype, 4)[2][:4]
    dout[:, :, 100:] = 0.0
    dS0 = torch.empty_like(SN)
    dq, dk, dv = la.la_decay_backward(q, k, v, dout, g, 0.25, dS0=dS0)
    part = [_np(t[:, :, :100]) for t in (q, k, v, dout)]
    refs = decay.backward(*part, gn, 0.25)
    hs = decay.backward(*(np.abs(t) for t in part), gn, 0.25)
    for name, got, r, h in zip(("dq", "dk", "dv"), (dq, dk, dv), refs, hs):
        _rows(name, got[:, :, :100], r, h, K, dtype)
    assert not dk[:, :, 100:].any() and not dv[:, :, 100:].any()
    _close("dS0", dS0, refs[3], K * U * hs[3])


@pytest.mark.parametrize("dtype", DTYPES)
def test_growing_states_that_are_small(dtype):
    """a^n over a segment is past fp32's range, its product with a small state is not."""
    H, N, (q, k, v, dout, S0, dSN, _) = _growing(dtype, 5)
    S0, dSN = 1e-30 * S0, 1e-30 * dSN
    K = _k(N, 16)
    qn, kn, vn, Sn, En = (_np(t) for t in (q, k, v, S0, dSN))
    ab = [np.abs(t) for t in (qn, kn, vn, Sn, En)]
    n = 500                                     # a segment of 384 and the next
    g = torch.full((H,), 0.25, device=DEV)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    SN = torch.empty_like(S0)
    out = la.la_decay_forward(q, torch.zeros_like(k), v, g, 0.25, S0=S0, SN=SN, lens=lens)
    ref, refS = decay.forward(qn, 0 * kn, vn, _np(g), 0.25, Sn, [n])
    H_, HS = decay.forward(ab[0], 0 * kn, ab[2], _np(g), 0.25, ab[3], [n])
    _rows("out", out, ref, H_, K, dtype)
    _close("SN", SN, refS, K * U * HS)
    n, by = (620, 0.2) if dtype == torch.float32 else (1100, 0.11)     # backward segments of 512 and 896
    g, lens = torch.full((H,), by, device=DEV), torch.tensor([n], dtype=torch.int32, device=DEV)
    dS0 = torch.empty_like(S0)
    _, dk, dv = la.la_decay_backward(q, k, v, torch.zeros_like(dout), g, 0.25, dSN=dSN, dS0=dS0, lens=lens)
    refs = decay.backward(qn, kn, vn, 0 * vn, _np(g), 0.25, None, En, [n])
    hs = decay.backward(*ab[:3], 0 * vn, _np(g), 0.25, None, ab[4], [n])
    for name, got, r, h in zip(("dk", "dv"), (dk, dv), refs[1:], hs[1:]):
        _rows(name, got, r, h, K, dtype)
    _close("dS0", dS0, refs[3], K * U * hs[3])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [None, [31], [97]])
def test_growing_states(lens, dtype):
    check(1, 2, 150, 64, 64, dtype, decays=[0.5, 0.1], lens=lens)
