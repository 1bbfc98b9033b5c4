"""Pins of the fp64 oracle of the attention with decays and of the norm and
rotation (CPU): the quadratic definition, closed forms, finite differences,
chaining, and planted mistakes."""
import numpy as np
import pytest

from oracle import decay


def _draw(seed, B=2, H=3, N=7, D=4, M=5):
    r = np.random.default_rng(seed)
    q, k = r.standard_normal((2, B, H, N, D))
    v, dout = r.standard_normal((2, B, H, N, M))
    S0, dSN = r.standard_normal((2, B, H, D, M))
    return q, k, v, dout, S0, dSN, np.log(r.uniform(0.2, 1.0, H))


def _quadratic(q, k, v, g, scale, S0, skip_diagonal=False):
    """The definition with the sum over j <= i written out."""
    N = q.shape[2]
    i, j = np.arange(N)[:, None], np.arange(N)[None]
    with np.errstate(over="ignore", invalid="ignore"):
        W = np.where(j < i + (not skip_diagonal), np.exp(g[:, None, None] * np.abs(i - j)), 0.0)
    out = np.einsum("bhij,hij,bhjm->bhim", np.einsum("bhid,bhjd->bhij", q, k), W, v)
    seen = np.exp(g[:, None] * (np.arange(N) + 1))
    return scale * (out + np.einsum("hi,bhid,bhdm->bhim", seen, q, S0))


@pytest.mark.parametrize("seed", range(3))
def test_the_recurrence_is_the_quadratic_form(seed):
    q, k, v, _, S0, _, g = _draw(seed)
    out, _ = decay.forward(q, k, v, g, 0.7, S0)
    assert np.abs(out - _quadratic(q, k, v, g, 0.7, S0)).max() < 1e-12
    assert np.abs(out - _quadratic(q, k, v, g, 0.7, S0, skip_diagonal=True)).max() > 0.1


def test_extremes_of_the_decay():
    q, k, v, _, S0, _, _ = _draw(4)
    none = decay.forward(q, k, v, np.full(3, -np.inf), 1.0, S0)[0]       # the token alone
    assert np.abs(none - np.einsum("bhnd,bhnd->bhn", q, k)[..., None] * v).max() < 1e-12
    ever = decay.forward(q, k, v, np.zeros(3), 1.0, S0)[1]               # everything
    assert np.abs(ever - (S0 + np.einsum("bhnd,bhnm->bhdm", k, v))).max() < 1e-12


def test_lengths_end_a_sequence():
    q, k, v, dout, S0, dSN, g = _draw(5, B=4)
    lens = [0, 3, 7, 9]
    out, S = decay.forward(q, k, v, g, 1.0, S0, lens)
    grads = decay.backward(q, k, v, dout, g, 1.0, S0, dSN, lens)
    for b, n in enumerate([0, 3, 7, 7]):
        o, s = decay.forward(*(t[b:b + 1, :, :n] for t in (q, k, v)), g, 1.0, S0[b:b + 1])
        assert np.array_equal(out[b:b + 1, :, :n], o) and not out[b, :, n:].any() and np.array_equal(S[b:b + 1], s)
        part = decay.backward(*(t[b:b + 1, :, :n] for t in (q, k, v, dout)), g, 1.0, S0[b:b + 1], dSN[b:b + 1])
        for a, p in zip(grads[:3], part[:3]):
            assert np.array_equal(a[b:b + 1, :, :n], p) and not a[b, :, n:].any()
        assert np.array_equal(grads[3][b:b + 1], part[3])
    assert np.array_equal(S[0], S0[0]) and np.array_equal(grads[3][0], dSN[0])


def test_gradients_by_differences():
    q, k, v, dout, S0, dSN, g = _draw(6, N=5)

    def loss(q, k, v, S0):
        out, S = decay.forward(q, k, v, g, 0.6, S0)
        return (out * dout).sum() + (S * dSN).sum()
    grads = decay.backward(q, k, v, dout, g, 0.6, S0, dSN)
    rng = np.random.default_rng(0)
    for i, grad in enumerate(grads):
        args = [q, k, v, S0]
        step = rng.standard_normal(args[i].shape)
        h = 1e-6
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * step, args[i] - h * step
        want = (loss(*up) - loss(*down)) / (2 * h)
        assert abs(want - (grad * step).sum()) < 1e-6 * (1 + abs(want)), i


def test_segments_chain():
    q, k, v, dout, S0, dSN, g = _draw(7)
    whole, SN = decay.forward(q, k, v, g, 1.0, S0)
    a, S = decay.forward(*(t[:, :, :3] for t in (q, k, v)), g, 1.0, S0)
    b, S1 = decay.forward(*(t[:, :, 3:] for t in (q, k, v)), g, 1.0, S)
    assert np.abs(np.concatenate([a, b], 2) - whole).max() < 1e-12 and np.abs(S1 - SN).max() < 1e-12
    grads = decay.backward(q, k, v, dout, g, 1.0, S0, dSN)
    late = decay.backward(*(t[:, :, 3:] for t in (q, k, v, dout)), g, 1.0, S, dSN)
    early = decay.backward(*(t[:, :, :3] for t in (q, k, v, dout)), g, 1.0, S0, late[3])
    for w, e, l in zip(grads[:3], early, late):
        assert np.abs(np.concatenate([e, l], 2) - w).max() < 1e-12
    assert np.abs(early[3] - grads[3]).max() < 1e-12


@pytest.mark.parametrize("pairs", ["half", "adjacent"])
def test_rotation(pairs):
    r = np.random.default_rng(8)
    x = r.standard_normal((2, 3, 5, 8))
    pos = r.integers(-9, 9, (2, 2, 5))
    freq = np.array([1.0, 0.25, 0.5], dtype=np.float32)
    ang = decay.angles(pos, freq, [0, 1, 1])
    assert np.abs(np.cos(ang[..., 1]) - np.cos(0.25 * pos[1])).max() < 1e-14
    y = decay.turn(x, ang, pairs)
    assert np.abs((y * y).sum(-1) - (x * x).sum(-1)).max() < 1e-12       # lengths stay
    assert np.array_equal(y[..., 6:], x[..., 6:])                        # the rest stays
    assert np.abs(decay.turn(y, -ang, pairs) - x).max() < 1e-12
    # products depend on the difference of positions alone
    one = decay.angles(np.full((2, 2, 5), 3), freq, [0, 1, 1])
    shifted = decay.turn(x, ang + one, pairs) * decay.turn(x[::-1], ang + one, pairs)
    assert np.abs(shifted.sum(-1) - (y * decay.turn(x[::-1], ang, pairs)).sum(-1)).max() < 1e-12
    # a quarter turn of (1, 0) is (0, 1)
    e = np.zeros((1, 1, 1, 4))
    e[..., 0] = 1.0
    got = decay.turn(e, np.full((1, 1, 2), np.pi / 2), pairs)
    want = np.zeros(4)
    want[2 if pairs == "half" else 1] = 1.0
    assert np.abs(got[0, 0, 0] - want).max() < 1e-15


@pytest.mark.parametrize("pairs", ["half", "adjacent"])
@pytest.mark.parametrize("norm", [True, False])
def test_rotation_gradients_by_differences(pairs, norm):
    r = np.random.default_rng(9)
    x, dy, step = r.standard_normal((3, 2, 3, 4, 6))
    w, dw = r.standard_normal((2, 6))
    ang = r.uniform(-3, 3, (2, 4, 2))
    w = w if norm else None

    def loss(x, w):
        return (decay.rotate(x, ang, w, 0.1, norm, pairs) * dy).sum()
    gx, gw = decay.rotate_backward(dy, x, ang, w, 0.1, norm, pairs)
    h = 1e-6
    want = (loss(x + h * step, w) - loss(x - h * step, w)) / (2 * h)
    assert abs(want - (gx * step).sum()) < 1e-6 * (1 + abs(want))
    if norm:
        want = (loss(x, w + h * dw) - loss(x, w - h * dw)) / (2 * h)
        assert abs(want - (gw * dw).sum()) < 1e-6 * (1 + abs(want))
