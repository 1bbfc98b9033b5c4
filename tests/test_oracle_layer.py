"""The oracle of the operators around the attention (oracle/layer.py) pinned by
closed forms, finite differences and planted mistakes (CPU)."""
import numpy as np
import pytest

from oracle import layer

GATES = ["decay", "log", "sigmoid"]


def _case(seed, shape=(2, 2, 7, 3)):
    rng = np.random.default_rng(seed)
    x, dout = rng.standard_normal(shape), rng.standard_normal(shape)
    state = shape[:2] + shape[3:]
    return x, rng.uniform(-0.9, 0.9, shape), dout, rng.standard_normal(state), rng.standard_normal(state)


def test_constant_decay_is_a_geometric_sum():
    x = np.ones((1, 1, 20, 1))
    out, hN = layer.recurrence(x, np.full_like(x, 0.5), "decay")
    np.testing.assert_allclose(out[0, 0, :, 0], 2.0 - 0.5 ** np.arange(20), rtol=1e-15)
    assert hN[0, 0, 0] == out[0, 0, -1, 0]


def test_sigmoid_gate_is_a_weighted_mean():
    """u = (1 - a) x: a constant input that is also the state stays where it is."""
    x = np.full((1, 1, 9, 2), 3.0)
    out, _ = layer.recurrence(x, np.random.default_rng(0).standard_normal(x.shape), "sigmoid", np.full((1, 1, 2), 3.0))
    np.testing.assert_allclose(out, 3.0, rtol=1e-14)


def test_lengths_bound_the_sequences():
    x, g, _, h0, _ = _case(1)
    out, hN = layer.recurrence(x, g, "decay", h0, lens=[0, 4])
    assert not out[0].any() and not out[1, :, 4:].any()
    np.testing.assert_array_equal(hN[0], h0[0])
    part, hp = layer.recurrence(x[1:, :, :4], g[1:, :, :4], "decay", h0[1:])
    np.testing.assert_array_equal(out[1:, :, :4], part)
    np.testing.assert_array_equal(hN[1:], hp)


def _num(f, v, h=1e-6):
    d = np.zeros_like(v)
    for i in np.ndindex(v.shape):
        p, m = v.copy(), v.copy()
        p[i] += h
        m[i] -= h
        d[i] = (f(p) - f(m)) / (2 * h)
    return d


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("lens", [None, [3, 7]])
def test_recurrence_backward_matches_differences(gate, lens):
    x, g, dout, h0, dhN = _case(2)

    def loss(x, g, h0):
        out, hN = layer.recurrence(x, g, gate, h0, lens)
        return float((out * dout).sum() + (hN * dhN).sum())
    got = layer.recurrence_backward(x, g, gate, dout, h0, dhN, lens)
    want = (_num(lambda v: loss(v, g, h0), x), _num(lambda v: loss(x, v, h0), g), _num(lambda v: loss(x, g, v), h0))
    for a, b in zip(got, want):
        np.testing.assert_allclose(a, b, rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("mistake", ["no carry", "h of this token", "gate of this token"])
def test_planted_recurrence_mistake_is_caught(mistake):
    x, g, dout, h0, dhN = _case(3)
    dx, dg, _ = layer.recurrence_backward(x, g, "decay", dout, h0, dhN)
    if mistake == "no carry":
        bad, ref = dout, dx
    elif mistake == "h of this token":
        bad, ref = dx * layer.recurrence(x, g, "decay", h0)[0], dg
    else:
        shifted = np.concatenate([g[:, :, :1], g[:, :, :-1]], axis=2)
        bad, ref = layer.recurrence_backward(x, shifted, "decay", dout, h0, dhN)[0], dx
    assert np.abs(bad - ref).max() > 1e-2


def test_layernorm_rows_have_mean_b_and_deviation_w():
    rng = np.random.default_rng(4)
    y, mean, rstd = layer.layernorm(5.0 + 3.0 * rng.standard_normal((4, 4000)), eps=0.0)
    np.testing.assert_allclose(y.mean(axis=1), 0.0, atol=1e-12)
    np.testing.assert_allclose(y.std(axis=1), 1.0, rtol=1e-12)
    np.testing.assert_allclose(mean, 5.0, atol=0.2)
    np.testing.assert_allclose(rstd, 1 / 3.0, rtol=0.05)


def test_layernorm_backward_matches_differences():
    rng = np.random.default_rng(5)
    s, dy, dsum = rng.standard_normal((3, 3, 5))
    w, b = rng.standard_normal((2, 5))

    def loss(s, w, b):
        return float((layer.layernorm(s, w, b, 1e-3)[0] * dy).sum() + (s * dsum).sum())
    got = layer.layernorm_backward(dy, s, w, 1e-3, dsum)
    want = (_num(lambda v: loss(v, w, b), s), _num(lambda v: loss(s, v, b), w), _num(lambda v: loss(s, w, v), b))
    for a, r in zip(got, want):
        np.testing.assert_allclose(a, r, rtol=1e-6, atol=1e-8)


def test_global_norm():
    assert layer.global_norm([np.array([3.0]), np.array([[4.0], [12.0]]), np.zeros(0)]) == 13.0
