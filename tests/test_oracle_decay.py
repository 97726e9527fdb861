"""Pins the float64 oracle of the decayed layer and of the group norm: closed
sums over pairs of tokens, agreement with the undecayed layer's oracle, and
central differences of every gradient."""
import numpy as np
import pytest

import oracle

RNG = np.random.default_rng(11)


def _case(H=2, T=7, dk=3, dv=4):
    q, k, v, dO = (RNG.standard_normal((H, T, d)) for d in (dk, dk, dv, dv))
    return q, k, v, dO, np.array([-0.7, -0.05])[:H], RNG.standard_normal((H, dv, dk)), RNG.standard_normal((H, dv, dk))


def test_forward_is_the_sum_over_pairs():
    q, k, v, _, ld, W0, _ = _case()
    o, W = oracle.decay_forward_f64(q, k, v, ld, 0.3, W0)
    T = q.shape[1]
    for h in range(2):
        g = np.exp(ld[h])
        for t in range(T):
            ref = g ** (t + 1) * W0[h] @ q[h, t]
            for s in range(t + 1):
                ref = ref + 0.3 * g ** (t - s) * (q[h, t] @ k[h, s]) * v[h, s]
            np.testing.assert_allclose(o[h, t], ref, rtol=0, atol=1e-12)
        end = g ** T * W0[h] + sum(0.3 * g ** (T - 1 - s) * np.outer(v[h, s], k[h, s]) for s in range(T))
        np.testing.assert_allclose(W[h], end, rtol=0, atol=1e-12)


def test_without_decay_it_is_the_plain_layer():
    q, k, v, dO, _, W0, dWT = _case()
    o, W = oracle.decay_forward_f64(q, k, v, np.zeros(2), 0.25, W0)
    o2, W2, _ = oracle.ttt_recurrence_f64(q[None], k[None], v[None], 0.25, S0=W0[None])
    np.testing.assert_allclose(o, o2[0], atol=1e-13)
    np.testing.assert_allclose(W, W2[0], atol=1e-13)
    g = oracle.decay_backward_f64(q, k, v, dO, np.zeros(2), 0.25, W0, dWT)
    r = oracle.ttt_backward_f64(q[None], k[None], v[None], 0.25, dO[None], dW_T=dWT[None], S0=W0[None])
    for n in ("dq", "dk", "dv", "dW0"):
        np.testing.assert_allclose(g[n], r[n][0], atol=1e-12)


def test_infinite_decay_sees_one_token():
    q, k, v, _, _, W0, _ = _case()
    o, _ = oracle.decay_forward_f64(q, k, v, np.array([-np.inf, -np.inf]), 0.5, W0)
    np.testing.assert_allclose(o, 0.5 * np.einsum("htd,htd->ht", q, k)[..., None] * v, atol=1e-13)


def _differences(f, x, g, h=1e-6):
    """<g, d> against the central difference of f along random directions d."""
    for _ in range(3):
        d = RNG.standard_normal(x.shape)
        num = (f(x + h * d) - f(x - h * d)) / (2 * h)
        assert abs(num - np.sum(g * d)) <= 1e-7 * (1.0 + np.abs(g * d).sum())


def test_layer_gradient_by_differences():
    q, k, v, dO, ld, W0, dWT = _case()

    def loss(q_, k_, v_, w_):
        o, W = oracle.decay_forward_f64(q_, k_, v_, ld, -0.4, w_)
        return np.sum(o * dO) + np.sum(W * dWT)

    g = oracle.decay_backward_f64(q, k, v, dO, ld, -0.4, W0, dWT)
    _differences(lambda x: loss(x, k, v, W0), q, g["dq"])
    _differences(lambda x: loss(q, x, v, W0), k, g["dk"])
    _differences(lambda x: loss(q, k, x, W0), v, g["dv"])
    _differences(lambda x: loss(q, k, v, x), W0, g["dW0"])


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("gated", [True, False])
def test_group_norm_gradient_by_differences(silu, gated):
    x, dy = RNG.standard_normal((2, 5, 6)), RNG.standard_normal((2, 5, 6))
    gate = RNG.standard_normal(x.shape) if gated else None
    w, b = RNG.standard_normal(6), RNG.standard_normal(6)

    def loss(x_, w_, b_, z_):
        return np.sum(oracle.group_norm_f64(x_, 3, w_, b_, z_, silu)[0] * dy)

    _, mean, rstd = oracle.group_norm_f64(x, 3, w, b, gate, silu)
    g = oracle.group_norm_backward_f64(dy, x, 3, mean, rstd, w, b, gate, silu)
    _differences(lambda t: loss(t, w, b, gate), x, g["dx"])
    _differences(lambda t: loss(x, t, b, gate), w, g["dweight"])
    _differences(lambda t: loss(x, w, t, gate), b, g["dbias"])
    if gated:
        _differences(lambda t: loss(x, w, b, t), gate, g["dgate"])


def test_group_norm_by_hand():
    x = np.array([[[1.0, 3.0, 10.0, 10.0]]])
    y, mean, rstd = oracle.group_norm_f64(x, 2, silu=False, eps=0.0625)
    np.testing.assert_allclose(mean, [[2.0, 10.0]])
    np.testing.assert_allclose(rstd, [[1 / np.sqrt(1.0625), 4.0]])
    np.testing.assert_allclose(y[0, 0], [-1 / np.sqrt(1.0625), 1 / np.sqrt(1.0625), 0.0, 0.0])
