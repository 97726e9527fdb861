"""Float64 CPU oracle for the layer with a decay for each head, its gradient,
and the output group norm with its gradient.

TEST INFRASTRUCTURE ONLY: nothing on the product path imports this module.  It
shares no code with the CUDA library.

The layer, token by token (gamma_h = exp(log_decay[h]), a = sigma * eta):

  W_t = gamma W_{t-1} + a v_t k_t^T ,   o_t = W_t q_t

and its gradient for dO and dL/dW_T, with G_t = dL/dW_t (everything W_t
reaches: o_t and W_{t+1}):

  G_t = gamma G_{t+1} + do_t q_t^T  (gamma G_{T+1} := dL/dW_T)
  dq_t = W_t^T do_t ,  dv_t = a G_t k_t ,  dk_t = a G_t^T v_t ,  dW_0 = gamma G_1

Arrays are [..., H, T, d] with log_decay [H]; states [..., H, d_v, d_k].
``tests/test_oracle_decay.py`` pins both by closed sums over pairs of tokens
and by central differences.
"""
from __future__ import annotations

import numpy as np

__all__ = ["decay_forward_f64", "decay_backward_f64", "group_norm_f64", "group_norm_backward_f64"]


def _gamma(log_decay):
    return np.exp(np.asarray(log_decay, dtype=np.float64))[..., None, None]


def decay_forward_f64(q, k, v, log_decay, a, W0=None):
    """(o, W_T) by the recurrence."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    lead, T = q.shape[:-2], q.shape[-2]
    W = np.zeros(lead + (v.shape[-1], q.shape[-1])) if W0 is None else np.array(W0, dtype=np.float64)
    g = _gamma(log_decay)
    o = np.zeros(v.shape)
    for t in range(T):
        W = g * W + a * v[..., t, :, None] * k[..., t, None, :]
        o[..., t, :] = np.einsum("...vk,...k->...v", W, q[..., t, :])
    return o, W


def decay_backward_f64(q, k, v, dO, log_decay, a, W0=None, dW_T=None):
    """A dict with dq, dk, dv and dW0."""
    q, k, v, dO = (np.asarray(x, dtype=np.float64) for x in (q, k, v, dO))
    lead, T = q.shape[:-2], q.shape[-2]
    shape = lead + (v.shape[-1], q.shape[-1])
    W = np.zeros(shape) if W0 is None else np.array(W0, dtype=np.float64)
    G = np.zeros(shape) if dW_T is None else np.array(dW_T, dtype=np.float64)
    g = _gamma(log_decay)
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for t in range(T):
        W = g * W + a * v[..., t, :, None] * k[..., t, None, :]
        dq[..., t, :] = np.einsum("...vk,...v->...k", W, dO[..., t, :])
    for t in range(T - 1, -1, -1):
        G = G + dO[..., t, :, None] * q[..., t, None, :]
        dv[..., t, :] = a * np.einsum("...vk,...k->...v", G, k[..., t, :])
        dk[..., t, :] = a * np.einsum("...vk,...v->...k", G, v[..., t, :])
        G = g * G
    return {"dq": dq, "dk": dk, "dv": dv, "dW0": G}


def _sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def group_norm_f64(x, groups, weight=None, bias=None, gate=None, silu=True, eps=1e-5):
    """(y, mean, rstd) of x [N, ..., C], channels last: statistics over each
    (sample, group); y = act(t) or t * act(gate), t = hat * weight + bias."""
    x = np.asarray(x, dtype=np.float64)
    n, c = x.shape[0], x.shape[-1]
    xg = x.reshape(n, -1, groups, c // groups)
    mean = xg.mean(axis=(1, 3))
    rstd = 1.0 / np.sqrt(((xg - mean[:, None, :, None]) ** 2).mean(axis=(1, 3)) + eps)
    t = ((xg - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(x.shape)
    t = t * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)
    z = t if gate is None else np.asarray(gate, dtype=np.float64)
    act = z * _sigmoid(z) if silu else z
    return (act if gate is None else t * act), mean, rstd


def group_norm_backward_f64(dy, x, groups, mean, rstd, weight=None, bias=None, gate=None, silu=True):
    """A dict with dx, dweight, dbias and dgate (None without a gate), from
    the given statistics."""
    x, dy = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    n, c = x.shape[0], x.shape[-1]
    shape = (n, -1, groups, c // groups)
    w = np.ones(c) if weight is None else np.asarray(weight, dtype=np.float64)
    b = np.zeros(c) if bias is None else np.asarray(bias, dtype=np.float64)
    mean, rstd = (np.asarray(s, dtype=np.float64)[:, None, :, None] for s in (mean, rstd))
    hat = ((x.reshape(shape) - mean) * rstd).reshape(x.shape)
    t = hat * w + b
    z = t if gate is None else np.asarray(gate, dtype=np.float64)
    s = _sigmoid(z)
    slope = s * (1.0 + z * (1.0 - s)) if silu else np.ones_like(z)
    dgate = None
    if gate is None:
        dt = dy * slope
    else:
        dt = dy * (z * s if silu else z)
        dgate = dy * t * slope
    dh, hg = (dt * w).reshape(shape), hat.reshape(shape)
    dx = rstd * (dh - dh.mean(axis=(1, 3), keepdims=True) - hg * (dh * hg).mean(axis=(1, 3), keepdims=True))
    axes = tuple(range(x.ndim - 1))
    return {"dx": dx.reshape(x.shape), "dweight": (dt * hat).sum(axis=axes), "dbias": dt.sum(axis=axes),
            "dgate": dgate}
