"""The layer with a decay for each head: binding of ttt_la_forward_decay,
ttt_la_backward_decay and ttt_la_decode_step_decay (include/ttt_la.h).

    W_t = gamma_h W_{t-1} + a v_t k_t^T ,  o_t = W_t q_t ,  gamma_h = exp(log_decay[h])

q, k [B,H,T,d_k] and v [B,H,T,d_v] may have any memory order whose features
are contiguous and whose rows start on 16 bytes: ``x.view(B, T, H, d)
.transpose(1, 2)`` of a projection's output goes in as it is, and outputs come
back in the order of their inputs.  With ``cu_seqlens`` (int32 CUDA tensor of
N + 1 row offsets) B is 1 and the T rows hold N sequences one behind another.
The tensors' device need not be the current one; work goes to ``stream``, by
default the current stream of that device.
"""
from __future__ import annotations

import math

import torch

from . import _abi
from ._call import FORMATS, check, check_distinct_rows, check_rows, launch_on, on_stream, run, run_with_workspace
from .norm import check_group_norm, group_norm

_FORWARD = FORMATS["ttt_la_decay_args"].pack
_BACKWARD = FORMATS["ttt_la_decay_grad_args"].pack
_STEP = FORMATS["ttt_la_decay_decode_args"].pack


def _shapes(q, k, v, log_decay, cu_seqlens):
    if q.dim() != 4 or k.shape != q.shape or v.dim() != 4 or v.shape[:3] != q.shape[:3]:
        raise ValueError("q, k: [B,H,T,d_k]; v: [B,H,T,d_v]")
    B, H, T, dk = q.shape
    dev, N = q.device, B
    if cu_seqlens is not None:
        if B != 1 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("packed sequences: B = 1 and cu_seqlens of N + 1 offsets")
        N = cu_seqlens.numel() - 1
        check(cu_seqlens, "cu_seqlens", torch.int32, dev)
    check(log_decay, "log_decay", torch.float32, dev, (H,))
    return N, H, T, dk, v.shape[-1], dev


def _default_eta(eta_const, dk):
    return 1.0 / math.sqrt(dk) if eta_const is None else float(eta_const)


def forward_decay(q, k, v, log_decay, eta_const=None, ascent=False, cu_seqlens=None, state_in=None,
                  return_state=True, out=None, state_out=None, workspace=None, segment_tokens=0, clear_rest=False,
                  stream=None):
    """Whole sequences (ttt_la_forward_decay).  Returns (o, W_T), W_T None
    when not requested.  ``eta_const`` defaults to 1/sqrt(d_k).  ``out``,
    ``state_out`` (which may be ``state_in``) and ``workspace`` may be
    preallocated; ``segment_tokens`` (a multiple of 64) overrides the
    automatic split of long sequences; with ``clear_rest`` the rows of o in no
    packed sequence are zeros instead of what was there."""
    N, H, T, dk, dv, dev = _shapes(q, k, v, log_decay, cu_seqlens)
    dt, code, state_shape = q.dtype, _abi._dtype_code(q), (N, H, dv, dk)

    def call(handle):
        nonlocal out, state_out
        if out is None:
            out = torch.empty_like(v)
        else:
            check_distinct_rows(out, "out")
        if return_state and state_out is None:
            state_out = torch.empty(state_shape, device=dev, dtype=torch.float32)
        (pq, sq), (pk, sk) = check_rows(q, "q", dt, dev, q.shape), check_rows(k, "k", dt, dev, q.shape)
        (pv, sv), (po, so) = check_rows(v, "v", dt, dev, v.shape), check_rows(out, "out", dt, dev, v.shape)
        block = _FORWARD(
            N, H, T, dk, dv, code, pq, pk, pv, po, *sq[:3], *sk[:3], *sv[:3], *so[:3], log_decay.data_ptr(),
            0 if cu_seqlens is None else cu_seqlens.data_ptr(), _default_eta(eta_const, dk), 1 if ascent else 0,
            check(state_in, "state_in", torch.float32, dev, state_shape),
            check(state_out, "state_out", torch.float32, dev, state_shape) if return_state else 0, int(segment_tokens),
            1 if clear_rest else 0)
        run_with_workspace("ttt_la_forward_decay", "ttt_la_decay_workspace_size", block, workspace, dev, handle)

    launch_on(dev, stream, call)
    return out, state_out if return_state else None


def backward_decay(q, k, v, grad_o, log_decay, eta_const=None, ascent=False, cu_seqlens=None, state_in=None,
                   grad_state=None, workspace=None, segment_tokens=0, stream=None):
    """Gradients of forward_decay (ttt_la_backward_decay) for dL/do and,
    optionally, dL/dW_T: a dict with dq, dk, dv (dtype and memory order of q,
    k, v) and dW0 [N,H,d_v,d_k] fp32."""
    N, H, T, dk, dv, dev = _shapes(q, k, v, log_decay, cu_seqlens)
    dt, code, state_shape = q.dtype, _abi._dtype_code(q), (N, H, dv, dk)
    g = {}

    def call(handle):
        ins = [check_rows(*x) for x in ((q, "q", dt, dev, q.shape), (k, "k", dt, dev, q.shape),
                                        (v, "v", dt, dev, v.shape), (grad_o, "grad_o", dt, dev, v.shape))]
        g.update(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
                 dW0=torch.empty(state_shape, device=dev, dtype=torch.float32))
        ts = ins + [(g[n].data_ptr(), g[n].stride()) for n in ("dq", "dk", "dv")]
        block = _BACKWARD(
            N, H, T, dk, dv, code, *(p for p, _ in ts), *(x for _, st in ts for x in st[:3]), log_decay.data_ptr(),
            0 if cu_seqlens is None else cu_seqlens.data_ptr(), _default_eta(eta_const, dk), 1 if ascent else 0,
            check(state_in, "state_in", torch.float32, dev, state_shape),
            check(grad_state, "grad_state", torch.float32, dev, state_shape), g["dW0"].data_ptr(), int(segment_tokens))
        run_with_workspace("ttt_la_backward_decay", "ttt_la_backward_decay_workspace_size", block, workspace, dev, handle)

    launch_on(dev, stream, call)
    return g


def decode_step_decay(q, k, v, log_decay, state, eta_const=None, ascent=False, out=None, stream=None):
    """One new token of each of N sequences (ttt_la_decode_step_decay): q, k
    [N,H,d_k], v [N,H,d_v]; state [N,H,d_v,d_k] fp32, updated in place.  d_k
    is 32, 64 or 128 (a prompt takes more widths than the step), d_v any.
    Returns o [N,H,d_v]."""
    if q.dim() != 3 or k.shape != q.shape or v.dim() != 3 or v.shape[:2] != q.shape[:2]:
        raise ValueError("q, k: [N,H,d_k]; v: [N,H,d_v]")
    N, H, dk = q.shape
    dv, dev, dt = v.shape[-1], q.device, q.dtype
    code = _abi._dtype_code(q)

    def call(handle):
        nonlocal out
        if out is None:
            out = torch.empty_like(v)
        else:
            check_distinct_rows(out, "out")
        (pq, sq), (pk, sk) = check_rows(q, "q", dt, dev, q.shape), check_rows(k, "k", dt, dev, q.shape)
        (pv, sv), (po, so) = check_rows(v, "v", dt, dev, v.shape), check_rows(out, "out", dt, dev, v.shape)
        run("ttt_la_decode_step_decay", _STEP(
            N, H, dk, dv, code, pq, pk, pv, po, *sq[:2], *sk[:2], *sv[:2], *so[:2],
            check(log_decay, "log_decay", torch.float32, dev, (H,)), _default_eta(eta_const, dk), 1 if ascent else 0,
            check(state, "state", torch.float32, dev, (N, H, dv, dk))), handle)

    launch_on(dev, stream, call)
    return out


def forward_decay_norm(q, k, v, log_decay, gate=None, weight=None, bias=None, activation="silu", eps=1e-5, stream=None,
                       **kw):
    """The layer and its output norm: forward_decay, then every head's output
    of a token normalised by itself and gated (group_norm with one group a
    head).  gate [B,T,H*d_v] or None, in any memory order (one that is not
    contiguous, or starts off 16 bytes, is copied); weight, bias [H*d_v] or
    None.  Keyword arguments as forward_decay.  Returns (y [B,T,H*d_v], W_T),
    y empty where there are no rows.  What either operator refuses is refused
    before the layer runs."""
    B, H, T, dv = v.shape
    if gate is not None and tuple(gate.shape) != (B, T, H * dv):
        raise ValueError("gate: [B,T,H*d_v]")
    if kw.pop("out", None) is not None:
        raise ValueError("forward_decay_norm allocates its output")
    rows = (B * T, 1, H * dv)
    with on_stream(v.device, stream):  # all of the call: a copy made here is read, and its memory used again, there
        if gate is not None:
            gate = gate.contiguous()
            gate = (gate.clone() if gate.data_ptr() % 16 else gate).view(rows)
        o = torch.empty(B, T, H, dv, device=v.device, dtype=v.dtype)
        x, y = o.view(rows), torch.empty(rows, device=v.device, dtype=v.dtype)
        # before the layer, which may update its state in place
        check_group_norm(x, H, weight, bias, gate, activation, eps)
        # (the norm reads all rows)
        _, W = forward_decay(q, k, v, log_decay, out=o.transpose(1, 2), stream=stream, **{**kw, "clear_rest": True})
        if B * T > 0:
            group_norm(x, H, weight, bias, gate=gate, activation=activation, eps=eps, out=y, stream=stream)
    return y.view(B, T, H * dv), W
