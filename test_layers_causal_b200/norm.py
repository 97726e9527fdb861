"""Group norm over channels-last data with its activation: binding of
ttt_la_group_norm and ttt_la_group_norm_backward (include/ttt_la.h)."""
from __future__ import annotations

import ctypes

import torch

from . import _abi

_byref = ctypes.byref
_ACTIVATIONS = {None: 0, "none": 0, "silu": 1}


def _describe(x, num_groups, weight, bias, gate, activation):
    from .decay import need
    if x.dim() < 2:
        raise ValueError("x: [N, ..., C], channels last")
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation: one of {sorted(map(str, _ACTIVATIONS))}")
    N, C = x.shape[0], x.shape[-1]
    if N < 1 or C < 1 or x.numel() == 0:
        raise ValueError("x is empty")
    G = int(num_groups)
    if G < 1 or C % G:
        raise ValueError("num_groups must divide the channels")
    dev, dt = x.device, x.dtype
    params = [p for p in (weight, bias) if p is not None]
    pdt = params[0].dtype if params else torch.float32
    if pdt not in (torch.float32, dt):
        raise TypeError("weight and bias: fp32 or the dtype of x")
    pointers = (need(x, "x", dt, dev), need(gate, "gate", dt, dev, tuple(x.shape)),
                need(weight, "weight", pdt, dev, (C,)), need(bias, "bias", pdt, dev, (C,)))
    return N, x.numel() // (N * C), C, G, _abi._dtype_code(x), _abi.BF16 if pdt == torch.bfloat16 else _abi.F32, \
        _ACTIVATIONS[activation], pointers, pdt


def group_norm(x, num_groups, weight=None, bias=None, gate=None, activation="silu", eps=1e-5, out=None,
               workspace=None, stream=None):
    """y = act(t), or t * act(gate), of t = (x - mean) * rstd * weight + bias,
    the statistics over each (sample, group) of x [N, ..., C]
    (ttt_la_group_norm).  activation: "silu" or None.  Returns (y, mean, rstd)
    with mean, rstd fp32 [N,G], which the gradient takes."""
    from .decay import _workspace, launch_on, need
    N, L, C, G, code, pcode, act, (px, pg, pw, pb), _ = _describe(x, num_groups, weight, bias, gate, activation)
    dev = x.device
    stats = None

    def call(handle):
        nonlocal out, stats
        if out is None:
            out = torch.empty_like(x)
        stats = torch.empty((2, N, G), device=dev, dtype=torch.float32)
        a = _abi.TttGroupNormArgs(N, L, C, G, code, pcode, act, float(eps), px, pg, pw, pb,
                                  need(out, "out", x.dtype, dev, tuple(x.shape)), stats[0].data_ptr(),
                                  stats[1].data_ptr())
        lib = _abi.lib()
        nbytes = lib.ttt_la_group_norm_workspace_size(_byref(a))
        if nbytes:
            w = _workspace(workspace, nbytes, dev)
            a.workspace, a.workspace_bytes = w.data_ptr(), w.numel() * w.element_size()
        _abi._check("ttt_la_group_norm", lib.ttt_la_group_norm(_byref(a), handle))

    launch_on(dev, stream, call)
    return out, stats[0], stats[1]


def group_norm_backward(grad_y, x, num_groups, mean, rstd, weight=None, bias=None, gate=None, activation="silu",
                        workspace=None, stream=None):
    """Gradients of group_norm (ttt_la_group_norm_backward) from what the
    forward took and its mean and rstd: a dict with dx, dgate (None without a
    gate), dweight and dbias (None without the parameter)."""
    from .decay import _workspace, launch_on, need
    N, L, C, G, code, pcode, act, (px, pg, pw, pb), pdt = _describe(x, num_groups, weight, bias, gate, activation)
    dev = x.device
    out = {}

    def call(handle):
        pgy = need(grad_y, "grad_y", x.dtype, dev, tuple(x.shape))
        pm = need(mean, "mean", torch.float32, dev, (N, G))
        pr = need(rstd, "rstd", torch.float32, dev, (N, G))
        new = lambda like: None if like is None else torch.empty_like(like)  # noqa: E731
        out.update(dx=new(x), dgate=new(gate), dweight=new(weight), dbias=new(bias))
        ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        a = _abi.TttGroupNormGradArgs(N, L, C, G, code, pcode, act, pgy, px, pg, pw, pb, pm, pr, ptr(out["dx"]),
                                      ptr(out["dgate"]), ptr(out["dweight"]), ptr(out["dbias"]))
        lib = _abi.lib()
        nbytes = lib.ttt_la_group_norm_backward_workspace_size(_byref(a))
        if nbytes:
            w = _workspace(workspace, nbytes, dev)
            a.workspace, a.workspace_bytes = w.data_ptr(), w.numel() * w.element_size()
        _abi._check("ttt_la_group_norm_backward", lib.ttt_la_group_norm_backward(_byref(a), handle))

    launch_on(dev, stream, call)
    return out
