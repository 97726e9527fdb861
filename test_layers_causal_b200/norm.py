"""Group norm over channels-last data with its activation: binding of
ttt_la_group_norm and ttt_la_group_norm_backward (include/ttt_la.h)."""
from __future__ import annotations

import torch

from . import _abi
from ._call import FORMATS, check, launch_on, run_with_workspace

_FORWARD = FORMATS["ttt_la_group_norm_args"].pack
_BACKWARD = FORMATS["ttt_la_group_norm_grad_args"].pack
_ACTIVATIONS = {None: 0, "none": 0, "silu": 1}


def _describe(x, num_groups, weight, bias, gate, activation, empty=False):
    if x.dim() < 2:
        raise ValueError("x: [N, ..., C], channels last")
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation: one of {sorted(map(str, _ACTIVATIONS))}")
    N, C = x.shape[0], x.shape[-1]
    if C < 1 or (x.numel() == 0 and not empty):
        raise ValueError("x is empty")
    G = int(num_groups)
    if G < 1 or C % G:
        raise ValueError("num_groups must divide the channels")
    dev, dt = x.device, x.dtype
    params = [p for p in (weight, bias) if p is not None]
    pdt = params[0].dtype if params else torch.float32
    if pdt not in (torch.float32, dt):
        raise TypeError("weight and bias: fp32 or the dtype of x")
    pointers = (check(x, "x", dt, dev), check(gate, "gate", dt, dev, x.shape),
                check(weight, "weight", pdt, dev, (C,)), check(bias, "bias", pdt, dev, (C,)))
    return N, x.numel() // max(N * C, 1), C, G, _abi._dtype_code(x), _abi.BF16 if pdt == torch.bfloat16 else _abi.F32, \
        _ACTIVATIONS[activation], pointers, pdt


def check_group_norm(x, num_groups, weight, bias, gate, activation, eps):
    """Refuses what group_norm refuses, without a launch, for callers whose own
    work comes before the norm; x may hold no rows."""
    G = _describe(x, num_groups, weight, bias, gate, activation, empty=True)[3]
    if not 0 <= eps < 2.0 ** 128:
        raise _abi.TttError("ttt_la_group_norm", _abi.ERR_INVALID_ARG)
    if G > 4096:
        raise _abi.TttError("ttt_la_group_norm", _abi.ERR_UNSUPPORTED)


def group_norm(x, num_groups, weight=None, bias=None, gate=None, activation="silu", eps=1e-5, out=None,
               workspace=None, stream=None):
    """y = act(t), or t * act(gate), of t = (x - mean) * rstd * weight + bias,
    the statistics over each (sample, group) of x [N, ..., C]
    (ttt_la_group_norm).  activation: "silu" or None.  Returns (y, mean, rstd)
    with mean, rstd fp32 [N,G], which the gradient takes."""
    N, L, C, G, code, pcode, act, (px, pg, pw, pb), _ = _describe(x, num_groups, weight, bias, gate, activation)
    dev = x.device
    stats = None

    def call(handle):
        nonlocal out, stats
        if out is None:
            out = torch.empty_like(x)
        stats = torch.empty((2, N, G), device=dev, dtype=torch.float32)
        mean = stats.data_ptr()
        block = _FORWARD(N, L, C, G, code, pcode, act, eps, px, pg, pw, pb, check(out, "out", x.dtype, dev, x.shape), mean,
                         mean + 4 * N * G)
        run_with_workspace("ttt_la_group_norm", "ttt_la_group_norm_workspace_size", block, workspace, dev, handle)

    launch_on(dev, stream, call)
    mean, rstd = stats.unbind(0)
    return out, mean, rstd


def group_norm_backward(grad_y, x, num_groups, mean, rstd, weight=None, bias=None, gate=None, activation="silu",
                        workspace=None, stream=None):
    """Gradients of group_norm (ttt_la_group_norm_backward) from what the
    forward took and its mean and rstd: a dict with dx, dgate (None without a
    gate), dweight and dbias (None without the parameter)."""
    N, L, C, G, code, pcode, act, (px, pg, pw, pb), pdt = _describe(x, num_groups, weight, bias, gate, activation)
    dev = x.device
    out = {}

    def call(handle):
        pgy = check(grad_y, "grad_y", x.dtype, dev, x.shape)
        pm = check(mean, "mean", torch.float32, dev, (N, G))
        pr = check(rstd, "rstd", torch.float32, dev, (N, G))
        new = lambda like: None if like is None else torch.empty_like(like)  # noqa: E731
        out.update(dx=new(x), dgate=new(gate), dweight=new(weight), dbias=new(bias))
        ptr = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
        block = _BACKWARD(N, L, C, G, code, pcode, act, pgy, px, pg, pw, pb, pm, pr, ptr(out["dx"]), ptr(out["dgate"]),
                          ptr(out["dweight"]), ptr(out["dbias"]))
        run_with_workspace("ttt_la_group_norm_backward", "ttt_la_group_norm_backward_workspace_size", block, workspace, dev,
                           handle)

    launch_on(dev, stream, call)
    return out
