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

import contextlib
import ctypes
import math

import torch

from . import _abi
from .norm import group_norm

_I3 = ctypes.c_int64 * 3
_I2 = ctypes.c_int64 * 2
_byref = ctypes.byref


@contextlib.contextmanager
def on_stream(device, stream):
    """The tensors' device and the call's stream made current, so that what the
    call allocates belongs to the stream that uses it; yields the handle."""
    if stream is None:
        with torch.cuda.device(device):
            yield torch.cuda.current_stream(device).cuda_stream
    else:
        if stream.device != device:
            raise ValueError("stream belongs to another device than the tensors")
        with torch.cuda.stream(stream):
            yield stream.cuda_stream


def launch_on(device, stream, call):
    """call(handle) with the tensors' device and the call's stream current
    (on_stream without its cost where they already are)."""
    if stream is None and torch.cuda.current_device() == device.index:
        return call(torch.cuda.current_stream().cuda_stream)
    with on_stream(device, stream) as handle:
        return call(handle)


def need(t, name, dtype, device, shape=None, contiguous=True):
    """Refuses a tensor that is not what the library would read or write."""
    if t is None:
        return None
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name}: all tensors must be on one CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, dtype, device, shape):
    """Pointer and strides of a [.., d] tensor whose features are contiguous;
    the strides of dimensions of size 1 are not read."""
    p = need(t, name, dtype, device, shape, contiguous=False)
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return p


def _distinct_rows(t, name):
    """An output whose rows overlap would be written twice."""
    size, at = t.shape[:-1], 1
    for stride, n in sorted((t.stride(i), n) for i, n in enumerate(size) if n > 1):
        if stride < at * (t.shape[-1] if at == 1 else 1):
            raise ValueError(f"{name}: rows overlap")
        at = stride * n


def _shapes(q, k, v, log_decay, cu_seqlens):
    if q.dim() != 4 or k.shape != q.shape or v.dim() != 4 or v.shape[:3] != q.shape[:3]:
        raise ValueError("q, k: [B,H,T,d_k]; v: [B,H,T,d_v]")
    B, H, T, dk = q.shape
    dev, N = q.device, B
    if cu_seqlens is not None:
        if B != 1 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("packed sequences: B = 1 and cu_seqlens of N + 1 offsets")
        N = cu_seqlens.numel() - 1
        need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    need(log_decay, "log_decay", torch.float32, dev, (H,))
    return N, H, T, dk, v.shape[-1], dev


def _default_eta(eta_const, dk):
    return 1.0 / math.sqrt(dk) if eta_const is None else float(eta_const)


def _workspace(workspace, nbytes, device):
    if workspace is not None:
        need(workspace, "workspace", workspace.dtype, device)
    if workspace is None or workspace.numel() * workspace.element_size() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return workspace


def forward_decay(q, k, v, log_decay, eta_const=None, ascent=False, cu_seqlens=None, state_in=None,
                  return_state=True, out=None, state_out=None, workspace=None, segment_tokens=0, stream=None):
    """Whole sequences (ttt_la_forward_decay).  Returns (o, W_T), W_T None
    when not requested.  ``eta_const`` defaults to 1/sqrt(d_k).  ``out``,
    ``state_out`` (which may be ``state_in``) and ``workspace`` may be
    preallocated; ``segment_tokens`` (a multiple of 64) overrides the
    automatic split of long sequences."""
    N, H, T, dk, dv, dev = _shapes(q, k, v, log_decay, cu_seqlens)
    dt, code, state_shape = q.dtype, _abi._dtype_code(q), (N, H, dv, dk)

    def call(handle):
        nonlocal out, state_out
        if out is None:
            out = torch.empty_like(v)
        else:
            _distinct_rows(out, "out")
        if return_state and state_out is None:
            state_out = torch.empty(state_shape, device=dev, dtype=torch.float32)
        a = _abi.TttDecayArgs(
            N, H, T, dk, dv, code, _rows(q, "q", dt, dev, q.shape), _rows(k, "k", dt, dev, q.shape),
            _rows(v, "v", dt, dev, v.shape), _rows(out, "out", dt, dev, v.shape),
            _I3(*q.stride()[:3]), _I3(*k.stride()[:3]), _I3(*v.stride()[:3]), _I3(*out.stride()[:3]),
            log_decay.data_ptr(), None if cu_seqlens is None else cu_seqlens.data_ptr(), _default_eta(eta_const, dk),
            1 if ascent else 0, need(state_in, "state_in", torch.float32, dev, state_shape),
            need(state_out, "state_out", torch.float32, dev, state_shape) if return_state else None,
            int(segment_tokens))
        L = _abi.lib()
        nbytes = L.ttt_la_decay_workspace_size(_byref(a))
        if nbytes:
            w = _workspace(workspace, nbytes, dev)
            a.workspace, a.workspace_bytes = w.data_ptr(), w.numel() * w.element_size()
        _abi._check("ttt_la_forward_decay", L.ttt_la_forward_decay(_byref(a), handle))

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
        ins = (_rows(q, "q", dt, dev, q.shape), _rows(k, "k", dt, dev, q.shape), _rows(v, "v", dt, dev, v.shape),
               _rows(grad_o, "grad_o", dt, dev, v.shape))
        g.update(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
                 dW0=torch.empty(state_shape, device=dev, dtype=torch.float32))
        a = _abi.TttDecayGradArgs(
            N, H, T, dk, dv, code, *ins, g["dq"].data_ptr(), g["dk"].data_ptr(), g["dv"].data_ptr(),
            *(_I3(*t.stride()[:3]) for t in (q, k, v, grad_o, g["dq"], g["dk"], g["dv"])),
            log_decay.data_ptr(), None if cu_seqlens is None else cu_seqlens.data_ptr(), _default_eta(eta_const, dk),
            1 if ascent else 0, need(state_in, "state_in", torch.float32, dev, state_shape),
            need(grad_state, "grad_state", torch.float32, dev, state_shape), g["dW0"].data_ptr(), int(segment_tokens))
        L = _abi.lib()
        nbytes = L.ttt_la_backward_decay_workspace_size(_byref(a))
        if nbytes:
            w = _workspace(workspace, nbytes, dev)
            a.workspace, a.workspace_bytes = w.data_ptr(), w.numel() * w.element_size()
        _abi._check("ttt_la_backward_decay", L.ttt_la_backward_decay(_byref(a), handle))

    launch_on(dev, stream, call)
    return g


def decode_step_decay(q, k, v, log_decay, state, eta_const=None, ascent=False, out=None, stream=None):
    """One new token of each of N sequences (ttt_la_decode_step_decay): q, k
    [N,H,d_k], v [N,H,d_v]; state [N,H,d_v,d_k] fp32, updated in place.
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
            _distinct_rows(out, "out")
        a = _abi.TttDecayDecodeArgs(
            N, H, dk, dv, code, _rows(q, "q", dt, dev, q.shape), _rows(k, "k", dt, dev, q.shape),
            _rows(v, "v", dt, dev, v.shape), _rows(out, "out", dt, dev, v.shape),
            _I2(*q.stride()[:2]), _I2(*k.stride()[:2]), _I2(*v.stride()[:2]), _I2(*out.stride()[:2]),
            need(log_decay, "log_decay", torch.float32, dev, (H,)), _default_eta(eta_const, dk), 1 if ascent else 0,
            need(state, "state", torch.float32, dev, (N, H, dv, dk)))
        _abi._check("ttt_la_decode_step_decay", _abi.lib().ttt_la_decode_step_decay(_byref(a), handle))

    launch_on(dev, stream, call)
    return out


def forward_decay_norm(q, k, v, log_decay, gate=None, weight=None, bias=None, activation="silu", eps=1e-5, stream=None,
                       **kw):
    """The layer and its output norm: forward_decay, then every head's output
    of a token normalised by itself and gated (group_norm with one group a
    head).  gate [B,T,H*d_v] or None; weight, bias [H*d_v] or None.  Keyword
    arguments as forward_decay.  Returns (y [B,T,H*d_v], W_T)."""
    B, H, T, dv = v.shape
    if gate is not None and tuple(gate.shape) != (B, T, H * dv):
        raise ValueError("gate: [B,T,H*d_v]")
    if kw.pop("out", None) is not None:
        raise ValueError("forward_decay_norm allocates its output")
    with on_stream(v.device, stream):
        o = torch.empty(B, T, H, dv, device=v.device, dtype=v.dtype)
        if kw.get("cu_seqlens") is not None:
            o.zero_()  # rows in no sequence: the norm reads them
    _, W = forward_decay(q, k, v, log_decay, out=o.transpose(1, 2), stream=stream, **kw)
    rows = (B * T, 1, H * dv)
    y, _, _ = group_norm(o.view(rows), H, weight, bias, gate=None if gate is None else gate.reshape(rows),
                         activation=activation, eps=eps, stream=stream)
    return y.view(B, T, H * dv), W
