"""What the bindings of the decayed layer and the group norm share: checks of
tensors, the stream a call goes to, argument blocks and workspaces.

Argument blocks are packed with ``struct`` in the layout of the C structs of
include/ttt_la.h (``tests/test_decay_host.py`` holds the formats to them): a
call for one token spends most of its time here, and filling a ctypes structure
of 25 fields takes several microseconds.
"""
from __future__ import annotations

import contextlib
import ctypes
import struct

import torch

from . import _abi

# Formats of the C structs, without the trailing workspace and workspace_bytes where there are such.
FORMATS = {
    "ttt_la_decay_args": struct.Struct("<6i4Q12q2Qfi2Q2i"),
    "ttt_la_decay_grad_args": struct.Struct("<6i7Q21q2Qfi3Qi4x"),
    "ttt_la_decay_decode_args": struct.Struct("<5i4x4Q8qQfiQ"),
    "ttt_la_group_norm_args": struct.Struct("<7if7Q"),
    "ttt_la_group_norm_grad_args": struct.Struct("<7i4x11Q"),
}
_WORKSPACE = struct.Struct("<2Q")
_functions = {}
# the current stream's handle without a Stream object around it
_current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _function(name, restype):
    f = _functions.get(name)
    if f is None:
        f = _abi.lib()[name]  # an object of its own: the block goes in as bytes
        f.restype = restype
        f.argtypes = [ctypes.c_void_p] if restype is ctypes.c_size_t else [ctypes.c_void_p, ctypes.c_void_p]
        _functions[name] = f
    return f


def run(name, block, handle):
    """The entry point `name` on an argument block without a workspace."""
    code = _function(name, ctypes.c_int)(block, handle)
    if code:
        raise _abi.TttError(name, code)


def run_with_workspace(name, size_name, block, workspace, device, handle):
    """The same where the block ends in a workspace, allocated unless the
    caller's is large enough."""
    need_bytes = _function(size_name, ctypes.c_size_t)(block + _WORKSPACE.pack(0, 0))
    if not need_bytes:
        return run(name, block + _WORKSPACE.pack(0, 0), handle)
    if workspace is not None:
        check(workspace, "workspace", workspace.dtype, device)
    if workspace is None or workspace.numel() * workspace.element_size() < need_bytes:
        workspace = torch.empty(need_bytes, dtype=torch.uint8, device=device)
    size = workspace.numel() * workspace.element_size()
    run(name, block + _WORKSPACE.pack(workspace.data_ptr(), size), handle)


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
    (on_stream without its cost where they already are).  A value that
    its field of the block cannot hold (2^31 positions and more) is refused as
    an argument."""
    if device.type != "cuda":
        raise ValueError("all tensors must be on one CUDA device")
    try:
        if stream is None and torch.cuda.current_device() == device.index:
            return call(_current_handle(device.index))
        with on_stream(device, stream) as handle:
            return call(handle)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"an argument does not fit its field: {e}") from None


def check(t, name, dtype, device, shape=None, contiguous=True):
    """Refuses a tensor that is not what the library would read or write;
    returns its address, 0 for None."""
    if t is None:
        return 0
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name}: all tensors must be on one CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def check_rows(t, name, dtype, device, shape):
    """Address and strides of a [.., d] tensor whose features are contiguous;
    the strides of dimensions of size 1 are not read."""
    if t.dtype != dtype or t.shape != shape or t.device != device:
        check(t, name, dtype, device, shape, contiguous=False)
    s = t.stride()
    if s[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t.data_ptr(), s


def check_distinct_rows(t, name):
    """An output whose rows overlap would be written twice."""
    size, at = t.shape[:-1], 1
    for stride, n in sorted((t.stride(i), n) for i, n in enumerate(size) if n > 1):
        if stride < at * (t.shape[-1] if at == 1 else 1):
            raise ValueError(f"{name}: rows overlap")
        at = stride * n
