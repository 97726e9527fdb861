"""Host-side checks of the decayed layer and the group norm (no GPU needed,
nothing is launched): struct layouts, refusals of the C ABI and of the
binding, and the split of sequences into segments."""
import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def abi():
    from test_layers_causal_b200 import _abi
    from test_layers_causal_b200.build import build
    build()
    _abi.lib()
    return _abi


def test_struct_layouts_match_c(abi):
    pairs = {"ttt_la_decay_args": abi.TttDecayArgs, "ttt_la_decay_grad_args": abi.TttDecayGradArgs,
             "ttt_la_decay_decode_args": abi.TttDecayDecodeArgs, "ttt_la_group_norm_args": abi.TttGroupNormArgs,
             "ttt_la_group_norm_grad_args": abi.TttGroupNormGradArgs}
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "ttt_la.h"', "int main(void) {"]
    for c, py in pairs.items():
        src.append(f'printf("{c} %zu\\n", sizeof({c}));')
        src += [f'printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    src.append("return 0; }")
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "p.c"), os.path.join(d, "p")
        open(c, "w").write("\n".join(src))
        subprocess.run(["gcc", "-I" + os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split("\n")
    for line in filter(None, out):
        key, v = line.split()
        if "." in key:
            s, f = key.split(".")
            assert getattr(pairs[s], f).offset == int(v), key
        else:
            assert ctypes.sizeof(pairs[key]) == int(v), key


def test_packed_blocks_are_the_structs(abi):
    """The struct formats the bindings pack, against the ctypes mirrors (which
    the test above holds to the C layout)."""
    from test_layers_causal_b200._call import FORMATS
    mirrors = {"ttt_la_decay_args": abi.TttDecayArgs, "ttt_la_decay_grad_args": abi.TttDecayGradArgs,
               "ttt_la_decay_decode_args": abi.TttDecayDecodeArgs, "ttt_la_group_norm_args": abi.TttGroupNormArgs,
               "ttt_la_group_norm_grad_args": abi.TttGroupNormGradArgs}
    assert set(FORMATS) == set(mirrors)
    for name, fmt in FORMATS.items():
        cls = mirrors[name]
        fields = [f for f, _ in cls._fields_ if f not in ("workspace", "workspace_bytes")]
        has_workspace = len(fields) < len(cls._fields_)
        assert fmt.size + (16 if has_workspace else 0) == ctypes.sizeof(cls)
        flat, n = [], 0
        for f, t in cls._fields_:
            if f in fields:
                count = t._length_ if hasattr(t, "_length_") else 1
                base = t._type_ if count > 1 else t
                values = [0.5] if base is ctypes.c_float else list(range(n + 1, n + 1 + count))
                flat.append((f, values))
                n += count
        block = cls.from_buffer_copy(fmt.pack(*(x for _, v in flat for x in v)) + b"\0" * (16 if has_workspace else 0))
        for f, v in flat:
            got = getattr(block, f)
            assert (list(got) if hasattr(got, "__len__") else [got]) == v, (name, f)


I3, I2 = ctypes.c_int64 * 3, ctypes.c_int64 * 2


def _fwd(abi, **kw):
    a = abi.TttDecayArgs()
    a.N, a.H, a.T, a.d_k, a.d_v, a.dtype = 2, 3, 1000, 64, 128, abi.BF16
    a.q, a.k, a.v, a.o = 0x10000, 0x20000, 0x30000, 0x40000  # never dereferenced: each case is refused
    a.q_stride = a.k_stride = I3(192000, 64000, 64)
    a.v_stride = a.o_stride = I3(384000, 128000, 128)
    a.log_decay, a.eta_const = 0x50000, 0.1
    a.workspace, a.workspace_bytes = 0x100000, 1 << 40
    for n, x in kw.items():
        setattr(a, n, x)
    return a


INVALID = [dict(N=0), dict(H=0), dict(T=-1), dict(T=0), dict(d_k=0), dict(d_v=-8), dict(dtype=2), dict(q=None),
           dict(o=None), dict(k=0x20008), dict(o=0x30000), dict(log_decay=None), dict(log_decay=0x50002),
           dict(cu_seqlens=0x60002), dict(state_in=0x70004), dict(state_out=0x70008), dict(segment_tokens=32),
           dict(segment_tokens=-64), dict(q_stride=I3(192000, 64000, 60)), dict(v_stride=I3(384000, 0, 128)),
           dict(o_stride=I3(384000, -128000, 128)), dict(workspace=None, segment_tokens=64),
           dict(workspace_bytes=16, segment_tokens=64), dict(workspace=0x100004, segment_tokens=64)]


@pytest.mark.parametrize("bad", INVALID, ids=str)
def test_forward_refuses(abi, bad):
    assert abi.lib().ttt_la_forward_decay(ctypes.byref(_fwd(abi, **bad)), None) == abi.ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(d_k=60), dict(d_v=264), dict(d_k=512), dict(d_k=66, dtype=0)], ids=str)
def test_widths_that_are_not_there(abi, bad):
    assert abi.lib().ttt_la_forward_decay(ctypes.byref(_fwd(abi, **bad)), None) == abi.ERR_UNSUPPORTED
    assert abi.lib().ttt_la_decay_workspace_size(ctypes.byref(_fwd(abi, **bad))) == 0


def test_null_arguments(abi):
    L = abi.lib()
    for f in ("forward_decay", "backward_decay", "decode_step_decay", "group_norm", "group_norm_backward"):
        assert getattr(L, "ttt_la_" + f)(None, None) == abi.ERR_INVALID_ARG
    for f in ("decay", "backward_decay", "group_norm", "group_norm_backward"):
        assert getattr(L, f"ttt_la_{f}_workspace_size")(None) == 0


def _bwd(abi, **kw):
    a = abi.TttDecayGradArgs()
    a.N, a.H, a.T, a.d_k, a.d_v, a.dtype = 2, 3, 1000, 64, 128, abi.BF16
    a.q, a.k, a.v, a.grad_o = 0x10000, 0x20000, 0x30000, 0x40000
    a.grad_q, a.grad_k, a.grad_v = 0x80000, 0x90000, 0xa0000
    a.q_stride = a.k_stride = a.grad_q_stride = a.grad_k_stride = I3(192000, 64000, 64)
    a.v_stride = a.grad_o_stride = a.grad_v_stride = I3(384000, 128000, 128)
    a.log_decay, a.eta_const = 0x50000, 0.1
    a.workspace, a.workspace_bytes = 0x100000, 1 << 40
    for n, x in kw.items():
        setattr(a, n, x)
    return a


@pytest.mark.parametrize("bad", [dict(N=0), dict(T=0), dict(grad_o=None), dict(grad_q=0x10000), dict(grad_k=0x80000),
                                 dict(grad_v=0xa0008), dict(grad_state=0x4), dict(grad_state_in=0xb0000, grad_state=0xb0000),
                                 dict(grad_state_in=0xb0000, state_in=0xb0000), dict(log_decay=None),
                                 dict(grad_k_stride=I3(192000, 64000, 0)), dict(workspace=None, segment_tokens=64)], ids=str)
def test_backward_refuses(abi, bad):
    assert abi.lib().ttt_la_backward_decay(ctypes.byref(_bwd(abi, **bad)), None) == abi.ERR_INVALID_ARG


def _step(abi, **kw):
    a = abi.TttDecayDecodeArgs()
    a.N, a.H, a.d_k, a.d_v, a.dtype = 4, 2, 128, 128, abi.BF16
    a.q, a.k, a.v, a.o, a.state, a.log_decay = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000
    a.q_stride = a.k_stride = a.v_stride = a.o_stride = I2(256, 128)
    for n, x in kw.items():
        setattr(a, n, x)
    return a


@pytest.mark.parametrize("bad", [dict(N=0), dict(d_v=0), dict(dtype=5), dict(q=None), dict(o=0x10000), dict(state=None),
                                 dict(state=0x50008), dict(log_decay=None), dict(q_stride=I2(256, 4)),
                                 dict(v=0x30002), dict(N=1 << 24, H=128)], ids=str)
def test_step_refuses(abi, bad):
    assert abi.lib().ttt_la_decode_step_decay(ctypes.byref(_step(abi, **bad)), None) == abi.ERR_INVALID_ARG


def test_step_width_that_is_not_there(abi):
    assert abi.lib().ttt_la_decode_step_decay(ctypes.byref(_step(abi, d_k=96)), None) == abi.ERR_UNSUPPORTED


def _norm(abi, **kw):
    a = abi.TttGroupNormArgs()
    a.N, a.L, a.C, a.G, a.dtype, a.param_dtype, a.activation, a.eps = 3, 50, 320, 32, abi.BF16, abi.F32, 1, 1e-5
    a.x, a.gate, a.weight, a.bias, a.y, a.mean, a.rstd = (0x10000 * i for i in range(1, 8))
    a.workspace, a.workspace_bytes = 0x100000, 1 << 40
    for n, x in kw.items():
        setattr(a, n, x)
    return a


@pytest.mark.parametrize("bad", [dict(N=0), dict(L=0), dict(G=0), dict(G=3), dict(dtype=4), dict(param_dtype=3),
                                 dict(activation=2), dict(eps=-1.0), dict(eps=float("nan")), dict(x=None), dict(y=0x10000),
                                 dict(y=0x20000), dict(mean=None), dict(x=0x10008), dict(weight=0x30002),
                                 dict(workspace=None), dict(workspace_bytes=8)], ids=str)
def test_norm_refuses(abi, bad):
    assert abi.lib().ttt_la_group_norm(ctypes.byref(_norm(abi, **bad)), None) == abi.ERR_INVALID_ARG


def test_norm_shapes_that_are_not_there(abi):
    for kw in (dict(C=8192 * 8, G=8192), dict(C=8192, G=8192)):
        assert abi.lib().ttt_la_group_norm(ctypes.byref(_norm(abi, **kw)), None) == abi.ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", [dict(grad_y=None), dict(grad_x=None), dict(grad_gate=None), dict(grad_x=0x20000),
                                 dict(grad_bias=0xb0000, grad_weight=0xb0000), dict(rstd=None), dict(workspace=None)], ids=str)
def test_norm_backward_refuses(abi, bad):
    a = abi.TttGroupNormGradArgs()
    a.N, a.L, a.C, a.G, a.dtype, a.param_dtype, a.activation = 3, 50, 320, 32, abi.BF16, abi.F32, 1
    names = ("grad_y", "x", "gate", "weight", "bias", "mean", "rstd", "grad_x", "grad_gate", "grad_weight", "grad_bias")
    for i, n in enumerate(names):
        setattr(a, n, 0x10000 * (i + 1))
    a.workspace, a.workspace_bytes = 0x1000000, 1 << 40
    for n, x in bad.items():
        setattr(a, n, x)
    assert abi.lib().ttt_la_group_norm_backward(ctypes.byref(a), None) == abi.ERR_INVALID_ARG


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import test_layers_causal_b200 as ttt
    z = torch.zeros
    with pytest.raises(ValueError):
        ttt.forward_decay(z(1, 2, 5, 64), z(1, 2, 5, 64), z(1, 2, 5, 64), z(2))  # not on a CUDA device
    with pytest.raises(ValueError):
        ttt.forward_decay(z(1, 2, 5, 64), z(1, 2, 4, 64), z(1, 2, 5, 64), z(2))
    with pytest.raises(ValueError):
        ttt.forward_decay(z(2, 2, 5, 64), z(2, 2, 5, 64), z(2, 2, 5, 64), z(2), cu_seqlens=z(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        ttt.decode_step_decay(z(2, 2, 64), z(2, 2, 64), z(2, 3, 64), z(2), z(2, 2, 64, 64))
    with pytest.raises(ValueError):
        ttt.group_norm(z(2, 5, 64), 3)
    with pytest.raises(ValueError):
        ttt.group_norm(z(2, 5, 64), 4)
    with pytest.raises(ValueError):
        ttt.group_norm(z(2, 0, 64), 4)
    with pytest.raises(ValueError):
        ttt.group_norm(z(2, 5, 64), 4, activation="relu")
    with pytest.raises(ValueError):
        ttt.forward_decay_norm(z(1, 2, 5, 64), z(1, 2, 5, 64), z(1, 2, 5, 64), z(2), gate=z(1, 5, 64))


def test_output_rows_that_overlap_are_refused():
    from test_layers_causal_b200._call import check_distinct_rows as _distinct_rows
    x = torch.zeros(2, 3, 4, 8)
    for good in (x, x.transpose(1, 2), x.transpose(0, 2), x[:, :1], x[..., :4], torch.zeros(1, 1, 1, 8).expand(1, 1, 1, 8)):
        _distinct_rows(good, "out")
    for bad in (x[:, :1].expand(2, 3, 4, 8), x.as_strided((2, 3, 4, 8), (96, 32, 4, 1)), x.as_strided((2, 3, 4, 8), (32, 32, 8, 1))):
        with pytest.raises(ValueError):
            _distinct_rows(bad, "out")


@pytest.mark.parametrize("packed", [False, True])
def test_workspace_grows_with_the_segments(abi, packed):
    size = lambda **kw: abi.lib().ttt_la_decay_workspace_size(ctypes.byref(_fwd(abi, **kw)))  # noqa: E731
    base = dict(cu_seqlens=0x60000, N=7) if packed else {}
    a, b = size(segment_tokens=64, **base), size(segment_tokens=512, **base)
    state = 64 * 128 * 4 * 3
    assert a % state == 0 and a > b > 0
    # every token in some segment, and each sequence with one at least
    assert a // state >= (1000 // 64 + 7 if packed else 2 * 16)
    back = abi.lib().ttt_la_backward_decay_workspace_size(ctypes.byref(_bwd(abi, segment_tokens=64, **base)))
    assert back >= 2 * a


def test_norm_checks_come_before_the_layer():
    """forward_decay_norm refuses what its norm would refuse while nothing has
    been launched; no rows are no reason."""
    from test_layers_causal_b200 import _abi
    from test_layers_causal_b200.norm import _describe, check_group_norm
    x = torch.zeros(5, 1, 64)
    for G, act, eps, error in ((3, "silu", 1e-5, ValueError), (4, "relu", 1e-5, ValueError)):
        with pytest.raises(error):
            check_group_norm(x, G, None, None, None, act, eps)
    with pytest.raises(ValueError, match="empty"):
        _describe(x[:0], 4, None, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):  # the rows' number passes, their device does not
        check_group_norm(x[:0], 4, None, None, None, None, 1e-5)
    assert issubclass(_abi.TttError, RuntimeError)


@pytest.mark.parametrize("bad", [dict(q_stride=I2(256, 60)), dict(k_stride=I2(252, 128)), dict(v_stride=I2(256, 0)),
                                 dict(o_stride=I2(-20, 20)), dict(v_stride=I2(1 << 40, 20))], ids=str)
def test_step_strides_that_are_refused(abi, bad):
    assert abi.lib().ttt_la_decode_step_decay(ctypes.byref(_step(abi, **bad)), None) == abi.ERR_INVALID_ARG


def test_step_takes_values_of_any_width(abi):
    """Rows of v and o start anywhere. (A width of the keys that is not there
    is found behind the checks of the strides: nothing is launched.)"""
    for d_v in (1, 20, 33):
        block = _step(abi, d_k=96, d_v=d_v, v_stride=I2(2 * d_v, d_v), o_stride=I2(2 * d_v + 3, d_v + 1))
        assert abi.lib().ttt_la_decode_step_decay(ctypes.byref(block), None) == abi.ERR_UNSUPPORTED


@pytest.mark.parametrize("clear_rest", [2, -1])
def test_forward_refuses_a_clear_rest_that_is_no_truth_value(abi, clear_rest):
    assert abi.lib().ttt_la_forward_decay(ctypes.byref(_fwd(abi, clear_rest=clear_rest)), None) == abi.ERR_INVALID_ARG


def test_workspace_does_not_grow_with_short_sequences(abi):
    """Thousands of packed sequences of a few tokens: the workspace follows the
    tokens, as segments of sequences that are one need none; in place, where
    all start states go through it, each has a state."""
    L = abi.lib()
    kw = dict(N=4096, H=16, T=8192, d_k=128, d_v=128, cu_seqlens=0x60000, segment_tokens=64)
    state = 16 * 128 * 128 * 4
    assert 0 < L.ttt_la_decay_workspace_size(ctypes.byref(_fwd(abi, **kw))) <= (2 * 8192 // 64 + 1) * state
    assert 0 < L.ttt_la_backward_decay_workspace_size(ctypes.byref(_bwd(abi, **kw))) <= 2 * (2 * 8192 // 64 + 1) * state
    inplace = L.ttt_la_decay_workspace_size(ctypes.byref(_fwd(abi, state_in=0x70000, state_out=0x70000, **kw)))
    assert inplace >= 4096 * state
    # with the segments left to the library too
    kw.pop("segment_tokens")
    assert L.ttt_la_decay_workspace_size(ctypes.byref(_fwd(abi, **kw))) <= 4096 * state // 8
    # and however the tokens lie: one sequence of all of them, and N - 1 empty ones
    for N, T, S in ((1, 1000, 64), (2, 129, 64), (7, 1000, 64), (300, 12800, 128), (5, 64 * 50, 64)):
        kw = dict(N=N, H=1, T=T, d_k=64, d_v=64, cu_seqlens=0x60000, segment_tokens=S)
        slots = L.ttt_la_decay_workspace_size(ctypes.byref(_fwd(abi, **kw))) // (64 * 64 * 4)
        one = (T + S - 1) // S
        many = min(N, T // (S + 1))  # as many of two segments as there can be, the rest behind the first
        worst = max(one, 2 * (many - 1) + -(-(T - (many - 1) * (S + 1)) // S)) if many else one
        assert worst <= slots <= worst + 1, (N, T, S, worst, slots)


def test_sizes_past_their_field_are_refused_as_arguments(monkeypatch):
    from test_layers_causal_b200 import _call
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(_call, "_current_handle", lambda index: 0)
    for fmt in _call.FORMATS.values():
        n = len(fmt.unpack(bytes(fmt.size)))
        for bad in (1 << 31, -(1 << 31) - 1):
            with pytest.raises(ValueError, match="does not fit"):
                _call.launch_on(torch.device("cuda", 0), None, lambda handle: fmt.pack(bad, *[0] * (n - 1)))
    with pytest.raises(ValueError, match="does not fit"):
        _call.launch_on(torch.device("cuda", 0), None,
                        lambda handle: _call.FORMATS["ttt_la_group_norm_args"].pack(*[1] * 7, 1e40, *[0] * 7))
