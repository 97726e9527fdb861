"""GPU parity of the layer with a decay for each head (forward_decay,
backward_decay, decode_step_decay, forward_decay_norm) against the float64
oracle on the exact inputs given to the GPU.

Bounds, elementwise.  Every output is a sum of products x = sum s_i; let A be
the same sum of absolute values, which the oracle gives for absolute inputs.
u = 2^-8 is half a bf16 step relative to the value, e = 2^-24 half an fp32 step.
  fp32 inputs: sums of at most T + d terms in any order, each power of gamma
    off by less than 2 (T / 32 + 4) steps (at most T / 32 + 1 products of
    powers, each power within 2 steps and its exponent within one, x exp(-x) < 1):
    |err| <= (T + d + T / 8 + 32) e A for outputs and states.
  bf16 inputs: the same in fp32, and on the tensor cores a product chain has
    one rounding to bf16 (a weighted score, or the state as it is read) beside
    the result's: |err| <= u |x| + 2.1 u A leaves room for one more.  States
    take no rounding below 2^-16, and the tensor cores add in at least 22 bits:
    |err| <= (2^-16 + 2^-22 (T / 16 + 16)) A.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from tests.gpu_util import f64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import test_layers_causal_b200 as ttt

U, E = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(autouse=True)
def _no_timed_out_wait():
    yield
    assert ttt.device_status() == 0


def _log_decay(H):
    """From one that keeps everything to one that forgets at once."""
    half = np.linspace(0.0, 1.0, max(H, 2))[:H]
    ld = -np.exp2(2.0 - 12.0 * half)
    if H > 1:
        ld[-1] = 0.0
    if H > 2:
        ld[0] = -np.inf
    return torch.tensor(ld, dtype=torch.float32)


def _make(lens, H, dk, dv, dtype, packed, order, states, seed, extra=(0, 0)):
    """extra: rows before the first and behind the last packed sequence."""
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    B, T = (1, sum(lens) + sum(extra)) if packed else (len(lens), lens[0])

    def rows(d, unit):
        x = torch.randn(B, T, H, d, generator=g)
        if unit:
            x = x / x.norm(dim=-1, keepdim=True)
        if extra[0] and packed:
            x[:, :extra[0]] = float("nan")
        if extra[1] and packed:
            x[:, T - extra[1]:] = float("nan")
        x = x.to(dt).cuda().transpose(1, 2)
        return x if order == "tokens" else x.contiguous()

    c = dict(q=rows(dk, True), k=rows(dk, True), v=rows(dv, False), dO=rows(dv, False), ld=_log_decay(H).cuda(),
             W0=None, dW=None, cu=None, lens=lens, packed=packed, first=extra[0])
    if states:
        c["W0"] = (0.3 * torch.randn(len(lens), H, dv, dk, generator=g)).cuda()
        c["dW"] = torch.randn(len(lens), H, dv, dk, generator=g).cuda()
    if packed:
        c["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]) + extra[0], dtype=torch.int32).cuda()
    return c


def _of_seq(x, c, n):
    """[H, len, d] of sequence n."""
    if not c["packed"]:
        return x[n]
    a = c["first"] + sum(c["lens"][:n])
    return x[0, :, a:a + c["lens"][n]]


def _check(x, ref, A, what, dtype, T, d, state=False):
    x = f64(x)
    assert np.isfinite(x).all(), what
    if dtype == "f32":
        tol = (T + d + T / 8 + 32) * E * A
    elif state:
        tol = (2.0 ** -16 + 2.0 ** -22 * (T / 16 + 16)) * A
    else:
        tol = U * np.abs(ref) + 2.1 * U * A
    bad = np.abs(x - ref) - tol
    assert (bad <= 1e-30).all(), f"{what}: {np.abs(x - ref).max():.3e} off, {bad.max():.3e} past the bound"


def _abs(*xs):
    return [None if x is None else np.abs(x) for x in xs]


def _check_forward(c, o, W, dtype, a):
    H, dk, dv = c["q"].shape[1], c["q"].shape[-1], c["v"].shape[-1]
    ld = f64(c["ld"])
    for n, T in enumerate(c["lens"]):
        q, k, v = (f64(_of_seq(c[x], c, n)) for x in ("q", "k", "v"))
        W0 = None if c["W0"] is None else f64(c["W0"][n])
        ro, rW = oracle.decay_forward_f64(q, k, v, ld, a, W0)
        Ao, AW = oracle.decay_forward_f64(*_abs(q, k, v), ld, abs(a), None if W0 is None else np.abs(W0))
        _check(_of_seq(o, c, n), ro, Ao, f"o of sequence {n}", dtype, T, dk)
        if W is not None:
            _check(W[n], rW, AW, f"W_T of sequence {n}", dtype, T, dk, True)


def _check_backward(c, g, dtype, a):
    dk = c["q"].shape[-1]
    ld = f64(c["ld"])
    for n, T in enumerate(c["lens"]):
        x = [f64(_of_seq(c[y], c, n)) for y in ("q", "k", "v", "dO")]
        s = [None if c[y] is None else f64(c[y][n]) for y in ("W0", "dW")]
        ref = oracle.decay_backward_f64(*x, ld, a, *s)
        A = oracle.decay_backward_f64(*_abs(*x), ld, abs(a), *_abs(*s))
        for name in ("dq", "dk", "dv"):
            _check(_of_seq(g[name], c, n), ref[name], A[name], f"{name} of sequence {n}", dtype, T, dk)
        _check(g["dW0"][n], ref["dW0"], A["dW0"], f"dW0 of sequence {n}", dtype, T, dk, True)


CASES = [
    # lens, H, dk, dv, dtype, packed, order, states, segment_tokens
    ([1], 1, 64, 64, "bf16", False, "heads", False, 0),
    ([1], 3, 128, 128, "bf16", False, "tokens", True, 0),
    ([64, 64], 2, 64, 64, "bf16", False, "tokens", True, 0),
    ([129], 4, 64, 64, "bf16", False, "heads", True, 0),
    ([128], 2, 128, 64, "bf16", False, "tokens", False, 0),
    ([300, 300], 3, 128, 128, "bf16", False, "tokens", True, 0),
    ([513], 2, 128, 128, "bf16", False, "heads", True, 128),
    ([700], 3, 64, 128, "bf16", False, "tokens", True, 256),
    ([450], 2, 64, 64, "bf16", False, "heads", False, 64),
    ([390], 2, 128, 64, "bf16", False, "heads", True, 192),
    ([130, 0, 1, 65, 511, 127], 3, 128, 128, "bf16", True, "tokens", True, 0),
    ([130, 0, 1, 65, 511, 127], 3, 64, 64, "bf16", True, "tokens", True, 128),
    ([3, 400, 0, 77], 2, 64, 128, "bf16", True, "heads", False, 64),
    ([0, 256, 256], 2, 128, 64, "bf16", True, "tokens", True, 128),
    ([200], 2, 96, 80, "bf16", False, "tokens", True, 64),   # widths between the tiles'
    ([150, 60], 2, 8, 24, "bf16", True, "tokens", True, 64),
    ([140], 2, 256, 136, "bf16", False, "heads", True, 64),  # wider than the tiles
    ([1], 2, 32, 32, "f32", False, "heads", True, 0),
    ([95, 95], 2, 64, 64, "f32", False, "tokens", True, 64),
    ([257], 2, 32, 128, "f32", False, "heads", False, 0),
    ([33, 0, 200, 1], 3, 64, 32, "f32", True, "tokens", True, 64),
    ([70], 1, 4, 12, "f32", True, "heads", True, 64),
    ([100], 2, 256, 252, "f32", False, "heads", True, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
@pytest.mark.parametrize("ascent", [False, True])
def test_forward_matches_oracle(case, ascent):
    lens, H, dk, dv, dtype, packed, order, states, seg = case
    c = _make(lens, H, dk, dv, dtype, packed, order, states, seed=len(lens) + dk + 3 * dv)
    o, W = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], ascent=ascent, cu_seqlens=c["cu"], state_in=c["W0"],
                             segment_tokens=seg)
    assert o.stride() == c["v"].stride()
    a = np.float64(np.float32(1.0 / math.sqrt(dk)))
    _check_forward(c, o, W, dtype, -a if ascent else a)
    # the output alone, and the state in place, give the same bits
    o2, none = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], ascent=ascent, cu_seqlens=c["cu"], state_in=c["W0"],
                                 segment_tokens=seg, return_state=False)
    assert none is None and torch.equal(o, o2)
    if states:
        S = c["W0"].clone()
        o3, W3 = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], ascent=ascent, cu_seqlens=c["cu"], state_in=S,
                                   state_out=S, segment_tokens=seg)
        assert W3 is S and torch.equal(W3, W) and torch.equal(o3, o)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
def test_backward_matches_oracle(case):
    lens, H, dk, dv, dtype, packed, order, states, seg = case
    c = _make(lens, H, dk, dv, dtype, packed, order, states, seed=50 + len(lens) + dk + 3 * dv)
    g = ttt.backward_decay(c["q"], c["k"], c["v"], c["dO"], c["ld"], eta_const=0.2, cu_seqlens=c["cu"],
                           state_in=c["W0"], grad_state=c["dW"], segment_tokens=seg)
    assert g["dq"].stride() == c["q"].stride() and g["dv"].stride() == c["v"].stride()
    _check_backward(c, g, dtype, np.float64(np.float32(0.2)))


@pytest.mark.parametrize("lens,H,dk,dv,packed,seg", [
    ([300, 300], 3, 128, 128, False, 128), ([700], 2, 128, 128, False, 0), ([513], 2, 64, 64, False, 128),
    ([390], 2, 128, 64, False, 192), ([450], 2, 64, 128, False, 0), ([200], 2, 96, 80, False, 64),
    ([130, 0, 1, 65, 511, 127], 3, 128, 128, True, 128), ([3, 400, 0, 77], 2, 64, 64, True, 0)])
def test_outputs_take_one_rounding(lens, H, dk, dv, packed, seg):
    """bf16 on the tensor cores: an output's own rounding, u |x|, and beside it
    what two bf16 parts leave out.  A part is the upper half of a word, with 8
    bits, so two leave less than 2^-14: of a weighted score, or of the keys in
    the state and of the state as it is read, 2^-13 in all; sums are added in 22
    bits at least, (T / 16 + 16) terms deep, weights off by fewer steps than
    that.  |err| <= u |x| + (2^-13 + 2^-21 (T / 16 + 16)) A."""
    c = _make(lens, H, dk, dv, "bf16", packed, "tokens", True, seed=61 + dk)
    kw = dict(cu_seqlens=c["cu"], state_in=c["W0"], segment_tokens=seg, eta_const=0.25)
    o, _ = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], **kw)
    g = ttt.backward_decay(c["q"], c["k"], c["v"], c["dO"], c["ld"], grad_state=c["dW"], **kw)
    ld = f64(c["ld"])
    for n, T in enumerate(lens):
        q, k, v, dO = (f64(_of_seq(c[x], c, n)) for x in ("q", "k", "v", "dO"))
        W0, dW = f64(c["W0"][n]), f64(c["dW"][n])
        ref = dict(oracle.decay_backward_f64(q, k, v, dO, ld, 0.25, W0, dW), o=oracle.decay_forward_f64(q, k, v, ld, 0.25, W0)[0])
        A = dict(oracle.decay_backward_f64(*_abs(q, k, v, dO), ld, 0.25, *_abs(W0, dW)),
                 o=oracle.decay_forward_f64(*_abs(q, k, v), ld, 0.25, np.abs(W0))[0])
        for name, x in (("o", o), ("dq", g["dq"]), ("dk", g["dk"]), ("dv", g["dv"])):
            x = f64(_of_seq(x, c, n))
            tol = U * np.abs(ref[name]) + (2.0 ** -13 + 2.0 ** -21 * (T / 16 + 16)) * A[name]
            assert (np.abs(x - ref[name]) <= tol + 1e-30).all(), (name, n)


def test_gradient_agrees_with_differences():
    """<gradient, direction> against the fp32 layer's own central difference;
    the loss is a sum over o and W_T, linear in each input alone, so the
    difference's only error is the fp32 rounding of the two losses."""
    c = _make([70], 2, 32, 32, "f32", False, "heads", True, seed=7)
    g = ttt.backward_decay(c["q"], c["k"], c["v"], c["dO"], c["ld"], state_in=c["W0"], grad_state=c["dW"])

    def loss(**kw):
        x = {n: kw.get(n, c[n]) for n in ("q", "k", "v", "W0")}
        o, W = ttt.forward_decay(x["q"], x["k"], x["v"], c["ld"], state_in=x["W0"])
        return float((o.double() * c["dO"].double()).sum() + (W.double() * c["dW"].double()).sum())

    for n, gn in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("W0", "dW0")):
        d = torch.randn(c[n].shape, generator=torch.Generator().manual_seed(3)).cuda()
        num = (loss(**{n: c[n] + d}) - loss(**{n: c[n] - d})) / 2
        ref = float((g[gn].double() * d.double()).sum())
        # 4500 outputs of magnitude up to 10, each off by at most 150 steps of 2^-24
        assert abs(num - ref) <= 4500 * 10 * 150 * E, n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seg", [0, 64])
def test_rows_in_no_sequence(dtype, seg):
    """Rows before the first and behind the last sequence hold NaN and are
    neither read into a result nor written."""
    c = _make([70, 0, 200], 2, 64, 64, dtype, True, "tokens", True, seed=9, extra=(5, 37))
    out = torch.full_like(c["v"], 7.0)
    o, W = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], cu_seqlens=c["cu"], state_in=c["W0"], out=out,
                             segment_tokens=seg)
    a = np.float64(np.float32(1.0 / math.sqrt(64)))
    _check_forward(c, o, W, dtype, a)
    T = o.shape[2]
    assert (o[:, :, :5] == 7).all() and (o[:, :, T - 37:] == 7).all()
    g = ttt.backward_decay(c["q"], c["k"], c["v"], c["dO"], c["ld"], cu_seqlens=c["cu"], state_in=c["W0"],
                           grad_state=c["dW"], segment_tokens=seg)
    _check_backward(c, g, dtype, a)


@pytest.mark.parametrize("d", [64, 128])
def test_not_finite_stays_in_its_sequence_and_head(d):
    """Infinities and NaN in one (sequence, head), at its last row, reach no
    other, whose rows lie in the same tiles of memory."""
    c = _make([100, 90, 300], 2, d, d, "bf16", True, "tokens", True, seed=12)
    clean, Wc = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], cu_seqlens=c["cu"], state_in=c["W0"])
    v, k = c["v"].clone(memory_format=torch.preserve_format), c["k"].clone(memory_format=torch.preserve_format)
    v[0, 1, 189] = float("inf")
    v[0, 1, 100] = float("nan")
    k[0, 1, 150] = float("nan")
    o, W = ttt.forward_decay(c["q"], k, v, c["ld"], cu_seqlens=c["cu"], state_in=c["W0"])
    keep = torch.ones(o.shape[1:3], dtype=torch.bool, device="cuda")
    keep[1, 100:190] = False
    assert torch.equal(o[0][keep], clean[0][keep])
    ok = torch.ones(3, 2, dtype=torch.bool, device="cuda")
    ok[1, 1] = False
    assert torch.equal(W[ok], Wc[ok]) and not torch.isfinite(W[1, 1]).all()


@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 128, 128), ("bf16", 64, 96), ("f32", 32, 64)])
def test_prompt_then_steps_is_one_sequence(dtype, dk, dv):
    """A prompt and then single tokens give what the whole sequence gives."""
    T, P, H = 140, 133, 3
    c = _make([T, T], H, dk, dv, dtype, False, "tokens", True, seed=21)
    S = torch.empty_like(c["W0"])
    o, _ = ttt.forward_decay(c["q"][:, :, :P], c["k"][:, :, :P], c["v"][:, :, :P], c["ld"], state_in=c["W0"],
                             state_out=S)
    outs = [o]
    for t in range(P, T):
        outs.append(ttt.decode_step_decay(c["q"][:, :, t], c["k"][:, :, t], c["v"][:, :, t], c["ld"], S)[:, :, None])
    _check_forward(c, torch.cat(outs, 2), S, dtype, np.float64(np.float32(1.0 / math.sqrt(dk))))


@pytest.mark.parametrize("dtype,N,H,dk,dv", [("bf16", 1, 1, 128, 1), ("bf16", 5, 3, 64, 128), ("f32", 2, 2, 32, 40),
                                             ("bf16", 300, 7, 128, 64), ("f32", 97, 3, 64, 64)])
def test_step_matches_oracle(dtype, N, H, dk, dv):
    g = torch.Generator().manual_seed(N + dk)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    pad = 8  # rows longer than the features: strides are the caller's
    q, k = (torch.randn(N, H, dk + pad, generator=g).to(dt).cuda()[..., :dk] for _ in range(2))
    v = torch.randn(N, H, dv + pad + -dv % 8, generator=g).to(dt).cuda()[..., :dv]
    S = torch.randn(N, H, dv, dk, generator=g).cuda()
    ld = _log_decay(H).cuda()
    W0 = f64(S)
    ro, rW = oracle.decay_forward_f64(*(f64(x)[..., None, :] for x in (q, k, v)), f64(ld), -0.25, W0)
    Ao, AW = oracle.decay_forward_f64(*(np.abs(f64(x))[..., None, :] for x in (q, k, v)), f64(ld), 0.25, np.abs(W0))
    o = ttt.decode_step_decay(q, k, v, ld, S, eta_const=0.25, ascent=True)
    _check(S, rW, AW, "state", "f32", 1, 1)
    tol = (dk + 8) * E * Ao[..., 0, :] + (U * np.abs(ro[..., 0, :]) if dtype == "bf16" else 0)
    assert (np.abs(f64(o) - ro[..., 0, :]) <= tol * 1.001).all()


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("dtype,N,H,dk,dv", [("bf16", 300, 7, 64, 72), ("bf16", 1000, 5, 32, 40), ("f32", 300, 7, 64, 20),
                                             ("bf16", 5, 3, 64, 33), ("bf16", 700, 3, 128, 15), ("f32", 3, 2, 32, 1),
                                             ("bf16", 1500, 3, 32, 17)])
def test_step_of_any_value_width(dtype, N, H, dk, dv, padded):
    """Widths of v that a warp's rows do not divide: its accesses lie in two
    (sequence, head)s, or behind the last row; v and o with rows that do not
    start on 16 bytes; the memory around o stays as it is."""
    g = torch.Generator().manual_seed(N + dv)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k = (torch.randn(N, H, dk, generator=g).to(dt).cuda() for _ in range(2))
    pad = 3 if padded else 0
    v = torch.randn(N, H, dv + pad, generator=g).to(dt).cuda()[..., :dv]
    room = torch.full((N, H, dv + pad), 7.0, dtype=dt, device="cuda")
    S = torch.randn(N, H, dv, dk, generator=g).cuda()
    ld = _log_decay(H).cuda()
    W0 = f64(S)
    ro, rW = oracle.decay_forward_f64(*(f64(x)[..., None, :] for x in (q, k, v)), f64(ld), 0.25, W0)
    Ao, AW = oracle.decay_forward_f64(*(np.abs(f64(x))[..., None, :] for x in (q, k, v)), f64(ld), 0.25, np.abs(W0))
    S2 = S.clone()
    o = ttt.decode_step_decay(q, k, v, ld, S, eta_const=0.25)
    o2 = ttt.decode_step_decay(q, k, v, ld, S2, eta_const=0.25, out=room[..., :dv])
    assert torch.equal(o, o2) and torch.equal(S, S2) and (room[..., dv:] == 7).all()
    _check(S, rW, AW, "state", "f32", 1, 1)
    tol = (dk + 8) * E * Ao[..., 0, :] + (U * np.abs(ro[..., 0, :]) if dtype == "bf16" else 0)
    assert (np.abs(f64(o) - ro[..., 0, :]) <= tol * 1.001).all()


def test_streams_graphs_and_repeats_give_the_same_bits():
    c = _make([700, 700], 3, 128, 128, "bf16", False, "tokens", True, seed=30)
    kw = dict(state_in=c["W0"], segment_tokens=128)
    fwd = lambda: ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], **kw)  # noqa: E731
    bwd = lambda: ttt.backward_decay(c["q"], c["k"], c["v"], c["dO"], c["ld"], grad_state=c["dW"], **kw)  # noqa: E731
    flat = lambda: [*fwd(), *bwd().values()]  # noqa: E731
    a = flat()
    torch.cuda.synchronize()
    s, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = flat()
    b2 = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], stream=s2, **kw)  # another stream, beside the first
    torch.cuda.synchronize()
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d = flat()
    with torch.cuda.graph(g2):
        e = flat()
    for _ in range(2):
        g.replay()
        g2.replay()
    torch.cuda.synchronize()
    for x, *others in zip(a, b, d, e):
        assert all(torch.equal(x, y) for y in others)
    assert torch.equal(a[0], b2[0]) and torch.equal(a[1], b2[1])


def test_caller_workspace_and_out():
    c = _make([300], 2, 64, 64, "bf16", False, "heads", True, seed=31)
    o, W = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], state_in=c["W0"], segment_tokens=64)
    w = torch.full((1 << 21,), 255, dtype=torch.uint8, device="cuda")  # NaN where it is read unwritten
    out, S = torch.empty_like(c["v"]), torch.empty_like(c["W0"])
    o2, W2 = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], state_in=c["W0"], segment_tokens=64, out=out,
                               state_out=S, workspace=w)
    assert o2 is out and W2 is S and torch.equal(o, o2) and torch.equal(W, W2)


def test_many_short_sequences():
    lens = [(7 * i) % 40 for i in range(700)]
    c = _make(lens, 1, 64, 64, "bf16", True, "tokens", True, seed=33)
    o, W = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], cu_seqlens=c["cu"], state_in=c["W0"])
    _check_forward(c, o, W, "bf16", np.float64(0.125))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_rows_at_all(dtype):
    """Only empty sequences: the states pass through, forwards and backwards."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    z = torch.empty(1, 2, 0, 64, dtype=dt, device="cuda")
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    W0, dW = (torch.randn(3, 2, 64, 64, generator=torch.Generator().manual_seed(i)).cuda() for i in (1, 2))
    ld = _log_decay(2).cuda()
    o, W = ttt.forward_decay(z, z, z, ld, cu_seqlens=cu, state_in=W0)
    assert o.shape == z.shape and torch.equal(W, W0)
    g = ttt.backward_decay(z, z, z, z, ld, cu_seqlens=cu, state_in=W0, grad_state=dW)
    assert torch.equal(g["dW0"], dW)


def test_two_host_threads_on_two_streams():
    """Calls of two threads at once, each on its own stream, give the bits of
    one after the other."""
    import threading
    cs = [_make([500, 500], 2, 128, 128, "bf16", False, "tokens", True, seed=70 + i) for i in range(2)]

    def both(c):
        o, W = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], state_in=c["W0"])
        return [o, W, *ttt.backward_decay(c["q"], c["k"], c["v"], c["dO"], c["ld"], state_in=c["W0"]).values()]

    want = [both(c) for c in cs]
    torch.cuda.synchronize()
    got = [None, None]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                got[i] = both(cs[i])
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("cu", [[0, 500, 90, 200], [-7, 100, 100, 1 << 30], [200, 200, 0, 0]])
def test_offsets_outside_the_rows_touch_nothing_else(cu):
    """Offsets that leave the rows or decrease are clamped: the call returns,
    with memory around the output as it was."""
    c = _make([200], 2, 64, 64, "bf16", True, "tokens", False, seed=35)
    room = torch.full((3, 200, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(),
                      out=room[1:2].transpose(1, 2), segment_tokens=64)
    assert (room[0] == 5).all() and (room[2] == 5).all()


@pytest.mark.parametrize("packed", [False, True])
def test_layer_then_norm(packed):
    """The layer and its gated output norm in one call are the two calls."""
    c = _make([130, 60] if packed else [95, 95], 3, 64, 64, "bf16", packed, "tokens", True, seed=40)
    B, H, T, dv = c["v"].shape
    g = torch.Generator().manual_seed(1)
    gate = torch.randn(B, T, H * dv, generator=g).to(torch.bfloat16).cuda()
    w, b = (torch.randn(H * dv, generator=g).cuda() for _ in range(2))
    y, W = ttt.forward_decay_norm(c["q"], c["k"], c["v"], c["ld"], gate=gate, weight=w, bias=b, cu_seqlens=c["cu"],
                                  state_in=c["W0"])
    o, W2 = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], cu_seqlens=c["cu"], state_in=c["W0"])
    x = o.transpose(1, 2).reshape(B * T, 1, H * dv)
    y2, _, _ = ttt.group_norm(x, H, w, b, gate=gate.reshape(x.shape))
    assert torch.equal(y.view(x.shape), y2) and torch.equal(W, W2)


@pytest.mark.parametrize("layout", ["contiguous", "tokens outermost", "slice", "off 16 bytes"])
def test_layer_then_norm_on_a_stream(layout):
    """On a stream of the caller's, with a gate that this stream is still
    producing when the call is made, in any memory order: the two calls."""
    c = _make([95, 95], 3, 64, 64, "bf16", False, "tokens", True, seed=41)
    B, H, T, dv = c["v"].shape
    C = H * dv
    values = torch.randn(B, T, C, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    gate = {"contiguous": lambda: torch.empty(B, T, C, dtype=torch.bfloat16, device="cuda"),
            "tokens outermost": lambda: torch.empty(T, B, C, dtype=torch.bfloat16, device="cuda").transpose(0, 1),
            "slice": lambda: torch.empty(B, T, 3 * C, dtype=torch.bfloat16, device="cuda")[..., C:2 * C],
            "off 16 bytes": lambda: torch.empty(B * T * C + 1, dtype=torch.bfloat16, device="cuda")[1:].view(B, T, C)}[layout]()
    gate.fill_(float("nan"))
    o, W = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], state_in=c["W0"])
    want, _, _ = ttt.group_norm(o.transpose(1, 2).reshape(B * T, 1, C), H, gate=values.view(B * T, 1, C))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)  # some 25 ms
        gate.copy_(values)
    y, W2 = ttt.forward_decay_norm(c["q"], c["k"], c["v"], c["ld"], gate=gate, state_in=c["W0"], stream=s)
    after = [torch.full((B, T, C), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(4)]  # memory let go of
    torch.cuda.synchronize()
    assert torch.equal(y.view(want.shape), want) and torch.equal(W2, W) and len(after) == 4


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_then_norm_of_no_rows(dtype):
    """Only empty sequences: an empty output, the state as it was."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    z = torch.empty(1, 2, 0, 64, dtype=dt, device="cuda")
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    S = torch.randn(3, 2, 64, 64, generator=torch.Generator().manual_seed(1)).cuda()
    W0 = S.clone()
    y, W = ttt.forward_decay_norm(z, z, z, _log_decay(2).cuda(), gate=torch.empty(1, 0, 128, dtype=dt, device="cuda"),
                                  cu_seqlens=cu, state_in=S, state_out=S)
    assert y.shape == (1, 0, 128) and y.dtype == dt and W is S and torch.equal(S, W0)


@pytest.mark.parametrize("bad", ["activation", "eps", "eps nan", "eps large", "weight", "weight dtype", "gate dtype", "gate device"])
def test_layer_then_norm_refuses_before_the_state_moves(bad):
    c = _make([70], 2, 64, 64, "bf16", False, "tokens", True, seed=42)
    gate = torch.zeros(1, 70, 128, dtype=torch.bfloat16, device="cuda")
    kw = {"activation": dict(activation="relu"), "eps": dict(eps=-1e-5), "eps nan": dict(eps=float("nan")), "eps large": dict(eps=1e40),
          "weight": dict(weight=torch.ones(64, device="cuda")), "weight dtype": dict(weight=torch.ones(128, device="cuda").half()),
          "gate dtype": dict(gate=gate.float()), "gate device": dict(gate=gate.cpu())}[bad]
    S = c["W0"].clone()
    with pytest.raises((ValueError, TypeError, ttt.TttError)):
        ttt.forward_decay_norm(c["q"], c["k"], c["v"], c["ld"], state_in=S, state_out=S, **kw)
    torch.cuda.synchronize()
    assert torch.equal(S, c["W0"])


def test_a_wait_limit_covers_one_block_not_the_launches_before():
    """One block's 1024 tiles, some 4 ms, under a limit of 1 ms for each wait:
    launches that start early do not count that run against their waits."""
    T = 131072
    c = _make([T], 1, 64, 128, "bf16", False, "heads", True, seed=44)
    kw = dict(state_in=c["W0"], segment_tokens=T)
    both = lambda: [*ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], **kw),  # noqa: E731
                    *ttt.backward_decay(c["q"], c["k"], c["v"], c["dO"], c["ld"], grad_state=c["dW"], **kw).values()]
    want = both()
    torch.cuda.synchronize()
    ttt.set_wait_limit_ns(1_000_000)
    try:
        got = both()
        torch.cuda.synchronize()
    finally:
        ttt.set_wait_limit_ns(1_000_000_000)
    assert ttt.device_status() == 0
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("extra", [(0, 0), (5, 37), (0, 300), (90, 0)])
@pytest.mark.parametrize("dtype,dk,dv,order", [("bf16", 64, 64, "tokens"), ("bf16", 128, 80, "heads"), ("bf16", 16, 136, "tokens"),
                                               ("f32", 32, 12, "heads"), ("f32", 32, 64, "tokens")])
def test_rest_is_cleared_where_it_is_asked_for(dtype, dk, dv, order, extra):
    """Rows in no sequence become zeros, the others' bits stay, in a tensor
    whose neighbours keep theirs."""
    c = _make([70, 0, 200], 3, dk, dv, dtype, True, order, True, seed=45, extra=extra)
    want, W = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], cu_seqlens=c["cu"], state_in=c["W0"])
    T = want.shape[2]
    shape = (1, T, 3, 2 * dv) if order == "tokens" else (1, 3, T, 2 * dv)
    room = torch.full(shape, 7.0, dtype=c["v"].dtype, device="cuda")
    out = room[..., :dv]
    out = out.transpose(1, 2) if order == "tokens" else out
    o, W2 = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], cu_seqlens=c["cu"], state_in=c["W0"], out=out, clear_rest=True)
    a, b = extra[0], T - extra[1]
    assert torch.equal(o[:, :, a:b], want[:, :, a:b]) and torch.equal(W, W2)
    assert not o[:, :, :a].any() and not o[:, :, b:].any() and (room[..., dv:] == 7).all()


def test_rest_of_only_empty_sequences_and_of_equal_lengths():
    c = _make([0, 0], 2, 64, 64, "bf16", True, "tokens", True, seed=46, extra=(60, 80))
    o, W = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], cu_seqlens=c["cu"], state_in=c["W0"], clear_rest=True)
    assert not o.any() and torch.equal(W, c["W0"])
    c = _make([150, 150], 2, 64, 64, "bf16", False, "tokens", True, seed=47)  # nothing to clear
    a = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], state_in=c["W0"], clear_rest=True)
    b = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], state_in=c["W0"])
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_layer_then_norm_of_rows_in_no_sequence():
    """Zeros as the norm sees them, whatever memory the output comes to lie in."""
    c = _make([70, 0, 200], 2, 64, 64, "bf16", True, "tokens", True, seed=48, extra=(5, 37))
    T, C = c["v"].shape[2], 128
    b = torch.randn(C, generator=torch.Generator().manual_seed(3)).cuda()
    for fill in (float("nan"), 3.0):
        old = [torch.full((1, T, 2, 64), fill, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        del old  # the allocator hands it out again
        y, _ = ttt.forward_decay_norm(c["q"], c["k"], c["v"], c["ld"], bias=b, cu_seqlens=c["cu"], state_in=c["W0"])
        rest, _, _ = ttt.group_norm(torch.zeros(42, 1, C, dtype=torch.bfloat16, device="cuda"), 2, bias=b)
        assert torch.equal(torch.cat([y[0, :5], y[0, T - 37:]]), rest[:, 0])


def _exact_workspace(need):
    """A workspace of just the bytes, between others that are to stay."""
    room = torch.full((need + 8192,), 85, dtype=torch.uint8, device="cuda")
    return room, room[4096:4096 + need], lambda: bool((room[:4096] == 85).all() and (room[4096 + need:] == 85).all())


def _workspace_need(c, seg, in_place=False):
    """(forward's, gradient's) bytes, as the library asks for them."""
    import ctypes
    from test_layers_causal_b200 import _abi
    N, (_, H, T, dk), dv = len(c["lens"]), c["q"].shape, c["v"].shape[-1]
    out = []
    for cls, name in ((_abi.TttDecayArgs, "ttt_la_decay_workspace_size"), (_abi.TttDecayGradArgs, "ttt_la_backward_decay_workspace_size")):
        a = cls()
        a.N, a.H, a.T, a.d_k, a.d_v, a.dtype, a.segment_tokens = N, H, T, dk, dv, _abi._dtype_code(c["q"]), seg
        a.log_decay, a.cu_seqlens = c["ld"].data_ptr(), c["cu"].data_ptr()
        if in_place and cls is _abi.TttDecayArgs:
            a.state_in = a.state_out = c["W0"].data_ptr()
        out.append(getattr(_abi.lib(), name)(ctypes.byref(a)))
    return out


@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 64, 64), ("bf16", 64, 128), ("bf16", 16, 136), ("f32", 32, 36)])
def test_workspace_of_few_long_among_many_short(dtype, dk, dv):
    """Sequences of several segments here and there among hundreds of one, more
    than a block counts at once: each finds its slots, in just the bytes that
    the library asks for."""
    lens = [(7 * i) % 5 for i in range(900)]
    for i, n in ((0, 65), (31, 64), (32, 200), (33, 129), (607, 300), (608, 65), (899, 190)):
        lens[i] = n
    c = _make(lens, 1, dk, dv, dtype, True, "tokens", True, seed=51)
    need, back = _workspace_need(c, 64)
    T, state = sum(lens), dk * dv * 4
    assert 0 < need <= (2 * T // 64 + 1) * state < len(lens) * state
    room, w, whole = _exact_workspace(need)
    S = c["W0"].clone()
    o, W = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], cu_seqlens=c["cu"], state_in=c["W0"], segment_tokens=64, workspace=w)
    assert whole()
    _check_forward(c, o, W, dtype, np.float64(np.float32(1 / math.sqrt(dk))))
    if dtype == "bf16" and dv <= 128:
        room, w, whole = _exact_workspace(_workspace_need(c, 64, True)[0])
        o2, _ = ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], cu_seqlens=c["cu"], state_in=S, state_out=S, segment_tokens=64,
                                  workspace=w)
        assert whole() and torch.equal(o, o2) and torch.equal(S, W)
    room, w, whole = _exact_workspace(back)
    g = ttt.backward_decay(c["q"], c["k"], c["v"], c["dO"], c["ld"], cu_seqlens=c["cu"], state_in=c["W0"], grad_state=c["dW"],
                           segment_tokens=64, workspace=w)
    assert whole()
    _check_backward(c, g, dtype, np.float64(np.float32(1 / math.sqrt(dk))))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_of_more_segments_than_slots_stay_in_the_workspace(dtype):
    """Offsets that go back and forth over the rows: the call returns, the
    memory around its workspace and output as it was."""
    c = _make([640], 1, 32, 64, dtype, True, "tokens", False, seed=52)
    n = 3000
    c["cu"] = torch.randint(-50, 700, (n + 1,), dtype=torch.int32, generator=torch.Generator().manual_seed(1)).cuda()
    c["lens"] = [0] * n
    need, back = _workspace_need(c, 64)
    room, w, whole = _exact_workspace(need)
    rows = torch.full((3, 640, 1, 64), 5.0, dtype=c["v"].dtype, device="cuda")
    ttt.forward_decay(c["q"], c["k"], c["v"], c["ld"], cu_seqlens=c["cu"], out=rows[1:2].transpose(1, 2), segment_tokens=64,
                      workspace=w)
    assert whole() and (rows[0] == 5).all() and (rows[2] == 5).all()
    room, w, whole = _exact_workspace(back)
    ttt.backward_decay(c["q"], c["k"], c["v"], c["dO"], c["ld"], cu_seqlens=c["cu"], segment_tokens=64, workspace=w)
    assert whole()


def test_captured_packed_calls_follow_the_offsets():
    """A captured call of the layer, its gradient and its norm on packed
    sequences, replayed after the offsets, the inputs and the state changed,
    gives what a fresh call gives: nothing of the offsets is kept."""
    c = _make([300, 1, 0, 200], 2, 64, 128, "bf16", True, "tokens", True, seed=53, extra=(0, 20))
    C = 256
    gate = torch.randn(1, C, 521, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda().transpose(1, 2)

    def call():
        y, W = ttt.forward_decay_norm(c["q"], c["k"], c["v"], c["ld"], gate=gate, cu_seqlens=c["cu"], state_in=c["W0"],
                                      segment_tokens=64)
        g = ttt.backward_decay(c["q"], c["k"], c["v"], c["dO"], c["ld"], cu_seqlens=c["cu"], state_in=c["W0"],
                               grad_state=c["dW"], segment_tokens=64)
        return [y, W, *g.values()]

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for cu in ([0, 300, 301, 301, 501], [0, 64, 130, 130, 521], [3, 3, 503, 503, 504]):
        for n in ("q", "k", "v", "dO"):
            c[n].copy_(torch.randn(c[n].shape, generator=torch.Generator().manual_seed(cu[1])).to(torch.bfloat16) * 0.1)
        c["W0"].mul_(0.5)
        c["cu"].copy_(torch.tensor(cu, dtype=torch.int32))
        for t in got[2:5]:
            t.zero_()  # rows in no sequence are nobody's
        graph.replay()
        want = call()
        torch.cuda.synchronize()
        a, b = cu[0], cu[-1]
        for i, (x, y) in enumerate(zip(got, want)):
            if 2 <= i < 5:
                x, y = x[:, :, a:b], y[:, :, a:b]
            assert torch.equal(x, y), i


def test_past_2_31_elements():
    """q, k, v of 257 heads x 65536 tokens x 128 (2^31 elements and more):
    the last head against the oracle."""
    H, T, d = 257, 65536, 128
    c = _make([T], 1, d, d, "bf16", False, "heads", False, seed=60)
    x = {}
    for n in ("q", "k", "v"):
        x[n] = torch.zeros(1, H, T, d, dtype=torch.bfloat16, device="cuda")
        x[n][:, H - 1] = c[n][:, 0]
    ld = torch.full((H,), -0.01, device="cuda")
    o, W = ttt.forward_decay(x["q"], x["k"], x["v"], ld)
    c["ld"] = ld[-1:]
    _check_forward(c, o[:, H - 1:], W[:, H - 1:], "bf16", np.float64(np.float32(1.0 / math.sqrt(d))))
    assert not o[:, :H - 1].any() and not W[:, :H - 1].any()
