"""GPU parity of group_norm and group_norm_backward against the float64 oracle
on the exact inputs given to the GPU.

Bounds (e = 2^-24, u = 2^-8, m = L * C/G values a group): mean and variance
come from pairwise-joined fp32 sums of at most 256 terms each, so hat = (x -
mean) rstd is off by at most 64 steps of (|hat| + |mean| rstd + 1), and what is
made of it by 64 steps of its terms' absolute sum; silu's sigmoid (one
exponential, one division) by 8 steps relative.  A bf16 result adds u |y|.
Gradients add the group's two sums: 64 steps of their absolute sums; dweight
and dbias sum n terms in at least 64 strands: (n / 64 + 128) steps of the
absolute sum (bf16 parameters add u).
"""
import numpy as np
import pytest
import torch

import oracle
from tests.gpu_util import f64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import test_layers_causal_b200 as ttt

U, E = 2.0 ** -8, 2.0 ** -24

CASES = [
    # shape, groups, dtype, param dtype or None, gated, activation, shift of the mean
    ((1, 1, 8), 1, "bf16", "f32", True, "silu", 0.0),
    ((5, 1, 256), 2, "bf16", "f32", True, "silu", 0.0),
    ((33, 1, 2048), 16, "bf16", "bf16", True, "silu", 0.3),
    ((33, 2048), 32, "bf16", None, False, None, 0.0),
    ((1000, 1, 128), 1, "bf16", "f32", False, "silu", 0.0),
    ((7, 1, 1536), 3, "bf16", "f32", True, "silu", 0.0),        # a group of 64 units: wider than a warp
    ((9, 1, 320), 10, "f32", "f32", True, None, 0.0),
    ((4, 1, 64), 32, "f32", "f32", False, "silu", 0.0),         # two values a group
    ((3, 1, 192), 2, "f32", "f32", True, "silu", 0.0),          # 24 lanes: not a power of two
    ((2, 65, 65, 320), 32, "f32", "f32", False, "silu", 100.0),
    ((3, 77, 320), 32, "bf16", "f32", True, "silu", 0.0),
    ((2, 4099, 8), 8, "bf16", "bf16", False, "silu", 0.0),      # one channel a group
    ((2, 50, 2056), 1, "bf16", "f32", False, "silu", 4.0),      # more units than a block has threads
    ((1, 3000, 48), 16, "f32", None, True, "silu", 0.0),        # three channels a group
    ((600, 3, 64), 4, "bf16", "f32", False, "silu", 0.0),
    ((5, 7, 8192), 4096, "bf16", "f32", True, "silu", 0.0),     # the most groups
    ((70, 1, 3200), 25, "bf16", "f32", True, "silu", 0.0),      # a row in two columns of blocks
    ((11, 1, 192), 8, "bf16", "f32", True, None, 0.0),          # three units a group: not a power of two
    ((3, 77, 3), 1, "bf16", "bf16", True, "silu", 0.0),         # rows that do not start on 16 bytes
    ((2, 501, 10), 2, "bf16", "f32", False, "silu", 1.0),
    ((5, 1, 7), 7, "f32", None, False, None, 0.0),
    ((2, 33, 2), 1, "f32", "f32", True, "silu", 0.0),
    ((4, 2, 301), 1, "bf16", "f32", True, None, 0.0),
    ((40, 1, 192), 24, "bf16", "bf16", False, "silu", 0.0),     # one unit a group, rows side by side in a block
]


def _make(case, seed=0):
    shape, G, dtype, pd, gated, act, shift = case
    g = torch.Generator().manual_seed(seed + shape[-1] + shape[0])
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = (torch.randn(shape, generator=g) * 1.5 + shift).to(dt)
    gate = torch.randn(shape, generator=g).to(dt) if gated else None
    dy = torch.randn(shape, generator=g).to(dt)
    w = b = None
    if pd:
        p = torch.bfloat16 if pd == "bf16" else torch.float32
        w, b = ((1.0 if i == 0 else 0.0) + 0.3 * torch.randn(shape[-1], generator=g) for i in range(2))
        w, b = w.to(p), b.to(p)
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    return [cuda(t) for t in (x, dy, w, b, gate)]


def _spread(s, G, shape):
    """[N, G] -> the shape of x."""
    n, c = shape[0], shape[-1]
    s = np.repeat(s, c // G, axis=1).reshape((n,) + (1,) * (len(shape) - 2) + (c,))
    return np.broadcast_to(s, shape)


ids = lambda c: "-".join(str(x).replace(" ", "") for x in c)  # noqa: E731


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_forward_matches_oracle(case):
    shape, G, dtype, pd, gated, act, shift = case
    x, _, w, b, gate = _make(case)
    y, mean, rstd = ttt.group_norm(x, G, w, b, gate=gate, activation=act)
    X, W, B, Z = f64(x), f64(w), f64(b), f64(gate)
    ry, rm, rr = oracle.group_norm_f64(X, G, W, B, Z, silu=act == "silu")
    top = np.abs(X).reshape(shape[0], -1, G, shape[-1] // G).max(axis=(1, 3))
    assert (np.abs(f64(mean) - rm) <= 64 * E * top).all()
    # rstd = (var + eps)^(-1/2): half the relative error of var, itself 128 steps of top sigma and of var
    assert (np.abs(f64(rstd) - rr) <= 128 * E * rr * (1 + top * rr)).all()
    hat = (X - _spread(rm, G, shape)) * _spread(rr, G, shape)
    slack = np.abs(hat) * 3 + _spread(np.abs(rm) * rr, G, shape) + 1
    t = np.abs(hat * (1 if W is None else W)) + (0 if B is None else np.abs(B))
    dt = 64 * E * (slack * (1 if W is None else np.abs(W)) + t)
    if gated:
        act_z = np.abs(Z / (1 + np.exp(-Z)) if act else Z)
        tol = dt * act_z + 8 * E * (t * act_z)
    else:
        tol = 1.1 * dt + 8 * E * t  # silu's slope is below 1.1
    if dtype == "bf16":
        tol = tol + U * np.abs(ry)
    bad = np.abs(f64(y) - ry) - tol
    assert (bad <= 1e-30).all(), bad.max()


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_backward_matches_oracle(case):
    shape, G, dtype, pd, gated, act, shift = case
    x, dy, w, b, gate = _make(case, 7)
    _, mean, rstd = ttt.group_norm(x, G, w, b, gate=gate, activation=act)
    g = ttt.group_norm_backward(dy, x, G, mean, rstd, w, b, gate=gate, activation=act)
    X, W, B, Z, D, M, R = (f64(t) for t in (x, w, b, gate, dy, mean, rstd))
    ref = oracle.group_norm_backward_f64(D, X, G, M, R, W, B, Z, silu=act == "silu")
    r = _spread(R, G, shape)
    hat = (X - _spread(M, G, shape)) * r
    w1 = np.ones(shape[-1]) if W is None else np.abs(W)
    t_abs = np.abs(hat) * w1 + (0 if B is None else np.abs(B))
    # |dt| before its slope (at most 1.1 for silu), with everything it is made of
    up = np.abs(D) * (1.1 if not gated else np.abs(Z) if act else np.abs(Z))
    # hat's own error (64 steps of |hat| + |mean| rstd + 1) moves silu's slope by at most half of it
    hat_err = np.abs(hat) + _spread(np.abs(M) * R, G, shape) + 1
    dt_err = 64 * E * (up + np.abs(D) * (0 if gated else 1) * hat_err * w1 * 0.6 + up * 0.1)
    means = lambda a: _spread(a.reshape(shape[0], -1, G, shape[-1] // G).mean(axis=(1, 3)), G, shape)  # noqa: E731
    dh_err, dh = dt_err * w1, up * w1
    s1_err = means(dh_err) + 64 * E * means(dh)
    s2_err = means(dh_err * np.abs(hat) + 64 * E * dh * hat_err)
    s2 = means(dh * np.abs(hat))
    tol = r * (dh_err + s1_err + np.abs(hat) * s2_err + 64 * E * hat_err * s2 + 8 * E * (dh + means(dh) + np.abs(hat) * s2))
    if dtype == "bf16":
        tol = tol + U * np.abs(ref["dx"])
    bad = np.abs(f64(g["dx"]) - ref["dx"]) - tol
    assert (bad <= 1e-30).all(), bad.max()
    axes, n = tuple(range(len(shape) - 1)), x.numel() // shape[-1]
    if pd:
        steps = (n / 64 + 128) * E
        for name, err, size in (("dweight", dt_err * np.abs(hat) + 64 * E * up * hat_err, up * np.abs(hat)),
                                ("dbias", dt_err, up)):
            tol = err.sum(axis=axes) + steps * size.sum(axis=axes)
            if pd == "bf16":
                tol = tol + U * np.abs(ref[name])
            assert g[name].dtype == w.dtype
            assert (np.abs(f64(g[name]) - ref[name]) <= tol).all(), name
    else:
        assert g["dweight"] is None and g["dbias"] is None
    if gated:
        tol = 64 * E * np.abs(D) * 1.2 * (hat_err * w1 + t_abs)
        if dtype == "bf16":
            tol = tol + U * np.abs(ref["dgate"])
        assert (np.abs(f64(g["dgate"]) - ref["dgate"]) <= tol).all()
    else:
        assert g["dgate"] is None


def test_extreme_activations():
    """silu far from zero: no overflow of its exponential becomes a NaN."""
    x = torch.tensor([-3.0, 1.0, 5.0, -1.0] * 8).reshape(4, 1, 8).cuda()
    w = torch.full((8,), 300.0).cuda()
    gate = torch.tensor([-1e30, 1e30, -200.0, 200.0] * 8).reshape(4, 1, 8).cuda()
    y, mean, rstd = ttt.group_norm(x, 1, w)
    assert torch.isfinite(y).all()
    y, _, _ = ttt.group_norm(x, 1, gate=gate)
    assert torch.isfinite(y).all() and (y[..., 0::4] == 0).all()
    g = ttt.group_norm_backward(torch.ones_like(x), x, 1, mean, rstd, w)
    assert all(torch.isfinite(t).all() for t in g.values() if t is not None)
    g = ttt.group_norm_backward(torch.ones_like(x), x, 1, mean, rstd, gate=gate)
    assert torch.isfinite(g["dgate"]).all()


def test_not_finite_stays_in_its_group():
    for shape in ((6, 1, 256), (2, 300, 64)):
        x = torch.randn(shape, generator=torch.Generator().manual_seed(4)).cuda()
        y, mean, rstd = ttt.group_norm(x, 4)
        x2 = x.clone()
        x2[1, 0, 0] = float("nan")
        x2[0, 0, shape[-1] - 1] = float("inf")
        y2, mean2, _ = ttt.group_norm(x2, 4)
        cg = shape[-1] // 4
        same = torch.ones(shape[0], 4, dtype=torch.bool, device="cuda")
        same[1, 0] = same[0, 3] = False
        assert torch.equal(mean[same], mean2[same]) and not torch.isfinite(mean2[~same]).any()
        by = lambda t: t.view(shape[0], -1, 4, cg).transpose(1, 2)  # noqa: E731
        assert torch.equal(by(y)[same], by(y2)[same])


@pytest.mark.parametrize("shape,G", [((40, 1, 512), 4), ((2, 700, 320), 32)])
def test_streams_graphs_and_repeats_give_the_same_bits(shape, G):
    case = (shape, G, "bf16", "f32", True, "silu", 0.0)
    x, dy, w, b, gate = _make(case)

    def both():
        y, mean, rstd = ttt.group_norm(x, G, w, b, gate=gate)
        return [y, mean, rstd, *ttt.group_norm_backward(dy, x, G, mean, rstd, w, b, gate=gate).values()]

    a = both()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        d = both()
    s.synchronize()
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        e = both()
    with torch.cuda.graph(g2):
        f = both()
    g.replay()
    g2.replay()
    torch.cuda.synchronize()
    for t, *others in zip(a, d, e, f):
        assert all(torch.equal(t, o) for o in others)


@pytest.mark.parametrize("shape,G,dtype,gated", [((2, 4225, 320), 32, "f32", False), ((2, 4225, 320), 32, "bf16", True),
                                                 ((3000, 1, 2048), 16, "bf16", True), ((6000, 1, 320), 10, "f32", False)])
def test_repeats_give_the_same_bits(shape, G, dtype, gated):
    """Many runs back to back: copies into the ring's places never overtake the
    reads of what was there."""
    x, dy, w, b, gate = _make((shape, G, dtype, "f32", gated, "silu", 0.5))

    def both():
        y, mean, rstd = ttt.group_norm(x, G, w, b, gate=gate)
        g = ttt.group_norm_backward(dy, x, G, mean, rstd, w, b, gate=gate)
        return [t for t in (y, mean, rstd, *g.values()) if t is not None]

    first = both()
    for _ in range(40):
        for t, o in zip(first, both()):
            assert torch.equal(t, o)


def test_past_2_31_elements():
    """2^31 elements and more: the last sample, whose offsets pass 32 bits."""
    n, c = (1 << 20) + 3, 2048
    x = torch.zeros(n, 1, c, dtype=torch.bfloat16, device="cuda")
    last = torch.randn(1, 1, c, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    x[-1] = last[0]
    y, mean, rstd = ttt.group_norm(x, 16)
    ry, rm, _ = oracle.group_norm_f64(f64(last), 16)
    assert (np.abs(f64(y[-1:]) - ry) <= U * np.abs(ry) + 1e-5).all()
    assert np.abs(f64(mean[-1:]) - rm).max() <= 1e-5 and not y[:-1].any()


def test_the_most_positions():
    """2^31 - 1 positions of one channel, all zero but the last: positions plus
    a step pass 31 bits.  The sums over the zeros are known."""
    L, n = (1 << 31) - 1, 3000
    g = torch.Generator().manual_seed(6)
    tail, dtail = (torch.randn(n, generator=g).to(torch.bfloat16) for _ in range(2))
    x = torch.zeros(1, L, 1, dtype=torch.bfloat16, device="cuda")
    x[0, L - n:, 0] = tail.cuda()
    y, mean, rstd = ttt.group_norm(x, 1, activation=None)
    X, D = f64(tail), f64(dtail)
    m = X.sum() / L
    r = ((X * X).sum() / L - m * m + 1e-5) ** -0.5
    top = np.abs(X).max()
    assert abs(f64(mean)[0, 0] - m) <= 64 * E * top
    assert abs(f64(rstd)[0, 0] - r) <= 128 * E * r * (1 + top * r)
    M, R = f64(mean)[0, 0], f64(rstd)[0, 0]
    hat = (X - M) * R
    tol = 64 * E * (3 * np.abs(hat) + abs(M) * R + 1) + U * np.abs(hat)
    assert (np.abs(f64(y[0, L - n:, 0]) - hat) <= tol).all()
    zero = y[0, 0, 0]  # what a zero becomes
    assert abs(float(zero) + M * R) <= 64 * E + U * abs(M) * R
    assert (y[0, :L - n, 0] == zero).all()
    del y
    dy = torch.zeros_like(x)
    dy[0, L - n:, 0] = dtail.cuda()
    dx = ttt.group_norm_backward(dy, x, 1, mean, rstd, activation=None)["dx"]
    s1, s2 = D.sum() / L, (D * hat).sum() / L
    a1, a2 = np.abs(D).sum() / L, (np.abs(D) * (np.abs(hat) + 1)).sum() / L
    want = R * (D - s1 - hat * s2)
    tol = R * (64 * E * (np.abs(D) + a1 + (np.abs(hat) + 1) * a2 * 3)) + U * np.abs(want)
    assert (np.abs(f64(dx[0, L - n:, 0]) - want) <= tol).all()
    assert (dx[0, :L - n, 0] == dx[0, 0, 0]).all()


@pytest.mark.parametrize("shape,G,dtype", [((2, 300, 64), 4, "f32"), ((3, 70, 48), 16, "bf16"), ((2, 9, 10), 2, "f32"),
                                           ((5, 1, 96), 2, "bf16"), ((5, 1, 256), 2, "f32"), ((2, 3000, 320), 32, "f32")])
def test_values_whose_square_is_too_large(shape, G, dtype):
    """Values around 2^66 with a spread of 2^60: the square of the mean passes
    the largest fp32 number, the variance does not.  Against the oracle, with
    the bounds of test_forward_matches_oracle."""
    g = torch.Generator().manual_seed(8)
    x = (torch.randn(shape, generator=g).double() * 2.0 ** 60 + 2.0 ** 66).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    y, mean, rstd = ttt.group_norm(x, G, activation=None)
    X = f64(x)
    ry, rm, rr = oracle.group_norm_f64(X, G, silu=False)
    top = np.abs(X).reshape(shape[0], -1, G, shape[-1] // G).max(axis=(1, 3))
    assert (np.abs(f64(mean) - rm) <= 64 * E * top).all()
    assert (np.abs(f64(rstd) - rr) <= 128 * E * rr * (1 + top * rr)).all()
    hat = (X - _spread(rm, G, shape)) * _spread(rr, G, shape)
    tol = 64 * E * (np.abs(hat) * 4 + _spread(np.abs(rm) * rr, G, shape) + 1) + (U * np.abs(ry) if dtype == "bf16" else 0)
    assert (np.abs(f64(y) - ry) <= tol).all()


@pytest.mark.parametrize("shape,G", [((2, 300, 64), 4), ((2, 9, 10), 2), ((5, 1, 96), 2), ((5, 1, 256), 2), ((2, 3000, 320), 32),
                                     ((1, 70, 8), 1)])
def test_variance_past_the_largest_number(shape, G):
    """Values of 2^70 here and there: the variance is past fp32, rstd 0, the
    group's outputs zeros and not NaN; NaN and infinities stay what they are."""
    g = torch.Generator().manual_seed(9)
    x = torch.randn(shape, generator=g)
    cg = shape[-1] // G
    x[0, ..., 1] = 2.0 ** 70 * torch.where(torch.arange(x[0, ..., 1].numel()) % 3 == 0, 1.0, -0.25).view(x[0, ..., 1].shape)
    y, mean, rstd = ttt.group_norm(x.cuda(), G, activation=None)
    assert rstd[0, 0] == 0 and torch.isfinite(mean).all() and torch.isfinite(rstd).all() and torch.isfinite(y).all()
    assert (y[0, ..., :cg] == 0).all()
    for bad in (float("nan"), float("inf")):
        x[0, ..., 0] = bad
        y, mean, rstd = ttt.group_norm(x.cuda(), G, activation=None)
        assert not torch.isfinite(mean[0, 0]) and torch.isnan(y[0, ..., :cg]).all()
        if G > 1:
            assert torch.isfinite(y[0, ..., cg:]).all()
