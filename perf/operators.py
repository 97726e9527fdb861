"""The decayed fast-weight layer and its output norm: the cases that are measured, and what they compute.

Operators (sigma = 1, a = 1/sqrt(d_k), gamma_h = exp(log_decay[h]) <= 1):

  prompt     W_t = gamma W_{t-1} + a v_t k_t^T ;  o_t = W_t q_t      whole sequences, equal or packed lengths
  gradient   dq, dk, dv, dW_0 of the same layer for dL/do and dL/dW_T
  step       the same for one new token of each of N sequences, the state updated in place
  norm       group norm over channels-last data, then silu, or times silu(gate)
  norm_grad  its gradients

A case is a dict of plain values.  `run` computes the plain form (elementary torch operations in 32 bits) or, where
`own` is set, makes the calls that a user of the package makes.
"""
import math

import numpy as np
import torch

own = False

CHUNK = 128  # tokens per block of the plain form


# ------------------------------------------------------------------ cases ----
def _prompt(name, op, lens, heads, d_k, d_v, dtype="bf16", packed=False, order="heads", state=True):
    """`lens`: tokens of each sequence; packed: one row of tokens, the sequences one after the other; order: which of
    heads and tokens is the outer dimension in memory."""
    return {"name": name, "op": op, "lens": ",".join(str(n) for n in lens), "heads": heads, "d_k": d_k, "d_v": d_v,
            "dtype": dtype, "packed": packed, "order": order, "state": state}


def _step(name, seqs, heads, d_k, d_v, dtype="bf16"):
    return {"name": name, "op": "step", "seqs": seqs, "heads": heads, "d_k": d_k, "d_v": d_v, "dtype": dtype}


def _norm(name, op, n, length, channels, groups, dtype="bf16", gate=False):
    return {"name": name, "op": op, "n": n, "length": length, "channels": channels, "groups": groups, "dtype": dtype,
            "gate": gate}


def listed():
    return [
        # one long document on a layer of few heads: the long-context layer of the benchmark
        _prompt("prompt_long_d128", "prompt", [65536], 8, 128, 128, state=False),
        # a training or scoring batch of the LLM-shaped layer, activations as a projection leaves them
        _prompt("prompt_llm_d64", "prompt", [4096] * 4, 16, 64, 64, order="tokens"),
        # a serving prefill: requests of different lengths packed into one row of tokens, none a multiple of a tile
        _prompt("prompt_packed_d128", "prompt", [17, 2501, 1, 640, 3999, 333, 1200, 65, 129, 3500], 16, 128, 128,
                packed=True, order="tokens"),
        # the smallest prompt, in 32 bits: launch latency
        _prompt("prompt_tiny_f32", "prompt", [256], 2, 32, 32, dtype="f32"),
        # a training step of the wide layer
        _prompt("gradient_train_d128", "gradient", [8192] * 2, 16, 128, 128, order="tokens"),
        # training on ragged packed documents, keys narrower than values
        _prompt("gradient_packed_d64_d128", "gradient", [1001, 77, 2047, 513, 3], 12, 64, 128, packed=True,
                order="tokens"),
        # a full decoding batch: the benchmark's 256 sequences x 16 heads
        _step("step_batch_d128", 256, 16, 128, 128),
        # a single conversation: latency
        _step("step_one_d64", 1, 16, 64, 64),
        # every head's output normalised and gated, for the training step above
        _norm("norm_heads_gated", "norm", 16384, 1, 2048, 16, gate=True),
        # the norm in front of a layer over images or latents (positions x channels), odd extent
        _norm("norm_spatial_f32", "norm", 6, 4225, 320, 32, dtype="f32"),
        # gradients of the two
        _norm("norm_grad_heads_gated", "norm_grad", 16384, 1, 2048, 16, gate=True),
        _norm("norm_grad_spatial", "norm_grad", 8, 4096, 512, 32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "gradient", "step", "norm", "norm_grad"])
    if op in ("prompt", "gradient"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        d_k, d_v = (rng.choice([64, 128]) for _ in range(2)) if dtype == "bf16" else (rng.choice([32, 64]),) * 2
        heads = rng.randint(1, 24)
        # tokens x heads at most: half of the longest listed prompt; a quarter of that for gradients, a 32nd in 32 bits
        most = 262144 // (4 if op == "gradient" else 1) // (8 if dtype == "f32" else 1)
        tokens = _log(rng, 1, max(2, most // heads))
        packed = rng.random() < 0.5
        if packed:
            n = min(tokens, rng.randint(1, 12))
            cuts = sorted(rng.sample(range(1, tokens), n - 1)) if n > 1 else []
            ends = cuts + [tokens]
            lens = [b - a for a, b in zip([0] + cuts, ends)]
            if rng.random() < 0.3:
                lens.insert(rng.randint(0, len(lens)), 0)  # a request with nothing new
        else:
            n = min(tokens, rng.randint(1, 4))
            lens = [max(1, tokens // n)] * n
        c = _prompt("", op, lens, heads, d_k, d_v, dtype, packed, rng.choice(["heads", "tokens"]),
                    state=rng.random() < 0.7)
    elif op == "step":
        d_k, d_v = (rng.choice([64, 128]) for _ in range(2))
        heads = rng.randint(1, 24)
        c = _step("", _log(rng, 1, 4096 // heads), heads, d_k, d_v, rng.choice(["bf16", "bf16", "f32"]))
    else:
        dtype = rng.choice(["bf16", "bf16", "f32"])
        gate = rng.random() < 0.5
        most = 33554432 // (1 if op == "norm" else 2)  # elements
        if rng.random() < 0.5:  # tokens x heads
            groups, width = rng.randint(1, 24), rng.choice([64, 128])
            channels = groups * width
            n, length = _log(rng, 1, most // channels // 2), 1
        else:  # positions x channels
            groups = rng.choice([1, 8, 16, 32])
            channels = groups * rng.choice([2, 3, 4, 8, 10, 16])
            n = rng.randint(1, 8)
            length = _log(rng, 1, max(2, min(16384, most // channels // n // 2)))
        c = _norm("", op, n, length, channels, groups, dtype, gate)
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs ----
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _log_decay(heads, gen):
    """Half-lives from about one token to a few thousand, spread over the heads."""
    at = (torch.arange(heads, device="cuda") + torch.rand(heads, device="cuda", generator=gen)) / heads
    return torch.log1p(-torch.exp2(-(1.0 + 10.0 * at))).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * (seed + 1) + 17)
    normal = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    unit = lambda x: x / torch.linalg.vector_norm(x, dim=-1, keepdim=True).clamp_min(1e-12)  # noqa: E731
    dt, op = _dtype(case), case["op"]
    s = {"op": op, "case": case}
    if op in ("prompt", "gradient"):
        lens, heads, d_k, d_v = _lens(case), case["heads"], case["d_k"], case["d_v"]
        batch, tokens = (1, sum(lens)) if case["packed"] else (len(lens), lens[0])

        def rows(x):  # [batch, tokens, heads, d] memory order or [batch, heads, tokens, d]; indexed [batch, heads, ...]
            x = x.to(dt)
            return x.transpose(1, 2) if case["order"] == "tokens" else x.transpose(1, 2).contiguous()

        s["q"] = rows(unit(normal(batch, tokens, heads, d_k)))
        s["k"] = rows(unit(normal(batch, tokens, heads, d_k)))
        s["v"] = rows(normal(batch, tokens, heads, d_v))
        s["log_decay"] = _log_decay(heads, gen)
        s["state"] = 0.1 * normal(len(lens), heads, d_v, d_k) if case["state"] else None
        s["cu_seqlens"] = None
        if case["packed"]:
            s["cu_seqlens"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
        if op == "gradient":
            s["grad_o"] = rows(normal(batch, tokens, heads, d_v))
            s["grad_state"] = normal(len(lens), heads, d_v, d_k) if case["state"] else None
        s["plan"] = _chunk_plan(lens)
    elif op == "step":
        n, heads, d_k, d_v = case["seqs"], case["heads"], case["d_k"], case["d_v"]
        s["q"] = unit(normal(n, heads, d_k)).to(dt)
        s["k"] = unit(normal(n, heads, d_k)).to(dt)
        s["v"] = normal(n, heads, d_v).to(dt)
        s["log_decay"] = _log_decay(heads, gen)
        s["state"] = 0.1 * normal(n, heads, d_v, d_k)
    else:
        shape = (case["n"], case["length"], case["channels"])
        s["x"] = (normal(*shape) * 1.5 + 0.3).to(dt)
        s["gate"] = normal(*shape).to(dt) if case["gate"] else None
        s["weight"] = 1.0 + 0.2 * normal(case["channels"])
        s["bias"] = 0.2 * normal(case["channels"])
        if op == "norm_grad":
            s["grad_y"] = normal(*shape).to(dt)
            x = s["x"].double().view(case["n"], case["length"], case["groups"], -1)  # what the forward pass kept
            var, mean = torch.var_mean(x, dim=(1, 3), correction=0)
            s["mean"], s["rstd"] = mean.float(), (var + 1e-5).rsqrt().float()
    return s


def _chunk_plan(lens):
    """The plain form's blocks of at most CHUNK tokens, none across two sequences: rows of each block, and where it lies."""
    first, seq, pos, size, row = [], [], [], [], 0
    for n, length in enumerate(lens):
        p = np.arange(0, length, CHUNK)
        first.append(row + p)
        seq.append(np.full(len(p), n))
        pos.append(p)
        size.append(np.minimum(CHUNK, length - p))
        row += length
    first, seq, pos, size = (np.concatenate(x) for x in (first, seq, pos, size))
    j = np.arange(CHUNK)
    valid = j[None, :] < size[:, None]
    index = np.where(valid, first[:, None] + j[None, :], 0)
    of_row = np.nonzero(valid.reshape(-1))[0]  # in the order of the rows
    cuda = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    return {"index": cuda(index), "valid": cuda(valid), "of_row": cuda(of_row), "seq": cuda(seq), "pos": cuda(pos),
            "size": cuda(size), "lens": cuda(np.array(lens))}


# ------------------------------------------------------------- plain form ----
def _blocks(x, plan):
    """[batch, heads, tokens, d] in any memory order -> fp32 [heads, blocks, CHUNK, d], zeros behind a block's end."""
    rows = x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3]).float()
    return rows[:, plan["index"]] * plan["valid"][None, :, :, None]


def _unblocks(y, like, plan):
    rows = y.reshape(y.shape[0], -1, y.shape[3])[:, plan["of_row"]]
    b, h, t, _ = like.shape
    return rows.view(h, b, t, -1).permute(1, 0, 2, 3).to(like.dtype)


def _power(log_decay, distance, keep):
    """gamma_h^distance where `keep`, else 0; the exponent in 64 bits: far positions."""
    d = distance.clamp_min(0).double()
    return (torch.exp(log_decay.double().view(-1, *([1] * d.dim())) * d) * keep).float()


def _plain_prompt(q, k, v, log_decay, state, plan, a):
    """o and W_T by blocks: inside a block (Q K^T * powers) V, between blocks the states."""
    Q, K, V = (_blocks(x, plan) for x in (q, k, v))
    seq, pos, size = plan["seq"], plan["pos"], plan["size"]
    i = torch.arange(CHUNK, device=q.device)
    inside = _power(log_decay, i[:, None] - i[None, :], i[:, None] >= i[None, :])       # [H, C, C]
    O = (Q @ K.transpose(2, 3) * inside[:, None] * a) @ V
    to_end = _power(log_decay, size[:, None] - 1 - i[None, :], plan["valid"])           # [H, M, C]
    delta = (V * (a * to_end[..., None])).transpose(2, 3) @ K                           # [H, M, dv, dk]
    before = (seq[:, None] == seq[None, :]) & (pos[:, None] > pos[None, :])
    reach = _power(log_decay, pos[:, None] - (pos + size)[None, :], before)             # [H, M, M]
    h, m, d_v, d_k = delta.shape
    start = (reach @ delta.view(h, m, -1)).view(delta.shape)
    n = torch.arange(len(plan["lens"]), device=q.device)
    of_seq = n[:, None] == seq[None, :]
    last = _power(log_decay, plan["lens"][:, None] - (pos + size)[None, :], of_seq)     # [H, N, M]
    end = (last @ delta.view(h, m, -1)).view(h, -1, d_v, d_k).transpose(0, 1)
    if state is not None:
        start = start + _power(log_decay, pos, torch.ones_like(pos))[..., None, None] * state.transpose(0, 1)[:, seq]
        end = end + _power(log_decay, plan["lens"], torch.ones_like(plan["lens"])).t()[..., None, None] * state
    O = O + _power(log_decay, i + 1, torch.ones_like(i))[:, None, :, None] * (Q @ start.transpose(2, 3))
    return _unblocks(O, v, plan), end


def _plain_gradient(q, k, v, grad_o, log_decay, state, grad_state, plan, a):
    w_t = None if state is None else state.transpose(2, 3)
    dq, _ = _plain_prompt(grad_o, v, k, log_decay, w_t, plan, a)  # dq_t = W_t^T do_t
    dq = dq.to(q.dtype)
    Q, K, V, G = (_blocks(x, plan) for x in (q, k, v, grad_o))
    seq, pos, size = plan["seq"], plan["pos"], plan["size"]
    i = torch.arange(CHUNK, device=q.device)
    inside = _power(log_decay, i[None, :] - i[:, None], i[:, None] <= i[None, :])       # [j, i]: gamma^(i - j)
    inside = inside[:, None] * a
    dV = (K @ Q.transpose(2, 3) * inside) @ G
    dK = (V @ G.transpose(2, 3) * inside) @ Q
    # dL/dW right behind a block's last token, from the later blocks and from dL/dW_T
    from_start = _power(log_decay, i + 1, torch.ones_like(i))[:, None, :, None]
    delta = (G * from_start).transpose(2, 3) @ Q                                        # [H, M, dv, dk]
    h, m, d_v, d_k = delta.shape
    after = (seq[:, None] == seq[None, :]) & (pos[:, None] < pos[None, :])
    reach = _power(log_decay, pos[None, :] - (pos + size)[:, None], after)
    end = (reach @ delta.view(h, m, -1)).view(delta.shape)
    n = torch.arange(len(plan["lens"]), device=q.device)
    of_seq = n[:, None] == seq[None, :]
    first = _power(log_decay, pos[None, :].expand(of_seq.shape), of_seq)
    dW0 = (first @ delta.view(h, m, -1)).view(h, -1, d_v, d_k).transpose(0, 1)
    if grad_state is not None:
        left = plan["lens"][seq] - (pos + size)
        end = end + _power(log_decay, left, torch.ones_like(left))[..., None, None] * grad_state.transpose(0, 1)[:, seq]
        dW0 = dW0 + _power(log_decay, plan["lens"], torch.ones_like(plan["lens"])).t()[..., None, None] * grad_state
    to_end = a * _power(log_decay, size[:, None] - 1 - i[None, :], plan["valid"])[..., None]
    dV = dV + to_end * (K @ end.transpose(2, 3))
    dK = dK + to_end * (V @ end)
    return {"dq": dq, "dk": _unblocks(dK, k, plan), "dv": _unblocks(dV, v, plan), "dW0": dW0}


def _plain_step(q, k, v, log_decay, state, a):
    state.mul_(torch.exp(log_decay)[None, :, None, None])
    state.add_((a * v.float())[..., :, None] * k.float()[..., None, :])
    o = (state @ q.float()[..., None])[..., 0]
    return o.to(v.dtype), state


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _plain_norm(x, groups, weight, bias, gate, eps):
    n, length, channels = x.shape
    xf = x.float().view(n, length, groups, channels // groups)
    mean = xf.mean(dim=(1, 3))
    centred = xf - mean[:, None, :, None]
    rstd = 1.0 / torch.sqrt(centred.square().mean(dim=(1, 3)) + eps)
    t = (centred * rstd[:, None, :, None]).view(x.shape) * weight + bias
    y = _silu(t) if gate is None else t * _silu(gate.float())
    return y.to(x.dtype), mean, rstd


def _plain_norm_grad(grad_y, x, groups, mean, rstd, weight, bias, gate):
    n, length, channels = x.shape
    by_group = (n, length, groups, channels // groups)
    hat = ((x.float().view(by_group) - mean[:, None, :, None]) * rstd[:, None, :, None]).view(x.shape)
    g, t, out = grad_y.float(), hat * weight + bias, {}
    z = t if gate is None else gate.float()
    sig = 1.0 / (1.0 + torch.exp(-z))
    slope = sig * (1.0 + z * (1.0 - sig))
    if gate is None:
        dt = g * slope
    else:
        dt = g * z * sig
        out["dgate"] = (g * t * slope).to(gate.dtype)
    out["dweight"] = (dt * hat).sum(dim=(0, 1))
    out["dbias"] = dt.sum(dim=(0, 1))
    dh = (dt * weight).view(by_group)
    hat = hat.view(by_group)
    centre = dh.mean(dim=(1, 3), keepdim=True) + hat * (dh * hat).mean(dim=(1, 3), keepdim=True)
    out["dx"] = ((dh - centre) * rstd[:, None, :, None]).view(x.shape).to(x.dtype)
    return out


# -------------------------------------------------------------------- run ----
def run(s):
    op, case = s["op"], s["case"]
    if own:
        import test_layers_causal_b200 as ttt
        if op == "prompt":
            o, W = ttt.forward_decay(s["q"], s["k"], s["v"], s["log_decay"], cu_seqlens=s["cu_seqlens"],
                                     state_in=s["state"])
            return {"o": o, "state": W}
        if op == "gradient":
            return ttt.backward_decay(s["q"], s["k"], s["v"], s["grad_o"], s["log_decay"], cu_seqlens=s["cu_seqlens"],
                                      state_in=s["state"], grad_state=s["grad_state"])
        if op == "step":
            o = ttt.decode_step_decay(s["q"], s["k"], s["v"], s["log_decay"], s["state"])
            return {"o": o, "state": s["state"]}
        if op == "norm":
            y, mean, rstd = ttt.group_norm(s["x"], case["groups"], s["weight"], s["bias"], gate=s["gate"],
                                           activation="silu", eps=1e-5)
            return {"y": y, "mean": mean, "rstd": rstd}
        g = ttt.group_norm_backward(s["grad_y"], s["x"], case["groups"], s["mean"], s["rstd"], s["weight"], s["bias"],
                                    gate=s["gate"], activation="silu")
        return {n: x for n, x in g.items() if x is not None}
    if op in ("prompt", "gradient", "step"):
        a = 1.0 / math.sqrt(case["d_k"])
    if op == "prompt":
        o, W = _plain_prompt(s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["plan"], a)
        return {"o": o, "state": W}
    if op == "gradient":
        return _plain_gradient(s["q"], s["k"], s["v"], s["grad_o"], s["log_decay"], s["state"], s["grad_state"],
                               s["plan"], a)
    if op == "step":
        o, W = _plain_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], a)
        return {"o": o, "state": W}
    if op == "norm":
        y, mean, rstd = _plain_norm(s["x"], case["groups"], s["weight"], s["bias"], s["gate"], 1e-5)
        return {"y": y, "mean": mean, "rstd": rstd}
    return _plain_norm_grad(s["grad_y"], s["x"], case["groups"], s["mean"], s["rstd"], s["weight"], s["bias"],
                            s["gate"])


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("prompt", "gradient"):
        lens, h, d_k, d_v = _lens(case), case["heads"], case["d_k"], case["d_v"]
        t, state = sum(lens), 4 * len(lens) * h * d_k * d_v
        if op == "prompt":  # update and read-out of the state: 2 products of d_k d_v per token and head
            return {"bytes": t * h * 2 * (d_k + d_v) * e + state * (2 if case["state"] else 1),
                    "flops": t * h * 4 * d_k * d_v}
        # q, k, v, do in, dq, dk, dv out; W and dL/dW updated, dq, dk, dv read out: 5 products
        return {"bytes": t * h * (4 * d_k + 3 * d_v) * e + state * (3 if case["state"] else 1),
                "flops": t * h * 10 * d_k * d_v}
    if op == "step":
        n, d_k, d_v = case["seqs"] * case["heads"], case["d_k"], case["d_v"]
        return {"bytes": n * (2 * 4 * d_k * d_v + 2 * (d_k + d_v) * e), "flops": n * 5 * d_k * d_v}
    count = case["n"] * case["length"] * case["channels"]
    stats = 8 * case["n"] * case["groups"]
    if op == "norm":
        return {"bytes": count * e * (3 if case["gate"] else 2) + stats + 8 * case["channels"], "flops": count * 12}
    return {"bytes": count * e * (5 if case["gate"] else 3) + stats + 16 * case["channels"], "flops": count * 25}


# ------------------------------------------------------------------ exact ----
def _walk(x, n, t0, t1, case, first):
    """Tokens [t0, t1) of sequence n as fp64 [heads, tokens, d]."""
    return (x[0, :, first[n] + t0:first[n] + t1] if case["packed"] else x[n, :, t0:t1]).double()


def _exact_prompt(s, case):
    """Runs of tokens in order, in fp64, the state carried from one run to the next; inside a run every pair."""
    lens, a = _lens(case), 1.0 / math.sqrt(case["d_k"])
    first = np.concatenate([[0], np.cumsum(lens)])
    ld, step = s["log_decay"].double(), 384
    o = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
    ends = []
    for n, length in enumerate(lens):
        W = torch.zeros(case["heads"], case["d_v"], case["d_k"], dtype=torch.float64, device="cuda")
        if s["state"] is not None:
            W = s["state"][n].double()
        for t0 in range(0, length, step):
            t1 = min(length, t0 + step)
            q, k, v = (_walk(s[x], n, t0, t1, case, first) for x in ("q", "k", "v"))
            t = torch.arange(t1 - t0, dtype=torch.float64, device="cuda")
            w = torch.tril(torch.exp(ld[:, None, None] * (t[:, None] - t[None, :]).clamp_min(0)))
            y = torch.einsum("hij,hij,hjd->hid", torch.einsum("hid,hjd->hij", q, k), w * a, v)
            y += torch.exp(ld[:, None] * (t + 1))[..., None] * torch.einsum("hid,hvd->hiv", q, W)
            if case["packed"]:
                o[0, :, first[n] + t0:first[n] + t1] = y
            else:
                o[n, :, t0:t1] = y
            tail = a * torch.exp(ld[:, None] * (t[-1] - t))
            W = torch.exp(ld * (t1 - t0))[:, None, None] * W + torch.einsum("hj,hjv,hjd->hvd", tail, v, k)
        ends.append(W)
    return {"o": o, "state": torch.stack(ends)}


def _exact_gradient(s, case):
    """The chain rule over runs of tokens in fp64: dL/dW carried from the last token to the first, W the other way."""
    lens, a = _lens(case), 1.0 / math.sqrt(case["d_k"])
    first = np.concatenate([[0], np.cumsum(lens)])
    ld, step = s["log_decay"].double(), 384
    grads = {g: torch.zeros(s[x].shape, dtype=torch.float64, device="cuda") for g, x in (("dq", "q"), ("dk", "k"), ("dv", "v"))}
    dW0 = []

    def put(name, n, t0, t1, value):
        if case["packed"]:
            grads[name][0, :, first[n] + t0:first[n] + t1] = value
        else:
            grads[name][n, :, t0:t1] = value

    for n, length in enumerate(lens):
        W = torch.zeros(case["heads"], case["d_v"], case["d_k"], dtype=torch.float64, device="cuda")
        G = W.clone()  # dL/dW behind the last token of the run
        if s["state"] is not None:
            W, G = s["state"][n].double(), s["grad_state"][n].double()
        starts = list(range(0, length, step))
        for t0 in starts:
            t1 = min(length, t0 + step)
            k, v, g = (_walk(s[x], n, t0, t1, case, first) for x in ("k", "v", "grad_o"))
            t = torch.arange(t1 - t0, dtype=torch.float64, device="cuda")
            w = a * torch.tril(torch.exp(ld[:, None, None] * (t[:, None] - t[None, :]).clamp_min(0)))
            dq = torch.einsum("hij,hij,hjd->hid", torch.einsum("hiv,hjv->hij", g, v), w, k)
            dq += torch.exp(ld[:, None] * (t + 1))[..., None] * torch.einsum("hiv,hvd->hid", g, W)
            put("dq", n, t0, t1, dq)
            tail = a * torch.exp(ld[:, None] * (t[-1] - t))
            W = torch.exp(ld * (t1 - t0))[:, None, None] * W + torch.einsum("hj,hjv,hjd->hvd", tail, v, k)
        for t0 in reversed(starts):
            t1 = min(length, t0 + step)
            q, k, v, g = (_walk(s[x], n, t0, t1, case, first) for x in ("q", "k", "v", "grad_o"))
            t = torch.arange(t1 - t0, dtype=torch.float64, device="cuda")
            w = a * torch.tril(torch.exp(ld[:, None, None] * (t[:, None] - t[None, :]).clamp_min(0)))
            tail = (a * torch.exp(ld[:, None] * (t[-1] - t)))[..., None]
            put("dv", n, t0, t1, torch.einsum("hij,hij,hiv->hjv", torch.einsum("hid,hjd->hij", q, k), w, g)
                + tail * torch.einsum("hvd,hjd->hjv", G, k))
            put("dk", n, t0, t1, torch.einsum("hij,hij,hid->hjd", torch.einsum("hiv,hjv->hij", g, v), w, q)
                + tail * torch.einsum("hvd,hjv->hjd", G, v))
            G = torch.exp(ld * (t1 - t0))[:, None, None] * G
            G += torch.einsum("hi,hiv,hid->hvd", torch.exp(ld[:, None] * (t + 1)), g, q)
        dW0.append(G)
    return {**grads, "dW0": torch.stack(dW0)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prompt":
        return _exact_prompt(s, case)
    if op == "gradient":
        return _exact_gradient(s, case)
    if op == "step":
        W = torch.einsum("h,nhvd->nhvd", s["log_decay"].double().exp(), s["state"].double())
        W += torch.einsum("nhv,nhd->nhvd", s["v"].double(), s["k"].double()) / math.sqrt(case["d_k"])
        return {"o": torch.einsum("nhvd,nhd->nhv", W, s["q"].double()), "state": W}
    n, length, channels, groups = case["n"], case["length"], case["channels"], case["groups"]
    x = s["x"].double().view(n, length, groups, channels // groups)
    weight, bias = (s[p].double().view(groups, -1) for p in ("weight", "bias"))
    gate = None if s["gate"] is None else s["gate"].double().view(x.shape)
    if op == "norm":
        var, mean = torch.var_mean(x, dim=(1, 3), correction=0, keepdim=True)
        t = (x - mean) * (var + 1e-5).rsqrt() * weight + bias
        y = t * torch.sigmoid(t) if gate is None else t * gate * torch.sigmoid(gate)
        return {"y": y.view(s["x"].shape), "mean": mean.view(n, groups), "rstd": (var + 1e-5).rsqrt().view(n, groups)}
    # the gradient with mean and rstd taken from x, differentiated by the tape
    x.requires_grad_(True)
    hat = (x - s["mean"].double().view(n, 1, groups, 1)) * s["rstd"].double().view(n, 1, groups, 1)
    g = s["grad_y"].double().view(x.shape)
    w, b = weight.clone().requires_grad_(True), bias.clone().requires_grad_(True)
    if gate is not None:
        gate.requires_grad_(True)
    h = hat.detach().requires_grad_(True)
    t = h * w + b
    y = t * torch.sigmoid(t) if gate is None else t * (gate * torch.sigmoid(gate))
    wanted = torch.autograd.grad(y, [h, w, b] + ([gate] if gate is not None else []), g)
    dh = wanted[0]
    h = h.detach()
    dx = dh - dh.mean(dim=(1, 3), keepdim=True) - h * (dh * h).mean(dim=(1, 3), keepdim=True)
    out = {"dx": (dx * s["rstd"].double().view(n, 1, groups, 1)).view(s["x"].shape), "dweight": wanted[1].reshape(-1),
           "dbias": wanted[2].reshape(-1)}
    if gate is not None:
        out["dgate"] = wanted[3].view(s["x"].shape)
    return out
