"""The attention operators as a user's program runs them, over the range of their real sizes.

Three operators: rotary positions (forward and backward), attention over grouped-tril, length and
sliding-window masks (prompts and single tokens over a cache) and attention's backward pass, which
recomputes the probabilities. Each case is a dict of plain values; ``prepare`` makes its inputs,
``run`` makes one pass (in plain torch operations, or through this framework's calls where ``own``
is true), ``exact`` computes the same outputs in 64 bits.

Row i of batch b stands at position r = offset_b + i, L = seq_lens[b]; entry (r, c) is kept iff
0 <= r < L and c <= r (mask 0), c < L (mask 1) or r - window < c <= r (mask 2). Rows that keep
nothing give o = 0, lse = -inf and no gradient.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _attention(op, name, B, Hq, Hkv, Sq, Skv, d, dtype, lens, mask=0, window=0, layout="bhsd"):
    c = {"op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "Sq": Sq, "Skv": Skv, "d": d, "dtype": dtype, "len_lo": lens[0],
         "len_hi": lens[1], "mask": mask, "window": window, "layout": layout}
    return {"name": name, **c} if name else c


def _rotary(op, name, B, Hq, Hkv, S, d, rot, dtype, first, interleaved=False, factor=1.0, layout="bhsd"):
    c = {"op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "S": S, "d": d, "rot": rot, "dtype": dtype, "first": first,
         "interleaved": interleaved, "factor": factor, "layout": layout}
    return {"name": name, **c} if name else c


def listed():
    return [
        # A training or prompt pass with shared heads; q, k and v are views of the projections' [B, S, H d] outputs.
        _attention("forward", "forward_shared_heads_d128", 4, 32, 8, 4096, 4096, 128, "bf16", (2500, 4096), layout="bshd"),
        # The benchmark's attention shape, [32, 16, 2048] with head dim 64 and lengths 1024..2048.
        _attention("forward", "forward_s2048_d64", 32, 16, 16, 2048, 2048, 64, "bf16", (1024, 2048)),
        # A long document under a local causal window.
        _attention("forward", "forward_long_window", 1, 16, 2, 16384, 16384, 128, "f16", (16384, 16384), 2, 1024),
        # Short padded sequences of odd lengths, all keys visible (an encoder's batch): latency counts.
        _attention("forward", "forward_short_padded", 3, 8, 8, 333, 333, 64, "f16", (118, 333), 1),
        # One new token for each of 64 sequences over their caches: serving under load.
        _attention("forward", "token_batch64", 64, 32, 8, 1, 8192, 128, "bf16", (700, 8192)),
        # One new token of one short sequence: the smallest call of a serving loop.
        _attention("forward", "token_single", 1, 16, 4, 1, 1025, 64, "f16", (1025, 1025)),
        # The backward pass of the benchmark's attention shape.
        _attention("backward", "backward_s2048_d64", 32, 16, 16, 2048, 2048, 64, "bf16", (1024, 2048)),
        # The backward pass of a training step with shared heads, on views of the projections.
        _attention("backward", "backward_shared_heads_d128", 2, 32, 8, 4096, 4096, 128, "bf16", (3500, 4096), layout="bshd"),
        # The backward pass of an odd length under a narrow window.
        _attention("backward", "backward_odd_window", 1, 12, 4, 2611, 2611, 128, "f16", (2611, 2611), 2, 256),
        # q and k of a training step or prompt, half layout, long-context frequencies.
        _rotary("rotary", "rotary_prompt", 4, 32, 8, 4096, 128, 128, "bf16", 0, factor=8.0, layout="bshd"),
        # q and k of one new token for each of 64 sequences, far into their contexts.
        _rotary("rotary", "rotary_token_batch64", 64, 32, 8, 1, 128, 128, "bf16", 100000, interleaved=True, factor=8.0),
        # The gradient of a partial rotation in 32 bits.
        _rotary("rotary_backward", "rotary_backward_partial", 2, 16, 16, 2048, 64, 32, "f32", 0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "token", "chunk", "backward", "backward", "rotary", "rotary_backward"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 8])
    Hq = Hkv * group
    if op in ("rotary", "rotary_backward"):
        S = _log_int(rng, 1, 8192)
        B = _log_int(rng, 1, max(1, min(64, 4 * 32 * 4096 // (S * Hq))))
        rot = rng.choice([d, d, d // 2, d // 4])
        return _rotary(op, None, B, Hq, Hkv, S, d, rot, rng.choice(["bf16", "f16", "f32"]), _log_int(rng, 1, 500000) - 1,
                       rng.choice([False, True]), rng.choice([1.0, 8.0]), rng.choice(["bhsd", "bshd"]))
    dtype, layout = rng.choice(["bf16", "f16"]), rng.choice(["bhsd", "bshd"])
    mask = rng.choice([0, 0, 1, 2])
    if op in ("token", "chunk"):
        Skv = _log_int(rng, 200, 16384)
        Sq = 1 if op == "token" else _log_int(rng, 2, min(700, Skv))
        B = _log_int(rng, 1, max(1, min(64, 4 * 32 * 4096 * 4096 // (Skv * max(Sq, 64) * Hq * 4))))
        return _attention("forward", None, B, Hq, Hkv, Sq, Skv, d, dtype, (max(Sq, Skv // rng.randint(1, 8)), Skv), mask,
                          _log_int(rng, 16, 4096) if mask == 2 else 0, layout)
    S = _log_int(rng, 30, 6000)
    B = _log_int(rng, 1, max(1, min(32, 2 * 32 * 4096 * 4096 // (S * S * Hq))))
    return _attention(op, None, B, Hq, Hkv, S, S, d, dtype, (max(1, S // rng.randint(1, 4)), S), mask,
                      _log_int(rng, 16, 2048) if mask == 2 else 0, layout)


def _lens(case):
    """Lengths spread evenly over [len_lo, len_hi], the long and the short ones mixed."""
    B, lo, hi = case["B"], case["len_lo"], case["len_hi"]
    return [hi - (hi - lo) * ((7 * b) % B) // max(1, B - 1) if B > 1 else hi for b in range(B)]


def _offsets(case):
    """None for whole sequences; otherwise the new tokens are the last Sq of each sequence."""
    if case["Sq"] == case["Skv"]:
        return None
    return [n - case["Sq"] for n in _lens(case)]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _heads(B, H, S, d, layout, dtype, gen, std=1.0):
    """[B, H, S, d] of N(0, std^2): contiguous, or a view of a [B, S, H, d] projection."""
    shape = (B, S, H, d) if layout == "bshd" else (B, H, S, d)
    t = (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)
    return t.transpose(1, 2) if layout == "bshd" else t


def _frequencies(rot, base, factor, low, high, original):
    """Inverse frequencies of the rotated pairs; long-context scaling by parts where factor != 1."""
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    wave = 2.0 * math.pi / f
    mix = np.clip((original / wave - low) / (high - low), 0.0, 1.0)
    return ((1.0 - mix) * f / factor + mix * f).astype(np.float32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    if case["op"].startswith("rotary"):
        B, S, d = case["B"], case["S"], case["d"]
        q = _heads(B, case["Hq"], S, d, case["layout"], dtype, gen)
        k = _heads(B, case["Hkv"], S, d, case["layout"], dtype, gen)
        first = case["first"] + torch.randint(0, 64, (B, 1), generator=gen, device="cuda")
        positions = (first + torch.arange(S, device="cuda")).to(torch.int32)
        f = torch.from_numpy(_frequencies(case["rot"], 500000.0, case["factor"], 1.0, 4.0, 8192)).cuda()
        return {"case": case, "q": q, "k": k, "positions": positions, "inv_freq": f}
    B, d = case["B"], case["d"]
    state = {"case": case, "scale": d ** -0.5}
    state["q"] = _heads(B, case["Hq"], case["Sq"], d, case["layout"], dtype, gen)
    state["k"] = _heads(B, case["Hkv"], case["Skv"], d, case["layout"], dtype, gen)
    state["v"] = _heads(B, case["Hkv"], case["Skv"], d, case["layout"], dtype, gen)
    state["seq_lens"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    off = _offsets(case)
    state["q_offsets"] = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    if case["op"] == "backward":
        state["dout"] = _heads(B, case["Hq"], case["Sq"], d, case["layout"], dtype, gen, 0.01)
        state["o"], state["lse"] = _plain_forward(state)   # what the forward pass left
    return state


# ---------------------------------------------------------------------------
# The plain forms, in 32 bits
# ---------------------------------------------------------------------------

def _plain_kept(state):
    """[B, 1, Sq, Skv] truth values of the kept entries."""
    case = state["case"]
    L = state["seq_lens"].long()[:, None, None, None]
    r = torch.arange(case["Sq"], device="cuda")[None, None, :, None]
    if state["q_offsets"] is not None:
        r = r + state["q_offsets"].long()[:, None, None, None]
    c = torch.arange(case["Skv"], device="cuda")[None, None, None, :]
    live = (r >= 0) & (r < L)
    if case["mask"] == 1:
        return live & (c < L)
    kept = live & (c <= r)
    return kept & (c > r - case["window"]) if case["mask"] == 2 else kept


def _plain_shared(state, name):
    """k or v in 32 bits with each head repeated for the query heads that share it."""
    t = state[name].float()
    group = state["case"]["Hq"] // state["case"]["Hkv"]
    return t if group == 1 else t.repeat_interleave(group, 1)


def _plain_scores(state):
    s = torch.matmul(state["q"].float(), _plain_shared(state, "k").transpose(-1, -2))
    return s.mul_(state["scale"]).masked_fill_(~_plain_kept(state), -math.inf)


def _plain_forward(state):
    s = _plain_scores(state)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = s.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, _plain_shared(state, "v")) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log()).squeeze(-1)
    return o.to(state["q"].dtype), lse


def _plain_backward(state):
    case, q, dout = state["case"], state["q"].float(), state["dout"].float()
    lse = state["lse"].unsqueeze(-1)
    p = _plain_scores(state).sub_(torch.where(lse == -math.inf, torch.zeros_like(lse), lse)).exp_()
    dv = torch.matmul(p.transpose(-1, -2), dout)
    ds = torch.matmul(dout, _plain_shared(state, "v").transpose(-1, -2))
    ds = ds.sub_((ds * p).sum(-1, keepdim=True)).mul_(p).mul_(state["scale"])
    dq = torch.matmul(ds, _plain_shared(state, "k"))
    dk = torch.matmul(ds.transpose(-1, -2), q)
    shape = (case["B"], case["Hkv"], case["Hq"] // case["Hkv"], case["Skv"], case["d"])
    t = state["q"].dtype
    return dq.to(t), dk.view(shape).sum(2).to(t), dv.view(shape).sum(2).to(t)


def _plain_rotate(case, x, cos, sin):
    rot, x32 = case["rot"], x.float()
    if case["interleaved"]:
        a, b = x32[..., 0:rot:2], x32[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x32[..., :rot // 2], x32[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x32[..., rot:]), -1).to(x.dtype)


def _plain_rotary(state):
    case = state["case"]
    angle = state["positions"].double()[:, None, :, None] * state["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    if case["op"] == "rotary_backward":
        sin = -sin
    return _plain_rotate(case, state["q"], cos, sin), _plain_rotate(case, state["k"], cos, sin)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    if case["op"] == "forward":
        o, lse = _plain_forward(state)
        return {"o": o, "lse": lse}
    if case["op"] == "backward":
        dq, dk, dv = _plain_backward(state)
        return {"dq": dq, "dk": dk, "dv": dv}
    yq, yk = _plain_rotary(state)
    return {"q": yq, "k": yk}


def _own(state, case):
    import masked_softmax_attention_gb300 as gtms

    if case["op"] == "forward":
        o, lse = gtms.attention_forward(state["q"], state["k"], state["v"], state["seq_lens"], state["scale"],
                                        mask_kind=case["mask"], window=case["window"], q_offsets=state["q_offsets"])
        return {"o": o, "lse": lse}
    if case["op"] == "backward":
        dq, dk, dv = gtms.attention_backward(state["q"], state["k"], state["v"], state["o"], state["lse"], state["dout"],
                                             state["seq_lens"], state["scale"], mask_kind=case["mask"],
                                             window=case["window"], q_offsets=state["q_offsets"])
        return {"dq": dq, "dk": dk, "dv": dv}
    call = gtms.rotary_forward if case["op"] == "rotary" else gtms.rotary_backward
    yq, yk = call(state["q"], state["positions"], state["inv_freq"], other=state["k"], interleaved=case["interleaved"])
    return {"q": yq, "k": yk}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def _kept_pairs(case):
    """Per batch: kept (row, column) pairs, live rows and keys that some row keeps."""
    found = []
    for n, off in zip(_lens(case), _offsets(case) or [0] * case["B"]):
        r = np.arange(case["Sq"], dtype=np.int64) + off
        r = r[(r >= 0) & (r < n)]
        if not r.size:
            found.append((0, 0, 0))
            continue
        if case["mask"] == 1:
            found.append((int(r.size) * n, int(r.size), n))
            continue
        lo = np.maximum(0, r - case["window"] + 1) if case["mask"] == 2 else np.zeros_like(r)
        found.append((int((r + 1 - lo).sum()), int(r.size), int(r[-1] + 1 - lo[0])))
    return found


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("rotary"):
        heads = case["B"] * (case["Hq"] + case["Hkv"]) * case["S"]
        return {"bytes": 2 * heads * case["d"] * e + 4 * case["B"] * case["S"], "flops": 3 * heads * case["rot"]}
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    pairs, rows, keys = (sum(x) for x in zip(*_kept_pairs(case)))
    q_out, k_out = case["B"] * Hq * case["Sq"] * d * e, case["B"] * Hkv * case["Skv"] * d * e
    q_in, k_in = rows * Hq * d * e, keys * Hkv * d * e
    if case["op"] == "forward":
        return {"bytes": q_in + 2 * k_in + q_out + 4 * case["B"] * Hq * case["Sq"], "flops": 4 * d * pairs * Hq}
    return {"bytes": 3 * q_in + 2 * k_in + 4 * rows * Hq + q_out + 2 * k_out, "flops": 10 * d * pairs * Hq}


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    if case["op"].startswith("rotary"):
        return _exact_rotary(state, case)
    q, k, v = (state[n].double() for n in ("q", "k", "v"))
    back = case["op"] == "backward"
    group, rows = case["Hq"] // case["Hkv"], 1024
    o, lse = torch.zeros_like(q), torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b, (n, off) in enumerate(zip(_lens(case), _offsets(case) or [0] * case["B"])):
        for i0 in range(max(0, -off), min(case["Sq"], n - off), rows):
            i1 = min(case["Sq"], n - off, i0 + rows)
            pos = torch.arange(off + i0, off + i1, device="cuda")[:, None]
            c0 = max(0, off + i0 - case["window"] + 1) if case["mask"] == 2 else 0
            c1 = n if case["mask"] == 1 else off + i1
            col = torch.arange(c0, c1, device="cuda")[None, :]
            out = torch.zeros((i1 - i0, c1 - c0), dtype=torch.bool, device="cuda")
            if case["mask"] != 1:
                out = col > pos
            if case["mask"] == 2:
                out = out | (col <= pos - case["window"])
            for g in range(case["Hkv"]):
                h = slice(g * group, (g + 1) * group)
                kk, vv = k[b, g, c0:c1], v[b, g, c0:c1]
                z = torch.einsum("hid,cd->hic", q[b, h, i0:i1], kk) * state["scale"]
                z.masked_fill_(out, -math.inf)
                norm = torch.logsumexp(z, -1)
                p = torch.exp(z - norm[..., None])
                y = torch.einsum("hic,cd->hid", p, vv)
                o[b, h, i0:i1], lse[b, h, i0:i1] = y, norm
                if back:
                    dy = state["dout"][b, h, i0:i1].double()
                    dz = p * (torch.einsum("hid,cd->hic", dy, vv) - (dy * y).sum(-1, keepdim=True)) * state["scale"]
                    dq[b, h, i0:i1] = torch.einsum("hic,cd->hid", dz, kk)
                    dk[b, g, c0:c1] += torch.einsum("hic,hid->cd", dz, q[b, h, i0:i1])
                    dv[b, g, c0:c1] += torch.einsum("hic,hid->cd", p, dy)
    return {"dq": dq, "dk": dk, "dv": dv} if back else {"o": o, "lse": lse}


def _exact_rotary(state, case):
    rot = case["rot"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       state["positions"].double()[:, None, :, None] * state["inv_freq"].double())
    if case["op"] == "rotary_backward":
        turn = turn.conj()
    got = {}
    for name in ("q", "k"):
        y = state[name].double().clone()
        if case["interleaved"]:
            z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * turn
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        else:
            z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        got[name] = y
    return got
