"""The operators of a serving loop's caches as a user's program runs them, over the range of their real sizes.

Three operators: attention for a batch whose sequences share long prefixes (samples of one prompt), the weight that
each key of a cache received (accumulated over query rows and the heads that share it), and the eviction of the keys
of least weight from a cache. Each case is a dict of plain values; ``prepare`` makes its inputs, ``run`` makes one
pass (in plain torch operations, or through this framework's calls where ``own`` is true), ``exact`` computes the same
outputs in 64 bits.

Row i of batch b stands at position r = offset_b + i of its own sequence, L = seq_lens[b]; its own entry (r, c) is
kept iff 0 <= r < L and c <= r (mask 0), c < L (mask 1) or r - window < c <= r (mask 2). Sequence b of a batch of
G n sequences also keeps the first prefix_lens[b / n] keys of prefix b / n, where 0 <= r < L.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _prefix(name, G, n, Hq, Hkv, Sq, P, Skv, d, dtype, prefix_lens, lens, mask=0, layout="bhsd"):
    c = {"op": "prefix", "G": G, "B": G * n, "Hq": Hq, "Hkv": Hkv, "Sq": Sq, "P": P, "Skv": Skv, "d": d, "dtype": dtype,
         "prefix_lo": prefix_lens[0], "prefix_hi": prefix_lens[1], "len_lo": lens[0], "len_hi": lens[1], "mask": mask,
         "window": 0, "layout": layout}
    return {"name": name, **c} if name else c


def _weights(name, B, Hq, Hkv, Sq, Skv, d, dtype, lens, mask=0, window=0, accumulate=False, layout="bhsd"):
    c = {"op": "weights", "B": B, "Hq": Hq, "Hkv": Hkv, "Sq": Sq, "Skv": Skv, "d": d, "dtype": dtype, "len_lo": lens[0],
         "len_hi": lens[1], "mask": mask, "window": window, "accumulate": accumulate, "layout": layout}
    return {"name": name, **c} if name else c


def _evict(name, B, H, S, keep, d, dtype, lens, first, recent, layout="bhsd"):
    c = {"op": "evict", "B": B, "H": H, "S": S, "keep": keep, "d": d, "dtype": dtype, "len_lo": lens[0], "len_hi": lens[1],
         "first": first, "recent": recent, "layout": layout}
    return {"name": name, **c} if name else c


def listed():
    return [
        # One new token for each of 64 samples of one prompt, their own tokens so far between 100 and 1024.
        _prefix("prefix_samples64", 1, 64, 32, 8, 1, 8192, 1024, 128, "bf16", (8192, 8192), (100, 1024)),
        # Four long documents with eight questions each, answers well under way.
        _prefix("prefix_documents", 4, 8, 16, 2, 1, 32768, 2048, 128, "f16", (20000, 32768), (300, 2048)),
        # Four samples of one short prompt: the smallest call of a serving loop.
        _prefix("prefix_small", 1, 4, 16, 4, 1, 500, 64, 64, "bf16", (500, 500), (3, 64)),
        # Five drafted tokens to be checked for each of 24 samples, odd lengths.
        _prefix("prefix_drafts", 1, 24, 12, 4, 5, 5003, 333, 64, "f16", (5003, 5003), (50, 333), layout="bshd"),
        # The prompts of 16 requests behind one instruction of 4096 tokens.
        _prefix("prefix_prompts", 1, 16, 32, 8, 512, 4096, 512, 128, "bf16", (4096, 4096), (300, 512), layout="bshd"),
        # What a whole prompt's rows paid to each key, before the cache is first cut.
        _weights("weights_prompt", 4, 32, 8, 4096, 4096, 128, "bf16", (2500, 4096), layout="bshd"),
        # The last 32 rows of eight long prompts, which stand for what later rows will ask for.
        _weights("weights_last_rows", 8, 32, 8, 32, 16384, 128, "bf16", (9000, 16384)),
        # The step of one new token for 64 sequences, added to what stands there.
        _weights("weights_token", 64, 32, 8, 1, 8192, 128, "bf16", (700, 8192), accumulate=True),
        # Two short sequences of odd lengths under a window: latency counts.
        _weights("weights_small", 2, 8, 2, 333, 333, 64, "f16", (118, 333), mask=2, window=100),
        # Half of the caches of 32 sequences goes; the shortest stay whole.
        _evict("evict_half", 32, 8, 16384, 8192, 128, "bf16", (7000, 16384), 4, 256),
        # One long sequence keeps a quarter of its cache.
        _evict("evict_long", 1, 8, 131072, 32768, 128, "f16", (131072, 131072), 16, 1024, layout="bshd"),
        # Three short sequences, head dim 64: latency counts.
        _evict("evict_small", 3, 4, 500, 201, 64, "bf16", (150, 500), 4, 33),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "prefix", "weights", "weights", "evict", "evict"])
    d, layout = rng.choice([64, 128]), rng.choice(["bhsd", "bshd"])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 8])
    dtype = rng.choice(["bf16", "f16"])
    if op == "evict":
        S, dtype = _log_int(rng, 16, 131072), rng.choice(["bf16", "f16", "f32"])
        B = _log_int(rng, 1, max(1, min(64, 32 * 8 * 16384 * 128 // (S * Hkv * d * (4 if dtype == "f32" else 2)))))
        keep = max(2, int(S * rng.uniform(0.05, 0.95)))
        first, recent = rng.randint(0, min(16, keep // 4)), rng.randint(0, keep // 4)
        return _evict(None, B, Hkv, S, keep, d, dtype, (max(1, S // rng.randint(1, 4)), S), first, recent, layout)
    if op == "prefix":
        Sq = rng.choice([1, 1, 1, _log_int(rng, 2, 16), _log_int(rng, 17, 600)])
        P = _log_int(rng, 1, 32768)
        Skv = _log_int(rng, Sq, max(Sq, 2048))
        most = 16 * 32 * 512 * 4608 * 64 // (Hq * max(Sq, 16) * (P + Skv) * d)
        G = min(rng.choice([1, 1, 2, 4]), max(1, most))
        n = _log_int(rng, 1, max(1, min(64, most // G)))
        return _prefix(None, G, n, Hq, Hkv, Sq, P, Skv, d, dtype, (max(1, P // rng.randint(1, 3)), P),
                       (max(Sq, Skv // rng.randint(1, 4)), Skv), rng.choice([0, 0, 1]), layout)
    Skv = _log_int(rng, 30, 16384)
    Sq = rng.choice([1, _log_int(rng, 2, min(64, Skv)), 0])
    if Sq == 0:   # a whole prompt
        Sq = Skv = _log_int(rng, 65, 5000)
    B = _log_int(rng, 1, max(1, min(64, 2 * 32 * 4096 * 4096 // (Hq * max(Sq, 16) * Skv))))
    mask = rng.choice([0, 0, 1, 2])
    return _weights(None, B, Hq, Hkv, Sq, Skv, d, dtype, (max(Sq if Sq <= 64 else 1, Skv // rng.randint(1, 4)), Skv), mask,
                    _log_int(rng, 16, 4096) if mask == 2 else 0, rng.choice([False, True]), layout)


def _spread(count, lo, hi):
    """Lengths spread evenly over [lo, hi], the long and the short ones mixed."""
    return [hi - (hi - lo) * ((7 * b) % count) // max(1, count - 1) if count > 1 else hi for b in range(count)]


def _lens(case):
    return _spread(case["B"], case["len_lo"], case["len_hi"])


def _prefix_lens(case):
    return _spread(case["G"], case["prefix_lo"], case["prefix_hi"])


def _offsets(case):
    """None for whole sequences; otherwise the new tokens are the last Sq of each sequence."""
    return None if case["Sq"] == case["Skv"] else [n - case["Sq"] for n in _lens(case)]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _heads(B, H, S, d, layout, dtype, gen):
    """[B, H, S, d] of N(0, 1): contiguous, or a view of a [B, S, H, d] projection or cache."""
    shape = (B, S, H, d) if layout == "bshd" else (B, H, S, d)
    t = torch.randn(shape, generator=gen, device="cuda").to(dtype)
    return t.transpose(1, 2) if layout == "bshd" else t


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    state = {"case": case, "seq_lens": _int32(_lens(case))}
    if case["op"] == "evict":
        B, H, S, keep, d, layout = (case[n] for n in ("B", "H", "S", "keep", "d", "layout"))
        state["k"], state["v"] = (_heads(B, H, S, d, layout, dtype, gen) for _ in range(2))
        # Few keys have most of the weight; some were never paid any and tie.
        w = torch.exp(2.0 * torch.randn((B, H, S), generator=gen, device="cuda"))
        state["weights"] = w * (torch.rand((B, H, S), generator=gen, device="cuda") > 0.02)
        # Entries have stood at these positions of their sequences since an earlier cut.
        state["positions"] = (3 * torch.arange(S, device="cuda", dtype=torch.int32) + 1).expand(B, H, S).contiguous()
        shape = (B, keep, H, d) if layout == "bshd" else (B, H, keep, d)
        k, v = (torch.zeros(shape, dtype=dtype, device="cuda") for _ in range(2))
        k, v = (t.transpose(1, 2) if layout == "bshd" else t for t in (k, v))
        state["out"] = (k, v, torch.zeros((B, H, keep), device="cuda"),
                        torch.zeros((B, H, keep), dtype=torch.int32, device="cuda"))
        return state
    B, d, layout = case["B"], case["d"], case["layout"]
    state["scale"] = d ** -0.5
    state["q"] = _heads(B, case["Hq"], case["Sq"], d, layout, dtype, gen)
    state["k"] = _heads(B, case["Hkv"], case["Skv"], d, layout, dtype, gen)
    off = _offsets(case)
    state["q_offsets"] = None if off is None else _int32(off)
    if case["op"] == "prefix":
        state["v"] = _heads(B, case["Hkv"], case["Skv"], d, layout, dtype, gen)
        state["k_prefix"], state["v_prefix"] = (_heads(case["G"], case["Hkv"], case["P"], d, layout, dtype, gen)
                                                for _ in range(2))
        state["prefix_lens"] = _int32(_prefix_lens(case))
        return state
    state["lse"] = torch.logsumexp(_plain_scores(state), -1)   # what attention left
    before = torch.rand((B, case["Hkv"], case["Skv"]), generator=gen, device="cuda")
    state["weights"] = before if case["accumulate"] else torch.empty_like(before)
    return state


# ---------------------------------------------------------------------------
# The plain forms, in 32 bits
# ---------------------------------------------------------------------------

def _plain_rows(state):
    """Positions [B, 1, Sq, 1] of the rows, and whether they are live."""
    r = torch.arange(state["case"]["Sq"], device="cuda")[None, None, :, None]
    if state["q_offsets"] is not None:
        r = r + state["q_offsets"].long()[:, None, None, None]
    return r, (r >= 0) & (r < state["seq_lens"].long()[:, None, None, None])


def _plain_kept(state):
    """[B, 1, Sq, Skv] truth values of the kept entries of the sequences' own keys."""
    case = state["case"]
    r, live = _plain_rows(state)
    c = torch.arange(case["Skv"], device="cuda")[None, None, None, :]
    if case["mask"] == 1:
        return live & (c < state["seq_lens"].long()[:, None, None, None])
    kept = live & (c <= r)
    return kept & (c > r - case["window"]) if case["mask"] == 2 else kept


def _plain_shared(state, name):
    """k or v in 32 bits with each head repeated for the query heads that share it."""
    group = state["case"]["Hq"] // state["case"]["Hkv"]
    return state[name].float().repeat_interleave(group, 1)


def _plain_scores(state):
    s = torch.matmul(state["q"].float(), _plain_shared(state, "k").transpose(-1, -2))
    return s.mul_(state["scale"]).masked_fill_(~_plain_kept(state), -math.inf)


def _by_prefix(case, x):
    """[B, Hq, Sq, x] as [G, Hkv, rows of the sequences and heads that share a prefix's head, x]."""
    n, group = case["B"] // case["G"], case["Hq"] // case["Hkv"]
    x = x.reshape(case["G"], n, case["Hkv"], group, case["Sq"], x.shape[-1])
    return x.transpose(1, 2).reshape(case["G"], case["Hkv"], n * group * case["Sq"], x.shape[-1])


def _by_sequence(case, x):
    """The inverse of _by_prefix."""
    n, group = case["B"] // case["G"], case["Hq"] // case["Hkv"]
    x = x.reshape(case["G"], case["Hkv"], n, group, case["Sq"], x.shape[-1])
    return x.transpose(1, 2).reshape(case["B"], case["Hq"], case["Sq"], x.shape[-1])


def _plain_prefix(state):
    """All rows of a prefix in one product with its keys; both parts under one maximum."""
    case = state["case"]
    s = torch.matmul(_by_prefix(case, state["q"].float()), state["k_prefix"].float().transpose(-1, -2)).mul_(state["scale"])
    behind = torch.arange(case["P"], device="cuda") >= state["prefix_lens"].long()[:, None]
    s.masked_fill_(behind[:, None, None, :], -math.inf)
    z = _plain_scores(state)
    top = torch.maximum(_by_sequence(case, s.amax(-1, keepdim=True)), z.amax(-1, keepdim=True))
    _, live = _plain_rows(state)
    top = torch.where(live, top, torch.zeros_like(top))
    e, f = s.sub_(_by_prefix(case, top)).exp_(), z.sub_(top).exp_()
    total = _by_sequence(case, e.sum(-1, keepdim=True)) + f.sum(-1, keepdim=True)
    o = _by_sequence(case, torch.matmul(e, state["v_prefix"].float())) + torch.matmul(f, _plain_shared(state, "v"))
    o = torch.where(live, o / total, torch.zeros_like(o)).to(state["q"].dtype)
    lse = torch.where(live, top + total.log(), torch.full_like(top, -math.inf)).squeeze(-1)
    return {"o": o, "lse": lse}


def _plain_weights(state):
    case = state["case"]
    lse = state["lse"][..., None]
    p = _plain_scores(state).sub_(torch.where(lse == -math.inf, torch.zeros_like(lse), lse)).exp_()
    w = p.sum(2).view(case["B"], case["Hkv"], case["Hq"] // case["Hkv"], case["Skv"]).sum(2)
    if case["accumulate"]:
        state["weights"].add_(w)
    else:
        state["weights"].copy_(w)
    return {"weights": state["weights"]}


def _plain_evict(state):
    case = state["case"]
    S, keep = case["S"], case["keep"]
    n = state["seq_lens"].long()[:, None, None]
    c = torch.arange(S, device="cuda")
    always = (c < case["first"]) | (c >= n - case["recent"])
    w = torch.where(always, torch.full_like(state["weights"], math.inf), state["weights"])
    w = torch.where(c < n, w, torch.full_like(w, -math.inf))
    at = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    lens = state["seq_lens"].clamp(max=keep)
    taken = torch.arange(keep, device="cuda") < lens.long()[:, None, None]
    at = torch.sort(torch.where(taken, at, torch.full_like(at, S)), dim=-1).values.clamp_(max=S - 1)
    k, v, weights, positions = state["out"]
    rows = at[..., None].expand(*at.shape, case["d"])
    k.copy_(torch.where(taken[..., None], torch.gather(state["k"], 2, rows), k))
    v.copy_(torch.where(taken[..., None], torch.gather(state["v"], 2, rows), v))
    weights.copy_(torch.where(taken, torch.gather(state["weights"], 2, at), weights))
    positions.copy_(torch.where(taken, torch.gather(state["positions"], 2, at), positions))
    return {"k": k, "v": v, "weights": weights, "positions": positions, "lens": lens}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return {"prefix": _plain_prefix, "weights": _plain_weights, "evict": _plain_evict}[case["op"]](state)


def _own(state, case):
    import masked_softmax_attention_gb300 as gtms

    if case["op"] == "prefix":
        o, lse = gtms.attention_shared_prefix(state["q"], state["k_prefix"], state["v_prefix"], state["k"], state["v"],
                                              state["seq_lens"], state["scale"], mask_kind=case["mask"],
                                              q_offsets=state["q_offsets"], prefix_lens=state["prefix_lens"])
        return {"o": o, "lse": lse}
    if case["op"] == "weights":
        w = gtms.attention_key_weights(state["q"], state["k"], state["lse"], state["seq_lens"], state["scale"],
                                       out=state["weights"], accumulate=case["accumulate"], mask_kind=case["mask"],
                                       window=case["window"], q_offsets=state["q_offsets"])
        return {"weights": w}
    k, v, weights, positions, lens = gtms.cache_evict(state["k"], state["v"], state["weights"], state["seq_lens"],
                                                      case["keep"], first=case["first"], recent=case["recent"],
                                                      positions=state["positions"], out=state["out"])
    return {"k": k, "v": v, "weights": weights, "positions": positions, "lens": lens}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def _kept_pairs(case):
    """Kept (row, own key) pairs of one query head, live rows of one query head and own keys that some row keeps, of
    all batches."""
    pairs = rows = keys = 0
    for n, off in zip(_lens(case), _offsets(case) or [0] * case["B"]):
        a, b = max(0, off), min(n, off + case["Sq"])   # live positions
        if a >= b:
            continue
        rows += b - a
        if case["mask"] == 1:
            pairs += (b - a) * n
            keys += n
        elif case["mask"] == 0:
            pairs += (a + 1 + b) * (b - a) // 2
            keys += b
        else:
            w = case["window"]
            pairs += sum(min(w, r + 1) for r in range(a, b))
            keys += b - max(0, a - w + 1)
    return pairs, rows, keys


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "evict":
        lens = _lens(case)
        kept = case["H"] * sum(min(n, case["keep"]) for n in lens)
        read = case["H"] * sum(n for n in lens if n > case["keep"]) * 4   # weights that are compared
        return {"bytes": 2 * kept * (2 * case["d"] * e + 8) + read, "flops": 0}
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    pairs, rows, keys = _kept_pairs(case)
    q_in, k_in = rows * Hq * d * e, keys * Hkv * d * e
    if case["op"] == "weights":
        w = case["B"] * Hkv * case["Skv"] * 4 if not case["accumulate"] else 2 * keys * Hkv * 4
        return {"bytes": q_in + rows * Hq * 4 + k_in + w, "flops": 2 * d * pairs * Hq}
    per = [0] * case["G"]
    for b, (n, off) in enumerate(zip(_lens(case), _offsets(case) or [0] * case["B"])):
        per[b // (case["B"] // case["G"])] += max(0, min(n, off + case["Sq"]) - max(0, off))
    shared = _prefix_lens(case)
    pairs += sum(r * p for r, p in zip(per, shared))
    out = case["B"] * Hq * case["Sq"] * (d * e + 4)
    return {"bytes": q_in + 2 * k_in + 2 * sum(shared) * Hkv * d * e + out, "flops": 4 * d * pairs * Hq}


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _exact_own(case, n, off, i0, i1):
    """Own keys [c0, c1) that rows i0 .. i1 - 1 may keep, and which of these entries they do not."""
    pos = torch.arange(off + i0, off + i1, device="cuda")[:, None]
    c0 = max(0, off + i0 - case["window"] + 1) if case["mask"] == 2 else 0
    c1 = n if case["mask"] == 1 else off + i1
    col = torch.arange(c0, c1, device="cuda")[None, :]
    out = torch.zeros((i1 - i0, c1 - c0), dtype=torch.bool, device="cuda")
    if case["mask"] != 1:
        out = col > pos
    if case["mask"] == 2:
        out = out | (col <= pos - case["window"])
    return c0, c1, out


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(state, case)
    q, k = state["q"].double(), state["k"].double()
    prefix = case["op"] == "prefix"
    group, rows = case["Hq"] // case["Hkv"], 1024
    if prefix:
        v, kp, vp = (state[name].double() for name in ("v", "k_prefix", "v_prefix"))
        o, lse = torch.zeros_like(q), torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    else:
        w = torch.zeros(k.shape[:3], dtype=torch.float64, device="cuda")
        if case["accumulate"]:
            w += state["weights"].double()
    for b, (n, off) in enumerate(zip(_lens(case), _offsets(case) or [0] * case["B"])):
        g = b // (case["B"] // case["G"]) if prefix else 0
        for i0 in range(max(0, -off), min(case["Sq"], n - off), rows):
            i1 = min(case["Sq"], n - off, i0 + rows)
            c0, c1, out = _exact_own(case, n, off, i0, i1)
            for hk in range(case["Hkv"]):
                h = slice(hk * group, (hk + 1) * group)
                keys = k[b, hk, c0:c1]
                if prefix:
                    shared = _prefix_lens(case)[g]
                    keys = torch.cat((kp[g, hk, :shared], keys))
                    out_all = torch.cat((torch.zeros((i1 - i0, shared), dtype=torch.bool, device="cuda"), out), 1)
                    z = torch.einsum("hid,cd->hic", q[b, h, i0:i1], keys) * state["scale"]
                    z.masked_fill_(out_all, -math.inf)
                    norm = torch.logsumexp(z, -1)
                    values = torch.cat((vp[g, hk, :shared], v[b, hk, c0:c1]))
                    o[b, h, i0:i1] = torch.einsum("hic,cd->hid", torch.exp(z - norm[..., None]), values)
                    lse[b, h, i0:i1] = norm
                else:
                    z = torch.einsum("hid,cd->hic", q[b, h, i0:i1], keys) * state["scale"]
                    z = torch.exp(z - state["lse"][b, h, i0:i1].double()[..., None]).masked_fill_(out, 0.0)
                    w[b, hk, c0:c1] += z.sum((0, 1))
    return {"o": o, "lse": lse} if prefix else {"weights": w}


def _exact_evict(state, case):
    k, v, weights, _ = (t.double() for t in state["out"])
    for b, n in enumerate(_lens(case)):
        m = min(n, case["keep"])
        a, z = case["first"], n - case["recent"]
        for h in range(case["H"]):
            if n <= case["keep"]:
                at = torch.arange(n, device="cuda")
            else:
                # Ties go to the lowest index: among equals, the one that stands further back comes first here.
                some = state["weights"][b, h, a:z].flip(0)
                best = a + (z - a - 1) - torch.argsort(some, stable=True)[-(m - a - case["recent"]):] \
                    if m > a + case["recent"] else torch.zeros(0, dtype=torch.long, device="cuda")
                at = torch.cat((torch.arange(a, device="cuda"), best.sort().values, torch.arange(z, n, device="cuda")))
            k[b, h, :m], v[b, h, :m] = state["k"][b, h, at].double(), state["v"][b, h, at].double()
            weights[b, h, :m] = state["weights"][b, h, at].double()
    return {"k": k, "v": v, "weights": weights, "positions": None, "lens": None}
