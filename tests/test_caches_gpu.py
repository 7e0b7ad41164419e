"""Attention over shared prefixes, key weights and cache eviction against their definitions (caches_reference.py)."""
import math
import os
import re

import pytest
import torch

import masked_softmax_attention_gb300 as gtms

from attention_reference import forward, kept
from caches_reference import evicted, joined, key_weights
from test_attention_gpu import BF16, F16, F32, LENGTH, TRIL, WINDOW, _close, _heads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    gtms.build_library()
    return torch.device("cuda:0")


def _int32(values):
    return None if values is None else torch.tensor(values, dtype=torch.int32, device="cuda")


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _captured(fn):
    """fn's call once by itself on a side stream, then captured: the graph and what its call returned."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fn()
    return graph, got


def _same_bits(a, b):
    bits = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return a.shape == b.shape and torch.equal(a.contiguous().view(bits), b.contiguous().view(bits))


# ---------------------------------------------------------------------------
# Shared prefixes
# ---------------------------------------------------------------------------

class Shared:
    def __init__(self, G, n, Hq, Hkv, Sq, P, Skv, d, dtype, prefix_lens, lens, offsets=None, mask=TRIL, layout="bhsd",
                 seed=1, scale=None, std=1.0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        B = G * n
        self.q = _heads(gen, B, Hq, Sq, d, dtype, layout, std)
        self.kp, self.vp = (_heads(gen, G, Hkv, P, d, dtype, layout, s) for s in (std, 1.0))
        self.k, self.v = (_heads(gen, B, Hkv, Skv, d, dtype, layout, s) for s in (std, 1.0))
        lens = [lens[b % len(lens)] for b in range(B)]
        self.lens, self.plens = _int32(lens), _int32(prefix_lens)
        self.off = _int32([x - Sq for x in lens] if offsets == "last" else offsets)
        self.scale, self.mask = d ** -0.5 if scale is None else scale, mask

    def __call__(self, **kw):
        return gtms.attention_shared_prefix(self.q, self.kp, self.vp, self.k, self.v, self.lens, self.scale,
                                            mask_kind=self.mask, q_offsets=self.off, prefix_lens=self.plens, **kw)

    def run(self, **kw):
        status = _status()
        o, lse = self(status=status, **kw)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        return o, lse

    def check(self, o, lse):
        ref, ref_lse, tol, tol_lse, live = joined(self.q, self.kp, self.vp, self.k, self.v, self.lens, self.scale,
                                                  self.plens, self.mask, self.off)
        live = live.expand_as(lse)
        _close("o", o, ref, tol)
        assert bool((lse[~live] == -math.inf).all())
        assert bool((o[~live].view(torch.int16) == 0).all()), "rows that keep nothing must be +0.0"
        _close("lse", lse[live], ref_lse[live], tol_lse[live])

    def spoil(self):
        """NaN wherever nothing is kept."""
        live = kept(self.lens, self.q.shape[2], self.k.shape[2], self.mask, 0, self.off).any(-1)[..., None]
        self.q.masked_fill_(~live, math.nan)
        for t, lens in ((self.k, self.lens), (self.v, self.lens), (self.kp, self.plens), (self.vp, self.plens)):
            if lens is not None:
                at = torch.arange(t.shape[2], device="cuda")[None, None, :, None]
                t.masked_fill_(at >= lens.clamp(min=0)[:, None, None, None], math.nan)


# G, n, Hq, Hkv, Sq, P, Skv, d, dtype, prefix_lens, lens, offsets, mask, layout
TOKENS = [
    (1, 1, 1, 1, 1, 1, 1, 64, BF16, None, (1,), "last", TRIL, "bhsd"),
    (1, 4, 4, 2, 1, 127, 9, 64, F16, None, (1, 9, 5, 0), "last", TRIL, "bhsd"),          # a sequence without keys
    (1, 64, 8, 2, 1, 700, 33, 128, BF16, (700,), (33, 1, 20), "last", TRIL, "bhsd"),
    (2, 3, 6, 2, 1, 300, 40, 128, F16, (0, 129), (40, 7), "last", TRIL, "bshd"),         # an empty prefix, three to a head
    (3, 2, 5, 1, 1, 1000, 130, 64, BF16, (1000, 1, 640), (130, 129), "last", LENGTH, "sliced"),
    (1, 100, 4, 1, 1, 257, 3, 128, BF16, (9000,), (3, 2), "last", TRIL, "bhsd"),         # lengths clamped, odd rows
    (2, 2, 4, 4, 1, 500, 64, 64, F16, (-7, 500), (64, 60), "last", TRIL, "bhsd"),
    (4, 1, 16, 2, 1, 385, 50, 128, BF16, (385, 256, 255, 384), (50,), "last", TRIL, "bshd"),
    (1, 24, 12, 4, 5, 1003, 33, 64, F16, None, (33, 5, 17), "last", TRIL, "bshd"),       # drafts
    (1, 7, 14, 2, 3, 640, 200, 128, BF16, (513,), (200, 3), "last", LENGTH, "bhsd"),
    (1, 3, 2, 1, 1, 20000, 17, 64, BF16, (19999,), (17,), "last", TRIL, "bhsd"),
    (1, 2, 128, 1, 2, 200, 12, 64, BF16, None, (12, 2), "last", TRIL, "bhsd"),           # 128 heads to a key
    (1, 2, 4, 2, 1, 0, 9, 128, BF16, None, (9, 4), "last", TRIL, "bhsd"),                # no prefix at all
    (1, 3, 4, 2, 2, 300, 40, 128, F16, None, (40, 40, 40), (38, -1, 41), TRIL, "bhsd"),  # rows before and behind the length
    (64, 2, 8, 8, 1, 300, 20, 128, F16, None, (20, 7), "last", TRIL, "bhsd"),            # more items than multiprocessors
    (48, 3, 16, 16, 1, 700, 20, 64, BF16, None, (20, 7, 0), "last", TRIL, "bshd"),
    (1, 2, 4, 1, 1, 3000, 5000, 128, BF16, None, (5000, 2100), "last", TRIL, "bhsd"),    # few long caches of their own
    (1, 2, 5, 1, 3, 3000, 4500, 64, F16, (2900,), (4500, 3), "last", TRIL, "bshd"),
    (2, 4, 4, 2, 1, 900, 20000, 64, BF16, None, (20000, 7000, 9, 0), "last", TRIL, "bhsd"),
    (1, 33, 2, 1, 1, 3000, 70, 128, BF16, None, (70, 1), "last", LENGTH, "bhsd"),
    # shapes as above at sizes that pack the rows
    (2, 30, 6, 2, 1, 3000, 40, 128, F16, (0, 1299), (40, 7), "last", TRIL, "bshd"),
    (3, 40, 5, 1, 1, 5000, 130, 64, BF16, (5000, 1, 640), (130, 129), "last", LENGTH, "sliced"),
    (4, 16, 16, 2, 1, 3850, 50, 128, BF16, (3850, 2560, 2559, 3841), (50, 0), "last", TRIL, "bshd"),
    (2, 60, 4, 4, 1, 5000, 64, 64, F16, (-7, 5000), (64, 60), "last", TRIL, "bhsd"),
    (1, 64, 12, 4, 5, 5003, 33, 64, F16, None, (33, 5, 17), "last", TRIL, "bshd"),
    (1, 40, 14, 2, 3, 6400, 200, 128, BF16, (5130,), (200, 3), "last", LENGTH, "bhsd"),
    (1, 20, 128, 1, 2, 4000, 12, 64, BF16, None, (12, 2), "last", TRIL, "bhsd"),
    (1, 60, 4, 2, 2, 6000, 40, 128, F16, None, (40,), (38, -1, 41) * 20, TRIL, "bhsd"),
]
PROMPTS = [
    (1, 2, 2, 1, 77, 130, 77, 64, BF16, None, (77, 41), None, TRIL, "bhsd"),
    (2, 2, 4, 2, 300, 513, 300, 128, F16, (513, 200), (300, 0, 129), None, TRIL, "bshd"),
    (1, 3, 6, 2, 128, 128, 128, 128, BF16, None, (128, 127, 1), None, LENGTH, "bhsd"),
    (1, 2, 4, 4, 257, 1000, 600, 64, F16, (999,), (600, 400), "last", TRIL, "sliced"),   # chunks over caches
    (2, 1, 3, 1, 520, 64, 520, 128, BF16, (0, 64), (520, 333), None, TRIL, "bhsd"),
    (1, 4, 8, 2, 40, 2000, 64, 64, BF16, None, (64, 40, 50), "last", TRIL, "bhsd"),
]


@pytest.mark.parametrize("case", TOKENS + PROMPTS, ids=str)
def test_shared_prefix_matches_reference(dev, case):
    c = Shared(*case)
    c.check(*c.run())


@pytest.mark.parametrize("case", TOKENS + PROMPTS, ids=str)
def test_shared_prefix_masked_places_may_hold_anything(dev, case):
    c = Shared(*case)
    want = c.run()
    c.spoil()
    for name, a, b in zip(("o", "lse"), c.run(), want):
        assert torch.equal(a, b), f"{name}: same inputs, same bits, whatever stands in masked places"


@pytest.mark.parametrize("scale,std", [(-0.2, 1.0), (0.0, 1.0), (1.0, 3.0), (0.125, 20.0)])
@pytest.mark.parametrize("case", [TOKENS[2], TOKENS[-6], TOKENS[-3], PROMPTS[1]], ids=str)
def test_shared_prefix_scales_and_steep_rows(dev, case, scale, std):
    c = Shared(*case, scale=scale, std=std)
    c.check(*c.run())


@pytest.mark.parametrize("case", [TOKENS[3], TOKENS[-5], TOKENS[-4], PROMPTS[1]], ids=str)
def test_shared_prefix_is_attention_over_the_keys_end_to_end(dev, case):
    """Beside the framework's own attention, for sequences whose prefix is full: within both calls' roundings."""
    c = Shared(*case[:9], None, *case[10:])
    n, P = case[1], case[5]
    o, lse = c.run()
    k, v = (torch.cat((p.repeat_interleave(n, 0), t), 2) for p, t in ((c.kp, c.k), (c.vp, c.v)))
    off = c.off if c.off is not None else torch.zeros_like(c.lens)
    o2, lse2 = gtms.attention_forward(c.q, k, v, c.lens + P * (c.lens > 0).int(), c.scale, mask_kind=c.mask, q_offsets=off + P)
    _, _, tol, tol_lse, live = joined(c.q, c.kp, c.vp, c.k, c.v, c.lens, c.scale, c.plens, c.mask, c.off)
    live = live.expand_as(lse)
    _close("o", o, o2.double(), 2 * tol)
    _close("lse", lse[live], lse2[live].double(), 2 * tol_lse[live])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P,Skv", [(1, 1), (2, 3), (129, 1), (100, 140)])
def test_shared_prefix_rounds_few_rows_once(dev, d, dtype, P, Skv):
    """Of few rows and keys o is its own rounding: beside half a step of o, (eps / 2)^2 of P's second rounding, below
    2^-16, scores off by at most 2^-16 (d terms of below 8 each, summed to 2^-23 of them, times d^-1/2), exponentials by
    2^-21 and sums of up to 256 terms by 2^-18, together below 2^-14 of sum p |v|. One rounding of P: eps / 2."""
    c = Shared(4, 2, 4, 2, 1, P, Skv, d, dtype, None, (Skv,), "last")
    o, _ = c.run()
    want, size = (joined(c.q, c.kp, vp, c.k, v, c.lens, c.scale, c.plens, c.mask, c.off)[0].double()
                  for vp, v in ((c.vp, c.v), (c.vp.abs(), c.v.abs())))
    half = torch.finfo(dtype).eps / 2
    bound = half * (want.abs() + 2.0 ** -14 * size) + 2.0 ** -14 * size + (2.0 ** -25 if dtype is F16 else 0.0)
    assert bool(((o.double() - want).abs() <= bound).all())


# G, n, Hq, Hkv, Sq, P, Skv ("tile": the rows of an item); whether P is two numbers
SMALL = [
    (4, 2, 4, 2, 1, 100, 140, True),            # 32 items
    (1, 11, 3, 1, 1, 100, 140, False),          # 33
    (1, 4, 8, 2, 1, 800, 96, True),             # 896 keys
    (1, 4, 8, 2, 1, 801, 96, False),            # 897
    (1, 2, 16, 4, "tile", 300, 300, True),      # 32 items of all their rows
    (1, 2, 16, 4, "tile + 1", 300, 300, False),
    (1, 1, 8, 2, 1, 57, 829, False),            # 886 keys, but packed at head dim 128
    (1, 4, 2, 1, 1, 3000, 64, False),           # packed
]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", SMALL, ids=str)
def test_shared_prefix_roundings_on_both_sides_of_their_rule(dev, case, d, dtype):
    """All within the bounds of P's one rounding; where P is two numbers within that of the last test: up to 160 products of
    16 terms cut 2^-23 each, 2^-15.7 in all, sums pass through 43 additions, and scores count twice, in a row's sum too: 2^-14."""
    G, n, Hq, Hkv, Sq, P, Skv, two = case
    Sq = {"tile": 2 * d, "tile + 1": 2 * d + 1}.get(Sq, Sq)
    c = Shared(G, n, Hq, Hkv, Sq, P, Skv, d, dtype, None, (Skv,), "last")
    o, lse = c.run()
    c.check(o, lse)
    if two:
        want, size = (joined(c.q, c.kp, vp, c.k, v, c.lens, c.scale, c.plens, c.mask, c.off)[0].double()
                      for vp, v in ((c.vp, c.v), (c.vp.abs(), c.v.abs())))
        half = torch.finfo(dtype).eps / 2
        bound = half * (want.abs() + 2.0 ** -14 * size) + 2.0 ** -14 * size + (2.0 ** -25 if dtype is F16 else 0.0)
        assert bool(((o.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("P,Skv,Sq", [(0, 0, 1), (300, 0, 1), (5000, 0, 3), (0, 40, 1), (0, 200, 200), (300, 20, 0)])
def test_shared_prefix_without_keys_or_rows(dev, P, Skv, Sq):
    """Without own keys no row is live, whatever the prefix; without a prefix it is attention over the own keys."""
    c = Shared(2, 40, 8, 2, Sq, P, Skv, 64, BF16, None, (Skv,), "last" if Skv != Sq else None)
    o, lse = c.run()
    if Skv == 0 or Sq == 0:
        assert o.shape == c.q.shape and bool((o == 0).all()) and bool((lse == -math.inf).all())
    else:
        o2, lse2 = gtms.attention_forward(c.q, c.k, c.v, c.lens, c.scale, q_offsets=c.off)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_shared_prefix_layouts_of_inputs_and_out(dev):
    """A prefix with one head for all, prefixes inside a fused buffer, an output of other strides."""
    c = Shared(1, 6, 4, 2, 1, 400, 20, 128, BF16, (390,), (20, 11), "last")
    one = c.kp[:, :1].contiguous()
    c.kp = one.expand(1, 2, 400, 128)
    fused = torch.stack((c.kp, c.vp), 3).contiguous()          # [1, 2, 400, 2, 128]
    c.vp = fused[:, :, :, 1]
    out = torch.zeros(6, 1, 4, 128, dtype=BF16, device="cuda").transpose(1, 2)
    o, lse = c.run(out=out)
    assert o.data_ptr() == out.data_ptr()
    c.check(o, lse)


@pytest.mark.parametrize("case", [TOKENS[2], TOKENS[8], TOKENS[-7], PROMPTS[0]], ids=str)
def test_shared_prefix_streams_and_graphs(dev, case):
    """On a side stream, two calls at once, and captured: always the bits of a call by itself."""
    c, e = Shared(*case), Shared(*case, seed=2)
    want, other = c.run(), e.run()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for s, call in zip(side, (c, e)):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(call())
        torch.cuda.synchronize()
        for a, b in zip(got[0] + got[1], want + other):
            assert torch.equal(a, b)
    graph, out = _captured(c)
    for t in out:
        t.zero_()
    c.q.copy_(e.q)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(out[0], want[0])
    c.check(*out)


# ---------------------------------------------------------------------------
# Key weights
# ---------------------------------------------------------------------------

class Weights:
    def __init__(self, B, Hq, Hkv, Sq, Skv, d, dtype, lens, mask=TRIL, window=0, offsets=None, layout="bhsd", seed=1,
                 scale=None, std=1.0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.q, self.k = _heads(gen, B, Hq, Sq, d, dtype, layout, std), _heads(gen, B, Hkv, Skv, d, dtype, layout, std)
        self.lens = _int32(lens)
        self.off = _int32([x - Sq for x in lens] if offsets == "last" else offsets)
        self.scale, self.mask, self.window = d ** -0.5 if scale is None else scale, mask, window
        self.keep = kept(self.lens, Sq, Skv, mask, window, self.off)
        self.lse = gtms.attention_forward(self.q, self.k, self.k, self.lens, self.scale, mask_kind=mask, window=window,
                                          q_offsets=self.off)[1]
        self.before = torch.rand(B, Hkv, Skv, generator=gen, device="cuda")

    def __call__(self, **kw):
        return gtms.attention_key_weights(self.q, self.k, self.lse, self.lens, self.scale, mask_kind=self.mask,
                                          window=self.window, q_offsets=self.off, **kw)

    def run(self, **kw):
        status = _status()
        w = self(status=status, **kw)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        return w

    def check(self, w, before=None):
        ref, tol = key_weights(self.q, self.k, self.lse, self.keep, self.scale)
        used = self.keep.any(-2).expand_as(w)
        if before is None:
            assert bool((w[~used].view(torch.int32) == 0).all()), "keys that no row keeps must be +0.0"
            _close("w", w, ref, tol)
        else:
            assert torch.equal(w[~used], before[~used]), "keys that no row keeps must stay"
            _close("w", w, before.double() + ref, tol + 2.0 ** -24 * (before.double() + ref))

    def spoil(self):
        """NaN wherever nothing is kept."""
        live = self.keep.any(-1)
        self.q.masked_fill_(~live[..., None], math.nan)
        self.lse.masked_fill_(~live.expand_as(self.lse), math.nan)
        at = torch.arange(self.k.shape[2], device="cuda")[None, None, :, None]
        self.k.masked_fill_(at >= self.lens.clamp(min=0)[:, None, None, None], math.nan)


# B, Hq, Hkv, Sq, Skv, d, dtype, lens, mask, window, offsets, layout
KEYS = [
    (1, 1, 1, 1, 1, 64, BF16, (1,), TRIL, 0, None, "bhsd"),
    (3, 4, 1, 1, 1000, 128, F16, (1000, 0, 17), TRIL, 0, "last", "bhsd"),
    (2, 16, 2, 1, 2049, 64, BF16, (2049, 1025), WINDOW, 300, "last", "bshd"),
    (2, 10, 2, 3, 700, 128, BF16, (700, 130), TRIL, 0, "last", "sliced"),
    (2, 6, 2, 11, 500, 64, F16, (500, 11), LENGTH, 0, "last", "bhsd"),
    (1, 8, 2, 32, 3000, 128, BF16, (2900,), TRIL, 0, "last", "bshd"),
    (2, 2, 1, 5, 5, 128, F16, (5, 3), TRIL, 0, None, "bhsd"),
    (3, 4, 2, 77, 77, 64, F16, (77, 0, 41), LENGTH, 0, None, "bshd"),
    (2, 3, 3, 128, 128, 128, BF16, (128, 127), TRIL, 0, None, "bhsd"),
    (2, 2, 2, 129, 129, 64, BF16, (129, 1), TRIL, 0, None, "sliced"),
    (2, 4, 1, 256, 256, 128, F16, (256, 130), LENGTH, 0, None, "bshd"),
    (1, 2, 2, 257, 257, 128, BF16, (257,), WINDOW, 1, None, "bhsd"),
    (2, 4, 2, 333, 333, 64, F16, (333, 200), WINDOW, 100, None, "bshd"),
    (2, 6, 2, 640, 640, 128, BF16, (640, 513), WINDOW, 128, None, "bhsd"),
    (1, 8, 2, 700, 700, 64, BF16, (700,), TRIL, 0, None, "sliced"),
    (1, 5, 1, 1025, 1025, 128, F16, (1025,), TRIL, 0, None, "bshd"),
    (2, 2, 2, 384, 384, 64, BF16, (9000, -4), TRIL, 0, None, "bhsd"),                # lengths clamped
    (2, 2, 2, 300, 300, 128, BF16, (300, 300), WINDOW, 5000, None, "bhsd"),          # a window wider than the rows
    (2, 4, 2, 130, 500, 64, BF16, (500, 213), TRIL, 0, (370, 83), "bhsd"),           # chunks over caches
    (2, 2, 1, 300, 900, 128, F16, (900, 450), WINDOW, 200, (600, 150), "bhsd"),
    (2, 2, 2, 200, 300, 128, BF16, (300, 100), TRIL, 0, (-50, 0), "bhsd"),           # rows before and behind the length
    (1, 140, 1, 3, 400, 64, BF16, (400,), TRIL, 0, "last", "bhsd"),                  # more heads to a key than a tile's rows
    (1, 32, 1, 600, 600, 128, BF16, (600,), TRIL, 0, None, "bhsd"),
    (1, 7, 1, 500, 4000, 64, F16, (4000,), LENGTH, 0, "last", "bshd"),
]


@pytest.mark.parametrize("case", KEYS, ids=str)
def test_key_weights_match_reference(dev, case):
    c = Weights(*case)
    w = c.run()
    c.check(w)
    assert torch.equal(c.run(out=torch.full_like(w, math.nan)), w), "same inputs, same bits, whatever out held"


@pytest.mark.parametrize("case", KEYS, ids=str)
def test_key_weights_accumulate(dev, case):
    c = Weights(*case)
    w = c.run(out=c.before.clone(), accumulate=True)
    c.check(w, c.before)


@pytest.mark.parametrize("case", KEYS, ids=str)
def test_key_weights_accumulate_leaves_places_behind_the_length(dev, case):
    """Bit for bit: a zero keeps its sign and a NaN its payload."""
    c = Weights(*case)
    bits = torch.tensor([-(1 << 31), 0x7fc01234, 0x7f801234, 1], dtype=torch.int32, device="cuda")   # -0, NaNs, the least number
    at = torch.arange(c.before.shape[2], device="cuda")
    behind = at >= c.lens.clamp(min=0)[:, None, None]
    before = torch.where(behind, bits[at % 4], c.before.view(torch.int32))
    w = c.run(out=before.clone().view(torch.float32), accumulate=True)
    assert torch.equal(w.view(torch.int32)[behind.expand_as(w)], before[behind.expand_as(w)])


@pytest.mark.parametrize("case", KEYS, ids=str)
def test_key_weights_masked_places_may_hold_anything(dev, case):
    c = Weights(*case)
    want = c.run()
    c.spoil()
    assert torch.equal(c.run(), want)


@pytest.mark.parametrize("scale,std", [(-0.2, 1.0), (0.0, 1.0), (1.0, 3.0), (0.125, 20.0)])
@pytest.mark.parametrize("case", [KEYS[3], KEYS[15]], ids=str)
def test_key_weights_scales_and_steep_rows(dev, case, scale, std):
    c = Weights(*case, scale=scale, std=std)
    c.check(c.run())


@pytest.mark.parametrize("case", [KEYS[1], KEYS[14]], ids=str)
def test_key_weights_rows_without_a_sum_add_nothing(dev, case):
    c = Weights(*case)
    c.lse[:, ::2] = -math.inf
    c.check(c.run())


@pytest.mark.parametrize("case", [KEYS[5], KEYS[15]], ids=str)
def test_key_weights_nan_stays_where_it_is(dev, case):
    """One in a live key reaches that key alone, one in a live row the keys that it keeps."""
    c = Weights(*case)
    want = c.run()
    c.k[0, 0, 200] = math.nan
    w = c.run()
    assert bool(torch.isnan(w[0, 0, 200])) and int(torch.isnan(w).sum()) == 1
    same = ~torch.isnan(w)
    assert torch.equal(w[same], want[same])
    c = Weights(*case)
    row = c.q.shape[2] // 2
    c.q[0, 0, row] = math.nan
    w = c.run()
    reach = c.keep[0, 0, row]
    assert torch.equal(torch.isnan(w[0, 0]), reach)
    assert torch.equal(w[0, 0][~reach], want[0, 0][~reach])


def test_key_weights_sum_to_the_rows(dev):
    """A row's probabilities sum to one: a head's weights to its live rows, within the bounds of the weights."""
    c = Weights(*KEYS[14])
    w = c.run()
    _, tol = key_weights(c.q, c.k, c.lse, c.keep, c.scale)
    _, _, _, tol_lse = forward(c.q, c.k, c.k, c.keep, c.scale)
    live = c.keep.any(-1).expand_as(c.lse)
    shape = w.shape[0], w.shape[1], -1
    rows = live.reshape(shape).sum(-1).double()
    off = torch.where(live, torch.expm1(tol_lse), 0.0).reshape(shape).sum(-1)   # lse's own error scales its row
    assert bool(((w.double().sum(-1) - rows).abs() <= tol.sum(-1) + off).all())


def test_key_weights_without_rows(dev):
    q, k = torch.zeros(2, 4, 0, 64, dtype=BF16, device="cuda"), torch.zeros(2, 2, 30, 64, dtype=BF16, device="cuda")
    lse = torch.zeros(2, 4, 0, device="cuda")
    out = torch.full((2, 2, 30), 3.0, device="cuda")
    gtms.attention_key_weights(q, k, lse, _int32((30, 5)), out=out, accumulate=True)
    assert bool((out == 3).all())
    gtms.attention_key_weights(q, k, lse, _int32((30, 5)), out=out)
    assert bool((out == 0).all())


@pytest.mark.parametrize("case", [KEYS[1], KEYS[5], KEYS[15], KEYS[13]], ids=str)
def test_key_weights_streams_and_graphs(dev, case):
    """On side streams, two calls at once, and captured: always the bits of a call by itself."""
    c, e = Weights(*case), Weights(*case, seed=2)
    want = c.run(), e.run()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for s, call in zip(side, (c, e)):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(call())
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph, w = _captured(c)
    w.zero_()
    c.q.copy_(e.q)
    c.k.copy_(e.k)
    c.lse.copy_(e.lse)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w, want[1])


class Broadcast(Weights):
    """q with a batch or head stride of 0."""

    def __init__(self, case, batch, heads):
        super().__init__(*case)
        q = self.q[:1] if batch else self.q
        self.q = (q[:, :1] if heads else q).expand(self.q.shape)
        self.lse = gtms.attention_forward(self.q, self.k, self.k, self.lens, self.scale, mask_kind=self.mask,
                                          window=self.window, q_offsets=self.off)[1]


@pytest.mark.parametrize("batch,heads", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("case", [KEYS[i] for i in (3, 4, 7, 8, 10, 13, 18, 19, 20, 21, 23)], ids=str)
def test_key_weights_of_broadcast_rows(dev, case, batch, heads):
    """One q for all batches or heads, of few rows and of many, and added to what stands there."""
    c = Broadcast(case, batch, heads)
    assert (c.q.stride(0) == 0 or c.q.shape[0] == 1 or not batch) and (c.q.stride(1) == 0 or c.q.shape[1] == 1 or not heads)
    w = c.run()
    c.check(w)
    assert torch.equal(c.run(), w)
    c.check(c.run(out=c.before.clone(), accumulate=True), c.before)
    if not heads:
        c.q = c.q.contiguous()
        assert torch.equal(c.run(), w), "the bits of rows of their own"


def test_key_weights_of_broadcast_heads_sum_two_million_rows(dev):
    """128 heads that share one q of zeros, 16384 rows: each of a key's 2^21 terms is p = exp(-lse), the same number, which
    a call of one row gives. Added up one after the other, 32 rows at a time, 32 p = 22.05 is rounded to a multiple of 1/8
    from 2^20 on, by 0.2 % of what it adds. In two steps a sum passes through 7 additions of a tile, those of 128 tiles and
    those of 512 such sums, each off by half a step at most: 647 2^-24 < 2^-14 of it."""
    rows, heads = 1 << 14, 128
    q = torch.zeros(1, 1, rows, 64, dtype=BF16, device="cuda").expand(1, heads, rows, 64)
    k = torch.randn(1, 1, rows, 64, dtype=F32, device="cuda").to(BF16)
    lse = torch.full((1, heads, rows), -math.log(22.05 / 32), device="cuda")
    lens = _int32((rows,))
    w = gtms.attention_key_weights(q, k, lse, lens, 1.0, mask_kind=LENGTH)
    one = gtms.attention_key_weights(q[:, :1, :1].contiguous(), k, lse[:, :1, :1].contiguous(), lens, 1.0, mask_kind=LENGTH)
    p = one[0, 0, 0].double()
    assert abs(float(p) - 22.05 / 32) < 2.0 ** -20 and bool((one == one[0, 0, 0]).all())
    off = (w.double() / (p * rows * heads) - 1).abs().max()
    assert float(off) <= 2.0 ** -14, float(off)


def test_key_weights_beyond_32_bit_offsets(dev):
    """Keys whose elements stand more than 2^32 elements into the cache."""
    B, H, S, d = 1, 2, 1 << 14, 128
    cache = torch.zeros(S * 180000 + 64, 1, dtype=BF16, device="cuda")[:, 0]   # 5.9 GB: rows 180000 elements apart
    k = cache.as_strided((B, H, S, d), (0, 128, 180000, 1))
    gen = torch.Generator(device="cuda").manual_seed(3)
    k.copy_(torch.randn(B, H, S, d, generator=gen, device="cuda"))
    lens = _int32((S,))
    for Sq in (1, 70):
        q = torch.randn(B, 4, Sq, d, generator=gen, device="cuda").to(BF16)
        off = _int32((S - Sq,))
        lse = gtms.attention_forward(q, k.contiguous(), k.contiguous(), lens, d ** -0.5, q_offsets=off)[1]
        a = gtms.attention_key_weights(q, k, lse, lens, d ** -0.5, q_offsets=off)
        b = gtms.attention_key_weights(q, k.contiguous(), lse, lens, d ** -0.5, q_offsets=off)
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# Eviction
# ---------------------------------------------------------------------------

class Cache:
    def __init__(self, B, H, S, d, dtype, lens, keep, first=0, recent=0, layout="bhsd", kind="spread", seed=1, more=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.k, self.v = (_heads(gen, B, H, S, d, dtype, layout) for _ in range(2))
        w = torch.exp(3 * torch.randn(B, H, S, generator=gen, device="cuda"))
        if kind == "ties":
            w = torch.randint(0, 3, (B, H, S), generator=gen, device="cuda").float()
        elif kind == "equal":
            w = torch.full((B, H, S), 0.25, device="cuda")
        elif kind == "special":
            w = torch.randn(B, H, S, generator=gen, device="cuda")
            odd = torch.tensor([math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-45, -1e-45, 3e38], device="cuda")
            pick = torch.randint(0, 24, (B, H, S), generator=gen, device="cuda")
            w = torch.where(pick < 8, odd[pick.clamp(max=7)], w)
        self.weights = w
        self.positions = torch.randint(0, 1 << 30, (B, H, S), generator=gen, device="cuda").to(torch.int32)
        self.lens, self.options = _int32(lens), dict(keep=keep, first=first, recent=recent)
        self.rows = min(keep, S) + more

    def buffers(self, fill=7):
        B, H, S, d = self.k.shape
        return (torch.full((B, H, self.rows, d), fill, dtype=self.k.dtype, device="cuda"),
                torch.full((B, H, self.rows, d), fill, dtype=self.k.dtype, device="cuda"),
                torch.full((B, H, self.rows), float(fill), device="cuda"),
                torch.full((B, H, self.rows), fill, dtype=torch.int32, device="cuda"))

    def call(self, positions=True, **kw):
        return gtms.cache_evict(self.k, self.v, self.weights, self.lens, positions=self.positions if positions else None,
                                **self.options, **kw)

    def check(self, got, before, positions=True):
        """Against the definition: `before` holds what stood in the outputs."""
        *out, lens = got
        B, H, S, d = self.k.shape
        w = self.weights.cpu().tolist()
        ns = [min(max(n, 0), S) for n in self.lens.tolist()]
        assert lens.tolist() == [min(n, self.options["keep"]) for n in ns]
        want = [t.clone() for t in before]
        src = self.k, self.v, self.weights, \
            self.positions if positions else torch.arange(S, device="cuda", dtype=torch.int32).expand(B, H, S)
        for b, n in enumerate(ns):
            for h in range(H):
                at = torch.tensor(evicted(w[b][h], n, **self.options), dtype=torch.long, device="cuda")
                for t, s in zip(want, src):
                    t[b, h, :at.numel()] = s[b, h, at]
        for name, a, b in zip(("k", "v", "weights", "positions"), out, want):
            assert a is None or _same_bits(a, b), name


# B, H, S, d, dtype, lens, keep, first, recent, layout, kind, seed, rows of the outputs beyond keep
CUTS = [
    (1, 1, 1, 64, BF16, (1,), 1, 0, 0, "bhsd", "spread", 1, 0),
    (1, 1, 2, 64, BF16, (2,), 1, 0, 0, "bhsd", "spread", 1, 0),
    (3, 2, 100, 64, F16, (100, 40, 41), 40, 3, 7, "bhsd", "spread", 1, 0),
    (2, 3, 333, 128, BF16, (333, 0), 332, 0, 0, "bshd", "ties", 2, 5),
    (2, 2, 500, 128, F32, (499, 500), 11, 4, 7, "bhsd", "spread", 3, 0),              # the ends alone
    (2, 2, 777, 64, BF16, (777, 600), 300, 1, 0, "sliced", "equal", 4, 1),
    (2, 4, 1000, 128, F16, (1000, 900), 500, 0, 100, "bshd", "special", 5, 0),
    (1, 2, 5000, 64, BF16, (5000,), 1234, 16, 33, "bhsd", "ties", 6, 0),
    (2, 1, 9000, 128, F16, (9000, 8191), 8000, 4, 64, "bhsd", "spread", 7, 0),
    (1, 1, 70001, 64, BF16, (70001,), 20000, 5, 999, "bhsd", "ties", 8, 0),           # a cluster to a row
    (1, 1, 400000, 64, BF16, (399999,), 1000, 5, 99, "bhsd", "spread", 9, 0),         # weights that no CTA holds
    (2, 2, 64, 8, BF16, (64, 50), 20, 2, 2, "bhsd", "spread", 10, 0),                 # rows of 16 bytes
    (2, 2, 64, 24, F32, (64, 50), 20, 2, 2, "bhsd", "spread", 11, 0),                 # of 6 units
    (1, 2, 200, 1024, F32, (200,), 77, 2, 2, "bshd", "spread", 12, 3),
    (2, 2, 64, 64, F16, (9999, -3), 20, 2, 2, "bhsd", "spread", 13, 0),               # lengths clamped
    (2, 2, 64, 64, F16, (64, 10), 100, 20, 80, "bhsd", "spread", 14, 0),              # room for all
    (40, 8, 300, 128, BF16, tuple(range(20, 300, 7)), 150, 4, 32, "bhsd", "spread", 15, 0),
    (1, 8, 3000, 128, BF16, (3000,), 2999, 0, 0, "bhsd", "spread", 16, 0),            # one goes
    (5, 10, 20000, 64, F16, (20000, 16400, 9000, 15000, 19999), 7000, 4, 64, "bhsd", "ties", 17, 0),   # two CTAs to a row
    (2, 8, 33000, 64, BF16, (33000, 20001), 4096, 0, 0, "bshd", "spread", 18, 0),     # eight
    (20, 4, 17000, 8, F32, tuple(range(7000, 17000, 500)), 5000, 1, 1, "bhsd", "ties", 19, 0),         # one, in shared memory
    (1, 1, 140000, 16, F16, (140000,), 131000, 100, 7, "bhsd", "ties", 20, 0),        # a cluster, in shared memory
    (40, 2, 41500, 8, F16, tuple(range(1500, 41500, 1000)), 30000, 5, 99, "bhsd", "spread", 21, 0),    # one, in memory
]


@pytest.mark.parametrize("case", CUTS, ids=str)
def test_evict_matches_definition(dev, case):
    c = Cache(*case)
    before = c.buffers()
    c.check(c.call(out=tuple(t.clone() for t in before)), before)


@pytest.mark.parametrize("case", CUTS, ids=str)
def test_evict_in_place(dev, case):
    c, e = Cache(*case), Cache(*case)
    before = tuple(t.clone() for t in (c.k, c.v, c.weights, c.positions))
    got = e.call(out=(e.k, e.v, e.weights, e.positions))
    assert got[0].data_ptr() == e.k.data_ptr()
    c.check(got, before)


@pytest.mark.parametrize("case", [CUTS[2], CUTS[6], CUTS[16]], ids=str)
def test_evict_some_in_place_some_not(dev, case):
    c, e = Cache(*case), Cache(*case)
    rows = e.k.shape[2]
    v = torch.zeros_like(e.v, memory_format=torch.contiguous_format)
    p = torch.zeros_like(e.positions)
    before = c.k.clone(), v.clone(), c.weights.clone(), p.clone()
    assert rows == v.shape[2]
    c.check(e.call(out=(e.k, v, e.weights, p)), before)


@pytest.mark.parametrize("case", [CUTS[2], CUTS[3], CUTS[14]], ids=str)
def test_evict_new_tensors_and_indices(dev, case):
    c = Cache(*case[:-1], 0)
    c.check(c.call(positions=False), c.buffers(0), positions=False)
    k, v, w, p = c.buffers()
    got = c.call(positions=False, out=(k, v, w, None))
    assert got[3] is None
    c.check(got, c.buffers(), positions=False)


def test_evict_keeps_nothing(dev):
    c = Cache(2, 2, 50, 64, BF16, (50, 0), 0)
    k, v, w, p, lens = c.call()
    assert k.shape[2] == 0 and lens.tolist() == [0, 0]


@pytest.mark.parametrize("case", [CUTS[6], CUTS[9]], ids=str)
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_streams_and_graphs(dev, case, in_place):
    c = Cache(*case)
    want = [t.clone() for t in c.call(out=c.buffers(0))]
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(c.call(out=c.buffers(0)))
    torch.cuda.synchronize()
    for g in got:
        assert all(_same_bits(a, b) for a, b in zip(g, want))
    e = Cache(*case)
    out = (e.k, e.v, e.weights, e.positions) if in_place else e.buffers(0)
    start = [t.clone() for t in (e.k, e.v, e.weights, e.positions)]
    graph, got = _captured(lambda: e.call(out=out))
    for t, s in zip((e.k, e.v, e.weights, e.positions), start):
        t.copy_(s)
    before = tuple(t.clone() for t in out)
    graph.replay()
    torch.cuda.synchronize()
    c.check(got, before)


def test_evict_beyond_32_bit_offsets(dev):
    """In place and elsewhere, rows that stand more than 2^32 bytes and elements into the cache."""
    B, H, S, d = 1, 1, 1 << 14, 64
    c = Cache(B, H, S, d, BF16, (S,), 5000, 3, 100)
    wide = torch.zeros(S * 300000, dtype=BF16, device="cuda")    # 9.8 GB
    k = wide.as_strided((B, H, S, d), (0, 0, 300000, 1))
    k.copy_(c.k)
    want = c.call(out=c.buffers(0))
    got = gtms.cache_evict(k, c.v, c.weights, c.lens, positions=c.positions, out=c.buffers(0), **c.options)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    gtms.cache_evict(k, c.v, c.weights, c.lens, positions=c.positions, out=(k, *(t.clone() for t in (c.v, c.weights, c.positions))),
                     **c.options)
    assert torch.equal(k[:, :, :5000], want[0])


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("d,dtype", [(64, F16), (128, BF16)])
def test_samples_of_a_prompt_with_caches_that_are_cut(dev, d, dtype):
    """Samples of two prompts: their own caches grow by chunks and tokens, collect weights and are cut; every output
    against 64 bits over the entries that stand in the caches."""
    G, n, Hq, Hkv, P, room = 2, 3, 4, 2, 300, 96
    B, gen = G * n, torch.Generator(device="cuda").manual_seed(5)
    scale = d ** -0.5
    kp, vp = (_heads(gen, G, Hkv, P, d, dtype, "bhsd") for _ in range(2))
    plens = _int32((300, 211))
    k, v = (torch.zeros(B, Hkv, room, d, dtype=dtype, device="cuda") for _ in range(2))
    weights = torch.zeros(B, Hkv, room, device="cuda")
    positions = torch.zeros(B, Hkv, room, dtype=torch.int32, device="cuda")
    lens = _int32((0,) * B)
    seen, cuts = 0, 0
    for new in (40, 1, 1, 30, 1, 2, 25, 1, 1, 20, 1):
        if int(lens.max()) + new > room:
            *_, lens = gtms.cache_evict(k, v, weights, lens, 48, first=2, recent=16, positions=positions,
                                        out=(k, v, weights, positions))
            cuts += 1
            assert lens.tolist() == [48] * B
            live = positions[:, :, :48]
            assert bool((live[:, :, 1:] > live[:, :, :-1]).all()) and int(live.max()) == seen - 1
        at = int(lens.max())
        for t in (k, v):
            t[:, :, at:at + new] = _heads(gen, B, Hkv, new, d, dtype, "bhsd")
        weights[:, :, at:at + new] = 0
        positions[:, :, at:at + new] = torch.arange(seen, seen + new, device="cuda", dtype=torch.int32)
        off, lens, seen = lens, lens + new, seen + new
        q = _heads(gen, B, Hq, new, d, dtype, "bhsd")
        o, lse = gtms.attention_shared_prefix(q, kp, vp, k, v, lens, scale, q_offsets=off, prefix_lens=plens)
        ref, ref_lse, tol, tol_lse, _ = joined(q, kp, vp, k, v, lens, scale, plens, TRIL, off)
        _close("o", o, ref, tol)
        _close("lse", lse, ref_lse, tol_lse)
        before = weights.clone()
        gtms.attention_key_weights(q, k, lse, lens, scale, out=weights, accumulate=True, q_offsets=off)
        w, tol = key_weights(q, k, lse, kept(lens, new, room, TRIL, 0, off), scale)
        _close("weights", weights, before.double() + w, tol + 2.0 ** -24 * (before.double() + w))
    assert cuts >= 1


def test_readme_serving_loop(dev):
    """The loop that README.md shows, run as it stands for two cuts."""
    text = open(os.path.join(os.path.dirname(gtms.__file__), "..", "README.md")).read()
    step = next(b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "cache_evict" in b)
    prompts, n, Hq, Hkv, P, d, limit, keep, dtype = 2, 3, 4, 2, 50, 64, 96, 80, BF16
    B, gen, scale = prompts * n, torch.Generator(device="cuda").manual_seed(9), d ** -0.5
    start = torch.tensor((80, 3, 41, 79, 80, 1), device="cuda", dtype=torch.int32)
    k_prompt, v_prompt = (_heads(gen, prompts, Hkv, P, d, dtype, "bhsd") for _ in range(2))
    k, v = (_heads(gen, B, Hkv, limit, d, dtype, "bhsd") for _ in range(2))
    weights = torch.zeros(B, Hkv, limit, device="cuda")
    positions = torch.arange(limit, device="cuda", dtype=torch.int32).expand(B, Hkv, limit).contiguous()
    names = dict(k_prompt=k_prompt, v_prompt=v_prompt, k=k, v=v, weights=weights, positions=positions, scale=scale, limit=limit,
                 keep=keep, lens=start.clone(), steps_since_last_cut=0, rows=torch.arange(B, device="cuda"))
    total = torch.zeros(B, Hkv, 256, dtype=torch.float64, device="cuda")   # by position
    bound = torch.zeros_like(total)
    stood = positions.clone()
    rows, cuts = torch.arange(B, device="cuda"), 0
    for t in range(40):
        names["lens"] = names["lens"] + 1
        names["steps_since_last_cut"] += 1
        names["token"] = start + t               # the new token's position
        slot = (names["lens"] - 1).long()
        k[rows, :, slot], v[rows, :, slot] = (_heads(gen, B, Hkv, 1, d, dtype, "bhsd")[:, :, 0] for _ in range(2))
        stood[rows, :, slot] = names["token"][:, None]
        names["q"] = q = _heads(gen, B, Hq, 1, d, dtype, "bhsd")
        lens, keys = names["lens"], k.clone()
        exec(step, names)
        w, tol = key_weights(q, keys, names["lse"], kept(lens, 1, limit, TRIL, 0, lens - 1), scale)
        at = stood.long()
        live = torch.arange(limit, device="cuda") < lens[:, None, None]
        total.scatter_add_(2, torch.where(live, at, 255), torch.where(live, w, 0.0))
        bound.scatter_add_(2, torch.where(live, at, 255), torch.where(live, tol, 0.0))
        bound += 2.0 ** -24 * total
        if names["lens"] is not lens:
            assert names["lens"].tolist() == [min(x, keep) for x in lens.tolist()]
            names["steps_since_last_cut"] = 0
            cuts += 1
            live = torch.arange(limit, device="cuda") < names["lens"][:, None, None]
            at = positions.long()
            stood = torch.where(live, positions, stood)
        live = live.expand_as(weights)
        at = torch.where(live, at, 255)
        _close("weights", weights[live], total.gather(2, at)[live], bound.gather(2, at)[live])
        assert torch.equal(positions[live], stood[live])
        assert bool((positions[rows, :, (names["lens"] - 1).long()] == names["token"][:, None]).all())
        assert bool(((positions[:, :, 1:] > positions[:, :, :-1]) | ~live[:, :, 1:]).all())
    assert cuts == 2
