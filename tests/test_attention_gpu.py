"""Attention, its backward pass and rotary positions against 64-bit references (attention_reference.py)."""
import math

import pytest
import torch

import masked_softmax_attention_gb300 as gtms

from attention_reference import TINY, UNIT, backward, forward, kept, rotate

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
TRIL, LENGTH, WINDOW = 0, 1, 2


@pytest.fixture(scope="module")
def dev():
    gtms.build_library()
    return torch.device("cuda:0")


def _heads(gen, B, H, S, d, dtype, layout, std=1.0):
    """[B, H, S, d] of N(0, std^2): contiguous ("bhsd"), a [B, S, H, d] view, or a slice of a wider buffer."""
    if layout == "bshd":
        return (torch.randn(B, S, H, d, generator=gen, device="cuda") * std).to(dtype).transpose(1, 2)
    if layout == "sliced":
        t = (torch.randn(B, S + 3, H + 2, d + 8, generator=gen, device="cuda") * std).to(dtype)
        return t[:, 2:S + 2, 1:H + 1, 8:].transpose(1, 2)
    return (torch.randn(B, H, S, d, generator=gen, device="cuda") * std).to(dtype)


class Case:
    def __init__(self, B, Hq, Hkv, Sq, Skv, d, dtype, lens, mask=TRIL, window=0, offsets=None, layout="bhsd", seed=1,
                 scale=None, std=1.0, dstd=1.0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.q = _heads(gen, B, Hq, Sq, d, dtype, layout, std)
        self.k = _heads(gen, B, Hkv, Skv, d, dtype, layout, std)
        self.v = _heads(gen, B, Hkv, Skv, d, dtype, layout)
        self.dout = _heads(gen, B, Hq, Sq, d, dtype, layout, dstd)
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
        self.scale = d ** -0.5 if scale is None else scale
        self.mask, self.window = mask, window
        self.keep = kept(self.lens, Sq, Skv, mask, window, self.off)

    @property
    def options(self):
        return dict(mask_kind=self.mask, window=self.window, q_offsets=self.off)

    def forward(self, **kw):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, lse = gtms.attention_forward(self.q, self.k, self.v, self.lens, self.scale, status=status, **self.options, **kw)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        return o, lse

    def backward(self, o, lse, **kw):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = gtms.attention_backward(self.q, self.k, self.v, o, lse, self.dout, self.lens, self.scale, status=status,
                                      **self.options, **kw)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        return got

    def check_forward(self, o, lse):
        ref, ref_lse, tol, tol_lse = forward(self.q, self.k, self.v, self.keep, self.scale)
        _close("o", o, ref, tol)
        dead = ~self.keep.any(-1).expand_as(lse)
        assert bool((lse[dead] == -math.inf).all())
        assert bool((o[dead].view(torch.int16) == 0).all()), "rows that keep nothing must be +0.0"
        _close("lse", lse[~dead], ref_lse[~dead], tol_lse[~dead])
        return ref, ref_lse

    def check_backward(self, got):
        refs, tols = backward(self.q, self.k, self.v, self.dout, self.keep, self.scale)
        for name, g, r, t in zip(("dq", "dk", "dv"), got, refs, tols):
            _close(name, g, r, t)
        rows = self.keep.any(-1)[..., None].expand_as(got[0])
        cols = self.keep.any(-2)[..., None].expand_as(got[1])
        for g, live in zip(got, (rows, cols, cols)):
            assert bool((g[~live].view(torch.int16) == 0).all()), "gradients of unused rows must be +0.0"

    def spoil(self):
        """NaN wherever nothing is kept."""
        rows, cols = self.keep.any(-1)[..., None], self.keep.any(-2)[..., None]
        beyond = torch.arange(self.k.shape[2], device="cuda")[None, None, :, None] >= self.lens.clamp(min=0)[:, None, None, None]
        for t, dead in ((self.q, ~rows), (self.dout, ~rows), (self.k, beyond), (self.v, beyond)):
            t.masked_fill_(dead.expand_as(t), math.nan)


def _close(name, got, ref, tol):
    assert got.shape == ref.shape
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    if bool(bad.any()):
        i = int(torch.argmax(torch.where(bad, torch.nan_to_num(err / tol, nan=math.inf), torch.zeros_like(err))))
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} out of tolerance; at {i}: got "
                             f"{float(got.reshape(-1)[i])}, want {float(ref.reshape(-1)[i])} +- {float(tol.reshape(-1)[i])}")


# B, Hq, Hkv, Sq, Skv, d, dtype, lens, mask, window, offsets, layout
SHAPES = [
    (1, 1, 1, 1, 1, 64, BF16, (1,), TRIL, 0, None, "bhsd"),
    (2, 2, 1, 5, 5, 128, F16, (5, 3), TRIL, 0, None, "bhsd"),
    (3, 4, 2, 77, 77, 64, F16, (77, 0, 41), LENGTH, 0, None, "bshd"),
    (2, 3, 3, 128, 128, 128, BF16, (128, 127), TRIL, 0, None, "bhsd"),
    (2, 2, 2, 129, 129, 64, BF16, (129, 1), TRIL, 0, None, "sliced"),
    (2, 4, 1, 256, 256, 128, F16, (256, 130), LENGTH, 0, None, "bshd"),
    (1, 2, 2, 257, 257, 128, BF16, (257,), WINDOW, 1, None, "bhsd"),
    (2, 4, 2, 333, 333, 64, F16, (333, 200), WINDOW, 100, None, "bshd"),
    (2, 2, 1, 640, 640, 128, BF16, (640, 513), WINDOW, 128, None, "bhsd"),
    (1, 8, 2, 700, 700, 64, BF16, (700,), TRIL, 0, None, "sliced"),
    (1, 3, 1, 1025, 1025, 128, F16, (1025,), TRIL, 0, None, "bshd"),
    (2, 2, 2, 384, 384, 64, BF16, (9000, -4), TRIL, 0, None, "bhsd"),                # lengths clamped
    (2, 2, 2, 300, 300, 128, BF16, (300, 300), WINDOW, 5000, None, "bhsd"),          # a window wider than the rows
    # rows at offsets: chunks of a sequence over its cache, rows before and behind the live length
    (2, 4, 2, 130, 500, 64, BF16, (500, 213), TRIL, 0, (370, 83), "bshd"),
    (2, 2, 1, 300, 900, 128, F16, (900, 450), WINDOW, 200, (600, 150), "bhsd"),
    (2, 2, 2, 200, 300, 128, BF16, (300, 100), TRIL, 0, (-50, 0), "bhsd"),
    (2, 2, 2, 140, 260, 64, F16, (200, 260), LENGTH, 0, (100, -3), "sliced"),
    (2, 2, 2, 64, 100, 64, BF16, (100, 90), TRIL, 0, (2 ** 31 - 1, -2 ** 31), "bhsd"),  # no row is alive
    (1, 2, 1, 400, 150, 64, BF16, (150,), TRIL, 0, None, "bhsd"),                    # more rows than keys
]
# new tokens over a cache: few rows, many keys
TOKENS = [
    (3, 4, 4, 1, 700, 64, BF16, (700, 1, 0), TRIL, 0, (699, 0, -1), "bhsd"),
    (2, 8, 2, 1, 1025, 128, F16, (1025, 64), TRIL, 0, (1024, 63), "bshd"),
    (2, 16, 1, 1, 2000, 128, BF16, (2000, 999), WINDOW, 300, (1999, 998), "bhsd"),
    (1, 32, 2, 1, 4097, 64, F16, (4097,), LENGTH, 0, (4096,), "sliced"),
    (2, 4, 1, 3, 515, 128, BF16, (515, 2), TRIL, 0, (512, -1), "bshd"),
    (2, 6, 2, 7, 1300, 64, F16, (1300, 640), WINDOW, 64, (1293, 633), "bhsd"),
    (1, 2, 2, 1, 20000, 128, BF16, (19999,), TRIL, 0, (19998,), "bhsd"),
    (5, 2, 1, 1, 1, 64, BF16, (1, 1, 0, 1, 1), TRIL, 0, None, "bhsd"),
    (1, 64, 1, 2, 300, 128, F16, (300,), TRIL, 0, (298,), "bhsd"),
    (1, 8, 1, 16, 5000, 128, BF16, (5000,), TRIL, 0, (4984,), "bshd"),
    # several tiles of 16 packed rows share the keys of a key/value head
    (1, 8, 2, 9, 3000, 64, F16, (2990,), TRIL, 0, (2981,), "bhsd"),
    (2, 12, 1, 5, 4001, 128, BF16, (4001, 7), WINDOW, 700, (3996, 2), "sliced"),
    (3, 4, 4, 33, 2500, 64, BF16, (2500, 33, 1200), LENGTH, 0, (2467, 0, 1167), "bshd"),
    # few key/value heads over many keys: clusters of more than eight
    (1, 8, 8, 1, 4500, 128, F16, (4499,), TRIL, 0, (4498,), "bshd"),
    (7, 2, 1, 1, 4700, 64, BF16, (4700, 0, 9, 4096, 1, 3000, 193), TRIL, 0, (4699, -1, 8, 4095, 0, 2999, 192), "bhsd"),
    (4, 4, 1, 2, 9000, 128, BF16, (9000, 5, 4095, 6000), WINDOW, 5000, (8998, 3, 4093, 5998), "sliced"),
    (1, 3, 1, 4, 16000, 64, F16, (15990,), LENGTH, 0, (15986,), "bhsd"),
    (11, 2, 1, 1, 4100, 128, BF16, tuple(range(4100, 0, -400)), TRIL, 0, tuple(range(4099, -1, -400)), "bhsd"),
    (3, 5, 5, 1, 600, 64, BF16, (600, 0, 111), LENGTH, 0, (599, 0, 110), "bshd"),
    (20, 2, 1, 1, 4200, 64, BF16, tuple(range(200, 4201, 210))[:20], WINDOW, 4150, tuple(range(199, 4200, 210))[:20], "bshd"),
    (15, 8, 4, 1, 2100, 64, F16, tuple(range(140, 2101, 140)), TRIL, 0, tuple(range(139, 2100, 140)), "bhsd"),
    (40, 4, 2, 1, 2100, 128, BF16, tuple(range(2100, 0, -53))[:40], TRIL, 0, tuple(range(2099, -1, -53))[:40], "bhsd"),
    # many rows, but few key/value heads and many keys
    (1, 4, 1, 150, 4000, 64, F16, (3990,), TRIL, 0, (3840,), "sliced"),
    (2, 2, 1, 300, 3500, 128, BF16, (3500, 2100), WINDOW, 2000, (3200, 1800), "bhsd"),
    (1, 1, 1, 700, 6000, 128, F16, (5999,), LENGTH, 0, (5299,), "bshd"),
    # more CTAs than run at once: sequences are taken by length, ties and empty ones among them
    (70, 8, 8, 1, 600, 64, BF16, tuple((97 * b) % 601 // 3 * 3 for b in range(70)), TRIL, 0,
     tuple((97 * b) % 601 // 3 * 3 - 1 for b in range(70)), "bshd"),
    (256, 2, 2, 1, 140, 128, F16, tuple(b % 140 for b in range(256)), LENGTH, 0, (0,) * 256, "bhsd"),
    (257, 4, 2, 2, 90, 64, BF16, tuple(90 - b % 70 for b in range(257)), WINDOW, 40, tuple(88 - b % 70 for b in range(257)), "bhsd"),
    (60, 1, 1, 1, 300, 128, F16, tuple(range(1, 301, 5)), TRIL, 0, tuple(range(0, 300, 5)), "bhsd"),
]
# longer sequences: many tiles to an item, many items to a multiprocessor
LONG = [
    (1, 4, 2, 2300, 2300, 128, BF16, (2190,), TRIL, 0, None, "bshd"),
    (1, 4, 1, 2300, 2300, 64, F16, (2300,), TRIL, 0, None, "bhsd"),
    (1, 2, 2, 2500, 2500, 64, BF16, (2500,), WINDOW, 300, None, "bshd"),
    (1, 2, 1, 2500, 2500, 128, F16, (2431,), LENGTH, 0, None, "bhsd"),
    (6, 16, 4, 300, 900, 128, F16, (900, 450, 301, 0, 777, 899), WINDOW, 200, (600, 150, 1, -300, 477, 599), "bshd"),
    (4, 16, 4, 260, 700, 64, BF16, (700, 261, 260, 500), TRIL, 0, (440, 1, 0, 240), "sliced"),
    (60, 16, 8, 20, 20, 64, BF16, tuple(1 + (7 * b) % 20 for b in range(60)), TRIL, 0, None, "bhsd"),
    (60, 16, 8, 150, 150, 128, F16, tuple((37 * b) % 151 for b in range(60)), TRIL, 0, None, "bshd"),
]


@pytest.mark.parametrize("case", SHAPES + TOKENS + LONG, ids=str)
def test_forward_matches_reference(dev, case):
    c = Case(*case)
    c.check_forward(*c.forward())


@pytest.mark.parametrize("case", SHAPES + TOKENS[:5] + LONG, ids=str)
def test_backward_matches_reference(dev, case):
    c = Case(*case, dstd=0.01)
    ref, ref_lse, _, _ = forward(c.q, c.k, c.v, c.keep, c.scale)
    c.check_backward(c.backward(ref.to(c.q.dtype), ref_lse.float()))


@pytest.mark.parametrize("case", [SHAPES[2], SHAPES[4], SHAPES[7], SHAPES[9], SHAPES[15], TOKENS[1], TOKENS[4]], ids=str)
def test_masked_places_may_hold_anything(dev, case):
    c = Case(*case)
    c.spoil()
    o, lse = c.forward()
    c.check_forward(o, lse)
    dead = ~c.keep.any(-1).expand_as(lse)
    o, lse = o.masked_fill(dead[..., None], math.nan), lse.masked_fill(dead, math.nan)
    c.check_backward(c.backward(o, lse))


@pytest.mark.parametrize("d,Sq,window,mask", [(64, 900, 40, WINDOW), (128, 900, 40, WINDOW), (128, 900, 0, TRIL),
                                              (64, 24, 9, WINDOW)])
def test_how_far_a_live_nan_reaches(dev, d, Sq, window, mask):
    """One in v: the rows that keep it, and at most those within 127 rows of one that keeps a key of its tile. One in
    k: the rows that keep it alone."""
    Skv, at = 900, 880 if Sq < 900 else 300
    c = Case(1, 2, 1, Sq, Skv, d, BF16, (Skv,), mask, window, (Skv - Sq,), "bhsd", seed=17)
    clean, _ = c.forward()
    keeps = c.keep.any(1)[0]                                                   # [Sq, Skv]
    near = keeps[:, at // 128 * 128:at // 128 * 128 + 128].any(1).nonzero()
    row = torch.arange(Sq, device="cuda")
    far = (row < near.min() - 127) | (row > near.max() + 127)
    for t, safe in ((c.v, far), (c.k, ~keeps[:, at])):
        old = t[:, :, at].clone()
        t[:, :, at] = math.nan
        o, _ = c.forward()
        t[:, :, at] = old
        assert bool(torch.isnan(o[:, :, keeps[:, at]]).all())
        assert bool(torch.isfinite(o[:, :, safe]).all())
        if t is c.v:                                                           # the scores are the same, and so are the bits
            assert torch.equal(o[:, :, safe], clean[:, :, safe])


@pytest.mark.parametrize("scale,std", [(-0.2, 1.0), (0.0, 1.0), (1.0, 3.0), (0.125, 20.0)])
def test_scales_and_steep_rows(dev, scale, std):
    c = Case(2, 2, 1, 300, 300, 64, BF16, (300, 211), scale=scale, std=std, seed=5)
    o, lse = c.forward()
    c.check_forward(o, lse)
    c.check_backward(c.backward(o, lse))


def test_scores_of_the_lowest_value(dev):
    """Rows whose every score is hugely negative still normalise to one."""
    c = Case(1, 2, 2, 200, 200, 64, BF16, (200,), scale=1.0)
    c.q.fill_(1000.0)
    c.k.fill_(-1000.0)
    c.k[:, :, ::3] = -999.0 * 1.0
    o, lse = c.forward()
    c.check_forward(o, lse)


@pytest.mark.parametrize("small", [1e-4, 1e-6])
def test_fp16_gradients_of_small_dout(dev, small):
    """ds far below fp16's range keeps its bits: dout of 1e-6 gives gradients as exact as dout of 1."""
    c = Case(1, 4, 2, 700, 700, 128, F16, (650,), seed=9, dstd=1.0)
    one = c.backward(*c.forward())
    c.dout = (c.dout.float() * 2.0 ** round(math.log2(small))).to(F16)
    o, lse = c.forward()
    c.check_backward(c.backward(o, lse))
    assert bool(torch.isfinite(one[0]).all())


@pytest.mark.parametrize("case", [SHAPES[5], SHAPES[9], TOKENS[3]], ids=str)
def test_same_inputs_same_bits(dev, case):
    c = Case(*case)
    o, lse = c.forward()
    first = c.backward(o, lse)
    for _ in range(3):
        o2, lse2 = c.forward()
        assert torch.equal(o2, o) and torch.equal(lse2, lse)
        for a, b in zip(first, c.backward(o, lse)):
            assert torch.equal(a, b)


def test_outputs_inside_one_fused_buffer(dev):
    """q, k, v and their gradients as parts of fused [B, S, (Hq + 2 Hkv) d] buffers; nothing else is written."""
    B, S, Hq, Hkv, d = 2, 301, 4, 2, 64
    H = Hq + 2 * Hkv

    def parts(t):
        t = t.view(B, S, H, d).transpose(1, 2)
        return t[:, :Hq], t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:]

    c = Case(B, Hq, Hkv, S, S, d, BF16, (301, 190))
    qkv = torch.randn(B, S, H * d, device=dev).to(BF16)
    c.q, c.k, c.v = parts(qkv)
    o, lse = c.forward()
    c.check_forward(o, lse)
    grads = torch.full((B, S + 1, H * d + 16), 7.0, dtype=BF16, device=dev)
    whole = grads[:, :S, 8:-8]
    out = tuple(whole[..., a * d:b * d].unflatten(-1, (b - a, d)).transpose(1, 2)
                for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, H)))
    c.check_backward(c.backward(o, lse, out=out))
    assert bool((grads[:, S:] == 7.0).all() & (grads[:, :, :8] == 7.0).all() & (grads[:, :, -8:] == 7.0).all())


def test_shared_and_broadcast_inputs(dev):
    """k and v expanded over batches and heads are read in place; autograd sums their gradients."""
    c = Case(3, 4, 4, 150, 150, 64, BF16, (150, 90, 12))
    k1, v1 = c.k[:1, :1].clone(), c.v[:1, :1].clone()
    c.k, c.v = k1.expand(3, 4, -1, -1), v1.expand(3, 4, -1, -1)
    o, lse = c.forward()
    c.check_forward(o, lse)
    refs, tols = backward(c.q, c.k, c.v, c.dout, c.keep, c.scale)
    leaf_k, leaf_v = k1.clone().requires_grad_(), v1.clone().requires_grad_()
    y = gtms.attention(c.q, leaf_k.expand(3, 4, -1, -1), leaf_v.expand(3, 4, -1, -1), c.lens, c.scale)
    y.backward(c.dout)
    for leaf, ref, tol in ((leaf_k, refs[1], tols[1]), (leaf_v, refs[2], tols[2])):
        total = ref.sum((0, 1), keepdim=True)
        # autograd sums the 12 rounded gradients in 16 bits: a rounding of every partial sum, each at
        # most the sum of the absolute values
        tol = tol.sum((0, 1), keepdim=True) + 12 * UNIT[BF16] * ref.abs().sum((0, 1), keepdim=True)
        _close("broadcast", leaf.grad, total, tol)


def _odd_gradients(dev, t):
    """Gradients of t's shape as autograd may hand them over: expanded, transposed, at an odd address, every other one."""
    B, H, S, d = t.shape
    rand = lambda *s: torch.randn(*s, device=dev).to(t.dtype)  # noqa: E731
    return (torch.ones((), dtype=t.dtype, device=dev).expand(t.shape), rand(1, 1, S, d).expand(t.shape),
            rand(B, H, 1, d).expand(t.shape), rand(B, H, d, S).transpose(2, 3),
            rand(B * H * S * d + 1)[1:].view(t.shape), rand(B, H, S, d + 4)[..., 4:], rand(B, H, S, 2 * d)[..., ::2])


def test_output_gradients_of_any_layout(dev):
    """autograd hands the backward expanded, transposed and sliced gradients: as good as contiguous ones."""
    c = Case(2, 4, 2, 70, 70, 64, BF16, (70, 41))
    f = gtms.rotary_frequencies(64, device=dev)
    pos = torch.arange(70, dtype=torch.int32, device=dev)
    leaves = [t.clone().requires_grad_() for t in (c.q, c.k, c.v)]
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    y = gtms.attention(*leaves, c.lens, c.scale, status=status)
    z = gtms.rotary(leaves[0], pos, f)
    y.sum().backward(retain_graph=True)
    first = [t.grad for t in leaves]
    for i, dy in enumerate(_odd_gradients(dev, y)):
        c.dout = dy.clone(memory_format=torch.contiguous_format)
        want = c.backward(*c.forward())
        got = torch.autograd.grad(y, leaves, dy, retain_graph=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        if i == 0:
            assert all(torch.equal(a, b) for a, b in zip(got, first))
        dx, = torch.autograd.grad(z, leaves[:1], dy, retain_graph=True)
        assert torch.equal(dx, gtms.rotary_backward(c.dout, pos, f))
    assert int(status) == 0


def test_gradients_against_differences(dev):
    """<dq, t> + <dk, t'> + <dv, t''> against central differences of the 64-bit forward pass."""
    c = Case(2, 4, 2, 90, 90, 64, BF16, (90, 55), mask=WINDOW, window=40)
    o, lse = c.forward()
    got = c.backward(o, lse)
    _, tols = backward(c.q, c.k, c.v, c.dout, c.keep, c.scale)
    gen = torch.Generator(device="cuda").manual_seed(3)
    steps = [torch.randn(t.shape, generator=gen, device="cuda").double() for t in (c.q, c.k, c.v)]
    rows, cols = c.keep.any(-1)[..., None], c.keep.any(-2)[..., None]

    def loss(h):
        q, k, v = (t.double() + h * s for t, s in zip((c.q, c.k, c.v), steps))
        s = torch.einsum("bhid,bhcd->bhic", q, k.repeat_interleave(2, 1)) * c.scale
        p = torch.softmax(torch.where(c.keep, s, -1e300), -1) * rows
        return (torch.einsum("bhic,bhcd->bhid", p, v.repeat_interleave(2, 1)) * c.dout.double()).sum()

    h = 1e-4
    want = (loss(h) - loss(-h)) / (2 * h)
    have = sum((g.double() * s).sum() for g, s in zip(got, steps))
    tol = sum((t * s.abs()).sum() for t, s in zip(tols, steps))
    assert abs(float(have - want)) <= float(tol) + 1e-5 * abs(float(want))
    assert bool(cols.any())


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_gradients_along_themselves(dev, dtype):
    """Each gradient g against a central difference of the 64-bit forward pass along g / |g|, which is |g|: the kernel's
    may be off by what its elements' bounds add up to along that step (2 to 5 % of |g| in bf16), so a zero gradient, one
    of the wrong sign or one without the term D is told from the right one."""
    c = Case(2, 4, 2, 90, 90, 64, dtype, (90, 55), mask=WINDOW, window=40)
    got = c.backward(*c.forward())
    refs, tols = backward(c.q, c.k, c.v, c.dout, c.keep, c.scale)
    rows = c.keep.any(-1)[..., None]

    def loss(q, k, v):
        s = torch.einsum("bhid,bhcd->bhic", q, k.repeat_interleave(2, 1)) * c.scale
        p = torch.softmax(torch.where(c.keep, s, -1e300), -1) * rows
        return float((torch.einsum("bhic,bhcd->bhid", p, v.repeat_interleave(2, 1)) * c.dout.double()).sum())

    for i, (g, ref, tol) in enumerate(zip(got, refs, tols)):
        step, h, ends = ref / ref.norm(), 1e-3, []
        for side in (h, -h):
            x = [t.double() for t in (c.q, c.k, c.v)]
            x[i] = x[i] + side * step
            ends.append(loss(*x))
        want = (ends[0] - ends[1]) / (2 * h)
        # the difference is off by h^2 / 6 times the third derivative, some 2e-10 of |g|, and by 1e-13 / h of the loss
        bound = float((tol * step.abs()).sum()) + 1e-6 * want
        assert bound <= 0.1 * want
        assert abs(float((g.double() * step).sum()) - want) <= bound


def test_on_a_side_stream(dev):
    c = Case(*SHAPES[9])
    want = c.forward()
    grads = c.backward(*want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o, lse = gtms.attention_forward(c.q, c.k, c.v, c.lens, c.scale, **c.options)
        got = gtms.attention_backward(c.q, c.k, c.v, o, lse, c.dout, c.lens, c.scale, **c.options)
    s.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert all(torch.equal(a, b) for a, b in zip(got, grads))


@pytest.mark.parametrize("d,dtype", [(64, F16), (128, BF16)])
def test_calls_one_after_the_other(dev, d, dtype):
    """The launches of a call overlap (few long items of dk and dv beside many short ones of dq), but what follows in
    the stream, the next call in the same memory too, stands behind all of them."""
    cases = [Case(1, 8, 1, S, S, d, dtype, (n,), TRIL, 0, None, "bhsd", seed=s) for s, (S, n) in
             enumerate([(1500, 1500), (1200, 1100), (900, 900)], 30)]
    first = []
    for c in cases:
        o, lse = c.forward()
        first.append((o, lse, [t.clone() for t in c.backward(o, lse)]))
    out = [torch.empty_like(t) for t in (cases[0].q, cases[0].k, cases[0].v)]
    for _ in range(6):
        seen = []
        for c, (o, lse, _g) in zip(cases, first):
            views = tuple(b.view(-1)[:t.numel()].view(t.shape) for b, t in zip(out, (c.q, c.k, c.v)))
            gtms.attention_backward(c.q, c.k, c.v, o, lse, c.dout, c.lens, c.scale, out=views, **c.options)
            seen.append([t.clone() for t in views])
        for got, (_o, _l, want) in zip(seen, first):
            for g, w in zip(got, want):
                assert torch.equal(g, w)


def test_calls_at_the_same_time(dev):
    """Calls on several streams at once, each with its own tensors, give what they give alone."""
    cases = [Case(*s, seed=i) for i, s in enumerate((SHAPES[9], SHAPES[7], SHAPES[8], TOKENS[1], LONG[0], LONG[1]))]
    want = []
    for c in cases:
        o, lse = c.forward()
        want.append((o, lse, *c.backward(o, lse)))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[] for _ in cases]
    for _ in range(5):
        for c, s, g in zip(cases, streams, got):
            with torch.cuda.stream(s):
                o, lse = gtms.attention_forward(c.q, c.k, c.v, c.lens, c.scale, **c.options)
                g.append((o, lse, *gtms.attention_backward(c.q, c.k, c.v, o, lse, c.dout, c.lens, c.scale, **c.options)))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for one in g:
            assert all(torch.equal(a, b) for a, b in zip(one, w))


_FIRST_CALL = """
import sys; sys.path.insert(0, {root!r})
import torch
import masked_softmax_attention_gb300 as gtms
q = torch.randn(1, 4, 200, 64, device="cuda").to(torch.bfloat16)
lens = torch.tensor([200], dtype=torch.int32, device="cuda")
pos = torch.arange(200, dtype=torch.int32, device="cuda")
f = gtms.rotary_frequencies(64, device="cuda")
def step():
    x, y = gtms.rotary_forward(q, pos, f, other=q)
    o, lse = gtms.attention_forward(x, y, q, lens, 0.125)
    return o, *gtms.attention_backward(x, y, q, o, lse, o, lens, 0.125)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step()))
print("same")
"""


def test_first_calls_of_a_process_may_be_captured(dev):
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", _FIRST_CALL.format(root=root)], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "same" in res.stdout, res.stderr[-2000:]


@pytest.mark.parametrize("case", [SHAPES[9], TOKENS[1]], ids=str)
def test_captured_and_replayed(dev, case):
    """Two graphs of the same calls, replayed after the inputs changed, give what eager calls give."""
    c = Case(*case)
    c.backward(*c.forward())
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, lse = gtms.attention_forward(c.q, c.k, c.v, c.lens, c.scale, **c.options)
            grads = gtms.attention_backward(c.q, c.k, c.v, o, lse, c.dout, c.lens, c.scale, **c.options)
        graphs.append((g, (o, lse, *grads)))
    for turn in range(2):
        c.q.copy_(c.q.flip(-1))
        c.lens.sub_(turn)
        if c.off is not None:
            c.off.sub_(turn)
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        o, lse = c.forward()
        want = (o, lse, *c.backward(o, lse))
        for _, got in graphs:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_rows_or_no_keys(dev):
    lens = torch.tensor([4, 0], dtype=torch.int32, device=dev)
    z = lambda *s: torch.zeros(s, dtype=BF16, device=dev)  # noqa: E731
    o, lse = gtms.attention_forward(z(2, 2, 3, 64).fill_(1), z(2, 2, 0, 64), z(2, 2, 0, 64), lens)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    got = gtms.attention_backward(z(2, 2, 3, 64).fill_(1), z(2, 2, 0, 64), z(2, 2, 0, 64), o, lse, o, lens)
    assert bool((got[0] == 0).all()) and got[1].numel() == 0
    q = z(2, 2, 0, 64)
    o, lse = gtms.attention_forward(q, z(2, 2, 5, 64), z(2, 2, 5, 64), lens)
    got = gtms.attention_backward(q, z(2, 2, 5, 64), z(2, 2, 5, 64), o, lse, q, lens, out=(
        q.clone(), z(2, 2, 5, 64).fill_(3), z(2, 2, 5, 64).fill_(3)))
    torch.cuda.synchronize()
    assert bool((got[1] == 0).all()) and bool((got[2] == 0).all())
    assert gtms.attention_forward(z(0, 2, 3, 64), z(0, 2, 3, 64), z(0, 2, 3, 64), lens[:0])[0].numel() == 0


@pytest.mark.parametrize("B,Hkv,d,window", [(16, 8, 128, 256), (9, 16, 64, 100)])
def test_capacity_behind_a_window_does_not_matter(dev, B, Hkv, d, window):
    """Work under a sliding window is shared out by the keys in it: with many heads, a token over a long cache takes the
    same launch, and gives the same bits, as over one that is hardly longer than the window."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    n = 500
    q = torch.randn(B, 2 * Hkv, 1, d, generator=gen, device=dev).to(BF16)
    k, v = (torch.randn(B, Hkv, n, d, generator=gen, device=dev).to(BF16) for _ in range(2))
    lens = n - torch.arange(B, dtype=torch.int32, device=dev)
    got = []
    for capacity in (n, 9000):
        ck, cv = (torch.full((B, Hkv, capacity, d), math.nan, dtype=BF16, device=dev) for _ in range(2))
        ck[:, :, :n], cv[:, :, :n] = k, v
        got.append(gtms.attention_forward(q, ck, cv, lens, d ** -0.5, mask_kind=WINDOW, window=window, q_offsets=lens - 1))
    ref, ref_lse, tol, tol_lse = forward(q, k, v, kept(lens, 1, n, WINDOW, window, lens - 1), d ** -0.5)
    for o, lse in got:
        _close("o", o, ref, tol)
        _close("lse", lse, ref_lse, tol_lse)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_cache_beyond_32_bit_offsets(dev):
    """The second sequence of a [2, 16, 2^20, 128] cache stands more than 2^31 elements in."""
    B, Hkv, S, d, L = 2, 16, 1 << 20, 128, 70001
    k = torch.empty(B, Hkv, S, d, dtype=BF16, device=dev)
    v = torch.empty(B, Hkv, S, d, dtype=BF16, device=dev)
    gen = torch.Generator(device="cuda").manual_seed(4)
    k[1, :, :L] = torch.randn(Hkv, L, d, generator=gen, device=dev).to(BF16)
    v[1, :, :L] = torch.randn(Hkv, L, d, generator=gen, device=dev).to(BF16)
    for Sq in (1, 150):
        q = torch.randn(B, Hkv, Sq, d, generator=gen, device=dev).to(BF16)
        lens = torch.tensor([0, L], dtype=torch.int32, device=dev)
        o, lse = gtms.attention_forward(q, k, v, lens, d ** -0.5, q_offsets=lens - Sq)
        assert bool((o[0] == 0).all())
        for h in (0, 15):
            at = slice(h, h + 1)
            keep = kept(lens[1:], Sq, L, 0, 0, lens[1:] - Sq)
            ref, ref_lse, tol, tol_lse = forward(q[1:, at], k[1:, at, :L], v[1:, at, :L], keep, d ** -0.5)
            _close("o", o[1:, at], ref, tol)
            _close("lse", lse[1:, at], ref_lse, tol_lse)


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------

# The angle is off by at most 2^-25 half turns in its last rounding (2^-25 pi < 2^-23) and the sine and
# cosine by an ulp or two: 2^-22 of the pair's length |x1| + |x2| with the products, then the dtype's
# own rounding.
ROT_UNIT = {F32: 2.0 ** -24, **UNIT}
ROT_TINY = {F32: 2.0 ** -149, **TINY}


def _rotary_tol(x, ref, inv_freq, interleaved, amplitude):
    R = 2 * inv_freq.numel()
    a = x.double().abs()
    size = torch.zeros_like(a)
    i1 = slice(0, R, 2) if interleaved else slice(0, R // 2)
    i2 = slice(1, R, 2) if interleaved else slice(R // 2, R)
    size[..., i1] = size[..., i2] = a[..., i1] + a[..., i2]
    return 2.0 ** -21 * abs(amplitude) * size + ROT_UNIT[x.dtype] * ref.abs() + ROT_TINY[x.dtype]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,H2,S,d,R,dtype,layout,first", [
    (1, 1, 0, 1, 64, 64, BF16, "bhsd", 0), (2, 4, 1, 33, 128, 128, F16, "bshd", 1000),
    (3, 2, 2, 17, 64, 16, F32, "sliced", 2 ** 31 - 200), (2, 3, 1, 5, 80, 40, BF16, "bhsd", 5),
    (1, 2, 1, 9, 34, 10, F32, "bhsd", 77), (4, 8, 2, 1, 128, 32, BF16, "bshd", 123456),
    (2, 2, 1, 300, 96, 96, F16, "bhsd", -150), (1, 2, 3, 8, 6, 0, F32, "bhsd", 3), (2, 40, 8, 130, 128, 64, BF16, "bhsd", 10 ** 6),
])
def test_rotary_matches_reference(dev, B, H, H2, S, d, R, dtype, layout, first, interleaved):
    gen = torch.Generator(device="cuda").manual_seed(11)
    x = _heads(gen, B, H, S, d, dtype, layout)
    other = _heads(gen, B, H2, S, d, dtype, layout) if H2 else None
    f = gtms.rotary_frequencies(R, 10000.0, device=dev)
    pos = (first + torch.arange(S, device=dev)[None] + 64 * torch.arange(B, device=dev)[:, None]).to(torch.int32)
    for inverse, call in ((False, gtms.rotary_forward), (True, gtms.rotary_backward)):
        got = call(x, pos, f, other=other, interleaved=interleaved, amplitude=1.25)
        for g, t in zip(got if H2 else (got,), (x, other) if H2 else (x,)):
            ref = rotate(t, pos, f, interleaved, 1.25, inverse)
            _close("rotary", g, ref, _rotary_tol(t, ref, f, interleaved, 1.25))
            assert torch.equal(g[..., R:], t[..., R:])


@pytest.mark.parametrize("layout", ["bhsd", "sliced"])
def test_rotary_in_place_and_shared_positions(dev, layout):
    gen = torch.Generator(device="cuda").manual_seed(12)
    x, k = (_heads(gen, 3, h, 50, 64, BF16, layout) for h in (4, 2))
    f = gtms.rotary_frequencies(32, 500000.0, gtms.GTMS_ROTARY_BY_PARTS, 8.0, device=dev)
    pos = torch.arange(50, dtype=torch.int32, device=dev)
    want = gtms.rotary_forward(x, pos, f, other=k)
    wide = gtms.rotary_forward(x, pos[None].expand(3, -1).contiguous(), f, other=k)
    got = gtms.rotary_forward(x, pos, f, other=k, out=x, out_other=k)
    for a, b, c in zip(want, wide, got):
        assert torch.equal(a, b) and torch.equal(a, c)
    assert got[0].data_ptr() == x.data_ptr() and got[1].data_ptr() == k.data_ptr()


def test_rotary_refuses_positions_of_another_shape(dev):
    x = torch.zeros(3, 2, 4, 64, dtype=BF16, device=dev)
    f = gtms.rotary_frequencies(64, device=dev)
    for shape in ((), (3,), (2, 4), (3, 3), (1, 1, 4), (3, 1, 4), (0, 4)):
        with pytest.raises(ValueError):
            gtms.rotary_forward(x, torch.zeros(shape, dtype=torch.int32, device=dev), f)
    for bad in (torch.zeros(4, dtype=torch.int64, device=dev), torch.zeros(4, dtype=torch.int32),
                torch.zeros(8, dtype=torch.int32, device=dev)[::2]):
        with pytest.raises(ValueError):
            gtms.rotary_forward(x, bad, f)


def test_rotary_in_place_inside_a_fused_buffer(dev):
    B, S, H, d = 2, 40, 6, 64
    qkv = torch.randn(B, S, H * d, device=dev).to(BF16)
    before = qkv.clone()
    heads = qkv.view(B, S, H, d).transpose(1, 2)
    q, k = heads[:, :3], heads[:, 3:4]
    f = gtms.rotary_frequencies(d, device=dev)
    pos = torch.arange(S, dtype=torch.int32, device=dev)
    old = before.view(B, S, H, d).transpose(1, 2)
    want = gtms.rotary_forward(old[:, :3], pos, f, other=old[:, 3:4])
    gtms.rotary_forward(q, pos, f, other=k, out=q, out_other=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(qkv[..., 4 * d:], before[..., 4 * d:])


# ---------------------------------------------------------------------------
# Together, as a layer uses them
# ---------------------------------------------------------------------------

def _layer(x, w, pos, f, lens, Hq, Hkv, d):
    B, S, _ = x.shape
    qkv = (x @ w).view(B, S, Hq + 2 * Hkv, d).transpose(1, 2)
    q, k = gtms.rotary(qkv[:, :Hq], pos, f, other=qkv[:, Hq:Hq + Hkv])
    return gtms.attention(q, k, qkv[:, Hq + Hkv:], lens, d ** -0.5)


def test_layer_gradients(dev):
    """Projection, rotary positions and attention through autograd against the same in 64 bits."""
    B, S, Hq, Hkv, d, n = 2, 150, 4, 2, 64, 32
    gen = torch.Generator(device="cuda").manual_seed(21)
    x = torch.randn(B, S, n, generator=gen, device=dev).to(BF16)
    w = (torch.randn(n, (Hq + 2 * Hkv) * d, generator=gen, device=dev) * n ** -0.5).to(BF16).requires_grad_()
    dy = torch.randn(B, Hq, S, d, generator=gen, device=dev).to(BF16)
    pos = torch.arange(S, dtype=torch.int32, device=dev)
    lens = torch.tensor([150, 97], dtype=torch.int32, device=dev)
    f = gtms.rotary_frequencies(d, device=dev)
    y = _layer(x, w, pos, f, lens, Hq, Hkv, d)
    y.backward(dy)

    w64 = w.detach().double().requires_grad_()
    qkv = (x.double() @ w64).view(B, S, Hq + 2 * Hkv, d).transpose(1, 2)
    qk = qkv[:, :Hq + Hkv]
    angle = pos.double()[:, None] * f.double()
    x1, x2 = qk[..., :d // 2], qk[..., d // 2:]
    qk = torch.cat((x1 * angle.cos() - x2 * angle.sin(), x2 * angle.cos() + x1 * angle.sin()), -1)
    s = torch.einsum("bhid,bhcd->bhic", qk[:, :Hq], qk[:, Hq:].repeat_interleave(2, 1)) * d ** -0.5
    keep = kept(lens, S, S)
    p = torch.softmax(torch.where(keep, s, -1e300), -1) * keep.any(-1)[..., None]
    ref = torch.einsum("bhic,bhcd->bhid", p, qkv[:, Hq + Hkv:].repeat_interleave(2, 1))
    ref.backward(dy.double())
    # Each 16-bit tensor on the way (qkv, rotated q and k, p, o; then ds, dq/dk/dv, their rotation, the
    # fused gradient) adds at most u of its size: ten roundings, random in sign, so the norm of the error
    # stays within 10 u of the result's norm times the amplification of at most 2 of softmax's derivative
    # at these scores (|s| is about 1).
    for got, want in ((y, ref), (w.grad, w64.grad)):
        assert float((got.detach().double() - want.detach()).norm() / want.detach().norm()) <= 20 * UNIT[BF16]


def test_token_by_token_equals_whole_sequence(dev):
    """Tokens one at a time over a cache give the rows of the whole pass."""
    B, S, Hq, Hkv, d = 2, 40, 4, 2, 64
    c = Case(B, Hq, Hkv, S, S, d, BF16, (S, S))
    f = gtms.rotary_frequencies(d, device=dev)
    pos = torch.arange(S, dtype=torch.int32, device=dev)
    q, k = gtms.rotary_forward(c.q, pos, f, other=c.k)
    whole, lse = gtms.attention_forward(q, k, c.v, c.lens, c.scale)
    cache_k, cache_v = (torch.full((B, Hkv, 64, d), math.nan, dtype=BF16, device=dev) for _ in range(2))
    ref, _, tol, tol_lse = forward(q, k, c.v, c.keep, c.scale)
    for t in range(S):
        step = torch.full((B, 1), t, dtype=torch.int32, device=dev)
        qt, kt = gtms.rotary_forward(c.q[:, :, t:t + 1], step, f, other=c.k[:, :, t:t + 1])
        cache_k[:, :, t:t + 1], cache_v[:, :, t:t + 1] = kt, c.v[:, :, t:t + 1]
        lens = torch.full((B,), t + 1, dtype=torch.int32, device=dev)
        o, l1 = gtms.attention_forward(qt, cache_k, cache_v, lens, c.scale, q_offsets=lens - 1)
        assert torch.equal(qt, q[:, :, t:t + 1])
        _close("token", o, ref[:, :, t:t + 1], tol[:, :, t:t + 1])
        assert bool(((l1 - lse[:, :, t:t + 1]).abs() <= 2 * tol_lse[:, :, t:t + 1]).all())
    _close("whole", whole, ref, tol)


def test_layer_step_captured_without_autograd_nodes(dev):
    """Rotary, attention and their gradients captured while an eager autograd graph of the same leaf lives."""
    B, S, Hq, Hkv, d = 1, 130, 4, 2, 64
    c = Case(B, Hq, Hkv, S, S, d, F16, (S,))
    f = gtms.rotary_frequencies(d, device=dev)
    pos = torch.arange(S, dtype=torch.int32, device=dev)
    leaf = c.q.clone().requires_grad_()
    alive = gtms.attention(*gtms.rotary(leaf, pos, f, other=c.k), c.v, c.lens, c.scale)

    def step():
        q, k = gtms.rotary_forward(leaf.detach(), pos, f, other=c.k)
        o, lse = gtms.attention_forward(q, k, c.v, c.lens, c.scale)
        dq, dk, dv = gtms.attention_backward(q, k, c.v, o, lse, c.dout, c.lens, c.scale)
        return (*gtms.rotary_backward(dq, pos, f, other=dk), dv)

    want = step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    alive.backward(c.dout)
    assert torch.equal(leaf.grad, want[0])


# ---------------------------------------------------------------------------
# Giving up
# ---------------------------------------------------------------------------

def _build_give_up_probe():
    """tests/attention_give_up_probe.cu (the attention kernels without their copies) as a library of its own."""
    import ctypes
    import os
    import subprocess

    from masked_softmax_attention_gb300 import _build as b

    src = os.path.join(b.ROOT, "tests", "attention_give_up_probe.cu")
    out_dir = os.path.join(b.ROOT, "_build", "test_probe")
    os.makedirs(out_dir, exist_ok=True)
    path = os.path.join(out_dir, "libgtms_attention_give_up_probe.so")
    deps = [src] + [os.path.join(b.CSRC, f) for f in os.listdir(b.CSRC)] + [os.path.join(b.INCLUDE, "gtms.h")]
    if not os.path.exists(path) or any(os.path.getmtime(d) > os.path.getmtime(path) for d in deps):
        tmp = path + f".{os.getpid()}.tmp"
        subprocess.run([b.nvcc_path(), *b.ARCH, *b.NVCC_FLAGS, "-shared", src, "-o", tmp], check=True,
                       capture_output=True, text=True)
        os.replace(tmp, path)
    fn = ctypes.CDLL(path).gtms_test_attention_no_loads
    vp, i32 = ctypes.c_void_p, ctypes.c_int32
    fn.argtypes = [vp, vp, vp, i32, i32, i32, i32, ctypes.c_float, vp, vp, vp, ctypes.c_uint64]
    fn.restype = ctypes.c_int
    return fn


@pytest.mark.parametrize("d", [64, 128])
def test_kernels_give_up_when_their_waits_run_out(dev, d):
    """Failure detection without a GPU fault: where no copy is issued, every wait runs out (after 200 us here).
    The launches must succeed, the grid must end promptly, also the CTAs that had not started, with
    GTMS_ERR_TIMEOUT in the status word, and a normal call right after it is exact."""
    import ctypes
    import time

    probe = _build_give_up_probe()
    B, H, S = 8, 16, 1000
    c = Case(B, H, H, S, S, d, BF16, (S,) * B)
    o, lse = c.forward()
    grads = [torch.zeros_like(t) for t in (c.q, c.k, c.v)]
    tensors = (ctypes.c_void_p * 8)(*(t.data_ptr() for t in (c.q, c.k, c.v, o.clone(), c.dout, *grads)))
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    work = torch.empty(1 << 22, dtype=torch.uint8, device=dev)
    for workspace in (None, work.data_ptr()):
        status.zero_()
        torch.cuda.synchronize()
        t0 = time.monotonic()
        rc = probe(tensors, lse.clone().data_ptr(), c.lens.data_ptr(), B, H, S, d, c.scale, status.data_ptr(), workspace,
                   torch.cuda.current_stream().cuda_stream, 200_000)
        torch.cuda.synchronize()
        assert rc == 0 and int(status.item()) == gtms.GTMS_ERR_TIMEOUT and time.monotonic() - t0 < 5.0
    o2, lse2 = c.forward()
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    c.backward(o, lse)
