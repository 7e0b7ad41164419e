"""Long sums: a million and more terms of one sign into one accumulator, and sums of several parts.

Tolerances. u is half a step of the type. The tensor cores' accumulators cut off: a product of 16 terms loses up to
2^-23 of the sum it goes into, and the kernels let no more than 2^15 terms in fp16 and 2^17 in bf16 (2^11 and 2^13
products) into one before they take its 16-bit part out (exactly, the rest stays in), so a sum is off by CUT = 2^-12 or
2^-10 of its terms' absolute sum, and by 2^-24 for each part. Softmax's fp32 sum takes one rounding a tile of 128 keys: 2^-24 Skv / 128, and 2^-15 covers exponentials,
scores and lse. P and ds are rounded once to the type (u), and o, from which D = do . o is formed, too.
"""
import math

import pytest
import torch

import masked_softmax_attention_gb300 as gtms

from attention_reference import UNIT
from test_attention_gpu import BF16, F16, LENGTH, TRIL, WINDOW, Case, _close

pytestmark = pytest.mark.gpu

CUT = {F16: 2.0 ** -12 + 2.0 ** -17, BF16: 2.0 ** -10 + 2.0 ** -17}   # 128 parts at most here


class OneSign:
    """Inputs for which every term of o, dq and dv has one sign, and every term of dk too, under the length mask:
    q, do > 0; v is larger for the first half of the keys than for the second, which makes ds positive and negative, and
    k has the sign of ds."""

    def __init__(self, Hq, Sq, Skv, d, dtype):
        gen = torch.Generator(device="cuda").manual_seed(Skv + d)
        rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        half = (torch.arange(Skv, device="cuda") < Skv // 2)[None, None, :, None]
        sign = torch.where(half, 1.0, -1.0)
        self.q, self.dout = ((0.5 + 0.2 * rand(1, Hq, Sq, d).abs()).to(dtype) for _ in range(2))
        self.k = (sign * (0.5 + 0.2 * rand(1, 1, Skv, d).abs())).to(dtype)
        self.v = (1.0 + 0.5 * sign + 0.1 * rand(1, 1, Skv, d)).to(dtype)
        self.lens = torch.tensor([Skv], dtype=torch.int32, device="cuda")
        self.off = self.lens - Sq
        self.scale, self.u = 1.0 / d, UNIT[dtype]
        self.cut, self.w = CUT[dtype], Skv / 128 * 2.0 ** -24 + 2.0 ** -15
        opts = dict(mask_kind=LENGTH, q_offsets=self.off)
        self.o, self.lse = gtms.attention_forward(self.q, self.k, self.v, self.lens, self.scale, **opts)
        self.grads = gtms.attention_backward(self.q, self.k, self.v, self.o, self.lse, self.dout, self.lens, self.scale, **opts)

    def check_row(self, h, i):
        """o and dq of one row."""
        q, do, k, v = self.q[0, h, i].double(), self.dout[0, h, i].double(), self.k[0, 0].double(), self.v[0, 0].double()
        p = torch.softmax(k @ q * self.scale, 0)
        o = p @ v
        _close("o", self.o[0, h, i], o, self.u * o.abs() + (self.u + self.cut + self.w) * (p @ v.abs()))
        dp, D = v @ do, do @ o
        ds = p * (dp - D)
        tol = ds.abs() * (self.u + self.cut + self.w) + p * (self.u * (do.abs() @ o.abs()) + 2.0 ** -15 * (v.abs() @ do.abs()))
        dq = self.scale * (ds @ k)
        _close("dq", self.grads[0][0, h, i], dq, self.u * dq.abs() + self.scale * (tol @ k.abs()))

    def check_key(self, c):
        """dk and dv of one key, all rows and heads live; D from each row's own o in 64 bits of the kernel's o."""
        k, v = self.k[0, 0, c].double(), self.v[0, 0, c].double()
        dk, dv, tk, tv = (torch.zeros_like(k) for _ in range(4))
        for h in range(self.q.shape[1]):
            q, do, o = self.q[0, h].double(), self.dout[0, h].double(), self.o[0, h].double()
            p = torch.exp(q @ k * self.scale - self.lse[0, h].double())
            dv += p @ do
            tv += (self.u + self.cut + self.w) * (p @ do.abs())
            ds = p * (do @ v - (do * o).sum(-1))
            dk += self.scale * (ds @ q)
            tk += self.scale * ((ds.abs() * (self.u + self.cut + self.w) + p * 2.0 ** -15 * (do.abs() @ v.abs())) @ q.abs())
        _close("dk", self.grads[1][0, 0, c], dk, self.u * dk.abs() + tk)
        _close("dv", self.grads[2][0, 0, c], dv, self.u * dv.abs() + tv)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_a_million_keys(dtype, d):
    c = OneSign(1, 4200, 1 << 20, d, dtype)
    for i in (0, 131, 4199):
        c.check_row(0, i)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_a_million_rows_of_shared_heads(dtype, d):
    c = OneSign(64, 16384, 16384, d, dtype)
    for key in (0, 5000, 16383):
        c.check_key(key)
    c.check_row(63, 16000)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_one_token_over_two_million_keys(dtype, d):
    """The kernel for few rows, its keys not split over CTAs since there are heads enough. Its sum of exponentials takes
    2^19 roundings of random sign, 2^-24 at most each: 2^-12 is eight times their standard deviation."""
    B, H, S = 8, 80, 1 << 21
    gen = torch.Generator(device="cuda").manual_seed(d)
    q = torch.randn(B, H, 1, d, generator=gen, device="cuda").to(dtype)
    k = torch.randn(1, 1, S, d, generator=gen, device="cuda").to(dtype)
    v = (1.0 + 0.3 * torch.randn(1, 1, S, d, generator=gen, device="cuda")).to(dtype)
    lens = torch.full((B,), S, dtype=torch.int32, device="cuda")
    o, _ = gtms.attention_forward(q, k.expand(B, H, -1, -1), v.expand(B, H, -1, -1), lens, d ** -0.5, q_offsets=lens - 1)
    for b, h in ((0, 0), (7, 79), (3, 40)):
        p = torch.softmax(k[0, 0].double() @ q[b, h, 0].double() * d ** -0.5, 0)
        want, size = p @ v[0, 0].double(), p @ v[0, 0].double().abs()
        u = UNIT[dtype]
        _close("o", o[b, h, 0], want, u * want.abs() + (u + CUT[dtype] + 2.0 ** -12 + 2.0 ** -15) * size)


# Several parts to a sum: keys (o and dq), then rows of shared heads (dk and dv). Sums of random sign under every mask,
# against the general bounds.
PARTS = [
    (1, 16, 1, 260, 70000, 64, F16, (69990,), TRIL, 0, (69730,), "bhsd"),
    (1, 16, 1, 260, 140000, 128, BF16, (140000,), LENGTH, 0, (139740,), "bshd"),
    (1, 16, 1, 260, 70000, 64, F16, (66000,), WINDOW, 40000, (65740,), "sliced"),
    (2, 16, 1, 260, 40000, 128, F16, (33100, 300), TRIL, 0, (32840, 40), "bhsd"),
    (1, 16, 1, 260, 140000, 64, BF16, (139000,), WINDOW, 133000, (138740,), "bhsd"),
    (1, 128, 1, 2300, 2300, 64, BF16, (2300,), TRIL, 0, None, "bshd"),
    (1, 32, 1, 2300, 2300, 128, F16, (2190,), LENGTH, 0, None, "sliced"),
    (1, 64, 2, 2100, 2100, 64, F16, (2100,), WINDOW, 1500, None, "bhsd"),
    (2, 80, 1, 1700, 1700, 128, BF16, (1700, 900), TRIL, 0, None, "bhsd"),
]


@pytest.mark.parametrize("case", PARTS, ids=str)
def test_sums_of_several_parts(case):
    c = Case(*case, dstd=0.01)
    o, lse = c.forward()
    c.check_forward(o, lse)
    c.check_backward(c.backward(o, lse))


@pytest.mark.parametrize("case", PARTS[::3], ids=str)
def test_sums_of_several_parts_beside_masked_nan(case):
    c = Case(*case)
    c.spoil()
    o, lse = c.forward()
    c.check_forward(o, lse)
    c.check_backward(c.backward(o, lse))


@pytest.mark.parametrize("scale,std,dstd", [(-0.3, 1.0, 1.0), (0.0, 1.0, 1.0), (0.125, 1.0, 1e-6), (1.0, 2.0, 100.0)])
def test_sums_of_several_parts_scaled(scale, std, dstd):
    """Raised maxima between the parts, scales of every sign, gradients far from 1."""
    for case in (PARTS[0], PARTS[7]):
        c = Case(*case, scale=scale, std=std, dstd=dstd)
        o, lse = c.forward()
        c.check_forward(o, lse)
        c.check_backward(c.backward(o, lse))


def test_maxima_that_rise_late():
    """The keys that count come last in the kernel's order, after parts have been carried at a far lower maximum."""
    c = Case(1, 16, 1, 260, 70000, 64, F16, (70000,), LENGTH, 0, (69740,), "bhsd")
    c.k[:, :, :3000] *= 4.0
    c.q.abs_()
    c.k[:, :, 1000].fill_(3.0)
    o, lse = c.forward()
    c.check_forward(o, lse)
    c.check_backward(c.backward(o, lse))
    assert math.isfinite(float(lse.max()))
