"""Attention, its gradients and rotary positions in 64 bits from their definitions, with error bounds.

Every function takes torch tensors and works in float64 on their device. The bounds count, for each
output element, the roundings a 16-bit kernel with fp32 sums cannot avoid (``u`` = half a step of the
dtype, every addition inside the tensor cores and every fp32 sum taken to lose at most 2^-23):

* a score sums d exact products: off by es = d 2^-23 scale sum |q||k|, plus 2^-22 of |s| and of the
  running maximum (or lse) it is compared with, when it is brought to base 2 and shifted;
* a probability is then off by that, relatively, and by 2^-21 for the exponential; rounded to 16 bits
  it is off by u more, or by 2^-25 where fp16 runs out of exponents (probabilities are at most 1 before
  they are normalised, and the sum they are divided by is at least 1);
* the exponential is zero where it would be below 2^-126, fp32's smallest normal number: p is off by up
  to 2^-126 there, and ds by 2^-126 |dp - D| (seen as a gradient of 2e-37 that came out as zero: one
  p of 2^-127 times dp - D and q of about 10 each);
* o divides by a sum with the same relative errors, sums n products (n 2^-23 of their absolute sum) and
  is rounded once: u |o|;
* D = do . o takes o rounded: u sum |do||o|, and d 2^-23 of that sum for the additions;
* ds = p (dp - D) carries p times the errors of dp and D, and |ds| times those of p, and is rounded once
  (u, or 2^-25 of the largest value 2^14 that fp16 holds it scaled to: 2^-38 of 4 max|do_i| max|v_c|,
  twice the bound of |dp - D|, since the scale is a power of two);
* dq, dk and dv sum n products and are rounded once.
"""
import math

import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step, relative to the value
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}  # half the smallest step
F = 2.0 ** -23
FLUSH = 2.0 ** -126


def kept(seq_lens, Sq, Skv, mask_kind=0, window=0, q_offsets=None):
    """[B, 1, Sq, Skv] truth values."""
    dev = seq_lens.device
    L = seq_lens.long().clamp(0, Skv)[:, None, None, None]
    r = torch.arange(Sq, device=dev)[None, None, :, None]
    if q_offsets is not None:
        r = r + q_offsets.long()[:, None, None, None]
    c = torch.arange(Skv, device=dev)[None, None, None, :]
    live = (r >= 0) & (r < L)
    if mask_kind == 1:
        return live & (c < L)
    keep = live & (c <= r)
    return keep & (c > r - window) if mask_kind == 2 else keep


def _spread(t, group):
    return t.double().repeat_interleave(group, 1)


def _scores(q, k, scale, keep):
    group = q.shape[1] // k.shape[1]
    qd, kd = q.double(), _spread(k, group)
    s = torch.einsum("bhid,bhcd->bhic", qd, kd) * scale
    mag = torch.einsum("bhid,bhcd->bhic", qd.abs(), kd.abs()) * abs(scale)
    return torch.where(keep, s, -math.inf), torch.where(keep, mag, 0.0)


def _clean(t, rows):
    """t with the rows that are not used (anything may stand there) zeroed."""
    return torch.where(rows, t.double(), 0.0)


def _live(keep):
    rows = keep.any(-1)[..., None]                 # [B, 1, Sq, 1]
    cols = keep.any(-2)[..., None]                 # [B, 1, Skv, 1]
    return rows, cols


def forward(q, k, v, keep, scale):
    """o, lse and their bounds."""
    u, tiny, d, n = UNIT[q.dtype], TINY[q.dtype], q.shape[3], keep.shape[3]
    dtype = q.dtype
    rows, cols = _live(keep)
    q, k, v = _clean(q, rows), _clean(k, cols), _clean(v, cols)
    group = q.shape[1] // k.shape[1]
    s, mag = _scores(q, k, scale, keep)
    lse = torch.logsumexp(s, -1)
    safe = torch.where(lse == -math.inf, 0.0, lse)
    p = torch.exp(s - safe[..., None])
    vd = _spread(v, group)
    o = torch.einsum("bhic,bhcd->bhid", p, vd)
    A = torch.einsum("bhic,bhcd->bhid", p, vd.abs())
    smax = torch.where(keep, s.abs(), 0.0).amax(-1)
    e = d * F * mag.amax(-1) + 2 * 2.0 ** -22 * smax + 2.0 ** -21
    tol = u * o.abs() + (u + 2 * e + 2 * n * F)[..., None] * A + tiny
    tol = tol + FLUSH * torch.einsum("bhic,bhcd->bhid", keep.double().expand_as(p), vd.abs())
    if dtype == torch.float16:
        tol = tol + tiny * torch.einsum("bhic,bhcd->bhid", keep.double().expand_as(p), vd.abs())
    tol_lse = e + n * F + 2.0 ** -22 * safe.abs()
    return o, lse, tol, tol_lse


def backward(q, k, v, dout, keep, scale):
    """dq, dk, dv and their bounds."""
    dtype, d, Sq, Skv = q.dtype, q.shape[3], keep.shape[2], keep.shape[3]
    u, tiny = UNIT[dtype], TINY[dtype]
    rows, cols = _live(keep)
    q, dout, k, v = _clean(q, rows), _clean(dout, rows), _clean(k, cols), _clean(v, cols)
    B, Hkv, group = q.shape[0], k.shape[1], q.shape[1] // k.shape[1]
    s, mag = _scores(q, k, scale, keep)
    lse = torch.logsumexp(s, -1)
    safe = torch.where(lse == -math.inf, 0.0, lse)[..., None]
    p = torch.exp(s - safe)
    kd, vd = _spread(k, group), _spread(v, group)
    dp = torch.einsum("bhid,bhcd->bhic", dout, vd)
    adp = torch.einsum("bhid,bhcd->bhic", dout.abs(), vd.abs())
    o = torch.einsum("bhic,bhcd->bhid", p, vd)
    D = (dout * o).sum(-1, keepdim=True)
    aD = (dout.abs() * o.abs()).sum(-1, keepdim=True)
    ds = p * (dp - D)
    ep = d * F * mag + 2.0 ** -22 * (torch.where(keep, s.abs(), 0.0) + 2 * safe.abs()) + 2.0 ** -20
    e_ds = p * (d * F * adp + (u + d * F) * aD) + ds.abs() * (ep + u + 2.0 ** -21)
    e_p = p * (u + ep) + keep * FLUSH
    e_ds = e_ds + keep * FLUSH * (dp - D).abs()
    if dtype == torch.float16:
        top = dout.norm(dim=-1).amax() * v.norm(dim=-1).amax()
        e_ds = e_ds + keep * (4 * top * 2.0 ** -38)
        e_p = e_p + keep * tiny

    def fold(t):
        return t.view(B, Hkv, group, Skv, d).sum(2)

    sc = abs(scale)
    dq = scale * torch.einsum("bhic,bhcd->bhid", ds, kd)
    tq = u * dq.abs() + sc * torch.einsum("bhic,bhcd->bhid", e_ds + 2 * Skv * F * ds.abs(), kd.abs()) + tiny
    n = 2 * Sq * group * F
    dk = scale * fold(torch.einsum("bhic,bhid->bhcd", ds, q))
    tk = u * dk.abs() + sc * fold(torch.einsum("bhic,bhid->bhcd", e_ds + n * ds.abs(), q.abs())) + tiny
    dv = fold(torch.einsum("bhic,bhid->bhcd", p, dout))
    tv = u * dv.abs() + fold(torch.einsum("bhic,bhid->bhcd", e_p + n * p, dout.abs())) + tiny
    return (dq, dk, dv), (tq, tk, tv)


def rotate(x, positions, inv_freq, interleaved=False, amplitude=1.0, inverse=False):
    """Rotary positions in 64 bits; positions [S] or [B, S]."""
    R = 2 * inv_freq.numel()
    pos = positions if positions.dim() == 2 else positions[None]
    angle = pos.double()[:, None, :, None] * inv_freq.double()
    cos, sin = amplitude * angle.cos(), amplitude * angle.sin() * (-1.0 if inverse else 1.0)
    y = x.double().clone()
    i1 = slice(0, R, 2) if interleaved else slice(0, R // 2)
    i2 = slice(1, R, 2) if interleaved else slice(R // 2, R)
    x1, x2 = x.double()[..., i1], x.double()[..., i2]
    y[..., i1], y[..., i2] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    return y
