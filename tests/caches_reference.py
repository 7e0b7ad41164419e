"""Attention over shared prefixes, key weights and cache eviction from their definitions, with error bounds.

Attention and its bounds are those of attention_reference.py over a prefix's keys and a sequence's own put end to end
(partial sums joined in fp32 add roundings of the kind that its bounds count per term). A key's weight sums
p = exp(s - lse) with lse given:

* the score sums d exact products: off by d 2^-23 scale sum |q||k|;
* scale and score, and lse, are brought to base 2 (log2 e, the scale times it, lse times it and the difference round
  once each): 2^-22 (|s| + |lse|), relative to p once exponentiated; the exponential itself 2^-21 at most;
* the exponential is zero below 2^-126;
* the sum of n terms in fp32: n 2^-23 of it.
"""
import math

import torch

from attention_reference import F, FLUSH, forward, kept


def joined(q, k_prefix, v_prefix, k, v, seq_lens, scale, prefix_lens=None, mask_kind=0, q_offsets=None):
    """o, lse and their bounds, and the truth values of live rows [B, 1, Sq]."""
    B, P, Skv, Sq = q.shape[0], k_prefix.shape[2], k.shape[2], q.shape[2]
    n = B // k_prefix.shape[0]
    own = kept(seq_lens, Sq, Skv, mask_kind, 0, q_offsets)
    live = own.any(-1)
    plens = torch.full((k_prefix.shape[0],), P, device=q.device) if prefix_lens is None else prefix_lens.long().clamp(0, P)
    seen = torch.arange(P, device=q.device) < plens.repeat_interleave(n)[:, None]
    keep = torch.cat((live[..., None] & seen[:, None, None, :], own), -1)
    kk = torch.cat((k_prefix.repeat_interleave(n, 0), k), 2)
    vv = torch.cat((v_prefix.repeat_interleave(n, 0), v), 2)
    # Keys behind a prefix's end are in no row's kept set and so are cleared with the rest.
    return forward(q, kk, vv, keep, scale) + (live,)


def key_weights(q, k, lse, keep, scale):
    """w [B, Hkv, Skv] and its bound."""
    B, Hq, Sq, d = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    group = Hq // Hkv
    rows = keep.any(-1)[..., None]
    q = torch.where(rows, q.double(), 0.0)
    k = torch.where(keep.any(-2)[..., None], k.double(), 0.0).repeat_interleave(group, 1)
    s = torch.einsum("bhid,bhcd->bhic", q, k) * scale
    mag = torch.einsum("bhid,bhcd->bhic", q.abs(), k.abs()) * abs(scale)
    z = lse.double()[..., None]
    counts = keep & (z != -math.inf)
    p = torch.where(counts, torch.exp(s - torch.where(counts, z, 0.0)), 0.0)
    e = d * F * mag + 2.0 ** -22 * (s.abs() + torch.where(counts, z.abs(), 0.0)) + 2.0 ** -21
    fold = lambda t: t.sum(2).view(B, Hkv, group, Skv).sum(2)  # noqa: E731
    w = fold(p)
    return w, fold(p * e) + Sq * group * (F * w + FLUSH)


def evicted(weights, n, keep, first, recent):
    """Indices that stay of one sequence's and head's n entries (a list of floats)."""
    if n <= keep:
        return list(range(n))
    middle = range(first, n - recent)
    top = sorted(middle, key=lambda c: (-math.inf if math.isnan(weights[c]) else -weights[c] + 0.0, c))
    # NaN counts above +infinity: those first, in order.
    nans = [c for c in middle if math.isnan(weights[c])]
    top = nans + [c for c in top if not math.isnan(weights[c])]
    return list(range(first)) + sorted(top[:keep - first - recent]) + list(range(n - recent, n))
