"""The 64-bit gradients that the GPU tests compare with, against autograd through a softmax written apart from them."""
import pytest
import torch

from attention_reference import backward, forward, kept


def attend(q, k, v, keep, scale):
    """Masked attention in 64 bits by torch's own softmax; rows that keep nothing give 0."""
    group = q.shape[1] // k.shape[1]
    s = torch.matmul(q, k.repeat_interleave(group, 1).transpose(-1, -2)) * scale
    p = torch.softmax(torch.where(keep, s, -1e300), -1) * keep.any(-1)[..., None]
    return torch.matmul(p, v.repeat_interleave(group, 1))


@pytest.mark.parametrize("Sq,Skv,lens,mask,window,offsets", [
    (60, 60, (60, 41), 0, 0, None), (47, 47, (47, 0), 1, 0, None), (60, 60, (60, 33), 2, 17, None),
    (9, 50, (50, 20), 0, 0, (41, 11)), (30, 40, (40, 25), 2, 6, (-4, 10))])
def test_gradient_formula_matches_autograd(Sq, Skv, lens, mask, window, offsets):
    gen = torch.Generator().manual_seed(7)
    q, k, v, dout = (torch.randn(2, H, n, 64, generator=gen).to(torch.bfloat16)
                     for H, n in ((6, Sq), (2, Skv), (2, Skv), (6, Sq)))
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32)
    keep, scale = kept(torch.tensor(lens, dtype=torch.int32), Sq, Skv, mask, window, off), 0.17
    leaves = [t.double().requires_grad_() for t in (q, k, v)]
    o = attend(*leaves, keep, scale)
    o.backward(dout.double())
    assert float((forward(q, k, v, keep, scale)[0] - o.detach()).abs().max()) <= 1e-12
    for leaf, want in zip(leaves, backward(q, k, v, dout, keep, scale)[0]):
        assert float((leaf.grad - want).abs().max()) <= 1e-12 * float(want.abs().max())
