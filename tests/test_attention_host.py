"""Host-side tests of the attention and rotary entry points (no GPU needed).

Every call here fails argument validation, or is an empty no-op, before the library touches CUDA; the
fake pointer values are never dereferenced.
"""
import ctypes
import math
import os

import pytest
import torch

import masked_softmax_attention_gb300 as gtms

OK, INVALID, UNSUPPORTED = gtms.GTMS_OK, gtms.GTMS_ERR_INVALID_ARG, gtms.GTMS_ERR_UNSUPPORTED
F32, BF16, F16 = gtms.GTMS_F32, gtms.GTMS_BF16, gtms.GTMS_F16
Q, K, V, O, DO, DQ, DK, DV, LSE, LENS, OFF, WORK, ST = (0x10_0000_0000 * i for i in range(1, 14))

pytestmark = pytest.mark.skipif(torch.cuda.is_available() or os.path.exists("/dev/nvidia0"),
                                reason="fake-pointer host tests run only without a GPU")


@pytest.fixture(scope="module", autouse=True)
def lib():
    gtms.build_library()
    return gtms.load_library()


def heads(data, H=4, S=200, d=64, strides=None):
    """Contiguous [B, H, S, d] heads at a fake address, or with given strides."""
    return None if data is None else gtms.Heads(data, *(strides or (H * S * d, S * d, d)))


def shape(B=2, Hq=4, Hkv=2, Sq=200, Skv=300, d=64, window=0, mask=0, dtype=BF16, scale=1.0):
    return gtms.AttentionShape(B, Hq, Hkv, Sq, Skv, d, window, mask, dtype, scale)


def fwd(s=None, q=None, k=None, v=None, o=None, lse=LSE, lens=LENS, off=None, status=None, **kw):
    return gtms.gtms_attention_forward(shape(**kw) if s is None else s, q or heads(Q), k or heads(K, 2, 300),
                                       v or heads(V, 2, 300), o or heads(O), lse, lens, off, status, None)


def bwd(s=None, q=None, k=None, v=None, o=None, lse=LSE, do=None, dq=None, dk=None, dv=None, lens=LENS, off=None,
        work=WORK, size=1 << 30, status=None, **kw):
    return gtms.gtms_attention_backward(shape(**kw) if s is None else s, q or heads(Q), k or heads(K, 2, 300),
                                        v or heads(V, 2, 300), o or heads(O), lse, do or heads(DO), dq or heads(DQ),
                                        dk or heads(DK, 2, 300), dv or heads(DV, 2, 300), lens, off, work, size, status,
                                        None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_shape_errors(call):
    assert call(B=-1) == INVALID and call(Sq=-1) == INVALID and call(Skv=-1) == INVALID and call(d=-64) == INVALID
    assert call(Hq=4, Hkv=3) == INVALID and call(Hq=4, Hkv=0) == INVALID and call(Hq=0, Hkv=2) == INVALID
    assert call(scale=math.nan) == INVALID and call(scale=math.inf) == INVALID
    assert call(mask=3) == UNSUPPORTED and call(mask=-1) == UNSUPPORTED
    assert call(mask=2, window=0) == INVALID
    assert call(dtype=F32) == UNSUPPORTED and call(dtype=7) == UNSUPPORTED
    assert call(d=32) == UNSUPPORTED and call(d=96) == UNSUPPORTED and call(d=256) == UNSUPPORTED
    assert call(Sq=gtms.GTMS_ATTENTION_MAX_S + 1) == UNSUPPORTED
    assert call(Skv=gtms.GTMS_ATTENTION_MAX_S + 1) == UNSUPPORTED
    assert call(B=1 << 40) == UNSUPPORTED                       # more work than a grid holds
    assert call(B=1 << 62, Hq=1 << 62, Hkv=1) == UNSUPPORTED


def test_null_arguments():
    assert gtms.gtms_attention_forward(None, heads(Q), heads(K), heads(V), heads(O), LSE, LENS, None, None, None) == INVALID
    for i in range(1, 5):
        args = [shape(), heads(Q), heads(K, 2, 300), heads(V, 2, 300), heads(O)]
        args[i] = None
        assert gtms.gtms_attention_forward(*args, LSE, LENS, None, None, None) == INVALID
        args[i] = gtms.Heads(None, 0, 0, 0)
        assert gtms.gtms_attention_forward(*args, LSE, LENS, None, None, None) == INVALID
    assert fwd(lens=None) == INVALID and bwd(lens=None) == INVALID
    assert bwd(lse=None) == INVALID and bwd(work=None) == INVALID
    for name in ("q", "k", "v", "o", "do", "dq", "dk", "dv"):
        assert bwd(**{name: gtms.Heads(None, 0, 0, 0)}) == INVALID


@pytest.mark.parametrize("call", [fwd, bwd])
def test_alignment_and_strides(call):
    assert call(q=heads(Q + 1)) == INVALID                                   # not element-aligned
    assert call(q=heads(Q + 8)) == UNSUPPORTED                               # not 16-byte aligned
    assert call(k=heads(K, 2, 300, strides=(2 * 300 * 64, 300 * 64, 68))) == UNSUPPORTED
    assert call(k=heads(K, 2, 300, strides=(-64, 300 * 64, 64))) == INVALID
    assert call(o=heads(O, strides=(1 << 62, 1 << 62, 64))) == INVALID       # the range overflows
    assert call(k=heads(K, 2, 300, strides=(2 * 300 * 64, 300 * 64, 0))) == UNSUPPORTED    # one row for every key
    assert call(k=heads(K, 2, 300, strides=(2 * 300 * 64, 300 * 64, 32))) == UNSUPPORTED   # rows that overlap
    assert call(v=heads(V, 2, 300, strides=(8, 300 * 64, 64))) == UNSUPPORTED
    assert call(v=heads(V, 2, 300, strides=(1 << 40, 300 * 64, 64))) == UNSUPPORTED        # a stride of 2^41 bytes
    assert call(lens=LENS + 2) == INVALID and call(off=OFF + 1) == INVALID and call(status=ST + 2) == INVALID
    assert call(lse=LSE + 2) == INVALID


def test_outputs_are_distinct():
    assert fwd(o=heads(O, strides=(0, 200 * 64, 64))) == INVALID             # batches written to one place
    assert fwd(o=heads(O, strides=(4 * 200 * 64, 0, 64))) == INVALID
    assert fwd(o=heads(O, strides=(4 * 200 * 64, 200 * 64, 32))) == INVALID  # rows that run into each other
    for name, t in (("dq", heads(DQ, strides=(0, 200 * 64, 64))), ("dk", heads(DK, strides=(64, 64, 64))),
                    ("dv", heads(DV, strides=(2 * 300 * 64, 0, 64)))):
        assert bwd(**{name: t}) == INVALID


def test_overlaps():
    assert fwd(o=heads(Q)) == INVALID and fwd(o=heads(K)) == INVALID and fwd(o=heads(V + 64)) == INVALID
    assert fwd(lse=O + 128) == INVALID and fwd(lens=O + 128) == INVALID and fwd(status=O) == INVALID
    assert fwd(off=O) == INVALID and fwd(lse=LENS) == INVALID and fwd(lse=Q) == INVALID and fwd(lse=K + 64) == INVALID
    for other in (Q, K, V, O, DO):
        assert bwd(dq=heads(other)) == INVALID
        assert bwd(dk=heads(other + 64, 2, 300)) == INVALID
    assert bwd(dk=heads(DQ, 2, 300)) == INVALID and bwd(dv=heads(DK + 128, 2, 300)) == INVALID
    assert bwd(work=DQ) == INVALID and bwd(work=Q) == INVALID and bwd(work=LENS) == INVALID and bwd(work=LSE) == INVALID
    assert bwd(work=WORK + 8) == INVALID
    assert bwd(lens=DV) == INVALID and bwd(lse=DQ) == INVALID and bwd(status=DK + 4) == INVALID


def test_parts_of_a_fused_projection_do_not_overlap():
    """Parts that run into each other are told from parts that do not (test_attention_gpu.py runs the latter)."""
    H, S, d, B = 8, 200, 64, 2
    st = (S * H * d, d, H * d)
    part = lambda base, h: heads(base + 2 * h * d, strides=st)  # noqa: E731
    q, k, v, o = part(Q, 0), part(Q, 4), part(Q, 6), heads(O)
    sh = dict(B=B, Hq=4, Hkv=2, Sq=S, Skv=S)
    bad = ctypes.c_uint64()
    assert gtms.gtms_attention_backward_workspace(shape(**sh), ctypes.byref(bad)) == OK
    need = bad.value
    assert need >= B * 4 * S * 4
    # a workspace that is too small is refused
    assert bwd(q=q, k=k, v=v, o=o, dq=part(DQ, 0), dk=part(DQ, 4), dv=part(DQ, 6), size=need - 1, **sh) == INVALID
    # parts that do run into each other are refused as overlaps with a workspace that is large enough
    assert bwd(q=q, k=k, v=v, o=o, dq=part(DQ, 0), dk=part(DQ, 3), dv=part(DQ, 6), size=need, **sh) == INVALID


def test_empty_work():
    none = gtms.Heads(None, 0, 0, 0)
    assert fwd(B=0, q=none, k=none, v=none, o=none, lens=None) == OK
    assert fwd(Sq=0, q=none, k=none, v=none, o=none, lens=None) == OK
    assert bwd(B=0, q=none, k=none, v=none, o=none, lens=None, work=None) == OK
    assert bwd(Sq=0, Skv=0, lens=None, work=None, lse=None) == OK
    n = ctypes.c_uint64(1)
    assert gtms.gtms_attention_backward_workspace(shape(Sq=0), ctypes.byref(n)) == OK
    assert gtms.gtms_attention_backward_workspace(shape(), None) == INVALID
    assert gtms.gtms_attention_backward_workspace(None, ctypes.byref(n)) == INVALID
    assert gtms.gtms_attention_backward_workspace(shape(d=32), ctypes.byref(n)) == UNSUPPORTED


def rot(x=Q, y=O, x2=None, y2=None, B=2, H=4, H2=0, S=10, d=64, R=64, pos=LENS, pb=1, freq=OFF, amp=1.0, dtype=BF16,
        sx=None, sy=None):
    return gtms.gtms_rotary(heads(x, H, S, d, sx), heads(y, H, S, d, sy), heads(x2, H2, S, d), heads(y2, H2, S, d), B, H,
                            H2, S, d, R, pos, pb, freq, 0, amp, 0, dtype, None)


def test_rotary_errors():
    assert rot(B=-1) == INVALID and rot(R=63) == INVALID and rot(R=66) == INVALID and rot(R=-2) == INVALID
    assert rot(amp=math.inf) == INVALID and rot(dtype=5) == UNSUPPORTED
    assert rot(d=1026, R=0) == UNSUPPORTED and rot(S=gtms.GTMS_ATTENTION_MAX_S + 1) == UNSUPPORTED
    assert rot(x=None) == INVALID and rot(y=None) == INVALID and rot(pos=None) == INVALID and rot(freq=None) == INVALID
    assert rot(pos=LENS + 2) == INVALID and rot(freq=OFF + 1) == INVALID and rot(pb=3) == INVALID
    assert rot(x=Q + 1) == INVALID and rot(x=Q + 2, dtype=F32) == INVALID
    assert rot(x2=K, H2=2) == INVALID and rot(y2=K, H2=2) == INVALID and rot(H2=2) == INVALID
    assert rot(y=Q + 128) == INVALID                                       # overlaps its input, not in place
    assert rot(x2=K, y2=O + 128, H2=2) == INVALID                          # the outputs overlap
    assert rot(x2=O, y2=K, H2=2) == INVALID                                # y over the second input
    assert rot(pos=O) == INVALID and rot(freq=O + 64) == INVALID
    assert rot(sy=(0, 640, 64)) == INVALID and rot(sx=(-1, 640, 64)) == INVALID
    assert rot(B=0, x=None, y=None, pos=None) == OK and rot(d=0, R=0, x=None, y=None) == OK
    assert rot(B=1 << 40) == UNSUPPORTED


def test_rotary_extents():
    many = gtms.GTMS_ATTENTION_MAX_S + 1
    assert rot(B=1, H=many, S=1, sx=(0, 64, 64), sy=(0, 64, 64), pb=1) == UNSUPPORTED
    assert rot(B=1 << 16, H=1, S=1 << 15, sx=(0, 0, 64), sy=(0, 64, 64), pb=1) == UNSUPPORTED   # 2^31 tokens


def test_rotary_frequencies():
    d, base = 128, 500000.0
    want = base ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    got = gtms.rotary_frequencies(d, base)
    assert torch.equal(got, want.float())
    assert torch.equal(gtms.rotary_frequencies(d, base, gtms.GTMS_ROTARY_LINEAR, 8.0), (want / 8).float())
    turns = 8192 * want / (2 * math.pi)
    m = ((turns - 1) / 3).clamp(0, 1)
    parts = gtms.rotary_frequencies(d, base, gtms.GTMS_ROTARY_BY_PARTS, 8.0, 1.0, 4.0, 8192)
    assert float((parts.double() / ((1 - m) * want / 8 + m * want) - 1).abs().max()) <= 2.0 ** -23
    assert torch.equal(parts[turns > 4], got[turns > 4]) and bool((parts[turns < 1] < got[turns < 1]).all())
    assert gtms.rotary_frequencies(0).numel() == 0
    for bad in (dict(rot_dim=7), dict(rot_dim=-2), dict(rot_dim=8, base=0.0), dict(rot_dim=8, base=math.inf),
                dict(rot_dim=8, factor=0.0, scaling=1), dict(rot_dim=8, scaling=3),
                dict(rot_dim=8, scaling=2, low_turns=4.0, high_turns=4.0), dict(rot_dim=8, scaling=2, original_length=0)):
        with pytest.raises(gtms.GtmsError):
            gtms.rotary_frequencies(**bad)


def test_tensor_api_refusals():
    z = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    lens = torch.ones(1, dtype=torch.int32)
    pos, f = torch.zeros(4, dtype=torch.int32), torch.ones(32)
    for call in (lambda: gtms.attention_forward(z, z, z, lens), lambda: gtms.attention(z, z, z, lens),
                 lambda: gtms.attention_backward(z, z, z, z, torch.zeros(1, 1, 4), z, lens),
                 lambda: gtms.rotary_forward(z, pos, f), lambda: gtms.rotary_backward(z, pos, f),
                 lambda: gtms.rotary(z[0], pos, f)):
        with pytest.raises(ValueError):
            call()


def test_differentiable_attention_hands_its_status_on(monkeypatch):
    """A wait that runs out in the forward or in the backward can be seen by the caller of attention()."""
    q = torch.zeros(1, 2, 3, 64, requires_grad=True)
    lens, status, seen = torch.ones(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), []

    def fwd_call(q, k, v, seq_lens, scale, status=None, **kw):
        seen.append(("forward", status))
        return torch.zeros_like(q), torch.zeros(q.shape[:3])

    def bwd_call(q, k, v, o, lse, dout, seq_lens, scale, status=None, **kw):
        seen.append(("backward", status))
        status.add_(4)
        return torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)

    monkeypatch.setattr(gtms, "attention_forward", fwd_call)
    monkeypatch.setattr(gtms, "attention_backward", bwd_call)
    gtms.attention(q, q.detach(), q.detach(), lens, status=status).sum().backward()
    assert [n for n, _ in seen] == ["forward", "backward"] and all(t is status for _, t in seen)
    assert int(status) == 4
