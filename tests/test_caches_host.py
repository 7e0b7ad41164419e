"""Host-side tests of the entry points on caches: refusals and workspaces (no GPU needed).

Every call here fails argument validation, or is an empty no-op, before the library touches CUDA; the fake pointer
values are never dereferenced.
"""
import ctypes
import math
import os

import pytest
import torch

import masked_softmax_attention_gb300 as gtms

from caches_reference import evicted

OK, INVALID, UNSUPPORTED = gtms.GTMS_OK, gtms.GTMS_ERR_INVALID_ARG, gtms.GTMS_ERR_UNSUPPORTED
F32, BF16, F16 = gtms.GTMS_F32, gtms.GTMS_BF16, gtms.GTMS_F16
Q, K, V, O, KP, VP, LSE, LENS, OFF, WORK, ST, PLENS, W, POS, KO, VO, WO, PO, LO = (0x10_0000_0000 * i for i in range(1, 20))
MAX = gtms.GTMS_ATTENTION_MAX_S

pytestmark = pytest.mark.skipif(torch.cuda.is_available() or os.path.exists("/dev/nvidia0"),
                                reason="fake-pointer host tests run only without a GPU")


@pytest.fixture(scope="module", autouse=True)
def lib():
    gtms.build_library()
    return gtms.load_library()


def heads(data, H, S, d=64, strides=None):
    return gtms.Heads(data, *(strides or (H * S * d, S * d, d)))


def shape(B=4, Hq=4, Hkv=2, Sq=20, Skv=300, d=64, window=0, mask=0, dtype=BF16, scale=1.0):
    return gtms.AttentionShape(B, Hq, Hkv, Sq, Skv, d, window, mask, dtype, scale)


# ---------------------------------------------------------------------------
# Shared prefixes
# ---------------------------------------------------------------------------

def prefix(s=None, G=2, P=500, lse=LSE, plens=PLENS, lens=LENS, off=OFF, work=WORK, size=1 << 40, status=ST, operands=None, **kw):
    t = {"q": heads(Q, 4, 20), "kp": heads(KP, 2, 500), "vp": heads(VP, 2, 500), "k": heads(K, 2, 300), "v": heads(V, 2, 300),
         "o": heads(O, 4, 20), **(operands or {})}
    return gtms.gtms_attention_shared_prefix(shape(**kw) if s is None else s, G, P, t["q"], t["kp"], t["vp"], t["k"], t["v"],
                                             t["o"], lse, plens, lens, off, work, size, status, None)


def test_prefix_shape_errors():
    assert prefix(B=-1) == INVALID and prefix(Sq=-1) == INVALID and prefix(Hkv=3) == INVALID and prefix(scale=math.nan) == INVALID
    assert prefix(G=-2) == INVALID and prefix(P=-1) == INVALID and prefix(G=0) == INVALID and prefix(G=3) == INVALID
    assert prefix(G=8) == INVALID                                 # fewer sequences than prefixes
    assert prefix(mask=2, window=10) == UNSUPPORTED and prefix(mask=5) == UNSUPPORTED
    assert prefix(P=MAX + 1) == UNSUPPORTED and prefix(dtype=F32) == UNSUPPORTED and prefix(d=96) == UNSUPPORTED
    assert prefix(B=1 << 40, G=1) == UNSUPPORTED


def test_prefix_null_and_misaligned_arguments():
    for name in ("q", "kp", "vp", "k", "v", "o"):
        assert prefix(operands={name: None}) == INVALID
        assert prefix(operands={name: gtms.Heads(None, 0, 0, 0)}) == INVALID
    assert gtms.gtms_attention_shared_prefix(None, 1, 1, *[None] * 6, *[None] * 5, 0, None, None) == INVALID
    assert prefix(lens=None) == INVALID
    for name in ("lse", "plens", "lens", "off", "status"):
        assert prefix(**{name: 0x10_0000_0002}) == INVALID
    at = heads(KP + 8, 2, 500)
    assert prefix(operands={"kp": at}) == UNSUPPORTED             # 8-byte aligned
    assert prefix(operands={"vp": heads(VP, 2, 500, strides=(64000, 32000, 60))}) == UNSUPPORTED
    assert prefix(operands={"vp": heads(VP, 2, 500, strides=(64000, 32000, -64))}) == INVALID
    assert prefix(operands={"o": heads(O, 4, 20, strides=(0, 1280, 64))}) == INVALID


def test_prefix_overlaps():
    row = 4 * 4 * 20 * 64 * 2                                     # bytes of o and of q
    for at in (Q, KP, VP, K, V):
        assert prefix(operands={"o": heads(at, 4, 20)}) == INVALID
    for name, size in (("lens", 16), ("off", 16), ("plens", 8), ("status", 4), ("lse", 4 * 4 * 20 * 4)):
        assert prefix(**{name: O + row - 4}) == INVALID
        if name != "lse":
            assert prefix(**{name: LSE + 4}) == INVALID
    for at in (Q, KP, VP, K, V):
        assert prefix(lse=at) == INVALID


def test_prefix_nothing_to_do():
    none = {n: None for n in ("q", "kp", "vp", "k", "v", "o")}
    assert prefix(B=0, G=0, operands=none, lens=None) == OK and prefix(Sq=0, operands=none, lens=None) == OK
    assert prefix(Hq=0, Hkv=0, operands=none, lens=None) == OK


@pytest.mark.parametrize("kw", [dict(), dict(Sq=1), dict(B=256, Sq=1, Hq=32, Hkv=8), dict(Sq=4000, Skv=4000)])
def test_prefix_workspace(kw):
    need = ctypes.c_uint64(123)
    s = shape(**kw)
    assert gtms.gtms_attention_shared_prefix_workspace(s, 2, 5000, ctypes.byref(need)) == OK
    assert need.value % 4 == 0 and need.value < 1 << 34
    operands = {"q": heads(Q, s.Hq, s.Sq), "o": heads(O, s.Hq, s.Sq), "kp": heads(KP, s.Hkv, 5000), "vp": heads(VP, s.Hkv, 5000),
                "k": heads(K, s.Hkv, s.Skv), "v": heads(V, s.Hkv, s.Skv)}
    if need.value:
        for bad in (dict(work=None), dict(size=need.value - 1), dict(work=WORK + 8), dict(work=O), dict(work=LSE), dict(work=Q),
                    dict(work=KP), dict(work=LENS)):
            assert prefix(s, P=5000, operands=operands, **bad) == INVALID
    assert gtms.gtms_attention_shared_prefix_workspace(s, 2, 5000, None) == INVALID
    assert gtms.gtms_attention_shared_prefix_workspace(s, 3, 5000, ctypes.byref(need)) == INVALID
    assert gtms.gtms_attention_shared_prefix_workspace(shape(mask=2, window=1), 2, 5000, ctypes.byref(need)) == UNSUPPORTED


def test_workspaces_of_any_shape():
    """Also without a prefix, own keys or rows; never negative or beyond what its parts can hold."""
    need = ctypes.c_uint64()
    for G, n in ((1, 1), (1, 64), (7, 3)):
        for Hq, Hkv in ((1, 1), (8, 2), (130, 1)):
            for Sq, Skv in ((0, 5), (1, 0), (1, 1), (1, 70000), (5, 300), (700, 700), (MAX, MAX)):
                for P in (0, 1, 500, 70000, MAX):
                    for d in (64, 128):
                        s = shape(B=G * n, Hq=Hq, Hkv=Hkv, Sq=Sq, Skv=Skv, d=d)
                        rc = gtms.gtms_attention_shared_prefix_workspace(s, G, P, ctypes.byref(need))
                        if G * n * Hq * ((max(Sq, Skv) + 63) // 64) >= 1 << 31:
                            assert rc == UNSUPPORTED
                            continue
                        # At most 2 parts of each of 512 + 31 splits of the prefix and 64 of the own keys.
                        assert rc == OK and need.value <= (2 * 543 + 64) * G * n * Hq * Sq * (d * 4 + 8)
                        assert need.value == 0 or P * Sq > 0
                        assert gtms.gtms_attention_key_weights_workspace(s, ctypes.byref(need)) == OK
                        assert need.value % 4 == 0 and (need.value == 0 or Sq * Skv > 0)


# ---------------------------------------------------------------------------
# Key weights
# ---------------------------------------------------------------------------

def weigh(s=None, q=Q, k=K, lse=LSE, w=W, accumulate=0, lens=LENS, off=OFF, work=WORK, size=1 << 40, status=ST, q_heads=None,
          k_heads=None, **kw):
    return gtms.gtms_attention_key_weights(shape(**kw) if s is None else s, q_heads or heads(q, 4, 20), k_heads or heads(k, 2, 300),
                                           lse, w, accumulate, lens, off, work, size, status, None)


def test_weights_errors():
    assert weigh(B=-1) == INVALID and weigh(Hkv=3) == INVALID and weigh(scale=math.inf) == INVALID
    assert weigh(mask=2) == INVALID and weigh(mask=3) == UNSUPPORTED
    assert weigh(dtype=F32) == UNSUPPORTED and weigh(d=32) == UNSUPPORTED and weigh(Skv=MAX + 1) == UNSUPPORTED
    assert weigh(q=None) == INVALID and weigh(k=None) == INVALID and weigh(lse=None) == INVALID and weigh(w=None) == INVALID
    assert weigh(lens=None) == INVALID
    for name in ("lse", "w", "lens", "off", "status"):
        assert weigh(**{name: 0x10_0000_0002}) == INVALID
    assert weigh(q=Q + 8) == UNSUPPORTED and weigh(k=K + 8) == UNSUPPORTED
    assert weigh(k_heads=heads(K, 2, 300, strides=(38400, 19200, -64))) == INVALID
    for name in ("q", "k", "lse", "lens", "off", "status"):
        assert weigh(**{name: W}) == INVALID                      # on the weights
    need = ctypes.c_uint64()
    s = shape(Sq=300)
    assert gtms.gtms_attention_key_weights_workspace(s, ctypes.byref(need)) == OK
    if need.value:
        for bad in (dict(work=None), dict(size=need.value - 1), dict(work=WORK + 4), dict(work=W), dict(work=LSE)):
            assert weigh(s, q_heads=heads(Q, 4, 300), **bad) == INVALID
    assert gtms.gtms_attention_key_weights_workspace(s, None) == INVALID
    assert gtms.gtms_attention_key_weights_workspace(shape(d=65), ctypes.byref(need)) == UNSUPPORTED


def test_weights_nothing_to_do():
    assert weigh(Skv=0, q=None, k=None, lse=None, w=None, lens=None) == OK
    assert weigh(B=0, q=None, k=None, lse=None, w=None, lens=None) == OK
    assert weigh(Sq=0, w=None) == INVALID                         # the weights are still to be zeroed


# ---------------------------------------------------------------------------
# Eviction
# ---------------------------------------------------------------------------

def evict(B=2, H=3, S=100, S_out=40, d=64, keep=40, first=2, recent=5, dtype=BF16, w=W, pos=POS, wo=WO, po=PO, lens=LENS, lo=LO,
          work=WORK, size=1 << 30, s=0, **operands):
    s = gtms.EvictShape(B, H, S, S_out, d, keep, first, recent, dtype) if s == 0 else s
    t = {"k": heads(K, H, S, d), "v": heads(V, H, S, d), "ko": heads(KO, H, S_out, d), "vo": heads(VO, H, S_out, d), **operands}
    return gtms.gtms_cache_evict(s, t["k"], t["v"], w, pos, t["ko"], t["vo"], wo, po, lens, lo, work, size, None)


def test_evict_sizes():
    assert evict(s=None) == INVALID
    for name in ("B", "H", "S", "S_out", "d", "keep", "first", "recent"):
        assert evict(**{name: -1}) == INVALID
    assert evict(first=36) == INVALID and evict(recent=41) == INVALID and evict(first=41, recent=0) == INVALID
    assert evict(first=(1 << 63) - 1, recent=(1 << 63) - 1) == INVALID
    assert evict(S_out=39) == INVALID and evict(S=30, keep=40, S_out=29) == INVALID
    assert evict(H=0) == INVALID                                  # nothing would write the lengths
    assert evict(dtype=7) == UNSUPPORTED and evict(d=1032) == UNSUPPORTED and evict(d=60) == UNSUPPORTED
    assert evict(d=2, dtype=F32) == UNSUPPORTED and evict(S=MAX + 1) == UNSUPPORTED and evict(S_out=MAX + 1) == UNSUPPORTED
    assert evict(B=1 << 40) == UNSUPPORTED and evict(B=1 << 62, H=1 << 62) == UNSUPPORTED
    assert evict(B=0) == OK


def test_evict_pointers():
    for name in ("k", "v", "ko", "vo"):
        assert evict(**{name: None}) == INVALID and evict(**{name: gtms.Heads(None, 0, 0, 0)}) == INVALID
        assert evict(**{name: heads(0x7000_0000_0008, 3, 100)}) == UNSUPPORTED
        assert evict(**{name: heads(0x7000_0000_0000, 3, 100, strides=(19200, 6400, -64))}) == INVALID
    for name in ("w", "wo", "lens", "lo", "work"):
        assert evict(**{name: None}) == INVALID
    for name in ("w", "wo", "pos", "po", "lens", "lo", "work"):
        assert evict(**{name: 0x7000_0000_0002}) == INVALID
    assert evict(work=WORK + 4) == INVALID and evict(size=2 * 3 * 40 * 4 - 1) == INVALID
    assert evict(ko=heads(KO, 3, 40, strides=(0, 2560, 64))) == INVALID                # an output on itself


def test_evict_overlaps():
    assert evict(ko=heads(K, 3, 40)) == INVALID                   # part of it, other strides
    assert evict(S_out=100, ko=heads(V, 3, 100)) == INVALID and evict(S_out=100, vo=heads(K, 3, 100)) == INVALID
    assert evict(ko=heads(KO, 3, 40), vo=heads(KO, 3, 40)) == INVALID
    assert evict(wo=W) == INVALID and evict(po=POS) == INVALID    # with S_out == S alone
    assert evict(S_out=100, wo=POS) == INVALID and evict(wo=PO) == INVALID and evict(wo=W + 400) == INVALID
    for name in ("w", "pos", "wo", "po", "lens", "work"):
        assert evict(**{name: LO}) == INVALID
    for name in ("wo", "po", "work", "lo"):
        assert evict(**{name: LENS}) == INVALID
    for name in ("w", "pos", "wo", "po", "lens", "lo"):
        assert evict(**{name: WORK}) == INVALID and evict(**{name: KO}) == INVALID
    for at in (K, V, KO, VO, W, POS, WO, PO):
        assert evict(work=at) == INVALID and evict(lo=at) == INVALID


def test_evict_workspace():
    need = ctypes.c_uint64()
    call = lambda *a: gtms.gtms_cache_evict_workspace(gtms.EvictShape(*a), ctypes.byref(need))  # noqa: E731
    assert call(2, 3, 100, 40, 64, 40, 0, 0, BF16) == OK and need.value >= 2 * 3 * 40 * 4
    assert call(2, 3, 30, 40, 64, 40, 0, 0, BF16) == OK and need.value >= 2 * 3 * 30 * 4
    assert call(2, 3, 30, 40, 64, 40, 30, 30, BF16) == INVALID
    assert gtms.gtms_cache_evict_workspace(None, ctypes.byref(need)) == INVALID
    assert gtms.gtms_cache_evict_workspace(gtms.EvictShape(2, 3, 100, 40, 64, 40, 0, 0, BF16), None) == INVALID


def test_what_stays_by_its_definition():
    w = [5.0, 1.0, 3.0, math.nan, 3.0, 0.0, -0.0, 9.0]
    assert evicted(w, 8, 8, 0, 0) == list(range(8)) and evicted(w, 3, 5, 1, 1) == [0, 1, 2]
    assert evicted(w, 8, 3, 0, 0) == [0, 3, 7] and evicted(w, 8, 3, 1, 1) == [0, 3, 7]
    assert evicted(w, 8, 4, 0, 0) == [0, 2, 3, 7] and evicted(w, 8, 3, 2, 1) == [0, 1, 7]
    assert evicted(w, 7, 6, 0, 0) == [0, 1, 2, 3, 4, 5]          # +0 and -0 tie


# ---------------------------------------------------------------------------
# The tensor calls' own checks
# ---------------------------------------------------------------------------

def test_tensor_calls_refuse_what_they_cannot_pass_on():
    q, k = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 9, 64, dtype=torch.bfloat16)
    lens = torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        gtms.attention_shared_prefix(q, k[:1], k[:1], k, k, lens)
    with pytest.raises(ValueError, match="CUDA"):
        gtms.attention_key_weights(q, k, torch.zeros(2, 4, 1), lens)
    with pytest.raises(ValueError, match="CUDA"):
        gtms.cache_evict(k, k, torch.zeros(2, 2, 9), lens, 4)
    with pytest.raises(ValueError, match="head_dim"):
        gtms.cache_evict(k[0], k, torch.zeros(2, 2, 9), lens, 4)
