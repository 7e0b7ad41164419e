"""The attention kernels' hand-offs and time limits: late warps, waits that are short beside an item."""
import ctypes
import os
import subprocess

import pytest
import torch

import masked_softmax_attention_gb300 as gtms

pytestmark = pytest.mark.gpu

TRIL, LENGTH = 0, 1


@pytest.fixture(scope="module")
def probe():
    """tests/attention_timing_probe.cu as a library of its own."""
    from masked_softmax_attention_gb300 import _build as b

    gtms.build_library()
    src = os.path.join(b.ROOT, "tests", "attention_timing_probe.cu")
    out_dir = os.path.join(b.ROOT, "_build", "test_probe")
    os.makedirs(out_dir, exist_ok=True)
    path = os.path.join(out_dir, "libgtms_attention_timing_probe.so")
    deps = [src] + [os.path.join(b.CSRC, f) for f in os.listdir(b.CSRC)] + [os.path.join(b.INCLUDE, "gtms.h")]
    if not os.path.exists(path) or any(os.path.getmtime(d) > os.path.getmtime(path) for d in deps):
        tmp = path + f".{os.getpid()}.tmp"
        subprocess.run([b.nvcc_path(), *b.ARCH, *b.NVCC_FLAGS, "-shared", src, "-o", tmp], check=True,
                       capture_output=True, text=True)
        os.replace(tmp, path)
    fn = ctypes.CDLL(path).gtms_test_attention_late
    vp, i32, u32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32
    fn.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, ctypes.c_float, i32, u32, u32, vp, vp, vp, ctypes.c_uint64]
    fn.restype = ctypes.c_int
    return fn


class Run:
    """One problem, its results from the normal build, and the probe's on the same inputs."""

    def __init__(self, B, Hq, Hkv, S, d, lens, mask, Sq=None):
        gen = torch.Generator(device="cuda").manual_seed(S + d)
        Sq = Sq or S
        self.q, self.k, self.v, self.dout = (
            torch.randn(B, H, n, d, generator=gen, device="cuda").to(torch.bfloat16)
            for H, n in ((Hq, Sq), (Hkv, S), (Hkv, S), (Hq, Sq)))
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.off = self.lens - Sq if Sq != S else torch.zeros_like(self.lens)
        self.mask, self.scale = mask, d ** -0.5
        options = dict(mask_kind=mask, q_offsets=self.off)
        self.o, self.lse = gtms.attention_forward(self.q, self.k, self.v, self.lens, self.scale, **options)
        self.grads = gtms.attention_backward(self.q, self.k, self.v, self.o, self.lse, self.dout, self.lens, self.scale,
                                             **options)

    def check(self, probe, backward, late_warps=0, late_ns=0, wait_ns=1_000_000_000):
        (B, Hq, Sq, d), (_, Hkv, S, _) = self.q.shape, self.k.shape
        o, lse = torch.full_like(self.o, 7.0), torch.full_like(self.lse, 7.0)
        grads = [torch.full_like(t, 7.0) for t in self.grads]
        tensors = (ctypes.c_void_p * 8)(*(t.data_ptr() for t in (
            self.q, self.k, self.v, self.o if backward else o, self.dout, *grads)))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        work = torch.empty(8 * (B * Hq * (Sq + 127) + 1024), dtype=torch.uint8, device="cuda")
        rc = probe(tensors, (self.lse if backward else lse).data_ptr(), self.lens.data_ptr(), self.off.data_ptr(), B, Hq,
                   Hkv, Sq, S, d, self.scale, self.mask, late_warps, late_ns, status.data_ptr(), work.data_ptr() if backward else None,
                   torch.cuda.current_stream().cuda_stream, wait_ns)
        torch.cuda.synchronize()
        assert rc == 0 and int(status.item()) == 0
        for got, want in zip(grads if backward else (o, lse), self.grads if backward else (self.o, self.lse)):
            assert torch.equal(got, want)


# Warps of a CTA, in order: 4 or 8 that work element by element (softmax, P and dS), then MMA, loads, deal.
@pytest.mark.parametrize("late", ["mma", "load", "deal", "first element-wise", "last element-wise", "mma and load"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("backward", [False, True])
def test_late_warps_change_nothing(probe, backward, d, late):
    """A role that is 20 us late at every wait, many times a tile's work, holds the others up and nothing else: no
    phase of a barrier may pass it by."""
    n = 8 if d == 128 else 4
    bits = {"mma": 1 << n, "load": 2 << n, "deal": 4 << n, "first element-wise": 1, "last element-wise": 1 << (n - 1),
            "mma and load": 3 << n}[late]
    Run(2, 4, 2, 700, d, (700, 613), TRIL).check(probe, backward, bits, 20_000)
    # sums of several parts: rows of many heads into dk and dv, many keys into o and dq
    if backward:
        Run(1, 130, 1, 1050, d, (1050,), LENGTH).check(probe, backward, bits, 5_000)
    Run(1, 16, 1, 140000, d, (140000,), LENGTH, 300).check(probe, backward, bits, 5_000)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("lens,mask", [((50000,), LENGTH), ((50000, 70), TRIL)])
def test_items_may_outlast_the_limit_of_a_wait(probe, lens, mask, backward, d):
    """The limit is that of a hand-off inside a tile (1 to 2 us of work), however many tiles an item has: here it is 120
    us and the items of some 400 tiles take three times that and more. There are more items than CTAs at once, so that
    the deal waits for whole items, and some in which a warp has no rows."""
    Run(len(lens), 2, 1, 50000, d, lens, mask).check(probe, backward, wait_ns=120_000)
