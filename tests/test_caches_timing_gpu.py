"""The hand-offs and time limits of the key-weight and shared-prefix kernels: late warps, waits that are short beside an
item, copies that never arrive."""
import ctypes
import os
import subprocess
import time

import pytest
import torch

import masked_softmax_attention_gb300 as gtms

pytestmark = pytest.mark.gpu

TRIL, LENGTH, WINDOW = 0, 1, 2
WEIGHTS, WHOLE, PACKED = 0, 1, 2


def _build(name, *flags):
    """tests/caches_probe.cu as a library of its own."""
    from masked_softmax_attention_gb300 import _build as b

    gtms.build_library()
    src = os.path.join(b.ROOT, "tests", "caches_probe.cu")
    out_dir = os.path.join(b.ROOT, "_build", "test_probe")
    os.makedirs(out_dir, exist_ok=True)
    path = os.path.join(out_dir, f"libgtms_{name}.so")
    deps = [src] + [os.path.join(b.CSRC, f) for f in os.listdir(b.CSRC)] + [os.path.join(b.INCLUDE, "gtms.h")]
    if not os.path.exists(path) or any(os.path.getmtime(d) > os.path.getmtime(path) for d in deps):
        tmp = path + f".{os.getpid()}.tmp"
        subprocess.run([b.nvcc_path(), *b.ARCH, *b.NVCC_FLAGS, *flags, "-shared", src, "-o", tmp], check=True,
                       capture_output=True, text=True)
        os.replace(tmp, path)
    fn = ctypes.CDLL(path).gtms_test_caches
    vp, i32, u32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32
    fn.argtypes = [i32, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, ctypes.c_float, i32, i32, u32, u32, vp, vp,
                   vp, ctypes.c_uint64]
    fn.restype = ctypes.c_int
    return fn


@pytest.fixture(scope="module")
def probe():
    return _build("caches_probe")


class Run:
    """One problem, its results from the normal build, and the probe's on the same inputs."""

    def __init__(self, what, B, Hq, Hkv, Sq, Skv, d, lens, mask=TRIL, window=0, G=1, P=0):
        gen = torch.Generator(device="cuda").manual_seed(Skv + d)
        self.q, self.k, self.v = (torch.randn(B, H, n, d, generator=gen, device="cuda").to(torch.bfloat16)
                                  for H, n in ((Hq, Sq), (Hkv, Skv), (Hkv, Skv)))
        self.kp, self.vp = (torch.randn(G, Hkv, P, d, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.off = self.lens - Sq if Sq != Skv else torch.zeros_like(self.lens)
        self.what, self.mask, self.window, self.scale = what, mask, window, d ** -0.5
        if what == WEIGHTS:
            self.lse = gtms.attention_forward(self.q, self.k, self.v, self.lens, self.scale, mask_kind=mask, window=window,
                                              q_offsets=self.off)[1]
            self.want = (gtms.attention_key_weights(self.q, self.k, self.lse, self.lens, self.scale, mask_kind=mask, window=window,
                                                    q_offsets=self.off),)
        else:
            self.want = gtms.attention_shared_prefix(self.q, self.kp, self.vp, self.k, self.v, self.lens, self.scale,
                                                     mask_kind=mask, q_offsets=self.off)

    def call(self, probe, late_warps=0, late_ns=0, wait_ns=1_000_000_000):
        """(status word, results)."""
        (B, Hq, Sq, d), (_, Hkv, Skv, _), (G, _, P, _) = self.q.shape, self.k.shape, self.kp.shape
        got = [torch.full_like(t, 7.0) for t in self.want]
        o = self.q if self.what == WEIGHTS else got[0]
        lse = self.lse if self.what == WEIGHTS else got[1]
        tensors = (ctypes.c_void_p * 6)(*(t.data_ptr() for t in (self.q, self.k, self.v, o, self.kp, self.vp)))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        work = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
        rc = probe(self.what, tensors, lse.data_ptr(), got[0].data_ptr(), self.lens.data_ptr(), self.off.data_ptr(), B, Hq, Hkv, Sq,
                   Skv, d, G, P, self.scale, self.mask, self.window, late_warps, late_ns, status.data_ptr(), work.data_ptr(),
                   torch.cuda.current_stream().cuda_stream, wait_ns)
        torch.cuda.synchronize()
        assert rc == 0
        return int(status.item()), got

    def check(self, probe, **kw):
        status, got = self.call(probe, **kw)
        assert status == 0
        for a, b in zip(got, self.want):
            assert torch.equal(a, b)


# Warps of a CTA, in order: 16 that sum, then MMA, loads, shifts, deal.
@pytest.mark.parametrize("late", [0x1, 0x8000, 0x00f0, 1 << 16, 1 << 17, 1 << 18, 1 << 19, 3 << 16, 5 << 16])
@pytest.mark.parametrize("d", [64, 128])
def test_late_warps_change_no_weights(probe, d, late):
    """A role that is 10 us late at every wait, many times a tile's work, holds the others up and nothing else: no phase of
    a barrier may pass it by."""
    Run(WEIGHTS, 2, 4, 2, 700, 700, d, (700, 613)).check(probe, late_warps=late, late_ns=10_000)
    Run(WEIGHTS, 2, 6, 2, 900, 900, d, (900, 300), WINDOW, 70).check(probe, late_warps=late, late_ns=10_000)
    Run(WEIGHTS, 8, 8, 4, 20, 9000, d, (9000, 700) * 4).check(probe, late_warps=late, late_ns=5_000)   # blocks put together


# 8 or 4 softmax warps, then MMA, loads, deal.
@pytest.mark.parametrize("late", ["mma", "load", "deal", "first softmax", "last softmax", "mma and load"])
@pytest.mark.parametrize("d", [64, 128])
def test_late_warps_change_no_rows_over_prefixes(probe, d, late):
    n = 8 if d == 128 else 4
    bits = {"mma": 1 << n, "load": 2 << n, "deal": 4 << n, "first softmax": 1, "last softmax": 1 << (n - 1),
            "mma and load": 3 << n}[late]
    Run(WHOLE, 4, 4, 2, 300, 300, d, (300, 0, 129, 7), G=2, P=600).check(probe, late_warps=bits, late_ns=20_000)
    Run(PACKED, 80, 16, 2, 1, 40, d, tuple(range(40)) * 2, G=2, P=5000).check(probe, late_warps=bits, late_ns=20_000)


# As above; a CTA's two tiles, where one holds all rows, on alternate tiles of keys, of which an item has 5 (one tile three
# of them, the other two) or 9; and P as two numbers, over 5 tiles of a prefix and 2 of a sequence's own keys.
@pytest.mark.parametrize("late", ["mma", "load", "deal", "first softmax", "last softmax", "mma and load", "one tile", "the other"])
@pytest.mark.parametrize("d", [64, 128])
def test_late_warps_change_no_small_calls_over_prefixes(probe, d, late):
    n = 8 if d == 128 else 4
    bits = {"mma": 1 << n, "load": 2 << n, "deal": 4 << n, "first softmax": 1, "last softmax": 1 << (n - 1),
            "mma and load": 3 << n, "one tile": 0x0f, "the other": 0xf0 if d == 128 else 0x01}[late]
    Run(PACKED, 16, 8, 2, 1, 40, d, tuple(range(25, 41)), G=2, P=5000).check(probe, late_warps=bits, late_ns=20_000)
    Run(PACKED, 32, 16, 8, 1, 40, d, tuple(range(9, 41)), G=4, P=3300).check(probe, late_warps=bits, late_ns=20_000)
    Run(WHOLE, 4, 4, 2, 1, 200, d, (200, 0, 129, 7), G=2, P=600).check(probe, late_warps=bits, late_ns=20_000)
    Run(WHOLE, 4, 4, 2, 100, 200, d, (200, 0, 129, 7), G=2, P=600).check(probe, late_warps=bits, late_ns=20_000)


@pytest.mark.parametrize("d", [64, 128])
def test_items_may_outlast_the_limit_of_a_wait(probe, d):
    """The limit is that of a hand-off inside a tile (1 to 2 us of work), however many tiles an item has: here it is 120 us,
    and items take several times that."""
    Run(WEIGHTS, 1, 16, 1, 30000, 30000, d, (30000,), LENGTH).check(probe, wait_ns=120_000)
    Run(WEIGHTS, 2, 64, 1, 20000, 20000, d, (20000, 300)).check(probe, wait_ns=120_000)
    Run(WHOLE, 1, 2, 1, 20000, 20000, d, (20000,), G=1, P=30000).check(probe, wait_ns=120_000)


@pytest.mark.parametrize("what", [WEIGHTS, WHOLE, PACKED])
@pytest.mark.parametrize("d", [64, 128])
def test_kernels_give_up_when_their_waits_run_out(probe, what, d):
    """Failure detection without a GPU fault: where no copy is issued, every wait runs out (after 200 us here). The launches
    must succeed, the grid must end promptly, also the CTAs that had not started, with GTMS_ERR_TIMEOUT in the status
    word, and a normal call right after it is exact."""
    without = _build("caches_no_loads_probe", "-DGTMS_ATTN_TMA_NO_LOADS=1")
    c = Run(what, 64, 32, 8, 1, 500, d, (500,) * 64, P=3000) if what == PACKED else \
        Run(what, 8, 16, 16, 1000, 1000, d, (1000,) * 8, P=0 if what == WEIGHTS else 500)
    t0 = time.monotonic()
    status, _ = c.call(without, wait_ns=200_000)
    assert status == gtms.GTMS_ERR_TIMEOUT and time.monotonic() - t0 < 5.0
    c.check(probe)
