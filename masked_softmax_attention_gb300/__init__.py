"""Grouped-tril masked softmax and attention for GB300 (sm_103a): thin Python binding of libgtms.

The compute runs in hand-written CUDA kernels behind the C ABI of
``include/gtms.h``. This module only marshals arguments: it passes device
pointers, sizes and the current CUDA stream to ``gtms_forward`` /
``gtms_backward`` and turns a non-zero status into an exception. There is no
CPU or PyTorch fallback: if ``libgtms.so`` is missing or cannot be loaded,
every call raises.

Operation ("Attention-Mask-Optimization" README, operator behaviour): for
X[B,M,S,S] and per-batch lengths L_b = seq_lens[b], row r keeps columns
c <= r when r < L_b; kept entries get softmax(scale * x), the rest +0.0.
Backward ("ops(8): self-attention 的 CUDA 实现及优化 (下)", section 2.1):
dx = scale * y * (dy - rowsum(dy * y)) on kept entries, +0.0 elsewhere.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

from ._build import LIB_PATH, build_library  # noqa: F401  (re-exported for build scripts)

GTMS_F32, GTMS_BF16, GTMS_F16 = 0, 1, 2
GTMS_OK, GTMS_ERR_INVALID_ARG, GTMS_ERR_UNSUPPORTED, GTMS_ERR_CUDA, GTMS_ERR_TIMEOUT = 0, 1, 2, 3, 4
GTMS_MAX_S = 65536
GTMS_MASK_GROUPED_TRIL, GTMS_MASK_LENGTH, GTMS_MASK_SLIDING_WINDOW = 0, 1, 2
GTMS_ATTENTION_MAX_S = 1 << 24
GTMS_ROTARY_PLAIN, GTMS_ROTARY_LINEAR, GTMS_ROTARY_BY_PARTS = 0, 1, 2

EXPORTED_SYMBOLS = ("gtms_forward", "gtms_backward", "gtms_status_string", "gtms_version",
                    "gtms_kernel_name", "gtms_kernel_name_masked", "gtms_kernel_name_explicit",
                    "gtms_device_pointer_of_host",
                    "gtms_forward_masked",
                    "gtms_backward_masked", "gtms_forward_explicit", "gtms_backward_explicit",
                    "gtms_attention_softmax_backward", "gtms_forward_staged",
                    "gtms_attention_forward", "gtms_attention_backward", "gtms_attention_backward_workspace",
                    "gtms_rotary", "gtms_rotary_frequencies",
                    "gtms_attention_shared_prefix", "gtms_attention_shared_prefix_workspace",
                    "gtms_attention_key_weights", "gtms_attention_key_weights_workspace",
                    "gtms_cache_evict", "gtms_cache_evict_workspace")

_lib = None
_lock = threading.Lock()


class Heads(ctypes.Structure):
    """``gtms_heads``: a strided [B, H, S, head_dim] tensor."""

    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64),
                ("stride_s", ctypes.c_int64)]


class AttentionShape(ctypes.Structure):
    """``gtms_attention_shape``: sizes and options of the attention calls."""

    _fields_ = [("B", ctypes.c_int64), ("Hq", ctypes.c_int64), ("Hkv", ctypes.c_int64), ("Sq", ctypes.c_int64),
                ("Skv", ctypes.c_int64), ("head_dim", ctypes.c_int64), ("window", ctypes.c_int64),
                ("mask_kind", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class EvictShape(ctypes.Structure):
    """``gtms_evict_shape``: sizes of an eviction from a cache."""

    _fields_ = [("B", ctypes.c_int64), ("H", ctypes.c_int64), ("S", ctypes.c_int64), ("S_out", ctypes.c_int64),
                ("head_dim", ctypes.c_int64), ("keep", ctypes.c_int64), ("first", ctypes.c_int64),
                ("recent", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class GtmsError(RuntimeError):
    """A libgtms call returned a non-zero status."""

    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libgtms.so (built in-tree by ``build_library``); raise if it is absent."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"libgtms.so not found at {p}: build it with "
                               "masked_softmax_attention_gb300.build_library() (needs nvcc); "
                               "there is no fallback implementation")
        lib = ctypes.CDLL(p)
        vp, i64 = ctypes.c_void_p, ctypes.c_int64
        lib.gtms_forward.argtypes = [vp, vp, vp, i64, i64, i64, ctypes.c_float, ctypes.c_int, vp]
        lib.gtms_forward.restype = ctypes.c_int
        lib.gtms_backward.argtypes = [vp, vp, vp, vp, i64, i64, i64, ctypes.c_float, ctypes.c_int, vp]
        lib.gtms_backward.restype = ctypes.c_int
        lib.gtms_forward_staged.argtypes = [vp, vp, vp, i64, i64, i64, ctypes.c_float, ctypes.c_int, vp]
        lib.gtms_forward_staged.restype = ctypes.c_int
        lib.gtms_forward_masked.argtypes = [vp, vp, vp, i64, i64, i64, ctypes.c_float, ctypes.c_int, i64,
                                            ctypes.c_int, vp]
        lib.gtms_forward_masked.restype = ctypes.c_int
        lib.gtms_backward_masked.argtypes = [vp, vp, vp, vp, i64, i64, i64, ctypes.c_float, ctypes.c_int, i64,
                                             ctypes.c_int, vp]
        lib.gtms_backward_masked.restype = ctypes.c_int
        lib.gtms_forward_explicit.argtypes = [vp, vp, vp, i64, i64, i64, i64, ctypes.c_float, ctypes.c_int, vp]
        lib.gtms_forward_explicit.restype = ctypes.c_int
        lib.gtms_backward_explicit.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, ctypes.c_float, ctypes.c_int, vp]
        lib.gtms_backward_explicit.restype = ctypes.c_int
        lib.gtms_attention_softmax_backward.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, ctypes.c_float,
                                                        ctypes.c_int, vp, vp]
        lib.gtms_attention_softmax_backward.restype = ctypes.c_int
        heads, shape = ctypes.POINTER(Heads), ctypes.POINTER(AttentionShape)
        lib.gtms_attention_forward.argtypes = [shape, heads, heads, heads, heads, vp, vp, vp, vp, vp]
        lib.gtms_attention_forward.restype = ctypes.c_int
        lib.gtms_attention_backward.argtypes = [shape, heads, heads, heads, heads, vp, heads, heads, heads, heads, vp,
                                                vp, vp, ctypes.c_uint64, vp, vp]
        lib.gtms_attention_backward.restype = ctypes.c_int
        lib.gtms_attention_backward_workspace.argtypes = [shape, ctypes.POINTER(ctypes.c_uint64)]
        lib.gtms_attention_backward_workspace.restype = ctypes.c_int
        lib.gtms_rotary.argtypes = [heads, heads, heads, heads, i64, i64, i64, i64, i64, i64, vp, i64, vp, ctypes.c_int,
                                    ctypes.c_float, ctypes.c_int, ctypes.c_int, vp]
        lib.gtms_rotary.restype = ctypes.c_int
        lib.gtms_rotary_frequencies.argtypes = [i64, ctypes.c_double, ctypes.c_int, ctypes.c_double, ctypes.c_double,
                                                ctypes.c_double, i64, vp]
        lib.gtms_rotary_frequencies.restype = ctypes.c_int
        u64p, evict = ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(EvictShape)
        lib.gtms_attention_shared_prefix.argtypes = [shape, i64, i64, heads, heads, heads, heads, heads, heads, vp, vp, vp,
                                                     vp, vp, ctypes.c_uint64, vp, vp]
        lib.gtms_attention_shared_prefix.restype = ctypes.c_int
        lib.gtms_attention_shared_prefix_workspace.argtypes = [shape, i64, i64, u64p]
        lib.gtms_attention_shared_prefix_workspace.restype = ctypes.c_int
        lib.gtms_attention_key_weights.argtypes = [shape, heads, heads, vp, vp, ctypes.c_int, vp, vp, vp, ctypes.c_uint64,
                                                   vp, vp]
        lib.gtms_attention_key_weights.restype = ctypes.c_int
        lib.gtms_attention_key_weights_workspace.argtypes = [shape, u64p]
        lib.gtms_attention_key_weights_workspace.restype = ctypes.c_int
        lib.gtms_cache_evict.argtypes = [evict, heads, heads, vp, vp, heads, heads, vp, vp, vp, vp, vp, ctypes.c_uint64, vp]
        lib.gtms_cache_evict.restype = ctypes.c_int
        lib.gtms_cache_evict_workspace.argtypes = [evict, u64p]
        lib.gtms_cache_evict_workspace.restype = ctypes.c_int
        lib.gtms_status_string.argtypes = [ctypes.c_int]
        lib.gtms_status_string.restype = ctypes.c_char_p
        lib.gtms_version.argtypes = []
        lib.gtms_version.restype = ctypes.c_int
        lib.gtms_kernel_name.argtypes = [ctypes.c_int, i64, ctypes.c_int, ctypes.c_int]
        lib.gtms_kernel_name.restype = ctypes.c_char_p
        lib.gtms_kernel_name_masked.argtypes = [ctypes.c_int, i64, ctypes.c_int, ctypes.c_int, ctypes.c_int, i64]
        lib.gtms_kernel_name_masked.restype = ctypes.c_char_p
        lib.gtms_kernel_name_explicit.argtypes = [ctypes.c_int, i64, ctypes.c_int]
        lib.gtms_kernel_name_explicit.restype = ctypes.c_char_p
        lib.gtms_device_pointer_of_host.argtypes = [vp, ctypes.POINTER(ctypes.c_void_p)]
        lib.gtms_device_pointer_of_host.restype = ctypes.c_int
        if path is None:
            _lib = lib
        return lib


# ---------------------------------------------------------------------------
# Raw C-ABI calls: integer pointers in, status code out.
# ---------------------------------------------------------------------------

def gtms_forward(x, y, seq_lens, B, M, S, scale, dtype, stream) -> int:
    return load_library().gtms_forward(x, y, seq_lens, B, M, S, scale, dtype, stream)


def gtms_backward(y, dy, dx, seq_lens, B, M, S, scale, dtype, stream) -> int:
    return load_library().gtms_backward(y, dy, dx, seq_lens, B, M, S, scale, dtype, stream)


def gtms_forward_staged(x, y, seq_lens, B, M, S, scale, dtype, stream) -> int:
    return load_library().gtms_forward_staged(x, y, seq_lens, B, M, S, scale, dtype, stream)


def gtms_forward_masked(x, y, seq_lens, B, M, S, scale, mask_kind, window, dtype, stream) -> int:
    return load_library().gtms_forward_masked(x, y, seq_lens, B, M, S, scale, mask_kind, window, dtype, stream)


def gtms_backward_masked(y, dy, dx, seq_lens, B, M, S, scale, mask_kind, window, dtype, stream) -> int:
    return load_library().gtms_backward_masked(y, dy, dx, seq_lens, B, M, S, scale, mask_kind, window, dtype, stream)


def gtms_forward_explicit(x, y, mask, mask_batches, B, M, S, scale, dtype, stream) -> int:
    return load_library().gtms_forward_explicit(x, y, mask, mask_batches, B, M, S, scale, dtype, stream)


def gtms_backward_explicit(y, dy, dx, mask, mask_batches, B, M, S, scale, dtype, stream) -> int:
    return load_library().gtms_backward_explicit(y, dy, dx, mask, mask_batches, B, M, S, scale, dtype, stream)


def gtms_attention_softmax_backward(p, dout, v, ds, seq_lens, B, M, S, head_dim, scale, dtype, status,
                                    stream) -> int:
    return load_library().gtms_attention_softmax_backward(p, dout, v, ds, seq_lens, B, M, S, head_dim, scale, dtype,
                                                          status, stream)


def gtms_attention_forward(shape, q, k, v, o, lse, seq_lens, q_offsets, status, stream) -> int:
    return load_library().gtms_attention_forward(shape, q, k, v, o, lse, seq_lens, q_offsets, status, stream)


def gtms_attention_backward(shape, q, k, v, o, lse, dout, dq, dk, dv, seq_lens, q_offsets, workspace, workspace_bytes,
                            status, stream) -> int:
    return load_library().gtms_attention_backward(shape, q, k, v, o, lse, dout, dq, dk, dv, seq_lens, q_offsets,
                                                  workspace, workspace_bytes, status, stream)


def gtms_attention_backward_workspace(shape, num_bytes) -> int:
    return load_library().gtms_attention_backward_workspace(shape, num_bytes)


def gtms_rotary(x, y, x2, y2, B, H, H2, S, head_dim, rot_dim, positions, position_batches, inv_freq, interleaved,
                amplitude, inverse, dtype, stream) -> int:
    return load_library().gtms_rotary(x, y, x2, y2, B, H, H2, S, head_dim, rot_dim, positions, position_batches,
                                      inv_freq, interleaved, amplitude, inverse, dtype, stream)


def gtms_rotary_frequencies(rot_dim, base, scaling, factor, low_turns, high_turns, original_length, inv_freq) -> int:
    return load_library().gtms_rotary_frequencies(rot_dim, base, scaling, factor, low_turns, high_turns,
                                                  original_length, inv_freq)


def gtms_attention_shared_prefix(shape, groups, prefix, q, k_prefix, v_prefix, k, v, o, lse, prefix_lens, seq_lens,
                                 q_offsets, workspace, workspace_bytes, status, stream) -> int:
    return load_library().gtms_attention_shared_prefix(shape, groups, prefix, q, k_prefix, v_prefix, k, v, o, lse,
                                                       prefix_lens, seq_lens, q_offsets, workspace, workspace_bytes,
                                                       status, stream)


def gtms_attention_shared_prefix_workspace(shape, groups, prefix, num_bytes) -> int:
    return load_library().gtms_attention_shared_prefix_workspace(shape, groups, prefix, num_bytes)


def gtms_attention_key_weights(shape, q, k, lse, weights, accumulate, seq_lens, q_offsets, workspace, workspace_bytes,
                               status, stream) -> int:
    return load_library().gtms_attention_key_weights(shape, q, k, lse, weights, accumulate, seq_lens, q_offsets,
                                                     workspace, workspace_bytes, status, stream)


def gtms_attention_key_weights_workspace(shape, num_bytes) -> int:
    return load_library().gtms_attention_key_weights_workspace(shape, num_bytes)


def gtms_cache_evict(shape, k, v, weights, positions, k_out, v_out, weights_out, positions_out, seq_lens, lens_out,
                     workspace, workspace_bytes, stream) -> int:
    return load_library().gtms_cache_evict(shape, k, v, weights, positions, k_out, v_out, weights_out, positions_out,
                                           seq_lens, lens_out, workspace, workspace_bytes, stream)


def gtms_cache_evict_workspace(shape, num_bytes) -> int:
    return load_library().gtms_cache_evict_workspace(shape, num_bytes)


def status_string(status: int) -> str:
    return load_library().gtms_status_string(status).decode()


def gtms_version() -> int:
    return load_library().gtms_version()


def kernel_name(direction: int, S: int, dtype: int, aligned16: bool = True) -> str:
    return load_library().gtms_kernel_name(direction, S, dtype, 1 if aligned16 else 0).decode()


def kernel_name_masked(direction: int, S: int, dtype: int, mask_kind: int, window: int = 0,
                       aligned16: bool = True) -> str:
    return load_library().gtms_kernel_name_masked(direction, S, dtype, 1 if aligned16 else 0, mask_kind,
                                                  window).decode()


def kernel_name_explicit(direction: int, S: int, dtype: int) -> str:
    return load_library().gtms_kernel_name_explicit(direction, S, dtype).decode()


def device_pointer_of_host(host_ptr: int) -> int:
    """Device address of a page-locked host buffer (``gtms_device_pointer_of_host``)."""
    out = ctypes.c_void_p()
    rc = load_library().gtms_device_pointer_of_host(host_ptr, ctypes.byref(out))
    if rc != GTMS_OK:
        raise GtmsError("gtms_device_pointer_of_host", rc)
    return out.value


# ---------------------------------------------------------------------------
# Tensor API (torch provides device memory and the stream, nothing else).
# ---------------------------------------------------------------------------

_dtype_codes: dict = {}


def _dtype_code(t) -> int:
    if not _dtype_codes:
        import torch

        _dtype_codes.update({torch.float32: GTMS_F32, torch.bfloat16: GTMS_BF16, torch.float16: GTMS_F16})
    code = _dtype_codes.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}; expected float32, bfloat16 or float16")
    return code


def _check_scores(name, t):
    if t.dim() != 4 or t.shape[-1] != t.shape[-2]:
        raise ValueError(f"{name} must be [B, M, S, S], got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_lens(seq_lens, B, device):
    import torch

    if seq_lens.dtype != torch.int32 or seq_lens.shape != (B,) or seq_lens.device != device \
            or not seq_lens.is_contiguous():
        raise ValueError("seq_lens must be a contiguous int32 CUDA tensor of shape [B] on the scores' device")


def forward(x, seq_lens, scale: float = 1.0, out=None, mask_kind: int = GTMS_MASK_GROUPED_TRIL, window: int = 0):
    """y = masked softmax(scale * x) (grouped tril by default); ``out`` may be ``x`` (in place)."""
    import torch

    _check_scores("x", x)
    B, M, S, _ = x.shape
    _check_lens(seq_lens, B, x.device)
    y = torch.empty_like(x) if out is None else out
    if y.shape != x.shape or y.dtype != x.dtype or y.device != x.device or not y.is_contiguous():
        raise ValueError("out must match x in shape, dtype, device and be contiguous")
    stream = torch.cuda.current_stream(x.device).cuda_stream
    rc = gtms_forward_masked(x.data_ptr(), y.data_ptr(), seq_lens.data_ptr(), B, M, S, float(scale),
                             int(mask_kind), int(window), _dtype_code(x), stream)
    if rc != GTMS_OK:
        raise GtmsError("gtms_forward_masked", rc)
    return y


def forward_staged(x, seq_lens, scale: float = 1.0, out=None):
    """``forward`` computed by the staged kernel (gtms_forward_staged: rows brought into shared
    memory by TMA bulk copies); the same values within the parity tolerances."""
    import torch

    _check_scores("x", x)
    B, M, S, _ = x.shape
    _check_lens(seq_lens, B, x.device)
    y = torch.empty_like(x) if out is None else out
    if y.shape != x.shape or y.dtype != x.dtype or y.device != x.device or not y.is_contiguous():
        raise ValueError("out must match x in shape, dtype, device and be contiguous")
    stream = torch.cuda.current_stream(x.device).cuda_stream
    rc = gtms_forward_staged(x.data_ptr(), y.data_ptr(), seq_lens.data_ptr(), B, M, S, float(scale), _dtype_code(x),
                             stream)
    if rc != GTMS_OK:
        raise GtmsError("gtms_forward_staged", rc)
    return y


def backward(y, dy, seq_lens, scale: float = 1.0, out=None, mask_kind: int = GTMS_MASK_GROUPED_TRIL,
             window: int = 0):
    """dx = scale * y * (dy - rowsum(dy * y)) under the mask; ``out`` may be ``y`` or ``dy``."""
    import torch

    _check_scores("y", y)
    _check_scores("dy", dy)
    if dy.shape != y.shape or dy.dtype != y.dtype or dy.device != y.device:
        raise ValueError("dy must match y in shape, dtype and device")
    B, M, S, _ = y.shape
    _check_lens(seq_lens, B, y.device)
    dx = torch.empty_like(y) if out is None else out
    if dx.shape != y.shape or dx.dtype != y.dtype or dx.device != y.device or not dx.is_contiguous():
        raise ValueError("out must match y in shape, dtype, device and be contiguous")
    stream = torch.cuda.current_stream(y.device).cuda_stream
    rc = gtms_backward_masked(y.data_ptr(), dy.data_ptr(), dx.data_ptr(), seq_lens.data_ptr(), B, M, S,
                              float(scale), int(mask_kind), int(window), _dtype_code(y), stream)
    if rc != GTMS_OK:
        raise GtmsError("gtms_backward_masked", rc)
    return dx


def _check_mask(mask, B, S, device):
    import torch

    if mask.dtype != torch.uint8 or mask.dim() != 3 or mask.shape[1:] != (S, S) or mask.shape[0] not in (1, B) \
            or mask.device != device or not mask.is_contiguous():
        raise ValueError("mask must be a contiguous uint8 CUDA tensor [1 or B, S, S] on the scores' device")


def forward_explicit(x, mask, scale: float = 1.0, out=None):
    """Softmax of scale * x over the entries whose mask byte is nonzero (mask uint8 [1 or B, S, S],
    shared by the heads); +0.0 elsewhere, all-masked rows zero. ``out`` may be ``x``."""
    import torch

    _check_scores("x", x)
    B, M, S, _ = x.shape
    _check_mask(mask, B, S, x.device)
    y = torch.empty_like(x) if out is None else out
    if y.shape != x.shape or y.dtype != x.dtype or y.device != x.device or not y.is_contiguous():
        raise ValueError("out must match x in shape, dtype, device and be contiguous")
    stream = torch.cuda.current_stream(x.device).cuda_stream
    rc = gtms_forward_explicit(x.data_ptr(), y.data_ptr(), mask.data_ptr(), mask.shape[0], B, M, S, float(scale),
                               _dtype_code(x), stream)
    if rc != GTMS_OK:
        raise GtmsError("gtms_forward_explicit", rc)
    return y


def backward_explicit(y, dy, mask, scale: float = 1.0, out=None):
    """Backward of forward_explicit over the same kept entries; ``out`` may be ``y`` or ``dy``."""
    import torch

    _check_scores("y", y)
    _check_scores("dy", dy)
    if dy.shape != y.shape or dy.dtype != y.dtype or dy.device != y.device:
        raise ValueError("dy must match y in shape, dtype and device")
    B, M, S, _ = y.shape
    _check_mask(mask, B, S, y.device)
    dx = torch.empty_like(y) if out is None else out
    if dx.shape != y.shape or dx.dtype != y.dtype or dx.device != y.device or not dx.is_contiguous():
        raise ValueError("out must match y in shape, dtype, device and be contiguous")
    stream = torch.cuda.current_stream(y.device).cuda_stream
    rc = gtms_backward_explicit(y.data_ptr(), dy.data_ptr(), dx.data_ptr(), mask.data_ptr(), mask.shape[0], B, M, S,
                                float(scale), _dtype_code(y), stream)
    if rc != GTMS_OK:
        raise GtmsError("gtms_backward_explicit", rc)
    return dx


def attention_softmax_backward(p, dout, v, seq_lens, scale: float = 1.0, out=None, status=None):
    """dS = scale * P * (dO V^T - rowsum(dO V^T * P)) on the grouped-tril kept entries, with the GEMM on the
    tensor cores; ``p`` [B,M,S,S], ``dout`` / ``v`` [B,M,S,d] (d 64 or 128), bf16 or fp16. ``status`` (an
    optional int32 CUDA tensor of one element, cleared before the call) receives ``GTMS_ERR_TIMEOUT`` if an internal
    wait of the kernel ran out."""
    import torch

    _check_scores("p", p)
    B, M, S, _ = p.shape
    for name, t in (("dout", dout), ("v", v)):
        if t.dim() != 4 or t.shape[:3] != p.shape[:3] or t.dtype != p.dtype or t.device != p.device \
                or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [B, M, S, d] tensor matching p")
    if dout.shape != v.shape:
        raise ValueError("dout and v must have the same shape")
    _check_lens(seq_lens, B, p.device)
    ds = torch.empty_like(p) if out is None else out
    if ds.shape != p.shape or ds.dtype != p.dtype or ds.device != p.device or not ds.is_contiguous():
        raise ValueError("out must match p in shape, dtype, device and be contiguous")
    stream = torch.cuda.current_stream(p.device).cuda_stream
    rc = gtms_attention_softmax_backward(p.data_ptr(), dout.data_ptr(), v.data_ptr(), ds.data_ptr(),
                                         seq_lens.data_ptr(), B, M, S, dout.shape[3], float(scale), _dtype_code(p),
                                         None if status is None else status.data_ptr(), stream)
    if rc != GTMS_OK:
        raise GtmsError("gtms_attention_softmax_backward", rc)
    return ds


def attention_softmax_backward_host(p, dout, v, seq_lens, scale: float = 1.0, out=None, status=None, device=None):
    """``attention_softmax_backward`` on pinned host tensors: the kernel reads P, dO, V and writes dS in host
    memory (see ``forward_host``). ``status``, if given, is an int32 CUDA tensor of one element."""
    import torch

    for name, t in (("p", p), ("dout", dout), ("v", v), ("seq_lens", seq_lens)):
        _check_pinned(name, t)
    if p.dim() != 4 or p.shape[-1] != p.shape[-2] or dout.dim() != 4 or dout.shape != v.shape \
            or dout.shape[:3] != p.shape[:3] or dout.dtype != p.dtype or v.dtype != p.dtype:
        raise ValueError("p must be [B, M, S, S]; dout and v [B, M, S, d] of p's dtype")
    if seq_lens.dtype != torch.int32 or seq_lens.shape != p.shape[:1]:
        raise ValueError("seq_lens must be int32 [B]")
    ds = torch.empty_like(p).pin_memory() if out is None else out
    _check_pinned("out", ds)
    B, M, S, _ = p.shape
    stream = torch.cuda.current_stream(device).cuda_stream
    dp = device_pointer_of_host
    rc = gtms_attention_softmax_backward(dp(p.data_ptr()), dp(dout.data_ptr()), dp(v.data_ptr()),
                                         dp(ds.data_ptr()), dp(seq_lens.data_ptr()), B, M, S, dout.shape[3],
                                         float(scale), _dtype_code(p), None if status is None else status.data_ptr(),
                                         stream)
    if rc != GTMS_OK:
        raise GtmsError("gtms_attention_softmax_backward", rc)
    return ds


def _check_pinned(name, t):
    if t.is_cuda or not t.is_pinned() or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous page-locked (pinned) CPU tensor")


def forward_host(x, seq_lens, scale: float = 1.0, out=None, device=None):
    """Forward on pinned host tensors: the kernels read x and write y in host memory.

    ``x`` [B,M,S,S], ``seq_lens`` int32 [B] and ``out`` (allocated pinned if
    omitted) stay in page-locked host memory; the call is enqueued on the
    current stream of ``device`` and returns at once (synchronise before
    reading ``out``).
    """
    import torch

    _check_pinned("x", x)
    _check_pinned("seq_lens", seq_lens)
    if x.dim() != 4 or x.shape[-1] != x.shape[-2] or seq_lens.dtype != torch.int32 or seq_lens.shape != x.shape[:1]:
        raise ValueError("x must be [B, M, S, S] and seq_lens int32 [B]")
    y = torch.empty_like(x).pin_memory() if out is None else out
    _check_pinned("out", y)
    B, M, S, _ = x.shape
    stream = torch.cuda.current_stream(device).cuda_stream
    rc = gtms_forward(device_pointer_of_host(x.data_ptr()), device_pointer_of_host(y.data_ptr()),
                      device_pointer_of_host(seq_lens.data_ptr()), B, M, S, float(scale), _dtype_code(x), stream)
    if rc != GTMS_OK:
        raise GtmsError("gtms_forward", rc)
    return y


def backward_host(y, dy, seq_lens, scale: float = 1.0, out=None, device=None):
    """Backward on pinned host tensors (see ``forward_host``)."""
    import torch

    for name, t in (("y", y), ("dy", dy), ("seq_lens", seq_lens)):
        _check_pinned(name, t)
    if dy.shape != y.shape or dy.dtype != y.dtype or y.dim() != 4 or seq_lens.dtype != torch.int32 \
            or seq_lens.shape != y.shape[:1]:
        raise ValueError("y and dy must be matching [B, M, S, S] tensors and seq_lens int32 [B]")
    dx = torch.empty_like(y).pin_memory() if out is None else out
    _check_pinned("out", dx)
    B, M, S, _ = y.shape
    stream = torch.cuda.current_stream(device).cuda_stream
    rc = gtms_backward(device_pointer_of_host(y.data_ptr()), device_pointer_of_host(dy.data_ptr()),
                       device_pointer_of_host(dx.data_ptr()), device_pointer_of_host(seq_lens.data_ptr()),
                       B, M, S, float(scale), _dtype_code(y), stream)
    if rc != GTMS_OK:
        raise GtmsError("gtms_backward", rc)
    return dx


def _autograd_function():
    import torch

    class GroupedTrilMaskSoftmax(torch.autograd.Function):
        """Autograd wrapper: forward and backward both run the CUDA kernels."""

        @staticmethod
        def forward(ctx, x, seq_lens, scale):
            y = forward(x.contiguous(), seq_lens, scale)
            ctx.save_for_backward(y, seq_lens)
            ctx.scale = scale
            return y

        @staticmethod
        def backward(ctx, dy):
            y, seq_lens = ctx.saved_tensors
            return backward(y, dy.contiguous(), seq_lens, ctx.scale), None, None

    return GroupedTrilMaskSoftmax


_fn = None


def grouped_tril_mask_softmax(x, seq_lens, scale: float = 1.0):
    """Differentiable op: ``y = grouped_tril_mask_softmax(x, seq_lens, scale)``."""
    global _fn
    if _fn is None:
        _fn = _autograd_function()
    return _fn.apply(x, seq_lens, float(scale))


# ---------------------------------------------------------------------------
# Attention and rotary positions: strided [B, H, S, head_dim] tensors.
# ---------------------------------------------------------------------------

_pack_heads = struct.Struct("@P3q").pack            # gtms_heads
_pack_shape = struct.Struct("@7q2if4x").pack        # gtms_attention_shape
_direct_calls: dict = {}


def _direct(name):
    """The entry point taking its structures as packed bytes (building ctypes objects costs more than a launch)."""
    fn = _direct_calls.get(name)
    if fn is None:
        lib = load_library()
        fn = lib[name]
        plain = getattr(lib, name).argtypes
        fn.argtypes = [ctypes.c_void_p if hasattr(t, "contents") else t for t in plain]
        fn.restype = ctypes.c_int
        _direct_calls[name] = fn
    return fn


def _heads(name, t, dtype, device):
    """Packed ``gtms_heads`` of a tensor, after the checks that only the tensor itself allows."""
    strides = t.stride()
    if len(strides) != 4:
        raise ValueError(f"{name} must be [B, H, S, head_dim], got {tuple(t.shape)}")
    if t.get_device() != device or device < 0:
        raise ValueError(f"{name} must be a CUDA tensor on the same device as the others")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be of the same dtype as the others")
    if strides[3] != 1 and t.shape[3] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return _pack_heads(t.data_ptr(), strides[0], strides[1], strides[2])


_int32_dtype = _uint8_dtype = None


def _uint8():
    global _uint8_dtype
    if _uint8_dtype is None:
        import torch

        _uint8_dtype = torch.uint8
    return _uint8_dtype


def _int32(name, t, shape, device):
    """Address of an optional contiguous int32 tensor."""
    global _int32_dtype
    if t is None:
        return None
    if _int32_dtype is None:
        import torch

        _int32_dtype = torch.int32
    if t.dtype is not _int32_dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor of shape {tuple(shape)} on the same device")
    return t.data_ptr()


def _launch(fn, device, *args):
    """The call on the current stream of the tensors' device, made the current one where it is not already."""
    import torch

    call, c = _direct_calls.get(fn) or _direct(fn), torch._C
    stream = c._cuda_getCurrentRawStream(device)
    if c._cuda_getDevice() == device:
        rc = call(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = call(*args, stream)
    if rc:
        raise GtmsError(fn, rc)


def _attention_shape(q, k, v, scale, mask_kind, window):
    B, Hq, Sq, d = q.shape
    kb, Hkv, Skv, kd = ks = k.shape
    if ks != v.shape or kb != B or kd != d:
        raise ValueError(f"k and v must be [B, Hkv, Skv, head_dim] matching q, got {tuple(ks)} and {tuple(v.shape)}")
    return B, Sq, _pack_shape(B, Hq, Hkv, Sq, Skv, d, int(window), int(mask_kind), _dtype_code(q), scale)


def attention_forward(q, k, v, seq_lens, scale: float = 1.0, out=None, mask_kind: int = GTMS_MASK_GROUPED_TRIL,
                      window: int = 0, q_offsets=None, status=None):
    """(o, lse) of attention under a mask family, the scores staying on the chip (gtms_attention_forward).

    ``q`` [B, Hq, Sq, d], ``k`` / ``v`` [B, Hkv, Skv, d] (bf16 or fp16, d 64 or 128, Hq a multiple of Hkv) with a
    contiguous last dimension, strides that are multiples of 8 elements and data on 16 bytes (a batch or head may be
    expanded); others are refused, not copied. ``o`` is laid out like ``q``, ``lse`` is fp32 [B, Hq, Sq]. Row i of
    batch b stands at position i, or ``q_offsets[b] + i``: for new tokens over a cache pass the cache as ``k`` and
    ``v``, the lengths with the new tokens as ``seq_lens`` and ``seq_lens - Sq`` as ``q_offsets``. Rows that keep
    nothing give o = 0 and lse = -inf. ``status`` as in ``attention_softmax_backward``."""
    import torch

    dtype, dev = q.dtype, q.get_device()
    q_, k_, v_ = _heads("q", q, dtype, dev), _heads("k", k, dtype, dev), _heads("v", v, dtype, dev)
    B, Sq, shape = _attention_shape(q, k, v, scale, mask_kind, window)
    lens, off = _int32("seq_lens", seq_lens, (B,), dev), _int32("q_offsets", q_offsets, (B,), dev)
    status = _int32("status", status, (1,), dev)
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape:
        raise ValueError("out must match q in shape")
    lse = torch.empty((B, q.shape[1], Sq), dtype=torch.float32, device=q.device)
    _launch("gtms_attention_forward", dev, shape, q_, k_, v_, _heads("out", out, dtype, dev), lse.data_ptr(), lens, off,
            status)
    return out, lse


def attention_backward(q, k, v, o, lse, dout, seq_lens, scale: float = 1.0, out=None,
                       mask_kind: int = GTMS_MASK_GROUPED_TRIL, window: int = 0, q_offsets=None, status=None):
    """(dq, dk, dv) of ``attention_forward``, the probabilities recomputed from ``lse`` (gtms_attention_backward);
    dk and dv are summed over the query heads that share them. The same inputs give the same bits. ``out`` is an
    optional triple of tensors to write to."""
    import torch

    dtype, dev, shape4 = q.dtype, q.get_device(), q.shape
    q_, k_, v_ = _heads("q", q, dtype, dev), _heads("k", k, dtype, dev), _heads("v", v, dtype, dev)
    B, _, shape = _attention_shape(q, k, v, scale, mask_kind, window)
    lens, off = _int32("seq_lens", seq_lens, (B,), dev), _int32("q_offsets", q_offsets, (B,), dev)
    status = _int32("status", status, (1,), dev)
    if o.shape != shape4 or dout.shape != shape4:
        raise ValueError("o and dout must match q in shape")
    if lse.dtype is not torch.float32 or lse.shape != shape4[:3] or lse.get_device() != dev or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 tensor [B, Hq, Sq] on q's device")
    if out is None:
        out = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dq, dk, dv = out
    if dq.shape != shape4 or dk.shape != k.shape or dv.shape != k.shape:
        raise ValueError("dq, dk and dv must match q, k and v in shape")
    need = ctypes.c_uint64()
    rc = _direct("gtms_attention_backward_workspace")(shape, ctypes.byref(need))
    if rc != GTMS_OK:
        raise GtmsError("gtms_attention_backward_workspace", rc)
    workspace = torch.empty(need.value, dtype=torch.uint8, device=q.device)
    _launch("gtms_attention_backward", dev, shape, q_, k_, v_, _heads("o", o, dtype, dev), lse.data_ptr(),
            _heads("dout", dout, dtype, dev), _heads("dq", dq, dtype, dev), _heads("dk", dk, dtype, dev),
            _heads("dv", dv, dtype, dev), lens, off, workspace.data_ptr(), need.value, status)
    return dq, dk, dv


# ---------------------------------------------------------------------------
# Caches: prefixes that a batch shares, the weight that keys received, eviction. Calls of serving: none of them is
# differentiable.
# ---------------------------------------------------------------------------

_pack_evict = struct.Struct("@8qi4x").pack          # gtms_evict_shape


_workspace_sizes: dict = {}


def _workspace(fn, like, *shape):
    """(tensor, address, bytes) of the workspace that a call of this shape needs, on the device of ``like``; the tensor
    is to outlive the call. The bytes follow from the shape alone, and asking costs as much as a launch's checks."""
    key = fn, *shape
    size = _workspace_sizes.get(key)
    if size is None:
        need = ctypes.c_uint64()
        rc = (_direct_calls.get(fn) or _direct(fn))(*shape, ctypes.byref(need))
        if rc != GTMS_OK:
            raise GtmsError(fn, rc)
        if len(_workspace_sizes) >= 1024:
            _workspace_sizes.clear()
        size = _workspace_sizes[key] = need.value
    if size == 0:
        return None, None, 0
    t = like.new_empty(size, dtype=_uint8())
    return t, t.data_ptr(), size


def _labels(name, t, dtype, shape, device):
    """Address of a contiguous tensor with one element to a cache entry."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {tuple(shape)} on the same device")
    return t.data_ptr()


def attention_shared_prefix(q, k_prefix, v_prefix, k, v, seq_lens, scale: float = 1.0, out=None,
                            mask_kind: int = GTMS_MASK_GROUPED_TRIL, q_offsets=None, prefix_lens=None, status=None):
    """(o, lse) of attention for a batch whose sequences share long prefixes (gtms_attention_shared_prefix): as
    ``attention_forward`` over the keys of a sequence's prefix and its own put end to end.

    ``k_prefix`` / ``v_prefix`` [G, Hkv, P, d]: of the batch of B = G n sequences, sequence b has prefix b // n, of
    which the first ``prefix_lens[b // n]`` keys (int32 [G]; all without it) are seen by each of its live rows.
    ``seq_lens`` and ``q_offsets`` count the sequences' own keys ``k`` / ``v`` [B, Hkv, Skv, d]. Masks: grouped tril or
    length. Everything else as in ``attention_forward``; like its, the results carry no gradient, whatever the inputs
    ask for (``attention`` over the keys put end to end has one)."""
    import torch

    dtype, dev = q.dtype, q.get_device()
    q_, k_, v_ = _heads("q", q, dtype, dev), _heads("k", k, dtype, dev), _heads("v", v, dtype, dev)
    kp_, vp_ = _heads("k_prefix", k_prefix, dtype, dev), _heads("v_prefix", v_prefix, dtype, dev)
    B, Sq, shape = _attention_shape(q, k, v, scale, mask_kind, 0)
    G, Hkv, P, d = ps = k_prefix.shape
    if ps != v_prefix.shape or Hkv != k.shape[1] or d != k.shape[3]:
        raise ValueError(f"k_prefix and v_prefix must be [G, Hkv, P, head_dim] matching k, got {tuple(ps)} and "
                         f"{tuple(v_prefix.shape)}")
    lens, off = _int32("seq_lens", seq_lens, (B,), dev), _int32("q_offsets", q_offsets, (B,), dev)
    plens, status = _int32("prefix_lens", prefix_lens, (G,), dev), _int32("status", status, (1,), dev)
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape:
        raise ValueError("out must match q in shape")
    lse = q.new_empty((B, q.shape[1], Sq), dtype=torch.float32)
    _keep, work, size = _workspace("gtms_attention_shared_prefix_workspace", q, shape, G, P)
    _launch("gtms_attention_shared_prefix", dev, shape, G, P, q_, kp_, vp_, k_, v_, _heads("out", out, dtype, dev),
            lse.data_ptr(), plens, lens, off, work, size, status)
    return out, lse


def attention_key_weights(q, k, lse, seq_lens, scale: float = 1.0, out=None, accumulate: bool = False,
                          mask_kind: int = GTMS_MASK_GROUPED_TRIL, window: int = 0, q_offsets=None, status=None):
    """The weight that each key received, fp32 [B, Hkv, Skv] (gtms_attention_key_weights): its probabilities summed over
    the rows that keep it and the query heads that share it, recomputed from the ``lse`` that ``attention_forward``
    (or ``attention_shared_prefix``) returned for these rows.

    ``out``, a contiguous fp32 tensor, receives the weights; with ``accumulate`` they are added to what stands there,
    and entries at and behind ``seq_lens`` stay: set those of new keys to 0 first, since after an eviction an older key's
    may stand in their place. The same inputs give the same bits. ``q``, ``k`` and the options as in
    ``attention_forward``."""
    import torch

    dtype, dev = q.dtype, q.get_device()
    q_, k_ = _heads("q", q, dtype, dev), _heads("k", k, dtype, dev)
    B, Sq, shape = _attention_shape(q, k, k, scale, mask_kind, window)
    lens, off = _int32("seq_lens", seq_lens, (B,), dev), _int32("q_offsets", q_offsets, (B,), dev)
    status = _int32("status", status, (1,), dev)
    lse_ = _labels("lse", lse, torch.float32, (B, q.shape[1], Sq), dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty(k.shape[:3], dtype=torch.float32, device=q.device)
    out_ = _labels("out", out, torch.float32, k.shape[:3], dev)
    _keep, work, size = _workspace("gtms_attention_key_weights_workspace", q, shape)
    _launch("gtms_attention_key_weights", dev, shape, q_, k_, lse_, out_, bool(accumulate), lens, off, work, size, status)
    return out


def cache_evict(k, v, weights, seq_lens, keep: int, first: int = 0, recent: int = 0, positions=None, out=None):
    """(k, v, weights, positions, lens) of a cache cut to ``keep`` entries a sequence and head (gtms_cache_evict).

    ``k`` / ``v`` [B, H, S, d], ``weights`` fp32 and ``positions`` int32 [B, H, S] (contiguous; without it an entry's
    index). Of a sequence of more than ``keep`` entries stay the first ``first``, the last ``recent`` and those of
    highest weight between them, ties to the lowest index, in their order; shorter ones stay whole. ``out``: four tensors
    of min(keep, S) or more rows to write to, whose rows behind the new lengths are left as they are; ``(k, v, weights,
    positions)`` themselves compact the cache in place, and None in the last place leaves positions out. Without it
    new ones of min(keep, S) rows are made, zero behind the new lengths. New tokens follow at ``lens``, for which
    ``attention_forward`` takes ``seq_lens`` and ``q_offsets``: rows go by places in the cache. Their weights (0, for
    ``attention_key_weights`` to add to) and positions are the caller's to set: compacted in place, the cache still has
    older entries' there."""
    import torch

    dtype, dev = k.dtype, k.get_device()
    k_, v_ = _heads("k", k, dtype, dev), _heads("v", v, dtype, dev)
    B, H, S, d = shape4 = k.shape
    if v.shape != shape4:
        raise ValueError("k and v must match in shape")
    weights_ = _labels("weights", weights, torch.float32, (B, H, S), dev)
    positions_ = None if positions is None else _labels("positions", positions, torch.int32, (B, H, S), dev)
    lens = _int32("seq_lens", seq_lens, (B,), dev)
    if out is None:
        rows = max(0, min(int(keep), S))
        out = (torch.zeros((B, H, rows, d), dtype=dtype, device=k.device), torch.zeros((B, H, rows, d), dtype=dtype, device=k.device),
               torch.zeros((B, H, rows), dtype=torch.float32, device=k.device),
               torch.zeros((B, H, rows), dtype=torch.int32, device=k.device))
    k_out, v_out, weights_out, positions_out = out
    rows = k_out.shape[2] if k_out.dim() == 4 else -1
    if k_out.shape != (B, H, rows, d) or v_out.shape != k_out.shape:
        raise ValueError("out's k and v must match k and v in every dimension but the rows")
    wo = _labels("out's weights", weights_out, torch.float32, (B, H, rows), dev)
    po = None if positions_out is None else _labels("out's positions", positions_out, torch.int32, (B, H, rows), dev)
    new = torch.empty_like(seq_lens)
    shape = _pack_evict(B, H, S, rows, d, int(keep), int(first), int(recent), _dtype_code(k))
    _keep, work, size = _workspace("gtms_cache_evict_workspace", k, shape)
    _launch("gtms_cache_evict", dev, shape, k_, v_, weights_, positions_, _heads("out's k", k_out, dtype, dev),
            _heads("out's v", v_out, dtype, dev), wo, po, lens, new.data_ptr(), work, size)
    return k_out, v_out, weights_out, positions_out, new


def rotary_frequencies(rot_dim: int, base: float = 10000.0, scaling: int = GTMS_ROTARY_PLAIN, factor: float = 1.0,
                       low_turns: float = 1.0, high_turns: float = 4.0, original_length: int = 8192, device=None):
    """Inverse frequencies [rot_dim / 2] (fp32) for ``rotary``, plain or scaled for long contexts
    (gtms_rotary_frequencies)."""
    import torch

    f = torch.empty(max(0, int(rot_dim)) // 2, dtype=torch.float32)
    rc = gtms_rotary_frequencies(int(rot_dim), float(base), int(scaling), float(factor), float(low_turns),
                                 float(high_turns), int(original_length), f.data_ptr())
    if rc != GTMS_OK:
        raise GtmsError("gtms_rotary_frequencies", rc)
    return f if device is None else f.to(device)


def _rotary(x, positions, inv_freq, other, interleaved, amplitude, out, out_other, inverse):
    import torch

    dtype, dev = x.dtype, x.get_device()
    x_ = _heads("x", x, dtype, dev)
    B, H, S, d = shape = x.shape
    pairs = inv_freq.numel()
    rows = positions.shape[0] if positions.dim() == 2 else 1
    if positions.dim() not in (1, 2) or rows != 1 and rows != B:
        raise ValueError(f"positions must be [S] or [B, S], got {tuple(positions.shape)}")
    pos = _int32("positions", positions, (S,) if positions.dim() == 1 else (rows, S), dev)
    if inv_freq.dtype is not torch.float32 or inv_freq.dim() != 1 or inv_freq.get_device() != dev \
            or not inv_freq.is_contiguous() or 2 * pairs > d:
        raise ValueError("inv_freq must be a contiguous fp32 CUDA tensor of at most head_dim / 2 elements on x's device")
    if out is None:
        out = torch.empty_like(x)
    elif out.shape != shape:
        raise ValueError("out must match x in shape")
    H2, other_, out2_ = 0, None, None
    if other is not None:
        other_ = _heads("other", other, dtype, dev)
        b2, H2, s2, d2 = other.shape
        if b2 != B or s2 != S or d2 != d:
            raise ValueError("other must match x in every dimension but the heads")
        if out_other is None:
            out_other = torch.empty_like(other)
        elif out_other.shape != other.shape:
            raise ValueError("out_other must match other in shape")
        out2_ = _heads("out_other", out_other, dtype, dev)
    _launch("gtms_rotary", dev, x_, _heads("out", out, dtype, dev), other_, out2_, B, H, H2, S, d, 2 * pairs, pos, rows,
            inv_freq.data_ptr(), bool(interleaved), amplitude, inverse, _dtype_code(x))
    return out if other is None else (out, out_other)


def rotary_forward(x, positions, inv_freq, other=None, interleaved: bool = False, amplitude: float = 1.0, out=None,
                   out_other=None):
    """Rotary positions on ``x`` [B, H, S, d] and, in the same launch, on ``other`` [B, H2, S, d] (q and k): the first
    ``2 * len(inv_freq)`` elements of each head turned by ``positions * inv_freq``, the rest copied (gtms_rotary).
    Returns y, or (y, y_other). ``out`` may be ``x`` itself, ``out_other`` may be ``other``."""
    return _rotary(x, positions, inv_freq, other, interleaved, amplitude, out, out_other, False)


def rotary_backward(dy, positions, inv_freq, other=None, interleaved: bool = False, amplitude: float = 1.0, out=None,
                    out_other=None):
    """Gradient of ``rotary_forward``: the inverse rotation of ``dy`` (and of ``other``'s gradient)."""
    return _rotary(dy, positions, inv_freq, other, interleaved, amplitude, out, out_other, True)


def _usable(t):
    """A gradient as the kernels take it: one that autograd expanded, or whose data stands at an odd place, is copied."""
    import torch

    aligned = 16 // t.element_size()
    ok = t.stride(3) == 1 and t.data_ptr() % 16 == 0 and all(n <= 1 or (s % aligned == 0 and s >= t.shape[3])
                                                            for n, s in zip(t.shape[:3], t.stride()[:3]))
    return t if ok else t.clone(memory_format=torch.contiguous_format)   # contiguous() keeps a dense tensor where it is


def _attention_functions():
    import torch
    from torch.autograd.function import once_differentiable

    class Attention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, seq_lens, q_offsets, scale, mask_kind, window, status):
            o, lse = attention_forward(q, k, v, seq_lens, scale, mask_kind=mask_kind, window=window,
                                       q_offsets=q_offsets, status=status)
            ctx.save_for_backward(q, k, v, o, lse, seq_lens, q_offsets)
            ctx.options = scale, mask_kind, window
            ctx.status = status   # written by both calls, so not one of the saved tensors, which must not change
            return o

        @staticmethod
        @once_differentiable
        def backward(ctx, dout):
            q, k, v, o, lse, seq_lens, q_offsets = ctx.saved_tensors
            scale, mask_kind, window = ctx.options
            dq, dk, dv = attention_backward(q, k, v, o, lse, _usable(dout), seq_lens, scale, mask_kind=mask_kind,
                                            window=window, q_offsets=q_offsets, status=ctx.status)
            return dq, dk, dv, None, None, None, None, None, None

    class Rotary(torch.autograd.Function):
        @staticmethod
        def forward(ctx, positions, inv_freq, interleaved, amplitude, x, *other):
            ctx.save_for_backward(positions, inv_freq)
            ctx.options = interleaved, amplitude
            return rotary_forward(x, positions, inv_freq, *other, interleaved=interleaved, amplitude=amplitude)

        @staticmethod
        @once_differentiable
        def backward(ctx, *dy):
            positions, inv_freq = ctx.saved_tensors
            interleaved, amplitude = ctx.options
            dy = [_usable(t) for t in dy]
            dx = rotary_backward(dy[0], positions, inv_freq, *dy[1:], interleaved=interleaved, amplitude=amplitude)
            return (None, None, None, None) + (dx if isinstance(dx, tuple) else (dx,))

    return Attention, Rotary


_attention_fns = None


def _attention_fn(i):
    global _attention_fns
    if _attention_fns is None:
        _attention_fns = _attention_functions()
    return _attention_fns[i]


def attention(q, k, v, seq_lens, scale: float = 1.0, mask_kind: int = GTMS_MASK_GROUPED_TRIL, window: int = 0,
              q_offsets=None, status=None):
    """Differentiable ``attention_forward`` (o alone); the backward is ``attention_backward``.

    ``status``, an int32 CUDA tensor of one element, is handed to both: cleared before the step and read after
    synchronising, it says whether a wait inside a kernel ran out, so that o or the gradients are incomplete
    (``GTMS_ERR_TIMEOUT``). Without it nothing says so.

    To capture a training step into a CUDA graph, capture ``attention_forward`` and ``attention_backward``
    (``rotary_forward`` and ``rotary_backward``) themselves, which make no autograd nodes."""
    return _attention_fn(0).apply(q, k, v, seq_lens, q_offsets, float(scale), int(mask_kind), int(window), status)


def rotary(x, positions, inv_freq, other=None, interleaved: bool = False, amplitude: float = 1.0):
    """Differentiable ``rotary_forward``: y, or (y, y_other). Gradients reach ``x`` and ``other`` alone. For a captured
    training step see ``attention``."""
    rest = () if other is None else (other,)
    return _attention_fn(1).apply(positions, inv_freq, bool(interleaved), float(amplitude), x, *rest)
