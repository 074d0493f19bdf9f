"""Python binding of the B200 NVFP4 W4A4 linear library (``include/nvfp4.h``).

Argument marshalling only: every step of the quantiser and of the linear runs in
the CUDA kernels of ``libnvfp4_w4a4.so``.  PyTorch supplies device memory (the
caller-side output buffers allocated here) and the current CUDA stream.  There is
no CPU fallback: if the library is missing or the device is not sm_100, calls raise.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Sequence

__all__ = [
    "lib", "NVFP4Error", "scale_bytes", "amax", "global_scale", "quantize", "quantize_fused", "linear",
    "linear_splitk", "linear_splitk_noalloc", "noalloc_default_splits", "splitk_default", "splitk_workspace_bytes",
    "NOALLOC_SCRATCH_BYTES", "fold_segments", "fp8_scale", "kv_cache_fp8", "gdn_recurrence",
    "device_status", "selftest_stalled_linear", "unswizzle_scales", "pack_weight", "NVFP4Tensor", "EPILOGUES", "OUT_KINDS",
    "BlockKVCache", "block_kv_cache", "rope_table", "qk_norm_rope", "kv_append", "attention",
    "attention_workspace_bytes", "matvec",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
# NVFP4_DEBUG=1 selects the bounds-checking build of the same library (built with
# ``python -m nvfp4_w4a4_quantized_02_b200.build --debug``).
DEBUG = os.environ.get("NVFP4_DEBUG", "0") not in ("", "0")
LIB_PATH = os.path.join(_PKG, "libnvfp4_w4a4_debug.so" if DEBUG else "libnvfp4_w4a4.so")

EPILOGUES = {"none": 0, "silu_mul": 1, "gdn_gates": 2}
OUT_KINDS = {"bf16": 0, "f32": 1, "nvfp4": 2}
MAX_SEGMENTS = 16
NOALLOC_SCRATCH_BYTES = 8 << 20  # NVFP4_NOALLOC_SCRATCH_BYTES of include/nvfp4.h

_c_i64 = ctypes.c_int64
_c_vp = ctypes.c_void_p


class Operand(ctypes.Structure):
    _fields_ = [("codes", _c_vp), ("scales", _c_vp), ("rows", _c_i64), ("K", _c_i64)]


class Segment(ctypes.Structure):
    _fields_ = [("n_begin", _c_i64), ("n_end", _c_i64), ("gs_w", _c_vp)]


class EpilogueParams(ctypes.Structure):
    _fields_ = [("beta_begin", _c_i64), ("alpha_begin", _c_i64), ("n_heads", _c_i64),
                ("A_log", _c_vp), ("dt_bias", _c_vp), ("beta_out", _c_vp), ("g_out", _c_vp),
                ("gs_out", _c_vp), ("out_scales", _c_vp)]


class BlockCache(ctypes.Structure):
    _fields_ = [("k", _c_vp), ("v", _c_vp), ("k_scales", _c_vp), ("v_scales", _c_vp), ("num_blocks", _c_i64),
                ("block_size", ctypes.c_int), ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int)]


class Batch(ctypes.Structure):
    _fields_ = [("cu_seqlens", _c_vp), ("kv_lens", _c_vp), ("block_table", _c_vp), ("n_seqs", _c_i64),
                ("tokens", _c_i64), ("max_blocks", _c_i64), ("ld_table", _c_i64)]


class NVFP4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_lib_status_string(status)} ({status})")


_LIB = None
SYMBOLS = ("nvfp4_status_string", "nvfp4_scale_bytes", "nvfp4_global_scale", "nvfp4_quantize",
           "nvfp4_quantize_rows", "nvfp4_linear", "nvfp4_linear_splitk", "nvfp4_splitk_workspace_bytes",
           "nvfp4_splitk_default", "nvfp4_linear_splitk_noalloc", "nvfp4_fold_segments",
           "nvfp4_fp8_scale", "nvfp4_kv_cache_fp8", "nvfp4_gdn_recurrence", "nvfp4_get_device_status",
           "nvfp4_selftest_stalled_linear", "nvfp4_unswizzle_scales", "nvfp4_pack_weight", "nvfp4_amax",
           "nvfp4_rope_table", "nvfp4_qk_norm_rope", "nvfp4_kv_append", "nvfp4_attention_workspace_bytes",
           "nvfp4_attention", "nvfp4_matvec")


def lib():
    """The loaded C library (ctypes), with argument types declared."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"NVFP4 CUDA library not built ({LIB_PATH} missing): "
            f"run `python -m nvfp4_w4a4_quantized_02_b200.build{' --debug' if DEBUG else ''}`")
    L = ctypes.CDLL(LIB_PATH)
    L.nvfp4_status_string.restype = ctypes.c_char_p
    L.nvfp4_status_string.argtypes = [ctypes.c_int]
    L.nvfp4_scale_bytes.restype = ctypes.c_size_t
    L.nvfp4_scale_bytes.argtypes = [_c_i64, _c_i64]
    L.nvfp4_amax.restype = ctypes.c_int
    L.nvfp4_amax.argtypes = [_c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp]
    L.nvfp4_global_scale.restype = ctypes.c_int
    L.nvfp4_global_scale.argtypes = [_c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp]
    L.nvfp4_quantize.restype = ctypes.c_int
    L.nvfp4_quantize.argtypes = [_c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp]
    L.nvfp4_quantize_rows.restype = ctypes.c_int
    L.nvfp4_quantize_rows.argtypes = [_c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_vp]
    L.nvfp4_linear.restype = ctypes.c_int
    L.nvfp4_linear.argtypes = [ctypes.POINTER(Operand), _c_vp, ctypes.POINTER(Operand),
                               ctypes.POINTER(Segment), ctypes.c_int, ctypes.c_int,
                               ctypes.POINTER(EpilogueParams), _c_vp, ctypes.c_int, _c_i64, _c_vp]
    L.nvfp4_linear_splitk.restype = ctypes.c_int
    L.nvfp4_linear_splitk.argtypes = [ctypes.POINTER(Operand), _c_vp, ctypes.POINTER(Operand),
                                      ctypes.POINTER(Segment), ctypes.c_int, ctypes.c_int,
                                      ctypes.POINTER(EpilogueParams), _c_vp, ctypes.c_int, _c_i64,
                                      ctypes.c_int, _c_vp, ctypes.c_size_t, _c_vp]
    L.nvfp4_splitk_workspace_bytes.restype = ctypes.c_size_t
    L.nvfp4_splitk_workspace_bytes.argtypes = [_c_i64, _c_i64, ctypes.c_int]
    L.nvfp4_splitk_default.restype = ctypes.c_int
    L.nvfp4_splitk_default.argtypes = [_c_i64, _c_i64, _c_i64]
    L.nvfp4_linear_splitk_noalloc.restype = ctypes.c_int
    L.nvfp4_linear_splitk_noalloc.argtypes = [ctypes.POINTER(Operand), _c_vp, ctypes.POINTER(Operand),
                                              ctypes.POINTER(Segment), ctypes.c_int, ctypes.c_int,
                                              ctypes.POINTER(EpilogueParams), _c_vp, ctypes.c_int, _c_i64,
                                              ctypes.c_int, _c_vp]
    L.nvfp4_fold_segments.restype = ctypes.c_int
    L.nvfp4_fold_segments.argtypes = [_c_vp, _c_i64, _c_i64, ctypes.POINTER(Segment), ctypes.c_int, _c_vp, _c_vp]
    L.nvfp4_fp8_scale.restype = ctypes.c_int
    L.nvfp4_fp8_scale.argtypes = [_c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp]
    L.nvfp4_kv_cache_fp8.restype = ctypes.c_int
    L.nvfp4_kv_cache_fp8.argtypes = [_c_vp, _c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp,
                                     _c_i64, _c_vp]
    L.nvfp4_gdn_recurrence.restype = ctypes.c_int
    L.nvfp4_gdn_recurrence.argtypes = [_c_vp, _c_vp, _c_i64, _c_vp, _c_i64, _c_vp, _c_vp, _c_i64, _c_vp, _c_i64,
                                       _c_i64, ctypes.c_int, ctypes.c_int, ctypes.c_int, _c_vp, ctypes.c_int,
                                       _c_vp, _c_i64, ctypes.c_int, _c_vp]
    L.nvfp4_get_device_status.restype = ctypes.c_int
    L.nvfp4_get_device_status.argtypes = [ctypes.POINTER(ctypes.c_int)]
    L.nvfp4_unswizzle_scales.restype = ctypes.c_int
    L.nvfp4_unswizzle_scales.argtypes = [_c_vp, _c_i64, _c_i64, _c_vp, _c_i64, _c_vp]
    L.nvfp4_pack_weight.restype = ctypes.c_int
    L.nvfp4_pack_weight.argtypes = [ctypes.POINTER(Operand), ctypes.c_int, _c_vp, _c_vp, _c_i64, _c_vp]
    L.nvfp4_selftest_stalled_linear.restype = ctypes.c_int
    L.nvfp4_selftest_stalled_linear.argtypes = [ctypes.POINTER(Operand), _c_vp, ctypes.POINTER(Operand),
                                                ctypes.POINTER(Segment), ctypes.c_int, _c_vp, _c_i64, ctypes.c_int,
                                                _c_vp]
    c_int, c_float = ctypes.c_int, ctypes.c_float
    L.nvfp4_rope_table.restype = c_int
    L.nvfp4_rope_table.argtypes = [_c_vp, _c_i64, c_int, ctypes.c_double, _c_vp]
    L.nvfp4_qk_norm_rope.restype = c_int
    L.nvfp4_qk_norm_rope.argtypes = [_c_vp, _c_i64, _c_vp, _c_i64, _c_i64, c_int, c_int, c_int, _c_vp, _c_vp, c_float,
                                     c_float, _c_vp, _c_vp, _c_i64, c_int, c_int, _c_vp, _c_i64, _c_vp, _c_i64, _c_vp]
    L.nvfp4_kv_append.restype = c_int
    L.nvfp4_kv_append.argtypes = [_c_vp, _c_i64, _c_vp, _c_i64, ctypes.POINTER(Batch), ctypes.POINTER(BlockCache),
                                  _c_vp]
    L.nvfp4_attention_workspace_bytes.restype = ctypes.c_size_t
    L.nvfp4_attention_workspace_bytes.argtypes = [_c_i64, _c_i64, c_int, c_int, c_int]
    L.nvfp4_attention.restype = c_int
    L.nvfp4_attention.argtypes = [_c_vp, _c_i64, c_int, ctypes.POINTER(Batch), ctypes.POINTER(BlockCache), c_float,
                                  c_int, _c_vp, c_int, _c_i64, _c_vp, ctypes.c_size_t, _c_vp]
    L.nvfp4_matvec.restype = c_int
    L.nvfp4_matvec.argtypes = [_c_vp, _c_i64, _c_i64, ctypes.POINTER(Operand), ctypes.POINTER(Segment), c_int, _c_vp,
                               c_int, _c_i64, _c_vp]
    _LIB = L
    return L


def _lib_status_string(status: int) -> str:
    try:
        return lib().nvfp4_status_string(status).decode()
    except Exception:  # pragma: no cover - message formatting only
        return "status"


def _check(status: int, what: str):
    if status != 0:
        raise NVFP4Error(status, what)


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return _c_vp(s.cuda_stream)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def scale_bytes(rows: int, cols: int) -> int:
    return int(lib().nvfp4_scale_bytes(rows, cols))


@dataclass
class NVFP4Tensor:
    """A quantised [rows x cols] matrix: packed codes, swizzled scales, global scale (device)."""
    codes: "torch.Tensor"   # uint8 [rows, cols/2]
    scales: "torch.Tensor"  # uint8 [scale_bytes(rows, cols)]
    gs: "torch.Tensor"      # float32 [1]
    rows: int
    cols: int


def amax(x, out=None, stream=None):
    """max|x| of a 2-D BF16 CUDA tensor, as a float32 [1] device tensor (calibration)."""
    import torch
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.is_cuda
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=x.device)
    _check(lib().nvfp4_amax(_c_vp(x.data_ptr()), x.shape[0], x.shape[1], x.stride(0), _c_vp(out.data_ptr()),
                            _stream(stream)), "nvfp4_amax")
    return out


def global_scale(x, out=None, stream=None):
    """gs = 2688 / max|x| of a 2-D BF16 CUDA tensor, as a float32 [1] device tensor."""
    import torch
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.is_cuda
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=x.device)
    _check(lib().nvfp4_global_scale(_c_vp(x.data_ptr()), x.shape[0], x.shape[1], x.stride(0),
                                    _c_vp(out.data_ptr()), _stream(stream)), "nvfp4_global_scale")
    return out


def quantize(x, gs=None, codes=None, scales=None, stream=None) -> NVFP4Tensor:
    """NVFP4-quantise a 2-D BF16 CUDA tensor (row stride x.stride(0), unit column stride).

    ``gs``: float32 [1] device tensor (static scale); None computes it from x first.
    """
    import torch
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.is_cuda and x.stride(1) == 1
    rows, cols = x.shape
    if gs is None:
        gs = global_scale(x, stream=stream)
    if codes is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(max(scale_bytes(rows, cols), 1), dtype=torch.uint8, device=x.device)
    _check(lib().nvfp4_quantize(_c_vp(x.data_ptr()), rows, cols, x.stride(0), _c_vp(gs.data_ptr()),
                                _c_vp(codes.data_ptr()), _c_vp(scales.data_ptr()), _stream(stream)),
           "nvfp4_quantize")
    return NVFP4Tensor(codes, scales, gs, rows, cols)


def quantize_fused(parts, gs_list=None, stream=None):
    """Quantise the modules of a fused weight, each with its own global scale, into one
    NVFP4 weight.  ``parts``: list of 2-D BF16 CUDA tensors (same cols).

    Returns ``(NVFP4Tensor, segments)`` with segments ``[(n_begin, n_end, gs), ...]``.
    """
    import torch
    cols = parts[0].shape[1]
    total = sum(p.shape[0] for p in parts)
    dev = parts[0].device
    codes = torch.empty((total, cols // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty(scale_bytes(total, cols), dtype=torch.uint8, device=dev)
    segs, n0 = [], 0
    for i, p in enumerate(parts):
        assert p.dtype == torch.bfloat16 and p.shape[1] == cols and p.stride(1) == 1
        gs = gs_list[i] if gs_list is not None else global_scale(p, stream=stream)
        _check(lib().nvfp4_quantize_rows(_c_vp(p.data_ptr()), p.shape[0], cols, p.stride(0),
                                         _c_vp(gs.data_ptr()), _c_vp(codes.data_ptr()),
                                         _c_vp(scales.data_ptr()), n0, total, _stream(stream)),
               "nvfp4_quantize_rows")
        segs.append((n0, n0 + p.shape[0], gs))
        n0 += p.shape[0]
    return NVFP4Tensor(codes, scales, segs[0][2], total, cols), segs


def _linear_args(a, w, segments, epilogue, out_dtype, out, ldo, gates, gs_out, out_scales):
    """Marshal the arguments shared by nvfp4_linear and nvfp4_linear_splitk."""
    import torch
    M, K = a.rows, a.cols
    N = w.rows
    if segments is None:
        segments = [(0, N, w.gs)]
    if len(segments) > MAX_SEGMENTS:
        raise ValueError("too many segments")
    segs = (Segment * len(segments))(*[Segment(int(n0), int(n1), _ptr(g)) for n0, n1, g in segments])
    nout = N // 2 if epilogue == "silu_mul" else N
    ep = EpilogueParams()
    if epilogue == "gdn_gates":
        g = gates or {}
        ep.beta_begin, ep.alpha_begin, ep.n_heads = int(g["beta_begin"]), int(g["alpha_begin"]), int(g["n_heads"])
        ep.A_log, ep.dt_bias = _ptr(g["A_log"]), _ptr(g["dt_bias"])
        ep.beta_out, ep.g_out = _ptr(g.get("beta_out")), _ptr(g.get("g_out"))
    if out_dtype == "nvfp4":
        if gs_out is None:
            raise ValueError("nvfp4 output needs gs_out")
        if out is None:
            out = torch.empty((M, nout // 2), dtype=torch.uint8, device=a.codes.device)
        if out_scales is None:
            out_scales = torch.empty(scale_bytes(M, nout), dtype=torch.uint8, device=a.codes.device)
        ep.gs_out, ep.out_scales = _ptr(gs_out), _ptr(out_scales)
        ldo = 0
        result = NVFP4Tensor(out, out_scales, gs_out, M, nout)
    else:
        dt = torch.bfloat16 if out_dtype == "bf16" else torch.float32
        if out is None:
            out = torch.empty((M, nout), dtype=dt, device=a.codes.device)
        ldo = out.stride(0) if ldo is None else ldo
        result = out
    A = Operand(a.codes.data_ptr(), a.scales.data_ptr(), M, K)
    W = Operand(w.codes.data_ptr(), w.scales.data_ptr(), N, w.cols)
    args = (ctypes.byref(A), _c_vp(a.gs.data_ptr()), ctypes.byref(W), segs, len(segments),
            EPILOGUES[epilogue], ctypes.byref(ep), _c_vp(out.data_ptr()), OUT_KINDS[out_dtype], int(ldo))
    keep = (A, W, segs, ep)  # keep the ctypes structures alive across the call
    return args, result, keep


def linear(a: NVFP4Tensor, w: NVFP4Tensor, segments: Optional[Sequence] = None, epilogue: str = "none",
           out_dtype: str = "bf16", out=None, ldo: Optional[int] = None, gates: Optional[dict] = None,
           gs_out=None, out_scales=None, stream=None):
    """Fused W4A4 linear ``epilogue(A @ W^T / (gs_a * gs_w[seg]))``.

    segments: list of ``(n_begin, n_end, gs_w_tensor)``; default one segment with ``w.gs``.
    gates (gdn_gates): dict with beta_begin, alpha_begin, n_heads, A_log, dt_bias
    [, beta_out, g_out] (float32 device tensors).
    out_dtype "nvfp4" returns an NVFP4Tensor quantised with ``gs_out``.
    """
    args, result, _keep = _linear_args(a, w, segments, epilogue, out_dtype, out, ldo, gates, gs_out, out_scales)
    _check(lib().nvfp4_linear(*args, _stream(stream)), "nvfp4_linear")
    return result


def splitk_default(M: int, N: int, K: int) -> int:
    return int(lib().nvfp4_splitk_default(M, N, K))


def splitk_workspace_bytes(M: int, N: int, split_k: int) -> int:
    return int(lib().nvfp4_splitk_workspace_bytes(M, N, split_k))


def linear_splitk(a: NVFP4Tensor, w: NVFP4Tensor, segments: Optional[Sequence] = None, epilogue: str = "none",
                  out_dtype: str = "bf16", out=None, ldo: Optional[int] = None, gates: Optional[dict] = None,
                  gs_out=None, out_scales=None, split_k: Optional[int] = None, workspace=None, stream=None):
    """``linear`` with K split over ``split_k`` units per output tile (decode regime).

    ``workspace``: a CUDA tensor of at least ``splitk_workspace_bytes(M, N, split_k)``
    bytes (allocated here when None).  ``split_k`` None: the library's choice.
    """
    import torch
    M, N, K = a.rows, w.rows, a.cols
    if split_k is None:
        split_k = splitk_default(M, N, K)
    need = splitk_workspace_bytes(M, N, split_k)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=a.codes.device)
    args, result, _keep = _linear_args(a, w, segments, epilogue, out_dtype, out, ldo, gates, gs_out, out_scales)
    _check(lib().nvfp4_linear_splitk(*args, int(split_k), _c_vp(workspace.data_ptr()),
                                     workspace.numel() * workspace.element_size(), _stream(stream)),
           "nvfp4_linear_splitk")
    return result


def noalloc_default_splits(M: int, N: int, K: int) -> int:
    """The library's default split count, lowered until the partial sums fit the fixed
    scratch array of ``linear_splitk_noalloc`` (never below 1; one split above 64 rows
    needs no scratch)."""
    s = max(splitk_default(M, N, K), 1)
    while s > 1 and splitk_workspace_bytes(M, N, s) > NOALLOC_SCRATCH_BYTES:
        s -= 1
    return s


def linear_splitk_noalloc(a: NVFP4Tensor, w: NVFP4Tensor, segments: Optional[Sequence] = None,
                          epilogue: str = "none", out_dtype: str = "bf16", out=None, ldo: Optional[int] = None,
                          gates: Optional[dict] = None, gs_out=None, out_scales=None,
                          split_k: Optional[int] = None, stream=None):
    """``linear_splitk`` whose partial sums live in the library's fixed scratch array
    (``NOALLOC_SCRATCH_BYTES``), for callers that cannot hand in a workspace.

    The library allocates nothing for it (the output buffers allocated here when
    ``out`` / ``out_scales`` are None are this wrapper's, not the entry point's).
    Calls that overlap on the GPU share the scratch and race: serialise them.
    """
    M, N, K = a.rows, w.rows, a.cols
    if split_k is None:
        split_k = noalloc_default_splits(M, N, K)
    args, result, _keep = _linear_args(a, w, segments, epilogue, out_dtype, out, ldo, gates, gs_out, out_scales)
    _check(lib().nvfp4_linear_splitk_noalloc(*args, int(split_k), _stream(stream)), "nvfp4_linear_splitk_noalloc")
    return result


def unswizzle_scales(t: NVFP4Tensor, out=None, stream=None):
    """The E4M3 block scales of ``t`` in logical order: uint8 [rows, cols/16] (device)."""
    import torch
    if out is None:
        out = torch.empty((t.rows, t.cols // 16), dtype=torch.uint8, device=t.scales.device)
    _check(lib().nvfp4_unswizzle_scales(_c_vp(t.scales.data_ptr()), t.rows, t.cols, _c_vp(out.data_ptr()),
                                        out.stride(0), _stream(stream)), "nvfp4_unswizzle_scales")
    return out


def pack_weight(parts: Sequence[NVFP4Tensor], rows_out: Optional[int] = None, stream=None):
    """Pack separately quantised modules (same cols) into one fused NVFP4 weight of
    ``rows_out`` rows (default: their total; extra rows are zero padding).  Returns
    ``(NVFP4Tensor, segments)`` with segments ``[(row0, row1, gs), ...]`` of the modules."""
    import torch
    cols = parts[0].cols
    total = sum(p.rows for p in parts)
    rows_out = total if rows_out is None else rows_out
    dev = parts[0].codes.device
    codes = torch.empty((rows_out, cols // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty(scale_bytes(rows_out, cols), dtype=torch.uint8, device=dev)
    ops = (Operand * len(parts))(*[Operand(p.codes.data_ptr(), p.scales.data_ptr(), p.rows, p.cols) for p in parts])
    _check(lib().nvfp4_pack_weight(ops, len(parts), _c_vp(codes.data_ptr()), _c_vp(scales.data_ptr()), rows_out,
                                   _stream(stream)), "nvfp4_pack_weight")
    segs, n0 = [], 0
    for p in parts:
        segs.append((n0, n0 + p.rows, p.gs))
        n0 += p.rows
    return NVFP4Tensor(codes, scales, parts[0].gs, rows_out, cols), segs


def fold_segments(w: NVFP4Tensor, segments: Sequence, gs_out=None, stream=None):
    """Fused-group repair in place: one global scale for all modules of ``w`` (the
    ratios folded into its block scales).  Returns the common scale (float32 [1] device
    tensor); afterwards ``linear(a, w, segments=[(0, w.rows, gs)])`` serves the weight."""
    import torch
    if gs_out is None:
        gs_out = torch.empty(1, dtype=torch.float32, device=w.codes.device)
    segs = (Segment * len(segments))(*[Segment(int(n0), int(n1), _ptr(g)) for n0, n1, g in segments])
    _check(lib().nvfp4_fold_segments(_c_vp(w.scales.data_ptr()), w.rows, w.cols, segs, len(segments),
                                     _c_vp(gs_out.data_ptr()), _stream(stream)), "nvfp4_fold_segments")
    return gs_out


def fp8_scale(x, out=None, stream=None):
    """Calibrated FP8 scale max|x| / 448 of a 2-D BF16 CUDA tensor (float32 [1] device tensor)."""
    import torch
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.is_cuda
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=x.device)
    _check(lib().nvfp4_fp8_scale(_c_vp(x.data_ptr()), x.shape[0], x.shape[1], x.stride(0), _c_vp(out.data_ptr()),
                                 _stream(stream)), "nvfp4_fp8_scale")
    return out


def kv_cache_fp8(k, v, k_scale, v_scale, slots, k_cache, v_cache, stream=None):
    """Write K / V token rows (BF16 [tokens, width]) into FP8 caches ([num_slots, width]
    uint8) at ``slots`` (int64 [tokens], negative = skip) with static scales."""
    import torch
    assert k.shape == v.shape and k.stride() == v.stride() and k.dtype == torch.bfloat16
    assert slots.dtype == torch.int64 and k_cache.shape == v_cache.shape
    _check(lib().nvfp4_kv_cache_fp8(_c_vp(k.data_ptr()), _c_vp(v.data_ptr()), k.shape[0], k.shape[1], k.stride(0),
                                    _c_vp(k_scale.data_ptr()), _c_vp(v_scale.data_ptr()), _c_vp(slots.data_ptr()),
                                    _c_vp(k_cache.data_ptr()), _c_vp(v_cache.data_ptr()), k_cache.shape[0],
                                    _stream(stream)), "nvfp4_kv_cache_fp8")


def gdn_recurrence(q, k, v, g, beta, cu_seqlens, state, *, initial_state=True, out=None, out_dtype="bf16",
                   stream=None):
    """Gated delta-rule recurrence of the GDN layers over packed sequences.

    q, k: BF16 [tokens, H_k * 128] (row-strided views allowed, e.g. column ranges of the
    fused in-projection output); v: BF16 [tokens, H_v * 128]; g, beta: FP32 [tokens, H_v]
    (row-strided, as the gate epilogue writes them); cu_seqlens: int32 [n_seqs + 1];
    state: FP32 [n_seqs, H_v, 128, 128] with state[s, h, j, i] = S[i, j], read as the
    initial state when ``initial_state`` and overwritten with the final one.  Returns
    out [tokens, H_v * 128] (BF16 or FP32), out[t, h*128 + j] = (S_t^T q_t)_j."""
    import torch
    tokens = q.shape[0]
    hk, hv = q.shape[1] // 128, v.shape[1] // 128
    assert q.dtype == k.dtype == v.dtype == torch.bfloat16 and q.shape == k.shape and q.stride() == k.stride()
    assert q.stride(1) == 1 and v.stride(1) == 1 and v.shape[0] == tokens
    assert g.dtype == beta.dtype == torch.float32 and g.stride() == beta.stride() and g.shape[1] >= hv
    assert cu_seqlens.dtype == torch.int32 and state.dtype == torch.float32 and state.is_contiguous()
    n_seqs = cu_seqlens.shape[0] - 1
    assert state.shape == (n_seqs, hv, 128, 128)
    if out_dtype not in ("bf16", "f32"):
        raise ValueError(f"out_dtype must be 'bf16' or 'f32', not {out_dtype!r}")
    kind = OUT_KINDS[out_dtype]
    if out is None:
        out = torch.empty((tokens, hv * 128), device=q.device,
                          dtype=torch.bfloat16 if out_dtype == "bf16" else torch.float32)
    _check(lib().nvfp4_gdn_recurrence(_c_vp(q.data_ptr()), _c_vp(k.data_ptr()), q.stride(0), _c_vp(v.data_ptr()),
                                      v.stride(0), _c_vp(g.data_ptr()), _c_vp(beta.data_ptr()), g.stride(0),
                                      _c_vp(cu_seqlens.data_ptr()), n_seqs, tokens, hk, hv, 128,
                                      _c_vp(state.data_ptr()), int(bool(initial_state)), _c_vp(out.data_ptr()),
                                      out.stride(0), kind, _stream(stream)), "nvfp4_gdn_recurrence")
    return out


@dataclass
class BlockKVCache:
    """A paged E4M3 K / V cache with one scale per (block of tokens, kv head)."""
    k: "torch.Tensor"         # uint8 [num_blocks, n_kv_heads, block_size, head_dim]
    v: "torch.Tensor"
    k_scales: "torch.Tensor"  # float32 [num_blocks, n_kv_heads]
    v_scales: "torch.Tensor"


def block_kv_cache(num_blocks: int, n_kv_heads: int, block_size: int, head_dim: int, device="cuda") -> BlockKVCache:
    """An empty cache (uninitialised memory; ``kv_append`` needs no more)."""
    import torch
    shape = (num_blocks, n_kv_heads, block_size, head_dim)
    k, v = (torch.empty(shape, dtype=torch.uint8, device=device) for _ in range(2))
    ks, vs = (torch.empty(shape[:2], dtype=torch.float32, device=device) for _ in range(2))
    return BlockKVCache(k, v, ks, vs)


# torch's types and the raw calls behind torch.cuda.current_stream / current_device, looked up
# once: the calls below take microseconds on the GPU, and a serving step makes hundreds.
_BF16 = _F32 = _U8 = _I32 = _I64 = _raw_stream = _current_device = None


def _bind_torch():
    global _BF16, _F32, _U8, _I32, _I64, _raw_stream, _current_device
    import torch
    _BF16, _F32, _U8, _I32, _I64 = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.int64
    _raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _rows(x, name: str, dtype, dev: int = -1) -> int:
    """Checks a matrix argument (CUDA, 2-D, unit column stride) and returns its row stride."""
    shape, stride, at = x.shape, x.stride(), x.get_device()
    if at < 0 or x.dtype != dtype or len(shape) != 2:
        raise ValueError(f"{name} must be a 2-D {dtype} CUDA tensor")
    if stride[1] != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have unit column stride")
    if at != dev and dev >= 0:
        raise ValueError(f"{name} is on another device")
    return stride[0] if shape[0] > 1 else shape[1]


def _made(dev: int, stream, make, *args, returned: bool = True, **kw):
    """``make(...)``'s buffer for a call on ``stream``, taken from that stream's memory: what the
    current stream's allocator hands out may still be in use by kernels queued there, and
    nothing orders ``stream`` behind them.  The caller has a ``returned`` buffer on the
    current stream, which the allocator has to know of."""
    if stream is not None and stream.device.index != dev:  # default streams have one handle on all devices
        raise ValueError("stream is on another device")
    if stream is None or stream.cuda_stream == _raw_stream(dev):
        return make(*args, **kw)
    import torch
    with torch.cuda.stream(stream):
        t = make(*args, **kw)
    if returned:
        t.record_stream(torch.cuda.current_stream(dev))
    return t


def _launch(what: str, fn, dev: int, stream, *args):
    """Calls an entry point with its device current, on ``stream`` (default: the device's
    current one)."""
    if stream is None:
        raw = _raw_stream(dev)
    elif stream.device.index != dev:
        raise ValueError("stream is on another device")
    else:
        raw = stream.cuda_stream
    if _current_device() == dev:
        status = fn(*args, raw)
    else:
        import torch
        with torch.cuda.device(dev):
            status = fn(*args, raw)
    if status != 0:
        raise NVFP4Error(status, what)


def _out_buffer(like, shape, out, out_dtype: str, stream):
    """(out, kind, row stride, whether it was allocated here) of a BF16 or FP32 result of ``shape``."""
    if out_dtype == "bf16":
        dtype, kind = _BF16, 0
    elif out_dtype == "f32":
        dtype, kind = _F32, 1
    else:
        raise ValueError(f"out_dtype must be 'bf16' or 'f32', not {out_dtype!r}")
    if out is None:
        if stream is None:
            out = like.new_empty(shape) if kind == 0 else like.new_empty(shape, dtype=dtype)
        else:
            out = _made(like.get_device(), stream, like.new_empty, shape, dtype=dtype)
        return out, kind, shape[1], True
    ld = _rows(out, "out", dtype, like.get_device())
    if out.shape != shape:
        raise ValueError(f"out must be {tuple(shape)}")
    return out, kind, ld, False


def _cache_struct(cache: BlockKVCache, dev: int) -> BlockCache:
    k, v, ks, vs = cache.k, cache.v, cache.k_scales, cache.v_scales
    shape = k.shape
    if len(shape) != 4 or k.dtype != _U8 or v.dtype != _U8 or v.shape != shape:
        raise ValueError("cache k / v must be uint8 [num_blocks, n_kv_heads, block_size, head_dim]")
    nb, hk, block, d = shape
    if ks.dtype != _F32 or vs.dtype != _F32 or ks.shape != (nb, hk) or vs.shape != (nb, hk):
        raise ValueError("cache scales must be float32 [num_blocks, n_kv_heads]")
    if not (k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()):
        raise ValueError("cache tensors must be contiguous")
    if not k.get_device() == v.get_device() == ks.get_device() == vs.get_device() == dev:
        raise ValueError("cache is on another device")
    return BlockCache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), nb, block, hk, d)


def _batch_struct(cu_seqlens, kv_lens, block_table, tokens: int, dev: int) -> Batch:
    ld = _rows(block_table, "block_table", _I32, dev)
    n, cols = block_table.shape
    if cu_seqlens.dtype != _I32 or kv_lens.dtype != _I32 or cu_seqlens.shape != (n + 1,) or kv_lens.shape != (n,):
        raise ValueError("cu_seqlens must be int32 [n_seqs + 1] and kv_lens int32 [n_seqs], n_seqs the rows of block_table")
    if not (cu_seqlens.is_contiguous() and kv_lens.is_contiguous()):
        raise ValueError("cu_seqlens and kv_lens must be contiguous")
    if cu_seqlens.get_device() != dev or kv_lens.get_device() != dev:
        raise ValueError("cu_seqlens / kv_lens are on another device")
    return Batch(cu_seqlens.data_ptr(), kv_lens.data_ptr(), block_table.data_ptr(), n, tokens, cols, ld)


def rope_table(max_positions: int, rot_dim: int, base: float = 10000.0, device="cuda", stream=None):
    """FP32 [max_positions, rot_dim] table of cosines and sines for ``qk_norm_rope``, angles
    p * base^(-2i / rot_dim) computed in FP64."""
    import torch
    if _BF16 is None:
        _bind_torch()
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError("device must be a CUDA device")
    dev = _current_device() if device.index is None else device.index
    table = _made(dev, stream, torch.empty, (max_positions, rot_dim), dtype=torch.float32, device=torch.device("cuda", dev))
    _launch("nvfp4_rope_table", lib().nvfp4_rope_table, dev, stream, table.data_ptr(), max_positions, rot_dim, float(base))
    return table


def qk_norm_rope(q, k, w_q, w_k, positions=None, table=None, *, eps: float = 1e-6, weight_offset: float = 0.0,
                 interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head and the position rotation, in one pass.

    q: BF16 [tokens, heads * head_dim], k: BF16 [tokens, kv_heads * head_dim] (column ranges
    of one projection's output allowed); w_q, w_k: BF16 [head_dim], used as
    ``weight_offset + w``; positions: int64 [tokens]; table: FP32 [max_positions, rot_dim]
    (``rope_table``), None for no rotation.  ``q_out`` / ``k_out`` may be ``q`` / ``k``.
    Returns ``(q_out, k_out)``."""
    if _BF16 is None:
        _bind_torch()
    bf16 = _BF16
    ld_q, dev = _rows(q, "q", bf16), q.get_device()
    ld_k = _rows(k, "k", bf16, dev)
    tokens, width_q = q.shape
    d, width_k = w_q.numel(), k.shape[1]
    if not (w_q.dtype == w_k.dtype == bf16 and w_q.dim() == 1 and w_q.shape == w_k.shape and d > 0
            and w_q.is_contiguous() and w_k.is_contiguous() and w_q.get_device() == w_k.get_device() == dev):
        raise ValueError("w_q and w_k must be BF16 [head_dim] on q's device")
    if k.shape[0] != tokens or width_q % d or width_k % d:
        raise ValueError("q and k must have the same rows, of whole heads")
    rot = most = p_pos = p_table = 0
    if table is not None:
        if table.dtype != _F32 or table.dim() != 2 or not table.is_contiguous() or table.get_device() != dev:
            raise ValueError("table must be a contiguous float32 [max_positions, rot_dim] tensor on q's device")
        if (positions is None or positions.dtype != _I64 or positions.shape != (tokens,)
                or not positions.is_contiguous() or positions.get_device() != dev):
            raise ValueError("positions must be a contiguous int64 [tokens] tensor on q's device")
        most, rot = table.shape
        p_pos, p_table = positions.data_ptr(), table.data_ptr()
    ld_qo, ld_ko = width_q, width_k
    if q_out is None:
        q_out = q.new_empty((tokens, width_q)) if stream is None else _made(dev, stream, q.new_empty, (tokens, width_q))
    else:
        ld_qo = _rows(q_out, "q_out", bf16, dev)
        if q_out.shape != q.shape:
            raise ValueError("q_out must have the shape of q")
    if k_out is None:
        k_out = q.new_empty((tokens, width_k)) if stream is None else _made(dev, stream, q.new_empty, (tokens, width_k))
    else:
        ld_ko = _rows(k_out, "k_out", bf16, dev)
        if k_out.shape != k.shape:
            raise ValueError("k_out must have the shape of k")
    if tokens:
        _launch("nvfp4_qk_norm_rope", lib().nvfp4_qk_norm_rope, dev, stream, q.data_ptr(), ld_q, k.data_ptr(),
                ld_k, tokens, width_q // d, width_k // d, d, w_q.data_ptr(), w_k.data_ptr(), weight_offset, eps,
                p_pos, p_table, most, rot, interleaved, q_out.data_ptr(), ld_qo, k_out.data_ptr(), ld_ko)
    return q_out, k_out


def kv_append(k, v, cu_seqlens, kv_lens, block_table, cache: BlockKVCache, stream=None):
    """Quantise the new tokens' K and V rows (BF16 [tokens, n_kv_heads * head_dim]) into the
    cache.  Sequence s has the rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1, the last of its
    kv_lens[s] tokens (int32 tensors); block_table: int32 [n_seqs, max_blocks]."""
    if _BF16 is None:
        _bind_torch()
    ld_k, dev = _rows(k, "k", _BF16), k.get_device()
    ld_v = _rows(v, "v", _BF16, dev)
    tokens, width = k.shape
    c = _cache_struct(cache, dev)
    if v.shape != k.shape or width != c.n_kv_heads * c.head_dim:
        raise ValueError("k and v must be [tokens, n_kv_heads * head_dim] of the cache")
    b = _batch_struct(cu_seqlens, kv_lens, block_table, tokens, dev)
    if tokens and b.n_seqs:
        _launch("nvfp4_kv_append", lib().nvfp4_kv_append, dev, stream, k.data_ptr(), ld_k, v.data_ptr(), ld_v, b, c)


def attention_workspace_bytes(tokens: int, n_seqs: int, n_heads: int, n_kv_heads: int, head_dim: int) -> int:
    return int(lib().nvfp4_attention_workspace_bytes(tokens, n_seqs, n_heads, n_kv_heads, head_dim))


def attention(q, cu_seqlens, kv_lens, block_table, cache: BlockKVCache, *, softmax_scale: Optional[float] = None,
              causal: bool = True, out=None, out_dtype: str = "bf16", workspace=None, stream=None):
    """Attention of the token rows q (BF16 [tokens, heads * head_dim]) over the cache that
    holds their K and V already (``kv_append``), prompts and single tokens alike.

    softmax_scale: default head_dim ** -0.5.  workspace: a contiguous CUDA tensor of at
    least ``attention_workspace_bytes(...)`` bytes (allocated here when None); calls that
    share one must not overlap on the GPU.  Returns out [tokens, heads * head_dim]."""
    if _BF16 is None:
        _bind_torch()
    ld_q, dev = _rows(q, "q", _BF16), q.get_device()
    tokens, width = q.shape
    c = _cache_struct(cache, dev)
    d = c.head_dim
    if d == 0 or width % d:
        raise ValueError("q must be [tokens, heads * head_dim] of the cache")
    b = _batch_struct(cu_seqlens, kv_lens, block_table, tokens, dev)
    out, kind, ld_out, made = _out_buffer(q, q.shape, out, out_dtype, stream)
    if tokens == 0 or b.n_seqs == 0:
        return out
    if not made and out.data_ptr() == q.data_ptr():
        raise ValueError("out must not be q")
    L = lib()
    if workspace is None:
        need = L.nvfp4_attention_workspace_bytes(tokens, b.n_seqs, width // d, c.n_kv_heads, d)
        need = max(need, 16)
        workspace = (q.new_empty(need, dtype=_U8) if stream is None
                     else _made(dev, stream, q.new_empty, need, dtype=_U8, returned=False))
    elif not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError("workspace must be contiguous, on q's device")
    _launch("nvfp4_attention", L.nvfp4_attention, dev, stream, q.data_ptr(), ld_q, width // d, b, c,
            d ** -0.5 if softmax_scale is None else softmax_scale, causal, out.data_ptr(), kind, ld_out,
            workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out


def _check_gs(g, dev: int):
    if g.get_device() != dev:
        raise ValueError("a global scale is on another device")
    if g.dtype is not _F32 or g.numel() < 1:
        raise ValueError("a global scale must be a float32 tensor of one value")


def matvec(x, w: NVFP4Tensor, segments: Optional[Sequence] = None, out_dtype: str = "bf16", out=None, stream=None):
    """x @ W^T for up to 16 token rows x (BF16 [tokens, K], not quantised) and an NVFP4
    weight.  segments: list of ``(n_begin, n_end, gs_w)``; default one with ``w.gs``.
    Returns out [tokens, N] (BF16 or FP32)."""
    if _BF16 is None:
        _bind_torch()
    ld_x, dev = _rows(x, "x", _BF16), x.get_device()
    codes, scales, rows, cols = w.codes, w.scales, w.rows, w.cols
    if x.shape[1] != cols:
        raise ValueError("x must have the weight's columns")
    if codes.get_device() != dev or scales.get_device() != dev:
        raise ValueError("the weight is on another device")
    if not (codes.dtype is scales.dtype is _U8 and codes.is_contiguous() and scales.is_contiguous()
            and codes.numel() >= rows * cols >> 1 and scales.numel() >= (rows + 127 >> 7) * (cols + 63 >> 6) << 9):
        raise ValueError("the weight must be contiguous uint8 codes [rows, cols / 2] and scales of scale_bytes(rows, cols)")
    out, kind, ldo, made = _out_buffer(x, (x.shape[0], rows), out, out_dtype, stream)
    if not made and out.data_ptr() == x.data_ptr():
        raise ValueError("out must not be x")
    if segments is None:
        g = w.gs
        _check_gs(g, dev)
        n, segs = 1, Segment(0, rows, g.data_ptr())
    else:
        n = len(segments)
        if n > MAX_SEGMENTS:
            raise ValueError("too many segments")
        for _, _, g in segments:
            _check_gs(g, dev)
        segs = (Segment * n)(*[Segment(n0, n1, g.data_ptr()) for n0, n1, g in segments])
    if x.shape[0] == 0:
        return out
    _launch("nvfp4_matvec", lib().nvfp4_matvec, dev, stream, x.data_ptr(), ld_x, x.shape[0],
            Operand(codes.data_ptr(), scales.data_ptr(), rows, cols), segs, n, out.data_ptr(), kind, ldo)
    return out


def device_status() -> int:
    """Read and clear the device status word (synchronises the device)."""
    code = ctypes.c_int(0)
    _check(lib().nvfp4_get_device_status(ctypes.byref(code)), "nvfp4_get_device_status")
    return code.value


def selftest_stalled_linear(a: NVFP4Tensor, w: NVFP4Tensor, stall_stage: int, stream=None):
    """Run the failure-detection self-test (``nvfp4_selftest_stalled_linear``): the 1-CTA
    GEMM with K tile ``stall_stage`` never loaded and short wait limits.  Returns the
    (meaningless) FP32 output; the timeout shows in ``device_status()``."""
    import torch
    out = torch.zeros((a.rows, w.rows), dtype=torch.float32, device=a.codes.device)
    segs = (Segment * 1)(Segment(0, w.rows, w.gs.data_ptr()))
    A = Operand(a.codes.data_ptr(), a.scales.data_ptr(), a.rows, a.cols)
    W = Operand(w.codes.data_ptr(), w.scales.data_ptr(), w.rows, w.cols)
    _check(lib().nvfp4_selftest_stalled_linear(ctypes.byref(A), _c_vp(a.gs.data_ptr()), ctypes.byref(W), segs, 1,
                                               _c_vp(out.data_ptr()), out.stride(0), int(stall_stage),
                                               _stream(stream)), "nvfp4_selftest_stalled_linear")
    return out
