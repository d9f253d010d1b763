"""Weight-only quantized linear for AMD Instinct MI355X (gfx950): thin Python binding.

Every function here has the name of a C entry point of ``include/qlinear.h`` and only marshals
arguments: it reads shapes, dtypes and data pointers of torch tensors (device memory), passes
torch's current HIP stream, and allocates outputs with torch when none are given.  All
computation runs in the HIP kernels of ``lib/libqlinear.so``; there is no CPU fallback.  If the
library has not been built, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import Optional, Sequence

__all__ = [
    "QLError",
    "QL_AFFINE",
    "QL_MXFP4",
    "QL_Q8_0",
    "QL_MXFP4_BLOCKS",
    "QL_Q4_K",
    "QL_Q6_K",
    "lib_path",
    "load_library",
    "qlinear_quantize",
    "qlinear_dequant",
    "qlinear_quantize_q8_0",
    "qlinear_take",
    "qlinear_transcode_gptq",
    "qlinear_transcode_gptq_planar",
    "qlinear_gptq_check_g_idx",
    "qlinear_transcode_awq",
    "qlinear_gemv",
    "qlinear_gemm",
    "qlinear_gemm_workspace_size",
    "qlinear_gemm_grouped",
    "qlinear_gemm_grouped_workspace_size",
    "qlinear_gemv_batched",
    "qlinear_gemv_batched_workspace_size",
    "qlinear_problem_list",
    "qlinear_route",
    "qlinear_apply_experts",
    "qlinear_apply_experts_workspace_size",
    "qlinear_apply_experts_noalloc",
    "qlinear_qk_norm_rope",
    "qlinear_kv_append",
    "qlinear_paged_attention",
    "qlinear_paged_attention_workspace_size",
    "qlinear_paged_cache_4bit",
    "qlinear_kv_append_4bit",
    "qlinear_kv_read_4bit",
    "qlinear_paged_attention_4bit",
    "qlinear_paged_attention_4bit_workspace_size",
    "qlinear_kv_extend",
    "qlinear_select_experts",
    "qlinear_combine_experts",
    "qlinear_version",
]

QL_AFFINE, QL_MXFP4, QL_Q8_0, QL_MXFP4_BLOCKS, QL_Q4_K, QL_Q6_K = 0, 1, 2, 3, 4, 5
_QL_F32, _QL_F16, _QL_BF16 = 0, 1, 2

_HERE = os.path.dirname(os.path.abspath(__file__))


def lib_path() -> str:
    return os.path.join(_HERE, "lib", "libqlinear.so")


class QLError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"[ql_status {status}] {message}")
        self.status = status


class _GemmWeight(ctypes.Structure):
    _fields_ = [
        ("packed", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("biases", ctypes.c_void_p),
        ("layer_bias", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("n", ctypes.c_int64),
    ]


class _Problem(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("packed", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("biases", ctypes.c_void_p),
        ("layer_bias", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("m", ctypes.c_int64),
        ("n", ctypes.c_int64),
        ("k", ctypes.c_int64),
        ("bits", ctypes.c_int32),
        ("group_size", ctypes.c_int32),
    ]


class _Heads(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("heads", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class _PagedCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + [
        (f, ctypes.c_int64)
        for f in ("n_pages", "page_size", "hk", "d", "page_stride", "token_stride", "head_stride")]


class _PagedCache4(ctypes.Structure):
    _fields_ = [(f, ctypes.c_void_p) for f in ("k_codes", "v_codes", "k_groups", "v_groups")] + [
        (f, ctypes.c_int64)
        for f in ("n_pages", "page_size", "hk", "d", "group_size", "page_stride", "token_stride", "head_stride",
                  "group_page_stride", "group_token_stride", "group_head_stride")]


class _NormRope(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("w_dtype", ctypes.c_int),
                ("eps", ctypes.c_float), ("positions", ctypes.c_void_p), ("cos_sin", ctypes.c_void_p),
                ("max_pos", ctypes.c_int64), ("rot", ctypes.c_int64), ("interleaved", ctypes.c_int)]


_LIB = None
_P, _I64, _INT, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t

_SIGNATURES = {
    "qlinear_quantize": (_INT, [_P, _I64, _I64, _INT, _INT, _INT, _P, _P, _P, _P]),
    "qlinear_dequant": (_INT, [_INT, _P, _P, _P, _INT, _I64, _I64, _INT, _INT, _P, _INT, _P]),
    "qlinear_quantize_q8_0": (_INT, [_P, _I64, _I64, _P, _P]),
    "qlinear_take": (_INT, [_P, _I64, _P, _I64, _I64, _P, _P]),
    "qlinear_transcode_gptq": (_INT, [_P, _P, _P, _INT, _I64, _I64, _INT, _INT, _INT, _P, _P, _P, _P]),
    "qlinear_transcode_gptq_planar": (_INT, [_P, _P, _P, _INT, _I64, _I64, _INT, _INT, _P, _P, _P, _P]),
    "qlinear_gptq_check_g_idx": (_INT, [_P, _I64, _INT]),
    "qlinear_transcode_awq": (_INT, [_P, _P, _P, _INT, _I64, _I64, _INT, _INT, _P, _P, _P, _P]),
    "qlinear_gemv": (_INT, [_P, _INT, _I64, _I64, _P, _P, _P, _INT, _I64, _INT, _INT, _P, _P, _INT, _P]),
    "qlinear_gemm_workspace_size": (_SZ, [_I64, _I64, _I64, _INT, _INT]),
    "qlinear_gemm": (_INT, [_P, _INT, _I64, _I64, _P, _P, _P, _INT, _I64, _INT, _INT, _P, _P, _INT, _P, _SZ, _P]),
    "qlinear_gemm_grouped_workspace_size": (_SZ, [_I64, _I64, ctypes.POINTER(_GemmWeight), _INT, _INT, _INT]),
    "qlinear_gemm_grouped": (_INT, [_P, _INT, _I64, _I64, ctypes.POINTER(_GemmWeight), _INT, _INT, _INT, _INT, _INT, _P,
                                    _SZ, _P]),
    "qlinear_gemv_batched_workspace_size": (_SZ, [ctypes.POINTER(_Problem), _INT]),
    "qlinear_gemv_batched": (_INT, [ctypes.POINTER(_Problem), _INT, _INT, _INT, _INT, _P, _SZ, _INT, _P]),
    "qlinear_route": (_INT, [_P, _I64, _I64, _P, _P, _P]),
    "qlinear_apply_experts_workspace_size": (_SZ, [_I64, _I64]),
    "qlinear_apply_experts": (_INT, [_INT, _P, _P, _I64, _I64, _I64, _P, _I64, _P, _INT, _I64, _P, _INT, _P, _SZ, _P]),
    "qlinear_apply_experts_noalloc": (_INT, [_INT, _P, _P, _I64, _I64, _I64, _P, _I64, _P, _INT, _I64, _P, _INT, _P]),
    "qlinear_qk_norm_rope": (_INT, [_P, _P, _P, _P, _INT, _I64, _I64, _P, _P]),
    "qlinear_kv_append": (_INT, [_P, _P, _P, _P, _P, _P, _INT, _I64, _P, _P]),
    "qlinear_paged_attention_workspace_size": (_SZ, [_I64] * 9),
    "qlinear_paged_attention": (_INT, [_P, _P, _INT, _I64, _P, _P, _I64, _I64, _P, _P, _I64, _I64, ctypes.c_float, _I64,
                                       _P, _P, _SZ, _P]),
    "qlinear_kv_append_4bit": (_INT, [_P, _P, _P, _P, _P, _P, _INT, _I64, _P, _P]),
    "qlinear_kv_read_4bit": (_INT, [_P, _P, _I64, _P, _P, _INT, _P]),
    "qlinear_paged_attention_4bit_workspace_size": (_SZ, [_I64] * 9),
    "qlinear_paged_attention_4bit": (_INT, [_P, _P, _INT, _I64, _P, _P, _I64, _I64, _P, _P, _I64, _I64, ctypes.c_float,
                                            _I64, _P, _P, _SZ, _P]),
    "qlinear_kv_extend": (_INT, [_P, _P, _I64, _P, _I64, _I64, _I64, _P, _I64, _P, _P, _P, _P, _P, _P, _I64, _P, _P]),
    "qlinear_select_experts": (_INT, [_P, _INT, _I64, _I64, _I64, _P, _INT, _I64, _I64, _INT, _I64, _INT, ctypes.c_float,
                                      _P, _P, _P, _P]),
    "qlinear_combine_experts": (_INT, [_P, _INT, _P, _P, _I64, _P, _I64, _I64, _I64, _P, _P]),
    "qlinear_last_error": (ctypes.c_char_p, []),
    "qlinear_version": (ctypes.c_char_p, []),
}


def load_library():
    """Load lib/libqlinear.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build the HIP library first (__graft_entry__.build())")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


def _check(status: int):
    if status != 0:
        raise QLError(status, load_library().qlinear_last_error().decode())


def _torch():
    import torch

    return torch


def _dt(t) -> int:
    torch = _torch()
    d = t if isinstance(t, torch.dtype) else t.dtype
    if d == torch.float32:
        return _QL_F32
    if d == torch.float16:
        return _QL_F16
    if d == torch.bfloat16:
        return _QL_BF16
    raise QLError(3, f"unsupported dtype {d}")


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream() -> int:
    return _torch().cuda.current_stream().cuda_stream


def qlinear_version() -> str:
    return load_library().qlinear_version().decode()


def qlinear_quantize(w, bits: int = 4, group_size: int = 64, param_dtype=None, packed=None, scales=None, biases=None):
    """Affine group quantize + pack of fp32 W [n, k] -> (packed u32 [n, k*bits/32] as int32,
    scales [n, k/g], biases [n, k/g] in param_dtype)."""
    torch = _torch()
    lib = load_library()
    param_dtype = param_dtype or torch.bfloat16
    n, k = w.shape
    if packed is None:
        packed = torch.empty((n, k * bits // 32), dtype=torch.int32, device=w.device)
    if scales is None:
        scales = torch.empty((n, k // group_size), dtype=param_dtype, device=w.device)
    if biases is None:
        biases = torch.empty((n, k // group_size), dtype=param_dtype, device=w.device)
    _check(lib.qlinear_quantize(_ptr(w), n, k, bits, group_size, _dt(param_dtype), _ptr(packed), _ptr(scales),
                                _ptr(biases), _stream()))
    return packed, scales, biases


def qlinear_quantize_q8_0(w, blocks=None):
    """quantize_q8_0 of fp32 W [rows, k] -> blocks uint8 [rows, k/32*34]."""
    torch = _torch()
    lib = load_library()
    rows, k = w.shape
    if blocks is None:
        blocks = torch.empty((rows, k // 32 * 34), dtype=torch.uint8, device=w.device)
    _check(lib.qlinear_quantize_q8_0(_ptr(w), rows, k, _ptr(blocks), _stream()))
    return blocks


def qlinear_take(pos, src, dst=None):
    """take: rows of `src` (its first axis; any dtype and trailing shape) at int64 positions
    `pos`, bytes copied with no value decoded; a position out of range gives a zero row."""
    torch = _torch()
    lib = load_library()
    n_pos = pos.numel()
    if dst is None:
        dst = torch.empty((n_pos,) + tuple(src.shape[1:]), dtype=src.dtype, device=src.device)
    row_bytes = math.prod(src.shape[1:]) * src.element_size()
    _check(lib.qlinear_take(_ptr(pos), n_pos, _ptr(src), src.shape[0], row_bytes, _ptr(dst), _stream()))
    return dst


def qlinear_gptq_check_g_idx(g_idx, group_size: int):
    """Raise QLError unless g_idx (int32 [k], any device; copied to host) is arange(k) //
    group_size: an activation-order map has no exact affine form."""
    import numpy as np
    lib = load_library()
    h = np.ascontiguousarray(np.asarray(g_idx.cpu() if hasattr(g_idx, "cpu") else g_idx, dtype=np.int32))
    _check(lib.qlinear_gptq_check_g_idx(h.ctypes.data, h.shape[0], group_size))


def qlinear_transcode_gptq(qweight, qzeros, scales, *, bits: int, group_size: int, v1_zeros: bool = False,
                           g_idx=None, packed=None, scales_out=None, biases_out=None):
    """GPTQ (continuous layout, contiguous groups) -> affine (packed [n, k*bits/32] int32, scales and
    biases [n, k/group_size] in scales' dtype).  qweight [k*bits/32, n], qzeros [G, n*bits/32]
    (int32), scales [G, n].  A g_idx, when given, is checked first (qlinear_gptq_check_g_idx)."""
    torch = _torch()
    lib = load_library()
    n = scales.shape[1]
    k = qweight.shape[0] * 32 // bits
    if g_idx is not None:
        qlinear_gptq_check_g_idx(g_idx, group_size)
    if packed is None:
        packed = torch.empty((n, qweight.shape[0]), dtype=torch.int32, device=qweight.device)
    so = scales_out if scales_out is not None else torch.empty((n, scales.shape[0]), dtype=scales.dtype,
                                                                device=qweight.device)
    bo = biases_out if biases_out is not None else torch.empty_like(so)
    _check(lib.qlinear_transcode_gptq(_ptr(qweight), _ptr(qzeros), _ptr(scales), _dt(scales), k, n, bits, group_size,
                                      1 if v1_zeros else 0, _ptr(packed), _ptr(so), _ptr(bo), _stream()))
    return packed, so, bo


def qlinear_transcode_gptq_planar(qweight, qzeros, scales, *, bits: int, group_size: int, g_idx=None, packed=None,
                                  scales_out=None, biases_out=None):
    """GPTQ_P (planar blocks, true zeros) -> affine (packed [n, k*tb/32] int32 with tb = 8 for 7-bit
    sources, else bits; scales and biases [n, k/group_size] in scales' dtype).  qweight
    [k*bits/32, n], qzeros [G, n*bits/32] (int32), scales [G, n].  A g_idx, when given, is checked
    first (qlinear_gptq_check_g_idx)."""
    torch = _torch()
    lib = load_library()
    n = scales.shape[1]
    k = qweight.shape[0] * 32 // bits
    if g_idx is not None:
        qlinear_gptq_check_g_idx(g_idx, group_size)
    tb = 8 if bits == 7 else bits
    if packed is None:
        packed = torch.empty((n, k * tb // 32), dtype=torch.int32, device=qweight.device)
    so = scales_out if scales_out is not None else torch.empty((n, scales.shape[0]), dtype=scales.dtype,
                                                                device=qweight.device)
    bo = biases_out if biases_out is not None else torch.empty_like(so)
    _check(lib.qlinear_transcode_gptq_planar(_ptr(qweight), _ptr(qzeros), _ptr(scales), _dt(scales), k, n, bits,
                                             group_size, _ptr(packed), _ptr(so), _ptr(bo), _stream()))
    return packed, so, bo


def qlinear_transcode_awq(qweight, qzeros, scales, *, bits: int, group_size: int, packed=None, scales_out=None,
                          biases_out=None):
    """AWQ GEMM (codes and zeros packed along the outputs) -> affine (packed [n, k*tb/32] int32 with
    tb = 8 for 7-bit sources, else bits; scales and biases [n, k/group_size] in scales' dtype).
    qweight [k, n*bits/32], qzeros [G, n*bits/32] (int32), scales [G, n]."""
    torch = _torch()
    lib = load_library()
    k, n = qweight.shape[0], scales.shape[1]
    tb = 8 if bits == 7 else bits
    if packed is None:
        packed = torch.empty((n, k * tb // 32), dtype=torch.int32, device=qweight.device)
    so = scales_out if scales_out is not None else torch.empty((n, scales.shape[0]), dtype=scales.dtype,
                                                                device=qweight.device)
    bo = biases_out if biases_out is not None else torch.empty_like(so)
    _check(lib.qlinear_transcode_awq(_ptr(qweight), _ptr(qzeros), _ptr(scales), _dt(scales), k, n, bits, group_size,
                                     _ptr(packed), _ptr(so), _ptr(bo), _stream()))
    return packed, so, bo


def qlinear_dequant(fmt: int, w0, w1=None, w2=None, *, rows: int, k: int, bits: int = 4, group_size: int = 64,
                    out_dtype=None, out=None):
    """dequant of an affine / MXFP4 / Q8_0 / MXFP4-blocks weight into out [rows, k] (out_dtype,
    default fp32)."""
    torch = _torch()
    lib = load_library()
    out_dtype = out_dtype or torch.float32
    if out is None:
        out = torch.empty((rows, k), dtype=out_dtype, device=w0.device)
    pdt = _dt(w1) if (fmt == QL_AFFINE and w1 is not None) else _QL_BF16
    _check(lib.qlinear_dequant(fmt, _ptr(w0), _ptr(w1), _ptr(w2), pdt, rows, k, bits, group_size, _ptr(out),
                               _dt(out), _stream()))
    return out


def qlinear_gemv(x, packed, scales, biases, *, bits: int, group_size: int, layer_bias=None, y_dtype=None, y=None):
    """y [m, n] = x [m, k] . dequant(W [n, k])^T (+ layer_bias)."""
    torch = _torch()
    lib = load_library()
    m, k = x.shape
    n = packed.shape[0]
    if y is None:
        y = torch.empty((m, n), dtype=y_dtype or x.dtype, device=x.device)
    _check(lib.qlinear_gemv(_ptr(x), _dt(x), m, k, _ptr(packed), _ptr(scales), _ptr(biases), _dt(scales), n, bits,
                            group_size, _ptr(layer_bias), _ptr(y), _dt(y), _stream()))
    return y


def qlinear_gemm_workspace_size(m: int, n: int, k: int, bits: int, group_size: int) -> int:
    return int(load_library().qlinear_gemm_workspace_size(m, n, k, bits, group_size))


def qlinear_gemm(x, packed, scales, biases, *, bits: int, group_size: int, layer_bias=None, y_dtype=None, y=None,
                 workspace=None):
    """Prefill product on the matrix cores; same result contract as qlinear_gemv."""
    torch = _torch()
    lib = load_library()
    m, k = x.shape
    n = packed.shape[0]
    if y is None:
        y = torch.empty((m, n), dtype=y_dtype or x.dtype, device=x.device)
    need = qlinear_gemm_workspace_size(m, n, k, bits, group_size)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    _check(lib.qlinear_gemm(_ptr(x), _dt(x), m, k, _ptr(packed), _ptr(scales), _ptr(biases), _dt(scales), n, bits,
                            group_size, _ptr(layer_bias), _ptr(y), _dt(y), _ptr(workspace), workspace.numel(),
                            _stream()))
    return y


def _gemm_weights(weights):
    arr = (_GemmWeight * max(1, len(weights)))()
    for i, w in enumerate(weights):
        arr[i] = _GemmWeight(_ptr(w["packed"]), _ptr(w["scales"]), _ptr(w["biases"]), _ptr(w.get("layer_bias")),
                             _ptr(w.get("y")), w["packed"].shape[0])
    return arr


def qlinear_gemm_grouped_workspace_size(m: int, k: int, weights: Sequence[dict], bits: int, group_size: int) -> int:
    return int(load_library().qlinear_gemm_grouped_workspace_size(m, k, _gemm_weights(weights), len(weights), bits,
                                                                  group_size))


def qlinear_gemm_grouped(x, weights: Sequence[dict], *, bits: int, group_size: int, y_dtype=None, workspace=None):
    """Prefill products of up to four weights that read the same x: each weight is a dict with
    tensors packed, scales, biases, optional layer_bias and optional output y (allocated here when
    absent).  Returns the list of outputs."""
    torch = _torch()
    lib = load_library()
    m, k = x.shape
    ws_in = [dict(w) for w in weights]
    for w in ws_in:
        if w.get("y") is None:
            w["y"] = torch.empty((m, w["packed"].shape[0]), dtype=y_dtype or x.dtype, device=x.device)
    arr = _gemm_weights(ws_in)
    if workspace is None:
        need = qlinear_gemm_grouped_workspace_size(m, k, ws_in, bits, group_size)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    ydt = ws_in[0]["y"] if ws_in else x
    _check(lib.qlinear_gemm_grouped(_ptr(x), _dt(x), m, k, arr, len(ws_in), _dt(ws_in[0]["scales"]) if ws_in else 2,
                                    bits, group_size, _dt(ydt), _ptr(workspace), workspace.numel(), _stream()))
    return [w["y"] for w in ws_in]


def qlinear_problem_list(problems):
    """Marshal a list of GEMV problems (dicts with tensors x, packed, scales, biases, y, optional
    layer_bias, and ints bits, group_size) into the C array qlinear_gemv_batched takes; pass the
    result instead of the list to skip re-marshalling on every call."""
    return _problem_array(problems)


def _problem_array(problems):
    if isinstance(problems, ctypes.Array):
        return problems
    arr = (_Problem * len(problems))()
    for i, p in enumerate(problems):
        x, packed, y = p["x"], p["packed"], p["y"]
        arr[i] = _Problem(_ptr(x), _ptr(packed), _ptr(p["scales"]), _ptr(p["biases"]), _ptr(p.get("layer_bias")),
                          _ptr(y), x.shape[0], packed.shape[0], x.shape[1], p["bits"], p["group_size"])
    return arr


def qlinear_gemv_batched_workspace_size(problems: Sequence[dict]) -> int:
    return int(load_library().qlinear_gemv_batched_workspace_size(_problem_array(problems), len(problems)))


def qlinear_gemv_batched(problems: Sequence[dict], *, x_dtype, param_dtype, y_dtype, workspace, upload: bool = True):
    """One launch (per class) over a list of GEMVs.  Each problem is a dict with tensors x, packed,
    scales, biases, y, optional layer_bias, and ints bits, group_size."""
    lib = load_library()
    arr = _problem_array(problems)
    _check(lib.qlinear_gemv_batched(arr, len(problems), _dt(x_dtype), _dt(param_dtype), _dt(y_dtype), _ptr(workspace),
                                    workspace.numel(), 1 if upload else 0, _stream()))


def qlinear_route(ids, e: int, offsets=None, perm=None):
    """Stable grouping of positions by expert id -> (offsets int32 [e+1], perm int32 [n_pos])."""
    torch = _torch()
    lib = load_library()
    n_pos = ids.numel()
    if offsets is None:
        offsets = torch.empty(e + 1, dtype=torch.int32, device=ids.device)
    if perm is None:
        perm = torch.full((max(n_pos, 1),), -1, dtype=torch.int32, device=ids.device)
    _check(lib.qlinear_route(_ptr(ids), n_pos, e, _ptr(offsets), _ptr(perm), _stream()))
    return offsets, perm


def qlinear_apply_experts_workspace_size(n_pos: int, e: int) -> int:
    return int(load_library().qlinear_apply_experts_workspace_size(n_pos, e))


def qlinear_apply_experts(fmt: int, w0, w1, ids, x, *, n: int, k: int, pos_per_row: int = 1, y_dtype=None, y=None,
                          workspace=None):
    """y [n_pos, n]: each position's x row through the expert its id names (zeros out of range)."""
    torch = _torch()
    lib = load_library()
    e = w0.shape[0]
    n_pos = ids.numel()
    if y is None:
        y = torch.empty((n_pos, n), dtype=y_dtype or x.dtype, device=x.device)
    need = qlinear_apply_experts_workspace_size(n_pos, e)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    _check(lib.qlinear_apply_experts(fmt, _ptr(w0), _ptr(w1), e, n, k, _ptr(ids), n_pos, _ptr(x), _dt(x), pos_per_row,
                                     _ptr(y), _dt(y), _ptr(workspace), workspace.numel(), _stream()))
    return y


def qlinear_apply_experts_noalloc(fmt: int, w0, w1, ids, x, *, n: int, k: int, y, pos_per_row: int = 1):
    """qlinear_apply_experts with the routing scratch in the library's built-in device array: no
    workspace, nothing allocated (y is the caller's output tensor [n_pos, n])."""
    lib = load_library()
    e = w0.shape[0]
    _check(lib.qlinear_apply_experts_noalloc(fmt, _ptr(w0), _ptr(w1), e, n, k, _ptr(ids), ids.numel(), _ptr(x), _dt(x),
                                             pos_per_row, _ptr(y), _dt(y), _stream()))
    return y


# ---- attention side.  These calls are short enough for the marshalling to show: the argument
# structures are kept, one set a thread, and messages are only put together for a refusal.
class _Args(threading.local):
    def __init__(self):
        self.q, self.q_out, self.k, self.v = _Heads(), _Heads(), _Heads(), _Heads()
        self.cache, self.cache4, self.nr = _PagedCache(), _PagedCache4(), _NormRope()
        self.at = {n: ctypes.addressof(getattr(self, n)) for n in ("q", "q_out", "k", "v", "cache", "cache4", "nr")}


_ARGS = _Args()


def _heads(h: _Heads, x, name: str, t: int, d: int, dtype, device: int):
    """Fill h from x [t, heads, d]."""
    shape = x.shape
    if len(shape) != 3 or shape[0] != t or shape[2] != d:
        raise QLError(2, f"{name} must be [{t}, heads, {d}], not {list(shape)}")
    if x.dtype is not dtype:
        raise QLError(3, f"{name} must have dtype {dtype}, not {x.dtype}")
    strides = x.stride()
    if strides[2] != 1 and d > 1:
        raise QLError(2, f"{name}'s last dimension must be contiguous")
    _same_device(x, name, device)
    h.p = x.data_ptr()
    h.heads = shape[1]
    # the stride of a dimension of one is free in torch: any legal value will do
    h.token_stride = strides[0] if t > 1 else 0
    h.head_stride = strides[1] if shape[1] > 1 else 0


def _same_device(x, name: str, device: int):
    if x.get_device() != device:
        raise QLError(2, f"every tensor must be on one GPU: {name} is on {x.device}")


def _array(x, name: str, dtype, shape, device: int):
    """Pointer of a contiguous tensor of the given dtype and shape (None: None)."""
    if x is None:
        return None
    if x.dtype is not dtype:
        raise QLError(3, f"{name} must have dtype {dtype}, not {x.dtype}")
    if x.shape != shape or not x.is_contiguous():
        raise QLError(2, f"{name} must be contiguous of shape {list(shape)}, not {list(x.shape)}")
    _same_device(x, name, device)
    return x.data_ptr()


def _result(x, name: str, dtype, shape, like, device: int):
    """An output and its pointer: x, checked, or a new tensor where like is."""
    if x is None:
        x = _torch().empty(shape, dtype=dtype, device=like.device)
        return x, x.data_ptr()
    return x, _array(x, name, dtype, shape, device)


def _paged_cache(c: _PagedCache, k_cache, v_cache, d: int, dtype, device: int):
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape or shape[3] != d:
        raise QLError(2, f"k_cache and v_cache must both be [n_pages, page_size, heads, {d}]")
    if k_cache.dtype is not dtype or v_cache.dtype is not dtype:
        raise QLError(3, f"the caches must have dtype {dtype}")
    sk, sv = k_cache.stride(), v_cache.stride()
    if sk != sv and any(a != b for a, b, n in zip(sk, sv, shape) if n > 1):
        raise QLError(2, "k_cache and v_cache must have the same strides")
    if d > 1 and (sk[3] != 1 or sv[3] != 1):
        raise QLError(2, "the caches' last dimension must be contiguous")
    _same_device(k_cache, "k_cache", device)
    _same_device(v_cache, "v_cache", device)
    c.k, c.v = k_cache.data_ptr(), v_cache.data_ptr()
    c.n_pages, c.page_size, c.hk, c.d = shape
    c.page_stride = sk[0] if shape[0] > 1 else 0
    c.token_stride = sk[1] if shape[1] > 1 else 0
    c.head_stride = sk[2] if shape[2] > 1 else 0


def _block_table(table, device: int):
    """(sequences, pages of a row, stride of the rows) of a block table."""
    if table.dim() != 2 or table.dtype is not _torch().int32:
        raise QLError(3, "block_table must be int32 [n_seqs, max_pages]")
    n_seqs, max_pages = table.shape
    row, place = table.stride()
    if place != 1 and max_pages > 1:
        raise QLError(2, "block_table's rows must be contiguous")
    _same_device(table, "block_table", device)
    return n_seqs, max_pages, row if n_seqs > 1 else max_pages


def _paged_cache4(c: _PagedCache4, cache, d: Optional[int], device: int):
    """Fill c from (k_codes, k_groups, v_codes, v_groups)."""
    torch = _torch()
    if len(cache) != 4:
        raise QLError(2, "cache must be (k_codes, k_groups, v_codes, v_groups)")
    kc, kg, vc, vg = cache
    i32, f16 = torch.int32, torch.float16
    if kc.dtype is not i32 or vc.dtype is not i32 or kg.dtype is not f16 or vg.dtype is not f16:
        raise QLError(3, "the cache's codes must be int32 and its groups float16")
    shape, groups = kc.shape, kg.shape
    if len(shape) != 4 or vc.shape != shape or (d is not None and shape[3] * 8 != d):
        raise QLError(2, f"the codes must both be [n_pages, page_size, heads, {d}/8]")
    n_pages, page_size, heads, words = shape
    if len(groups) != 5 or vg.shape != groups or groups[:3] != shape[:3] or groups[3] < 1 or groups[4] != 2 or \
            words * 8 % groups[3]:
        raise QLError(2, f"the groups must both be {list(shape[:3])} + [groups of a row, 2]")
    sk, sg, sv, sw = kc.stride(), kg.stride(), vc.stride(), vg.stride()
    if sk != sv or sg != sw:
        for a, b, x, name in ((sk, sv, shape, "codes"), (sg, sw, groups, "groups")):
            if any(i != j for i, j, n in zip(a, b, x) if n > 1):
                raise QLError(2, f"the {name} of k and v must have the same strides")
    if sk[3] != 1 and words > 1:
        raise QLError(2, "the last dimension of the codes must be contiguous")
    if sg[4] != 1 or (sg[3] != 2 and groups[3] > 1):
        raise QLError(2, "the last dimensions of the groups must be contiguous")
    if not (kc.get_device() == kg.get_device() == vc.get_device() == vg.get_device() == device):
        for x, name in zip(cache, ("k_codes", "k_groups", "v_codes", "v_groups")):
            _same_device(x, name, device)
    c.k_codes, c.k_groups, c.v_codes, c.v_groups = kc.data_ptr(), kg.data_ptr(), vc.data_ptr(), vg.data_ptr()
    c.n_pages, c.page_size, c.hk, c.d = n_pages, page_size, heads, words * 8
    c.group_size = words * 8 // groups[3]
    # the stride of a dimension of one is free in torch
    p, t, h = sk[0] if n_pages > 1 else 0, sk[1] if page_size > 1 else 0, sk[2] if heads > 1 else 0
    c.page_stride, c.token_stride, c.head_stride = 4 * p, 4 * t, 4 * h
    p, t, h = sg[0] if n_pages > 1 else 0, sg[1] if page_size > 1 else 0, sg[2] if heads > 1 else 0
    if (p | t | h) & 1:
        raise QLError(4, "the strides of the groups must be whole words")
    c.group_page_stride, c.group_token_stride, c.group_head_stride = p >> 1, t >> 1, h >> 1


def _norm_rope(n: _NormRope, t: int, d: int, q_weight, k_weight, eps, positions, cos_sin, interleaved, device: int):
    torch = _torch()
    w = q_weight if q_weight is not None else k_weight
    if w is not None:
        n.w_dtype = _dt(w)
    n.q_weight = _array(q_weight, "q_weight", w.dtype if w is not None else None, (d,), device)
    n.k_weight = _array(k_weight, "k_weight", w.dtype if w is not None else None, (d,), device)
    n.eps = eps
    n.positions = _array(positions, "positions", torch.int64, (t,), device)
    if cos_sin is None:
        n.cos_sin, n.max_pos, n.rot = None, 0, 0
    else:
        shape = cos_sin.shape
        if len(shape) != 2:
            raise QLError(2, "cos_sin must be [positions, rotated values]")
        n.cos_sin = _array(cos_sin, "cos_sin", torch.float32, shape, device)
        n.max_pos, n.rot = shape
    n.interleaved = 1 if interleaved else 0


def _stream_on(device: int) -> int:
    if device < 0:
        raise QLError(2, "every tensor must be on one GPU, not in host memory")
    cuda = _torch()._C
    if device != cuda._cuda_getDevice():
        raise QLError(2, f"the tensors are on cuda:{device}, which is not the current device")
    return cuda._cuda_getCurrentRawStream(device)


def qlinear_qk_norm_rope(q, k, *, q_weight=None, k_weight=None, eps: float = 1e-6, positions=None, cos_sin=None,
                         interleaved: bool = False, q_out=None, k_out=None):
    """RMS norms of q [t, hq, d] and k [t, hk, d] (either may be None) per head, then the rotation by
    the rows of cos_sin (fp32 [max_pos, rot]: rot/2 cosines, rot/2 sines) that positions (int64 [t])
    name -> (q_out, k_out).  q and k may be strided parts of one tensor, and q_out may be q."""
    torch = _torch()
    lib = load_library()
    x = q if q is not None else k
    if x is None or x.dim() != 3:
        raise QLError(2, "q or k must be given, [tokens, heads, d]")
    t, _, d = x.shape
    dtype, device, args = x.dtype, x.get_device(), _ARGS
    at = args.at
    if q is not None:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=dtype, device=q.device)
        _heads(args.q, q, "q", t, d, dtype, device)
        _heads(args.q_out, q_out, "q_out", t, d, dtype, device)
    if k is not None:
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=dtype, device=k.device)
        _heads(args.k, k, "k", t, d, dtype, device)
        _heads(args.v, k_out, "k_out", t, d, dtype, device)
    _norm_rope(args.nr, t, d, q_weight, k_weight, eps, positions, cos_sin, interleaved, device)
    status = lib.qlinear_qk_norm_rope(at["q"] if q is not None else None, at["q_out"], at["k"] if k is not None else None,
                                      at["v"], _dt(dtype), t, d, at["nr"], _stream_on(device))
    if status:
        _check(status)
    return q_out, k_out


def qlinear_kv_append(k, v, k_cache, v_cache, slots, *, q=None, q_out=None, q_weight=None, k_weight=None,
                      eps: float = 1e-6, positions=None, cos_sin=None, interleaved: bool = False):
    """Store k (normed and rotated as qlinear_qk_norm_rope does) and v [t, hk, d] at slots (int64 [t],
    slot = page * page_size + place; out of range: not stored) of the caches [n_pages, page_size,
    hk, d] (any strides), in one launch with q's norm and rotation where q [t, hq, d] is given
    -> q_out (None without q)."""
    torch = _torch()
    lib = load_library()
    if k.dim() != 3:
        raise QLError(2, "k must be [tokens, heads, d]")
    t, _, d = k.shape
    dtype, device, args = k.dtype, k.get_device(), _ARGS
    at = args.at
    if q is not None:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=dtype, device=q.device)
        _heads(args.q, q, "q", t, d, dtype, device)
        _heads(args.q_out, q_out, "q_out", t, d, dtype, device)
    _heads(args.k, k, "k", t, d, dtype, device)
    _heads(args.v, v, "v", t, d, dtype, device)
    _paged_cache(args.cache, k_cache, v_cache, d, dtype, device)
    slots_at = _array(slots, "slots", torch.int64, (t,), device)
    _norm_rope(args.nr, t, d, q_weight, k_weight, eps, positions, cos_sin, interleaved, device)
    status = lib.qlinear_kv_append(at["q"] if q is not None else None, at["q_out"], at["k"], at["v"], at["cache"],
                                   slots_at, _dt(dtype), t, at["nr"], _stream_on(device))
    if status:
        _check(status)
    return q_out if q is not None else None


def qlinear_paged_attention_workspace_size(q, k_cache, block_table, *, max_q: int, window: int = 0) -> int:
    t, hq, d = q.shape
    return int(load_library().qlinear_paged_attention_workspace_size(
        t, block_table.shape[0], hq, k_cache.shape[2], d, max_q, block_table.shape[1], k_cache.shape[1], window))


def qlinear_paged_attention(q, k_cache, v_cache, block_table, cu_q, kv_lens, *, max_q: int, scale=None,
                            window: int = 0, sinks=None, out=None, workspace=None):
    """Causal attention of new tokens q [t, hq, d] over the caches [n_pages, page_size, hk, d] that hold
    their k and v already.  Sequence s has the queries cu_q[s] .. cu_q[s+1] (int32 [n_seqs + 1]), which
    are the last of its kv_lens[s] positions (int32 [n_seqs]) in the pages block_table[s] (int32
    [n_seqs, max_pages]); max_q bounds a sequence's queries.  scale defaults to d^-1/2; window > 0: a
    query sees its last `window` positions; sinks fp32 [hq].  -> out [t, hq, d]."""
    torch = _torch()
    lib = load_library()
    if q.dim() != 3:
        raise QLError(2, "q must be [tokens, heads, d]")
    t, hq, d = q.shape
    dtype, device, args = q.dtype, q.get_device(), _ARGS
    at = args.at
    if out is None:
        out = torch.empty((t, hq, d), dtype=dtype, device=q.device)
    _heads(args.q, q, "q", t, d, dtype, device)
    _heads(args.q_out, out, "out", t, d, dtype, device)
    _paged_cache(args.cache, k_cache, v_cache, d, dtype, device)
    n_seqs, max_pages, row = _block_table(block_table, device)
    cu_at = _array(cu_q, "cu_q", torch.int32, (n_seqs + 1,), device)
    lens_at = _array(kv_lens, "kv_lens", torch.int32, (n_seqs,), device)
    sinks_at = _array(sinks, "sinks", torch.float32, (hq,), device)
    if workspace is None:
        need = qlinear_paged_attention_workspace_size(q, k_cache, block_table, max_q=max_q, window=window)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    elif not workspace.is_contiguous():
        raise QLError(2, "workspace must be contiguous")
    _same_device(workspace, "workspace", device)
    status = lib.qlinear_paged_attention(at["q"], at["q_out"], _dt(dtype), t, at["cache"], block_table.data_ptr(),
                                         row, max_pages, cu_at, lens_at, n_seqs, max_q,
                                         d ** -0.5 if scale is None else scale, window, sinks_at, workspace.data_ptr(),
                                         workspace.nbytes, _stream_on(device))
    if status:
        _check(status)
    return out


# ---- over a cache in 4 bits: four tensors (k_codes, k_groups, v_codes, v_groups), codes int32
# [n_pages, page_size, hk, d/8] and groups float16 [n_pages, page_size, hk, d/group_size, 2] (scale, bias).


def qlinear_paged_cache_4bit(n_pages: int, page_size: int, heads: int, d: int, group_size: int = 64, device="cuda"):
    """An empty cache in 4 bits -> (k_codes, k_groups, v_codes, v_groups).  Its pages are head-major in memory, so
    that a head's rows in a page are one run, which is what reads fastest."""
    torch = _torch()
    if group_size not in (32, 64, 128) or d % group_size:
        raise QLError(5, "group_size must be 32, 64 or 128 and divide d")
    codes = [torch.zeros((n_pages, heads, page_size, d // 8), dtype=torch.int32, device=device) for _ in range(2)]
    groups = [torch.zeros((n_pages, heads, page_size, d // group_size, 2), dtype=torch.float16, device=device)
              for _ in range(2)]
    return tuple(x.transpose(1, 2) for pair in zip(codes, groups) for x in pair)


def qlinear_kv_append_4bit(k, v, cache, slots, *, q=None, q_out=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                           positions=None, cos_sin=None, interleaved: bool = False):
    """qlinear_kv_append into a cache in 4 bits: the rows of k (normed and rotated) and v are quantized
    where they are stored -> q_out (None without q)."""
    torch = _torch()
    lib = load_library()
    if k.dim() != 3:
        raise QLError(2, "k must be [tokens, heads, d]")
    t, _, d = k.shape
    dtype, device, args = k.dtype, k.get_device(), _ARGS
    at = args.at
    if q is not None:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=dtype, device=q.device)
        _heads(args.q, q, "q", t, d, dtype, device)
        _heads(args.q_out, q_out, "q_out", t, d, dtype, device)
    _heads(args.k, k, "k", t, d, dtype, device)
    _heads(args.v, v, "v", t, d, dtype, device)
    _paged_cache4(args.cache4, cache, d, device)
    slots_at = _array(slots, "slots", torch.int64, (t,), device)
    _norm_rope(args.nr, t, d, q_weight, k_weight, eps, positions, cos_sin, interleaved, device)
    status = lib.qlinear_kv_append_4bit(at["q"] if q is not None else None, at["q_out"], at["k"], at["v"], at["cache4"],
                                        slots_at, _dt(dtype), t, at["nr"], _stream_on(device))
    if status:
        _check(status)
    return q_out if q is not None else None


def qlinear_kv_read_4bit(cache, slots, *, dtype=None, k_out=None, v_out=None):
    """The rows at slots (int64 [t]; out of range: zeros) of a cache in 4 bits as values -> (k_out, v_out)
    [t, hk, d] in dtype (default bfloat16, or that of k_out or v_out)."""
    torch = _torch()
    lib = load_library()
    device, args = slots.get_device(), _ARGS
    _paged_cache4(args.cache4, cache, None, device)
    t, hk, d = slots.shape[0], args.cache4.hk, args.cache4.d
    given = k_out if k_out is not None else v_out
    dtype = dtype or (given.dtype if given is not None else torch.bfloat16)
    if k_out is None:
        k_out = torch.empty((t, hk, d), dtype=dtype, device=slots.device)
    if v_out is None:
        v_out = torch.empty((t, hk, d), dtype=dtype, device=slots.device)
    _heads(args.k, k_out, "k_out", t, d, dtype, device)
    _heads(args.v, v_out, "v_out", t, d, dtype, device)
    slots_at = _array(slots, "slots", torch.int64, (t,), device)
    status = lib.qlinear_kv_read_4bit(args.at["cache4"], slots_at, t, args.at["k"], args.at["v"], _dt(dtype),
                                      _stream_on(device))
    if status:
        _check(status)
    return k_out, v_out


def qlinear_paged_attention_4bit_workspace_size(q, cache, block_table, *, max_q: int, window: int = 0) -> int:
    t, hq, d = q.shape
    return int(load_library().qlinear_paged_attention_4bit_workspace_size(
        t, block_table.shape[0], hq, cache[0].shape[2], d, max_q, block_table.shape[1], cache[0].shape[1], window))


def qlinear_paged_attention_4bit(q, cache, block_table, cu_q, kv_lens, *, max_q: int, scale=None, window: int = 0,
                                 sinks=None, out=None, workspace=None):
    """qlinear_paged_attention over a cache in 4 bits; q and out bfloat16 or float16 -> out [t, hq, d]."""
    torch = _torch()
    lib = load_library()
    if q.dim() != 3:
        raise QLError(2, "q must be [tokens, heads, d]")
    t, hq, d = q.shape
    dtype, device, args = q.dtype, q.get_device(), _ARGS
    at = args.at
    if out is None:
        out = torch.empty((t, hq, d), dtype=dtype, device=q.device)
    _heads(args.q, q, "q", t, d, dtype, device)
    _heads(args.q_out, out, "out", t, d, dtype, device)
    _paged_cache4(args.cache4, cache, d, device)
    n_seqs, max_pages, row = _block_table(block_table, device)
    cu_at = _array(cu_q, "cu_q", torch.int32, (n_seqs + 1,), device)
    lens_at = _array(kv_lens, "kv_lens", torch.int32, (n_seqs,), device)
    sinks_at = _array(sinks, "sinks", torch.float32, (hq,), device)
    if workspace is None:
        need = qlinear_paged_attention_4bit_workspace_size(q, cache, block_table, max_q=max_q, window=window)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    elif not workspace.is_contiguous():
        raise QLError(2, "workspace must be contiguous")
    _same_device(workspace, "workspace", device)
    status = lib.qlinear_paged_attention_4bit(at["q"], at["q_out"], _dt(dtype), t, at["cache4"], block_table.data_ptr(), row,
                                              max_pages, cu_at, lens_at, n_seqs, max_q, d ** -0.5 if scale is None else scale,
                                              window, sinks_at, workspace.data_ptr(), workspace.nbytes, _stream_on(device))
    if status:
        _check(status)
    return out


def qlinear_kv_extend(counts, lens, block_table, *, page_size: int, rows: int, free_pages=None, free_count=None,
                      lens_out=None, free_count_out=None, cu_q=None, positions=None, slots=None, info=None):
    """One step of a paged cache's tables on the device.  Sequence s, with lens[s] cached tokens in the pages
    block_table[s], brings counts[s] new ones (below 0: it is through, its pages go back); pages are
    taken from the top of free_pages[:free_count] and put back there -> (cu_q [n_seqs + 1], positions
    [rows], slots [rows], info [4] = tokens, pages taken, why refused (0: done), free pages left).
    lens and free_count (int32, as all but positions and slots) are updated in place unless lens_out and
    free_count_out are given.  A step that cannot be done changes nothing (see qlinear.h for why)."""
    torch = _torch()
    lib = load_library()
    device, i32, i64 = counts.get_device(), torch.int32, torch.int64
    if counts.dim() != 1:
        raise QLError(2, "counts must be [n_seqs]")
    n_seqs, max_pages, row = _block_table(block_table, device)
    cap = 0
    if (free_pages is None) != (free_count is None):
        raise QLError(1, "free_pages and free_count must be given together")
    if free_pages is not None:
        if free_pages.dim() != 1:
            raise QLError(2, "free_pages must be [entries]")
        cap = free_pages.shape[0]
    counts_at, lens_at = _array(counts, "counts", i32, (n_seqs,), device), _array(lens, "lens", i32, (n_seqs,), device)
    list_at, count_at = _array(free_pages, "free_pages", i32, (cap,), device), _array(free_count, "free_count", i32, (1,), device)
    if cap == 0 and free_pages is not None:
        list_at = count_at  # an empty tensor has no address: any that is not NULL, since no entry is touched
    lens_out_at = lens_at if lens_out is None else _array(lens_out, "lens_out", i32, (n_seqs,), device)
    count_out_at = count_at if free_count_out is None else _array(free_count_out, "free_count_out", i32, (1,), device)
    cu_q, cu_at = _result(cu_q, "cu_q", i32, (n_seqs + 1,), counts, device)
    positions, pos_at = _result(positions, "positions", i64, (rows,), counts, device)
    slots, slots_at = _result(slots, "slots", i64, (rows,), counts, device)
    info, info_at = _result(info, "info", i32, (4,), counts, device)
    status = lib.qlinear_kv_extend(counts_at, lens_at, n_seqs, block_table.data_ptr(), row, max_pages, page_size, list_at, cap,
                                   count_at, lens_out_at, count_out_at, cu_at, pos_at, slots_at, rows, info_at,
                                   _stream_on(device))
    if status:
        _check(status)
    return cu_q, positions, slots, info


def qlinear_select_experts(logits, k: int, *, sigmoid: bool = False, bias=None, n_groups: int = 1, top_groups: int = 1,
                           group_top: int = 1, renormalize: bool = True, scale: float = 1.0, n_rows=None, ids=None,
                           weights=None):
    """The k experts of each row of router logits [t, e] and their weights -> (ids int64 [t, k], weights
    fp32 [t, k]), for qlinear_apply_experts and qlinear_combine_experts.  Softmax or sigmoid scores; bias
    (fp32 [e]) counts in the choice only; the choice lies within the top_groups of n_groups groups with the
    largest score (or, group_top = 2, sum of two); n_rows (int32 [1], device): rows behind it get -1 and 0."""
    torch = _torch()
    lib = load_library()
    if logits.dim() != 2:
        raise QLError(2, "logits must be [tokens, experts]")
    t, e = logits.shape
    device = logits.get_device()
    row, place = logits.stride()
    if place != 1 and e > 1:
        raise QLError(2, "the rows of logits must be contiguous")
    ids, ids_at = _result(ids, "ids", torch.int64, (t, k), logits, device)
    weights, weights_at = _result(weights, "weights", torch.float32, (t, k), logits, device)
    status = lib.qlinear_select_experts(logits.data_ptr(), _dt(logits), t, e, row if t > 1 else e,
                                        _array(bias, "bias", torch.float32, (e,), device), 1 if sigmoid else 0, n_groups,
                                        top_groups, group_top, k, 1 if renormalize else 0, scale,
                                        _array(n_rows, "n_rows", torch.int32, (1,), device), ids_at, weights_at,
                                        _stream_on(device))
    if status:
        _check(status)
    return ids, weights


def qlinear_combine_experts(y, weights, *, ids=None, e: int = 0, residual=None, out=None):
    """residual [t, n] + the sum of y's k rows of each token (y [t * k, n], as qlinear_apply_experts gives them)
    times weights (fp32 [t, k]) -> out [t, n] in y's dtype.  Positions whose id (int64 [t, k]) lies outside
    [0, e) add nothing: ids and e, the number of experts, are given together.  out may be residual."""
    torch = _torch()
    lib = load_library()
    if weights.dim() != 2 or y.dim() != 2:
        raise QLError(2, "weights must be [tokens, k] and y [tokens * k, n]")
    if ids is not None and e < 1:
        raise QLError(2, "e, the number of experts, must be given with ids")
    (t, k), n = weights.shape, y.shape[1]
    device = y.get_device()
    out, out_at = _result(out, "out", y.dtype, (t, n), y, device)
    status = lib.qlinear_combine_experts(_array(y, "y", y.dtype, (t * k, n), device), _dt(y),
                                         _array(weights, "weights", torch.float32, (t, k), device),
                                         _array(ids, "ids", torch.int64, (t, k), device), e,
                                         _array(residual, "residual", y.dtype, (t, n), device), t, k, n, out_at,
                                         _stream_on(device))
    if status:
        _check(status)
    return out
