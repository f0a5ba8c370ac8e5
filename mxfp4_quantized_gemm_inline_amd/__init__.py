"""Inline-quantized A4W4 MXFP4 GEMM for MI355X (gfx950).

A thin Python binding over the C ABI in ``include/mx.h`` (``libmxgemm.so``, built
in-tree by ``python -m mxfp4_quantized_gemm_inline_amd.build``). Every function here
only marshals arguments: torch supplies device memory and the current HIP stream, and
all computation runs in the library's HIP kernels. There is no fallback: if the library
is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import functools
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmxgemm.so")

# Symbols declared in include/mx.h, with ctypes signatures.
_c_i64, _c_sz, _vp, _c_int = ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int
SIGNATURES = {
    "mx_status_string": (ctypes.c_char_p, [_c_int]),
    "mx_prepared_layout_version": (_c_int, []),
    "mx_prepared_weight_bytes": (_c_sz, [_c_i64, _c_i64]),
    "mx_prepare_weight": (_c_int, [_vp, _c_i64, _c_i64, _vp, _vp]),
    "mx_prepare_weight_packed": (_c_int, [_vp, _vp, _c_i64, _c_i64, _vp, _vp]),
    "mx_unprepare_weight": (_c_int, [_vp, _c_i64, _c_i64, _vp, _vp, _vp]),
    "mx_quant_act": (_c_int, [_vp, _c_i64, _c_i64, _vp, _vp, _vp]),
    "mx_a4w4_gemm_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_i64]),
    "mx_a4w4_gemm": (_c_int, [_vp, _vp, _vp, _c_i64, _c_i64, _c_i64, _vp, _c_sz, _vp]),
    "mx_a4w4_gemm_grouped": (_c_int, [_vp, _vp, _vp, _c_i64, _c_i64, _vp, _vp, _c_i64, _c_i64,
                                      _c_i64, _c_i64, _vp]),
    "mx_a4w4_gemm_plan": (_c_int, [_c_i64, _c_i64, _c_i64, _c_sz, ctypes.c_char_p, _c_sz]),
    "mx_a16w4_gemm_plan": (_c_int, [_c_i64, _c_i64, _c_i64, ctypes.c_char_p, _c_sz]),
    "mx_a4w4_gemm_grouped_plan": (_c_int, [_c_i64, _c_i64, _c_i64, _c_i64, _c_i64, _c_i64, ctypes.c_char_p,
                                           _c_sz]),
    "mx_a4w4_gemm_grouped_act_quant": (_c_int, [_vp, _vp, _vp, _c_i64, _c_i64, _vp, _c_i64, _c_i64, _c_i64,
                                                ctypes.c_int32, _c_i64, _vp, _vp, _vp]),
    "mx_a4w4_gemm_grouped_act_quant_plan": (_c_int, [_c_i64, _c_i64, _c_i64, _c_i64, ctypes.c_int32, _c_i64, ctypes.c_char_p,
                                                     _c_sz]),
    "mx_a4w4_gemm_grouped_mx": (_c_int, [_vp, _vp, _vp, _c_i64, _c_i64, _vp, _vp, _c_i64, _c_i64, _c_i64, _vp]),
    "mx_a4w4_gemm_grouped_mx_plan": (_c_int, [_c_i64, _c_i64, _c_i64, ctypes.c_char_p, _c_sz]),
    "mx_moe_combine": (_c_int, [_vp, _c_i64, _vp, _vp, _c_i64, _c_i64, _c_i64, _vp, _vp]),
    "mx_a16w4_gemm": (_c_int, [_vp, _vp, _vp, _c_i64, _c_i64, _c_i64, _vp]),
    "mx_a4w4_gemm_noalloc": (_c_int, [_vp, _vp, _vp, _c_i64, _c_i64, _c_i64, _vp]),
    "mx_noalloc_scratch_bytes": (_c_sz, []),
    "mx_kv_cache_bytes": (_c_sz, [_c_i64, _c_i64, _c_i64, _c_i64]),
    "mx_kv_tables": (_c_int, [_vp, _vp, _c_i64, _c_i64, _vp, _c_i64, _vp, _c_i64, _vp, _vp, _c_i64, _vp, _vp, _vp, _vp,
                              _vp, _c_sz, _vp]),
    "mx_kv_tables_workspace_bytes": (_c_sz, [_c_i64, _c_i64]),
    "mx_kv_write": (_c_int, [_vp, _c_i64, _vp, _c_i64, _vp, _c_i64, _vp, _c_i64, _c_i64, _c_i64, _c_i64, _vp]),
    "mx_kv_read": (_c_int, [_vp, _c_i64, _c_i64, _c_i64, _c_i64, _vp, _c_i64, _vp, _vp, _vp]),
    "mx_kv_attention": (_c_int, [_vp, _c_i64, _vp, _c_i64, _c_i64, _vp, _c_i64, _vp, _vp, _c_i64, _c_i64, _c_i64, _c_i64,
                                 _c_i64, _c_i64, _c_i64, ctypes.c_int32, _c_i64, ctypes.c_float, _vp, _c_i64, _vp, _c_sz,
                                 _vp]),
    "mx_kv_attention_workspace_bytes": (_c_sz, [_c_i64] * 8),
    "mx_kv_attention_plan": (_c_int, [_c_i64] * 8 + [_c_sz, ctypes.c_char_p, _c_sz]),
    "mx_moe_route": (_c_int, [_vp, _c_i64, _c_int, _vp, _c_i64, _c_i64, _c_i64, _c_int, _c_i64, _c_i64, _c_int, _c_int,
                              ctypes.c_float, _vp, _vp, _vp, _vp]),
    "mx_moe_sort": (_c_int, [_vp, _c_i64, _c_i64, _c_i64, _c_i64, _vp, _vp, _vp, _vp, _c_sz, _vp]),
    "mx_moe_sort_workspace_bytes": (_c_sz, [_c_i64] * 3),
    "mx_kv_append": (_c_int, [_vp, _c_i64, _vp, _c_i64, _vp, _c_i64, _vp, _vp, _c_i64, _c_i64, _c_i64, _c_i64, _vp, _c_i64,
                              _c_i64, _vp, _vp, ctypes.c_float, _vp, _c_i64, _c_int, ctypes.c_float, _vp, _c_i64, _vp]),
    "mx_verify_drafts": (_c_int, [_vp, _c_i64, _vp, _c_i64, _vp, _vp, _vp, _vp, _vp, _c_i64, _c_i64, _c_i64, _vp, _vp, _vp,
                                  _vp, _c_sz, _vp]),
    "mx_verify_drafts_workspace_bytes": (_c_sz, [_c_i64] * 2),
    "mx_calib_read": (_c_int, [_vp, _c_sz, _c_i64, _vp, _vp]),
    "mx_calib_mfma": (_c_int, [_c_i64, _c_i64, _vp, _vp]),
    "mx_calib_mfma_flops": (ctypes.c_double, [_c_i64, _c_i64]),
    "mx_calib_mfma_operands": (_c_int, [_vp, _c_sz, _c_i64, _c_i64, _vp, _vp]),
    "mx_calib_mfma_operands_flops": (ctypes.c_double, [_c_i64, _c_i64]),
    "mx_calib_mfma_operands_clock": (_c_int, [_vp, _c_sz, _c_i64, _c_i64, _vp, _vp, _vp]),
}

MX_OK, MX_ERR_NULL, MX_ERR_SHAPE, MX_ERR_ALIGN, MX_ERR_DEVICE, MX_ERR_WORKSPACE, MX_ERR_HIP = range(7)
MX_ACT_SILU, MX_ACT_SWIGLU = 0, 1
MX_SCORE_SOFTMAX, MX_SCORE_SIGMOID = 0, 1
MX_ROPE_HALVES, MX_ROPE_PAIRS = 0, 1

_lib = None


class MxError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing; build it with "
                              "`python -m mxfp4_quantized_gemm_inline_amd.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().mx_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != MX_OK:
        raise MxError(status, what)


# ----------------------------------------------------------------------------- torch marshalling

def _torch():
    import torch
    return torch


def _stream_ptr(stream=None) -> int:
    torch = _torch()
    if stream is None:
        # the handle alone where this torch gives it: its Stream object costs more than a small
        # call's checks together (2.7 against 0.1 us)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return int(raw(torch.cuda.current_device()))
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _need(t, name, dtype=None, shape=None, min_bytes=None, min_numel=None):
    """Validate a tensor argument from its metadata alone (type, dtype, shape, size), before
    any device pointer is taken: a short or mis-shaped buffer would otherwise be read or
    written out of bounds by the kernels, which receive only pointers and sizes."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(int(d) for d in shape):
        raise ValueError(f"{name} must have shape {tuple(int(d) for d in shape)}, got {tuple(t.shape)}")
    if min_bytes is not None and t.numel() * t.element_size() < min_bytes:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes, needs at least {min_bytes}")
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs at least {min_numel}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _dev(t, dtype, name):
    """Device pointer of a validated tensor (raises if it is not on the current device)."""
    torch = _torch()
    _need(t, name, dtype)
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.device.index is not None and t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, not on the current device cuda:{torch.cuda.current_device()}")
    return t.data_ptr()


def _dims2(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    return int(t.shape[0]), int(t.shape[1])


def mx_prepared_layout_version() -> int:
    return int(lib().mx_prepared_layout_version())


def mx_prepared_weight_bytes(N: int, K: int) -> int:
    return int(lib().mx_prepared_weight_bytes(int(N), int(K)))


def mx_a4w4_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().mx_a4w4_gemm_workspace_bytes(int(M), int(N), int(K)))


def mx_prepare_weight(w_bf16, out=None, stream=None):
    """W [N, K] bf16 -> opaque prepared MXFP4 blob (uint8, mx_prepared_weight_bytes(N, K))."""
    torch = _torch()
    _need(w_bf16, "w_bf16", torch.bfloat16)
    N, K = _dims2(w_bf16, "w_bf16")
    nbytes = mx_prepared_weight_bytes(N, K)
    if out is None:
        out = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=w_bf16.device)
    _need(out, "out", torch.uint8, min_bytes=nbytes)
    _check(lib().mx_prepare_weight(_dev(w_bf16, torch.bfloat16, "w_bf16"), N, K,
                                   _dev(out, torch.uint8, "w_prep"), _stream_ptr(stream)),
           "mx_prepare_weight")
    return out


def mx_prepare_weight_packed(w_fp4, w_scale, out=None, stream=None):
    """Caller-quantized weight -> prepared blob: w_fp4 uint8 [N, K/2] (low nibble = even k),
    w_scale uint8 [N, K/32] (E8M0)."""
    torch = _torch()
    _need(w_fp4, "w_fp4", torch.uint8)
    N, K2 = _dims2(w_fp4, "w_fp4")
    K = 2 * K2
    _need(w_scale, "w_scale", torch.uint8, shape=(N, K // 32))
    nbytes = mx_prepared_weight_bytes(N, K)
    if out is None:
        out = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=w_fp4.device)
    _need(out, "out", torch.uint8, min_bytes=nbytes)
    _check(lib().mx_prepare_weight_packed(_dev(w_fp4, torch.uint8, "w_fp4"), _dev(w_scale, torch.uint8, "w_scale"),
                                          N, K, _dev(out, torch.uint8, "w_prep"), _stream_ptr(stream)),
           "mx_prepare_weight_packed")
    return out


def mx_unprepare_weight(w_prep, N: int, K: int, stream=None):
    """Prepared blob -> canonical (payload uint8 [N, K/2], scales uint8 [N, K/32])."""
    torch = _torch()
    _need(w_prep, "w_prep", torch.uint8, min_bytes=mx_prepared_weight_bytes(N, K))
    q = torch.empty((N, K // 2), dtype=torch.uint8, device=w_prep.device)
    s = torch.empty((N, K // 32), dtype=torch.uint8, device=w_prep.device)
    _check(lib().mx_unprepare_weight(_dev(w_prep, torch.uint8, "w_prep"), N, K,
                                     _dev(q, None, "w_fp4"), _dev(s, None, "w_scale"),
                                     _stream_ptr(stream)), "mx_unprepare_weight")
    return q, s


def mx_quant_act(a_bf16, q_out=None, s_out=None, stream=None):
    """A [M, K] bf16 -> (payload uint8 [M, K/2], scales uint8 [M, K/32]), canonical layout."""
    torch = _torch()
    _need(a_bf16, "a_bf16", torch.bfloat16)
    M, K = _dims2(a_bf16, "a_bf16")
    q = q_out if q_out is not None else torch.empty((M, K // 2), dtype=torch.uint8, device=a_bf16.device)
    s = s_out if s_out is not None else torch.empty((M, K // 32), dtype=torch.uint8, device=a_bf16.device)
    _need(q, "a_fp4", torch.uint8, min_bytes=M * (K // 2))
    _need(s, "a_scale", torch.uint8, min_bytes=M * (K // 32))
    if M == 0:
        return q, s
    _check(lib().mx_quant_act(_dev(a_bf16, torch.bfloat16, "a_bf16"), M, K, _dev(q, torch.uint8, "a_fp4"),
                              _dev(s, torch.uint8, "a_scale"), _stream_ptr(stream)), "mx_quant_act")
    return q, s


def mx_a4w4_gemm(a_bf16, w_prep, N: int, out=None, workspace=None, stream=None):
    """C [M, N] bf16 = Q(A) Q(W)^T with A [M, K] bf16 and a prepared weight of shape [N, K].

    workspace: a device tensor for split-K partials, None to allocate
    mx_a4w4_gemm_workspace_bytes(M, N, K) bytes through torch, or False to pass none
    (the library then picks a configuration that needs no workspace).
    """
    torch = _torch()
    _need(a_bf16, "a_bf16", torch.bfloat16)
    M, K = _dims2(a_bf16, "a_bf16")
    _need(w_prep, "w_prep", torch.uint8, min_bytes=max(1, mx_prepared_weight_bytes(N, K)))
    c = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=a_bf16.device)
    _need(c, "out", torch.bfloat16, shape=(M, N))
    if M == 0:
        return c
    if workspace is None:
        nbytes = mx_a4w4_gemm_workspace_bytes(M, N, K)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=a_bf16.device) if nbytes else False
    ws_ptr, ws_bytes = (None, 0)
    if workspace is not False:
        ws_ptr, ws_bytes = _dev(workspace, None, "workspace"), workspace.numel() * workspace.element_size()
    _check(lib().mx_a4w4_gemm(_dev(a_bf16, torch.bfloat16, "a_bf16"), _dev(w_prep, torch.uint8, "w_prep"),
                              _dev(c, torch.bfloat16, "c_bf16"), M, int(N), K, ws_ptr, ws_bytes,
                              _stream_ptr(stream)), "mx_a4w4_gemm")
    return c


def mx_noalloc_scratch_bytes() -> int:
    """Size of the device scratch array mx_a4w4_gemm_noalloc uses in place of a workspace."""
    return int(lib().mx_noalloc_scratch_bytes())


def mx_a4w4_gemm_noalloc(a_bf16, w_prep, N: int, out, stream=None):
    """mx_a4w4_gemm without a caller workspace and without any allocation: the library's own
    device scratch array serves as the workspace (calls that overlap on one device share it).
    `out` [M, N] bf16 is required (allocating it here would defeat the purpose)."""
    torch = _torch()
    _need(a_bf16, "a_bf16", torch.bfloat16)
    M, K = _dims2(a_bf16, "a_bf16")
    _need(w_prep, "w_prep", torch.uint8, min_bytes=max(1, mx_prepared_weight_bytes(N, K)))
    _need(out, "out", torch.bfloat16, shape=(M, N))
    if M == 0:
        return out
    _check(lib().mx_a4w4_gemm_noalloc(_dev(a_bf16, torch.bfloat16, "a_bf16"), _dev(w_prep, torch.uint8, "w_prep"),
                                      _dev(out, torch.bfloat16, "c_bf16"), M, int(N), K, _stream_ptr(stream)),
           "mx_a4w4_gemm_noalloc")
    return out


def _grouped_tables(row_token, expert_offsets, w_prep_stacked, E, R_max, N, K):
    """The segment table, the row-to-token map and the stacked weights of a grouped call:
    expert_offsets [E+1] int32, row_token at least R_max int32 (when rows exist), E prepared
    weights of shape [N, K]."""
    torch = _torch()
    _need(expert_offsets, "expert_offsets", torch.int32, min_numel=int(E) + 1)
    if row_token is not None and R_max > 0:
        _need(row_token, "row_token", torch.int32, min_numel=int(R_max))
    _need(w_prep_stacked, "w_prep_stacked", torch.uint8,
          min_bytes=max(1, int(E) * mx_prepared_weight_bytes(N, K)))


def mx_a4w4_gemm_grouped(a_bf16, row_token, expert_offsets, E: int, R_max: int, w_prep_stacked,
                         N: int, rows_hint: int = 1, out=None, stream=None):
    """Grouped GEMM1: C [R_max, N] bf16, rows in expert-sorted order (rows >= R untouched)."""
    torch = _torch()
    _need(a_bf16, "a_bf16", torch.bfloat16)
    T, K = _dims2(a_bf16, "a_bf16")
    _grouped_tables(row_token, expert_offsets, w_prep_stacked, E, R_max, N, K)
    c = out if out is not None else torch.empty((R_max, N), dtype=torch.bfloat16, device=a_bf16.device)
    _need(c, "out", torch.bfloat16, shape=(R_max, N))
    _check(lib().mx_a4w4_gemm_grouped(
        _dev(a_bf16, torch.bfloat16, "a_bf16") if T > 0 else None,
        _dev(row_token, torch.int32, "row_token") if R_max > 0 else None,
        _dev(expert_offsets, torch.int32, "expert_offsets"), int(E), int(R_max),
        _dev(w_prep_stacked, torch.uint8, "w_prep_stacked"), _dev(c, torch.bfloat16, "c_bf16") if R_max > 0 else None,
        T, int(N), K, int(rows_hint), _stream_ptr(stream)), "mx_a4w4_gemm_grouped")
    return c


def mx_a4w4_gemm_grouped_act_quant(a_bf16, row_token, expert_offsets, E: int, R_max: int, w_prep_stacked,
                                   N: int, act: int = MX_ACT_SWIGLU, rows_hint: int = 1, h_fp4=None, h_scale=None,
                                   stream=None):
    """Grouped GEMM1 with fused SiLU / SwiGLU + MXFP4 quantization: returns (h_fp4 uint8
    [R_max, Nh/2], h_scale uint8 [R_max, Nh/32]) with Nh = N/2 (SwiGLU) or N (SiLU)."""
    torch = _torch()
    _need(a_bf16, "a_bf16", torch.bfloat16)
    T, K = _dims2(a_bf16, "a_bf16")
    _grouped_tables(row_token, expert_offsets, w_prep_stacked, E, R_max, N, K)
    Nh = N // 2 if act == MX_ACT_SWIGLU else N
    if h_fp4 is None:
        h_fp4 = torch.empty((R_max, Nh // 2), dtype=torch.uint8, device=a_bf16.device)
    if h_scale is None:
        h_scale = torch.empty((R_max, Nh // 32), dtype=torch.uint8, device=a_bf16.device)
    _need(h_fp4, "h_fp4", torch.uint8, min_bytes=R_max * (Nh // 2))
    _need(h_scale, "h_scale", torch.uint8, min_bytes=R_max * (Nh // 32))
    _check(lib().mx_a4w4_gemm_grouped_act_quant(
        _dev(a_bf16, torch.bfloat16, "a_bf16") if T > 0 else None,
        _dev(row_token, torch.int32, "row_token") if R_max > 0 else None,
        _dev(expert_offsets, torch.int32, "expert_offsets"), int(E), int(R_max),
        _dev(w_prep_stacked, torch.uint8, "w_prep_stacked"), T, int(N), K, int(act), int(rows_hint),
        _dev(h_fp4, torch.uint8, "h_fp4") if R_max > 0 else None,
        _dev(h_scale, torch.uint8, "h_scale") if R_max > 0 else None, _stream_ptr(stream)),
        "mx_a4w4_gemm_grouped_act_quant")
    return h_fp4, h_scale


def mx_a4w4_gemm_grouped_act_quant_plan(E: int, R_max: int, N: int, K: int, act: int = MX_ACT_SWIGLU,
                                        rows_hint: int = 1) -> str:
    """Kernel mx_a4w4_gemm_grouped_act_quant launches for this table size, shape and hint."""
    buf = ctypes.create_string_buffer(256)
    _check(lib().mx_a4w4_gemm_grouped_act_quant_plan(int(E), int(R_max), int(N), int(K), int(act), int(rows_hint),
                                                     buf, len(buf)),
           "mx_a4w4_gemm_grouped_act_quant_plan")
    return buf.value.decode()


def mx_a4w4_gemm_grouped_mx(a_fp4, a_scale, expert_offsets, E: int, R_max: int, w_prep_stacked, N: int,
                            rows_hint: int = 1, out=None, stream=None):
    """Second MoE GEMM on MXFP4 rows: a_fp4 uint8 [R_max, K/2], a_scale uint8 [R_max, K/32]
    -> C [R_max, N] bf16 (rows >= R untouched)."""
    torch = _torch()
    _need(a_fp4, "a_fp4", torch.uint8)
    rows, K2 = _dims2(a_fp4, "a_fp4")
    K = 2 * K2
    _need(a_scale, "a_scale", torch.uint8, shape=(rows, K // 32))
    if rows < R_max:
        raise ValueError(f"a_fp4 / a_scale hold {rows} rows, need at least R_max = {R_max}")
    _grouped_tables(None, expert_offsets, w_prep_stacked, E, R_max, N, K)
    c = out if out is not None else torch.empty((R_max, N), dtype=torch.bfloat16, device=a_fp4.device)
    _need(c, "out", torch.bfloat16, shape=(R_max, N))
    _check(lib().mx_a4w4_gemm_grouped_mx(
        _dev(a_fp4, torch.uint8, "a_fp4") if R_max > 0 else None,
        _dev(a_scale, torch.uint8, "a_scale") if R_max > 0 else None,
        _dev(expert_offsets, torch.int32, "expert_offsets"), int(E), int(R_max),
        _dev(w_prep_stacked, torch.uint8, "w_prep_stacked"), _dev(c, torch.bfloat16, "c_bf16") if R_max > 0 else None,
        int(N), K, int(rows_hint), _stream_ptr(stream)), "mx_a4w4_gemm_grouped_mx")
    return c


def mx_a4w4_gemm_grouped_mx_plan(N: int, K: int, rows_hint: int = 1) -> str:
    buf = ctypes.create_string_buffer(256)
    _check(lib().mx_a4w4_gemm_grouped_mx_plan(int(N), int(K), int(rows_hint), buf, len(buf)),
           "mx_a4w4_gemm_grouped_mx_plan")
    return buf.value.decode()


def mx_moe_combine(y_bf16, token_rows, token_weights, out=None, stream=None):
    """out [T, N] bf16 = sum_k token_weights[t, k] * y[token_rows[t, k]] (FP32, k order)."""
    torch = _torch()
    _need(y_bf16, "y_bf16", torch.bfloat16)
    R, N = _dims2(y_bf16, "y_bf16")
    _need(token_rows, "token_rows", torch.int32)
    T, topk = _dims2(token_rows, "token_rows")
    _need(token_weights, "token_weights", torch.float32, shape=(T, topk))
    o = out if out is not None else torch.empty((T, N), dtype=torch.bfloat16, device=token_rows.device)
    _need(o, "out", torch.bfloat16, shape=(T, N))
    _check(lib().mx_moe_combine(
        _dev(y_bf16, torch.bfloat16, "y_bf16") if R > 0 else None, R,
        _dev(token_rows, torch.int32, "token_rows") if T > 0 else None,
        _dev(token_weights, torch.float32, "token_weights") if T > 0 else None, T, topk, N,
        _dev(o, torch.bfloat16, "out_bf16") if T > 0 else None, _stream_ptr(stream)), "mx_moe_combine")
    return o


def mx_a16w4_gemm(a_bf16, w_prep, N: int, out=None, stream=None):
    """A16WFP4: A [M, K] bf16 (not quantized) x decoded prepared weight -> C [M, N] bf16."""
    torch = _torch()
    _need(a_bf16, "a_bf16", torch.bfloat16)
    M, K = _dims2(a_bf16, "a_bf16")
    _need(w_prep, "w_prep", torch.uint8, min_bytes=max(1, mx_prepared_weight_bytes(N, K)))
    c = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=a_bf16.device)
    _need(c, "out", torch.bfloat16, shape=(M, N))
    if M == 0:
        return c
    _check(lib().mx_a16w4_gemm(_dev(a_bf16, torch.bfloat16, "a_bf16"), _dev(w_prep, torch.uint8, "w_prep"),
                               _dev(c, torch.bfloat16, "c_bf16"), M, int(N), K, _stream_ptr(stream)),
           "mx_a16w4_gemm")
    return c


def mx_a4w4_gemm_plan(M: int, N: int, K: int, workspace_bytes=None) -> str:
    """Kernel(s) mx_a4w4_gemm launches for this shape; workspace_bytes defaults to what
    mx_a4w4_gemm allocates when given no workspace."""
    if workspace_bytes is None:
        workspace_bytes = mx_a4w4_gemm_workspace_bytes(M, N, K)
    buf = ctypes.create_string_buffer(256)
    _check(lib().mx_a4w4_gemm_plan(int(M), int(N), int(K), int(workspace_bytes), buf, len(buf)),
           "mx_a4w4_gemm_plan")
    return buf.value.decode()


def mx_a16w4_gemm_plan(M: int, N: int, K: int) -> str:
    """Kernel mx_a16w4_gemm launches for this shape."""
    buf = ctypes.create_string_buffer(256)
    _check(lib().mx_a16w4_gemm_plan(int(M), int(N), int(K), buf, len(buf)), "mx_a16w4_gemm_plan")
    return buf.value.decode()


def mx_a4w4_gemm_grouped_plan(E: int, R_max: int, T: int, N: int, K: int, rows_hint: int = 1) -> str:
    """Kernel mx_a4w4_gemm_grouped launches for this table size, token count and hint."""
    buf = ctypes.create_string_buffer(256)
    _check(lib().mx_a4w4_gemm_grouped_plan(int(E), int(R_max), int(T), int(N), int(K), int(rows_hint), buf,
                                           len(buf)), "mx_a4w4_gemm_grouped_plan")
    return buf.value.decode()


# ----------------------------------------------------------------------------- the MXFP4 key/value cache

def mx_kv_cache_bytes(num_pages: int, page_size: int, heads: int, D: int) -> int:
    """Bytes of a paged MXFP4 key/value cache (0 for sizes the library refuses)."""
    return int(lib().mx_kv_cache_bytes(int(num_pages), int(page_size), int(heads), int(D)))


@functools.lru_cache(maxsize=1024)
def _kv_page_bytes(page_size: int, heads: int, D: int) -> int:
    per = mx_kv_cache_bytes(1, page_size, heads, D)
    if per == 0:
        raise MxError(MX_ERR_SHAPE, f"kv cache with page_size={page_size}, heads={heads}, D={D}")
    return per


def _kv_pages(cache, page_size, heads, D):
    """Pages that fit the uint8 buffer `cache`."""
    _meta(cache, "cache", _torch().uint8)
    per = _kv_page_bytes(int(page_size), int(heads), int(D))
    pages = cache.numel() // per
    if pages < 1:
        raise ValueError(f"cache holds {cache.numel()} bytes, one page needs {per}")
    return pages


def _new(shape, dtype, like, stream):
    """A new tensor of the stream that the call runs on, so that torch neither hands out memory
    the current stream still uses nor reuses it under a kernel of `stream`."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _meta(t, name, dtype, least=0):
    """The checks of _need that the cache calls use, in one pass: a decoding step makes a few of
    these calls per layer, with up to ten tensors each."""
    try:
        if t.dtype is dtype and t.numel() >= least and t.is_contiguous():
            return
    except AttributeError:
        pass
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() < least:
        raise ValueError(f"{name} holds {t.numel()} elements, needs at least {least}")
    raise ValueError(f"{name} must be contiguous")


def _workspace_size(t):
    """Bytes of a workspace, a contiguous tensor of any type."""
    _meta(t, "workspace", getattr(t, "dtype", None))
    return t.numel() * t.element_size()


def _rows3(t, name):
    """(rows, heads, D, row stride) of a bf16 [rows, heads, D] tensor whose rows are dense (a
    slice of columns of a wider row-major tensor is)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D, got shape {tuple(t.shape)}")
    (T, H, D), (row, head, one) = t.shape, t.stride()
    if (D > 1 and one != 1) or (H > 1 and head != D):
        raise ValueError(f"{name} must have dense rows, got strides {t.stride()}")
    return T, H, D, row if T > 1 else H * D


def _pointers(names, *tensors):
    """Device pointers of tensors whose metadata was checked (None stays None): all of them on
    the current device. names: theirs, in one string."""
    current = _torch().cuda.current_device() if tensors[0].is_cuda else None
    out = []
    for i, t in enumerate(tensors):
        if t is None:
            out.append(None)
            continue
        if t.get_device() != current:
            name = names.split()[i]
            if not t.is_cuda:
                raise ValueError(f"{name} must be a device tensor")
            raise ValueError(f"{name} is on {t.device}, not on the current device cuda:{_torch().cuda.current_device()}")
        out.append(t.data_ptr())
    return out


@functools.lru_cache(maxsize=1024)
def _kv_workspace_bytes(call: str, *sizes: int) -> int:
    """The library's answer by the sizes' values (ints only: another number's hash may be its identity)."""
    return int(getattr(lib(), call)(*sizes))


def mx_kv_tables_workspace_bytes(B: int, max_rows: int) -> int:
    return _kv_workspace_bytes("mx_kv_tables_workspace_bytes", int(B), int(max_rows))


def mx_kv_tables(old_lens, new_lens, block_table, free_pages, free_count, page_size: int, max_rows: int, cu_q=None,
                 slots=None, positions=None, free_count_out=None, status=None, workspace=None, stream=None):
    """Block tables and slots from the requests' lengths (int32 [B], before and after the step):
    block_table [B, max_blocks] and the stack free_pages [capacity] (both int32) are updated in
    place. Returns (cu_q int32 [B+1], slots int64 [max_rows], positions int32 [max_rows],
    free_count_out int32 [1], status int32 [1]); status 0 means done (see mx.h for the rest)."""
    torch = _torch()
    i32 = torch.int32
    _meta(block_table, "block_table", i32)
    B, max_blocks = _dims2(block_table, "block_table")
    for t, name in ((old_lens, "old_lens"), (new_lens, "new_lens")):
        _meta(t, name, i32)
        if t.shape != (B,):
            raise ValueError(f"{name} must have shape {(B,)}, got {tuple(t.shape)}")
    _meta(free_pages, "free_pages", i32)
    _meta(free_count, "free_count", i32, 1)
    max_rows = int(max_rows)
    rows = max(max_rows, 0)
    if cu_q is None and positions is None and free_count_out is None and status is None:
        cu_q, positions, free_count_out, status = _new((B + rows + 3,), i32, block_table, stream).split((B + 1, rows, 1, 1))
    else:
        cu_q = cu_q if cu_q is not None else _new((B + 1,), i32, block_table, stream)
        positions = positions if positions is not None else _new((rows,), i32, block_table, stream)
        free_count_out = free_count_out if free_count_out is not None else _new((1,), i32, block_table, stream)
        status = status if status is not None else _new((1,), i32, block_table, stream)
        _meta(cu_q, "cu_q", i32, B + 1)
        _meta(positions, "positions", i32, max_rows)
        _meta(free_count_out, "free_count_out", i32, 1)
        _meta(status, "status", i32, 1)
    if slots is None:
        slots = _new((rows,), torch.int64, block_table, stream)
    else:
        _meta(slots, "slots", torch.int64, max_rows)
    nbytes, ws_bytes = mx_kv_tables_workspace_bytes(B, max_rows), 0
    if nbytes:
        workspace = workspace if workspace is not None else _new((nbytes,), torch.uint8, block_table, stream)
        ws_bytes = _workspace_size(workspace)
    else:
        workspace = None
    old_, new_, table_, stack_, count_, out_, cu_, slots_, pos_, status_, ws_ = _pointers(
        "old_lens new_lens block_table free_pages free_count free_count_out cu_q slots positions status workspace", old_lens,
        new_lens, block_table, free_pages, free_count, free_count_out, cu_q, slots, positions, status, workspace)
    _check(lib().mx_kv_tables(old_, new_, B, int(page_size), table_, max_blocks, stack_, free_pages.numel(), count_, out_,
                              max_rows, cu_, slots_, pos_, status_, ws_, ws_bytes, _stream_ptr(stream)), "mx_kv_tables")
    return cu_q, slots, positions, free_count_out, status


def mx_kv_write(k_bf16, v_bf16, slots, cache, page_size: int, stream=None) -> None:
    """Quantize keys and values [T, heads, D] bf16 (rows dense, any row stride) to MXFP4 into the
    cache's slots (int64 [T]; a slot outside the cache writes nothing)."""
    T, heads, D, k_stride = _rows3(k_bf16, "k_bf16")
    shape = (T, heads, D)
    *v_shape, v_stride = _rows3(v_bf16, "v_bf16")
    if tuple(v_shape) != shape:
        raise ValueError(f"v_bf16 must have shape {shape}, got {tuple(v_shape)}")
    _meta(slots, "slots", _torch().int64, T)
    pages = _kv_pages(cache, page_size, heads, D)
    if T == 0:
        return
    k_, v_, slots_, cache_ = _pointers("k_bf16 v_bf16 slots cache", k_bf16, v_bf16, slots, cache)
    _check(lib().mx_kv_write(k_, k_stride, v_, v_stride, slots_, T, cache_, pages, int(page_size), heads, D,
                             _stream_ptr(stream)), "mx_kv_write")


def mx_kv_read(cache, slots, heads: int, D: int, page_size: int, k_out=None, v_out=None, stream=None):
    """(k, v) bf16 [T, heads, D]: the values the cache holds at `slots` (int64 [T]); rows whose
    slot is outside the cache are left as they were."""
    torch = _torch()
    _meta(slots, "slots", torch.int64)
    pages = _kv_pages(cache, page_size, heads, D)
    shape = (slots.numel(), int(heads), int(D))
    k = k_out if k_out is not None else _new(shape, torch.bfloat16, cache, stream)
    v = v_out if v_out is not None else _new(shape, torch.bfloat16, cache, stream)
    for t, name in ((k, "k_out"), (v, "v_out")):
        _meta(t, name, torch.bfloat16)
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if shape[0] == 0:
        return k, v
    cache_, slots_, k_, v_ = _pointers("cache slots k_out v_out", cache, slots, k, v)
    _check(lib().mx_kv_read(cache_, pages, int(page_size), shape[1], shape[2], slots_, shape[0], k_, v_,
                            _stream_ptr(stream)), "mx_kv_read")
    return k, v


def mx_kv_attention_workspace_bytes(B: int, T: int, heads_q: int, heads: int, D: int, max_q: int, max_kv: int,
                                    window: int = 0) -> int:
    return _kv_workspace_bytes("mx_kv_attention_workspace_bytes", int(B), int(T), int(heads_q), int(heads), int(D), int(max_q),
                               int(max_kv), int(window))


def mx_kv_attention(q_bf16, cache, block_table, cu_q, kv_lens, heads: int, page_size: int, causal: bool = True,
                    window: int = 0, scale=None, max_q=None, max_kv=None, out=None, workspace=None, stream=None):
    """Attention of q [T, heads_q, D] bf16 (rows dense, any row stride) over the paged cache:
    request b's rows are cu_q[b] .. cu_q[b+1] - 1 (int32 [B+1]) over kv_lens[b] cached tokens
    (int32 [B]) in the pages block_table[b] (int32 [B, max_blocks]), its last row at the last
    token. Returns out [T, heads_q, D] bf16.

    scale defaults to D ** -0.5. max_q and max_kv (the most rows and the longest length of any
    request) choose the kernels and their cuts and change no result but its last bits. They default
    to T and to the table's width, for which a batch pays: 64 single rows over up to 8192 tokens take
    144 us and 43 MB of workspace without max_q, 75 us and 8.5 MB with max_q=1. workspace: a device
    tensor for partial results, None to allocate mx_kv_attention_workspace_bytes(...) bytes through
    torch, or False to pass none.
    """
    torch = _torch()
    i32 = torch.int32
    T, heads_q, D, q_stride = _rows3(q_bf16, "q_bf16")
    _meta(block_table, "block_table", i32)
    B, max_blocks = _dims2(block_table, "block_table")
    _meta(cu_q, "cu_q", i32, B + 1)
    _meta(kv_lens, "kv_lens", i32, B)
    page_size, heads, window = int(page_size), int(heads), int(window)
    pages = _kv_pages(cache, page_size, heads, D)
    if out is None:
        out, out_stride = _new((T, heads_q, D), torch.bfloat16, q_bf16, stream), heads_q * D
    else:
        *shape, out_stride = _rows3(out, "out")
        if tuple(shape) != (T, heads_q, D):
            raise ValueError(f"out must have shape {(T, heads_q, D)}, got {tuple(shape)}")
    if T == 0 or B == 0:
        return out
    max_q = int(max_q) if max_q is not None else T
    max_kv = int(max_kv) if max_kv is not None else max_blocks * page_size
    scale = float(scale) if scale is not None else D ** -0.5
    if workspace is None:
        nbytes = mx_kv_attention_workspace_bytes(B, T, heads_q, heads, D, max_q, max_kv, window)
        workspace = _new((nbytes,), torch.uint8, q_bf16, stream) if nbytes else None
    elif workspace is False:
        workspace = None
    ws_bytes = 0
    if workspace is not None:
        ws_bytes = _workspace_size(workspace)
    q_, cache_, table_, cu_, kv_, out_, ws_ = _pointers(
        "q_bf16 cache block_table cu_q kv_lens out workspace", q_bf16, cache, block_table, cu_q, kv_lens, out, workspace)
    _check(lib().mx_kv_attention(q_, q_stride, cache_, pages, page_size, table_, max_blocks, cu_, kv_, B, T, heads_q, heads,
                                 D, max_q, max_kv, 1 if causal else 0, window, scale, out_, out_stride, ws_, ws_bytes,
                                 _stream_ptr(stream)), "mx_kv_attention")
    return out


def mx_kv_attention_plan(B: int, T: int, heads_q: int, heads: int, D: int, max_q: int, max_kv: int, window: int = 0,
                         workspace_bytes=None) -> str:
    """Kernels mx_kv_attention launches for these sizes; workspace_bytes defaults to what it
    allocates when given no workspace."""
    if workspace_bytes is None:
        workspace_bytes = mx_kv_attention_workspace_bytes(B, T, heads_q, heads, D, max_q, max_kv, window)
    buf = ctypes.create_string_buffer(256)
    _check(lib().mx_kv_attention_plan(int(B), int(T), int(heads_q), int(heads), int(D), int(max_q), int(max_kv),
                                      int(window), int(workspace_bytes), buf, len(buf)), "mx_kv_attention_plan")
    return buf.value.decode()


def mx_kv_append(q_bf16, k_bf16, v_bf16, positions, slots, cache, page_size: int, inv_freq=None, rope: int = MX_ROPE_HALVES,
                 rope_scale: float = 1.0, q_weight=None, k_weight=None, eps: float = 1e-6, q_out=None, stream=None):
    """Queries [T, heads_q, D], keys and values [T, heads, D] (bf16, rows dense, any row stride) on their
    way from a projection to mx_kv_attention: each head of queries and keys normed (q_weight, k_weight
    float32 [D], or None), its first 2 * len(inv_freq) elements rotated by positions (int32 [T]; below 0:
    padding, skipped) times inv_freq (float32, or None), keys and values quantized into the cache's slots
    (int64 [T]). Returns the queries, bf16 [T, heads_q, D] (q_out, which may be q_bf16 itself).

    q_bf16 may be None (no queries); k_bf16, v_bf16, slots and cache may be None together (a layer that
    reads another's cache)."""
    torch = _torch()
    f32 = torch.float32
    T = heads_q = heads = q_stride = k_stride = v_stride = out_stride = pages = 0
    if q_bf16 is not None:
        T, heads_q, D, q_stride = _rows3(q_bf16, "q_bf16")
    elif q_out is not None:
        raise ValueError("q_out without q_bf16")
    if k_bf16 is not None:
        Tk, heads, Dk, k_stride = _rows3(k_bf16, "k_bf16")
        if q_bf16 is not None and (Tk, Dk) != (T, D):
            raise ValueError(f"k_bf16 must have shape {(T, heads, D)}, got {tuple(k_bf16.shape)}")
        T, D = Tk, Dk
        *v_shape, v_stride = _rows3(v_bf16, "v_bf16")
        if tuple(v_shape) != (T, heads, D):
            raise ValueError(f"v_bf16 must have shape {(T, heads, D)}, got {tuple(v_shape)}")
        _meta(slots, "slots", torch.int64, T)
        pages = _kv_pages(cache, page_size, heads, D)
    elif q_bf16 is None:
        raise ValueError("neither queries nor keys")
    elif v_bf16 is not None or slots is not None or cache is not None:
        raise ValueError("k_bf16, v_bf16, slots and cache go together")
    _meta(positions, "positions", torch.int32, T)
    if q_weight is not None:
        _meta(q_weight, "q_weight", f32, D)
    if k_weight is not None:
        _meta(k_weight, "k_weight", f32, D)
    rot = 0
    if inv_freq is not None:
        _meta(inv_freq, "inv_freq", f32)
        rot = 2 * inv_freq.numel()
    if q_bf16 is not None:
        if q_out is None:
            q_out, out_stride = _new((T, heads_q, D), torch.bfloat16, q_bf16, stream), heads_q * D
        else:
            *shape, out_stride = _rows3(q_out, "q_out")
            if tuple(shape) != (T, heads_q, D):
                raise ValueError(f"q_out must have shape {(T, heads_q, D)}, got {tuple(shape)}")
    if T == 0:
        return q_out
    pos_, q_, k_, v_, slots_, cache_, qw_, kw_, freq_, out_ = _pointers(
        "positions q_bf16 k_bf16 v_bf16 slots cache q_weight k_weight inv_freq q_out", positions, q_bf16, k_bf16, v_bf16, slots, cache,
        q_weight, k_weight, inv_freq, q_out)
    _check(lib().mx_kv_append(q_, q_stride, k_, k_stride, v_, v_stride, pos_, slots_, T, heads_q, heads, D, cache_, pages,
                              int(page_size), qw_, kw_, float(eps), freq_, rot, int(rope), float(rope_scale), out_, out_stride,
                              _stream_ptr(stream)), "mx_kv_append")
    return q_out


def mx_verify_drafts_workspace_bytes(B: int, V: int) -> int:
    return _kv_workspace_bytes("mx_verify_drafts_workspace_bytes", int(B), int(V))


def mx_verify_drafts(target_probs, draft_probs, tokens, cu_q, kv_lens, accept_random, sample_random, out_tokens=None, accepted=None,
                     new_lens=None, workspace=None, stream=None):
    """Drafts against the target's probabilities: request b's rows cu_q[b] .. cu_q[b+1] - 1 of tokens (int32
    [T]) are its last token and its drafts, target_probs and draft_probs (float32 [T, V]; draft_probs None
    for drafts without chance) the distributions after each row, accept_random [T] and sample_random [B]
    (float32) the numbers in [0, 1) that decide. Returns (out_tokens int32 [T]: accepted drafts, then the
    next token, then -1; accepted int32 [B]; new_lens int32 [B]: kv_lens less the refused drafts).

    Where neither outputs nor workspace are given they are parts of one allocation: an output that is kept
    keeps all of it, the workspace (mx_verify_drafts_workspace_bytes) too."""
    torch = _torch()
    i32, f32 = torch.int32, torch.float32
    T, V, p_stride = _rows2(target_probs, "target_probs", (f32,))
    q_stride = 0
    if draft_probs is not None:
        Tq, Vq, q_stride = _rows2(draft_probs, "draft_probs", (f32,))
        if (Tq, Vq) != (T, V):
            raise ValueError(f"draft_probs must have shape {(T, V)}, got {(Tq, Vq)}")
    _meta(tokens, "tokens", i32, T)
    _meta(kv_lens, "kv_lens", i32)
    B = kv_lens.numel()
    _meta(cu_q, "cu_q", i32, B + 1)
    _meta(accept_random, "accept_random", f32, T)
    _meta(sample_random, "sample_random", f32, B)
    nbytes = mx_verify_drafts_workspace_bytes(B, V)
    if workspace is None and nbytes and out_tokens is None and accepted is None and new_lens is None:
        # one allocation; the workspace first, where torch aligns it
        words = -(-nbytes // 4)
        workspace, out_tokens, accepted, new_lens = _new((words + T + 2 * B,), i32, target_probs, stream).split_with_sizes((words, T, B, B))
    else:
        out_tokens = out_tokens if out_tokens is not None else _new((T,), i32, target_probs, stream)
        accepted = accepted if accepted is not None else _new((B,), i32, target_probs, stream)
        new_lens = new_lens if new_lens is not None else _new((B,), i32, target_probs, stream)
        _meta(out_tokens, "out_tokens", i32, T)
        _meta(accepted, "accepted", i32, B)
        _meta(new_lens, "new_lens", i32, B)
        if nbytes and workspace is None:
            workspace = _new((nbytes,), torch.uint8, target_probs, stream)
    ws_bytes = 0
    if nbytes:
        ws_bytes = _workspace_size(workspace)
    else:
        workspace = None
    p_, q_, tokens_, cu_, kv_, accept_, sample_, out_, acc_, lens_, ws_ = _pointers(
        "target_probs draft_probs tokens cu_q kv_lens accept_random sample_random out_tokens accepted new_lens workspace",
        target_probs, draft_probs, tokens, cu_q, kv_lens, accept_random, sample_random, out_tokens, accepted, new_lens, workspace)
    _check(lib().mx_verify_drafts(p_, p_stride, q_, q_stride, tokens_, cu_, kv_, accept_, sample_, T, B, V, out_, acc_, lens_, ws_,
                                  ws_bytes, _stream_ptr(stream)), "mx_verify_drafts")
    return out_tokens, accepted, new_lens


# ----------------------------------------------------------------------------- routing to experts

def _rows2(t, name, dtype):
    """(rows, columns, row stride) of a 2-D tensor whose rows are dense."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtype:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtype)}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    (T, N), (row, one) = t.shape, t.stride()
    if N > 1 and one != 1:
        raise ValueError(f"{name} must have dense rows, got strides {t.stride()}")
    return T, N, row if T > 1 else N


def mx_moe_route(logits, topk: int, bias=None, score: int = MX_SCORE_SOFTMAX, groups: int = 1, topk_groups: int = 1,
                 group_top: int = 2, renormalize: bool = True, scale: float = 1.0, num_rows=None, ids=None, weights=None,
                 stream=None):
    """The topk experts of each token and their weights, (ids int32, weights float32) [T, topk], from a
    router's logits [T, E] (bf16 or float32, rows dense, any row stride).

    Experts are chosen by softmax or sigmoid score plus bias (float32 [E]), largest first, ties to the
    lower expert; with groups > 1 only among the topk_groups groups whose group_top best sum highest.
    Weights are the scores without the bias, over their sum where renormalize, times scale. Rows from
    num_rows (int32 [1], on the device) on are padding: id -1, weight 0, as for places that too few
    unmasked experts leave over."""
    torch = _torch()
    T, E, stride = _rows2(logits, "logits", (torch.bfloat16, torch.float32))
    topk = int(topk)
    shape = (T, max(topk, 0))
    if bias is not None:
        _meta(bias, "bias", torch.float32, E)
    if num_rows is not None:
        _meta(num_rows, "num_rows", torch.int32, 1)
    if ids is None:
        ids = _new(shape, torch.int32, logits, stream)
    elif _meta(ids, "ids", torch.int32) or ids.shape != shape:
        raise ValueError(f"ids must have shape {shape}, got {tuple(ids.shape)}")
    if weights is None:
        weights = _new(shape, torch.float32, logits, stream)
    elif _meta(weights, "weights", torch.float32) or weights.shape != shape:
        raise ValueError(f"weights must have shape {shape}, got {tuple(weights.shape)}")
    logits_, bias_, rows_, ids_, weights_ = _pointers("logits bias num_rows ids weights", logits, bias, num_rows, ids, weights)
    _check(lib().mx_moe_route(logits_, stride, 1 if logits.dtype is torch.float32 else 0, bias_, T, E, topk, int(score), int(groups),
                              int(topk_groups), int(group_top), 1 if renormalize else 0, float(scale), rows_, ids_, weights_,
                              _stream_ptr(stream)), "mx_moe_route")
    return ids, weights


def mx_moe_sort_workspace_bytes(T: int, topk: int, E: int) -> int:
    return _kv_workspace_bytes("mx_moe_sort_workspace_bytes", int(T), int(topk), int(E))


def mx_moe_sort(topk_ids, E: int, first_expert: int = 0, expert_offsets=None, row_token=None, token_rows=None, workspace=None,
                stream=None):
    """The tables of the grouped GEMMs and the combine for the E experts from first_expert on, from
    topk_ids (int32 [T, topk], contiguous; ids of other experts have no row): (expert_offsets int32
    [E + 1], row_token int32 [T * topk], token_rows int32 [T, topk]).

    Where neither outputs nor workspace are given they are parts of one allocation: an output that is kept
    keeps all of it, the workspace (mx_moe_sort_workspace_bytes) too."""
    torch = _torch()
    i32 = torch.int32
    _meta(topk_ids, "topk_ids", i32)
    T, topk = _dims2(topk_ids, "topk_ids")
    E = int(E)
    nbytes = mx_moe_sort_workspace_bytes(T, topk, E)
    if workspace is None and expert_offsets is None and row_token is None and token_rows is None:
        # one allocation; the workspace first, where torch aligns it
        sizes = (-(-nbytes // 4), max(E, 0) + 1, T * topk, T * topk)
        workspace, expert_offsets, row_token, token_rows = _new((sum(sizes),), i32, topk_ids, stream).split_with_sizes(sizes)
        token_rows = token_rows.view(T, topk)
    else:
        expert_offsets = expert_offsets if expert_offsets is not None else _new((max(E, 0) + 1,), i32, topk_ids, stream)
        row_token = row_token if row_token is not None else _new((T * topk,), i32, topk_ids, stream)
        token_rows = token_rows if token_rows is not None else _new((T, topk), i32, topk_ids, stream)
        _meta(expert_offsets, "expert_offsets", i32, E + 1)
        _meta(row_token, "row_token", i32, T * topk)
        _meta(token_rows, "token_rows", i32)
        if token_rows.shape != (T, topk):
            raise ValueError(f"token_rows must have shape {(T, topk)}, got {tuple(token_rows.shape)}")
        if nbytes and workspace is None:
            workspace = _new((nbytes,), torch.uint8, topk_ids, stream)
    ws_bytes = 0
    if nbytes:
        ws_bytes = _workspace_size(workspace)
    else:
        workspace = None
    ids_, offsets_, token_, rows_, ws_ = _pointers("topk_ids expert_offsets row_token token_rows workspace", topk_ids, expert_offsets,
                                                   row_token, token_rows, workspace)
    _check(lib().mx_moe_sort(ids_, T, topk, int(first_expert), E, offsets_, token_, rows_, ws_, ws_bytes, _stream_ptr(stream)),
           "mx_moe_sort")
    return expert_offsets, row_token, token_rows


def mx_calib_read(buf, ctas: int, sink, stream=None) -> None:
    """One streaming-read launch over the whole of `buf` (a contiguous device tensor whose
    byte size is a multiple of 16); `sink` is a device tensor of at least 4 bytes."""
    _dev(buf, None, "buf")
    _dev(sink, None, "sink")
    nbytes = buf.numel() * buf.element_size()
    if sink.numel() * sink.element_size() < 4:
        raise ValueError("sink must hold at least 4 bytes")
    _check(lib().mx_calib_read(buf.data_ptr(), nbytes, int(ctas), sink.data_ptr(), _stream_ptr(stream)),
           "mx_calib_read")


def mx_calib_mfma(ctas: int, iters: int, sink, stream=None) -> None:
    """One MFMA-only launch (ctas x 4 waves x iters x 8 FP4 MFMAs)."""
    _dev(sink, None, "sink")
    if sink.numel() * sink.element_size() < 4:
        raise ValueError("sink must hold at least 4 bytes")
    _check(lib().mx_calib_mfma(int(ctas), int(iters), sink.data_ptr(), _stream_ptr(stream)), "mx_calib_mfma")


def mx_calib_mfma_flops(ctas: int, iters: int) -> float:
    return float(lib().mx_calib_mfma_flops(int(ctas), int(iters)))


def mx_calib_mfma_operands(ops, ctas: int, iters: int, sink, stream=None) -> None:
    """The MFMA loop on the operand bytes of `ops` (a contiguous device tensor of at least
    16 KiB, e.g. a prepared weight); `sink` is a device tensor of at least 4 bytes."""
    _dev(ops, None, "ops")
    _dev(sink, None, "sink")
    if sink.numel() * sink.element_size() < 4:
        raise ValueError("sink must hold at least 4 bytes")
    _check(lib().mx_calib_mfma_operands(ops.data_ptr(), ops.numel() * ops.element_size(), int(ctas), int(iters),
                                        sink.data_ptr(), _stream_ptr(stream)), "mx_calib_mfma_operands")


def mx_calib_mfma_operands_flops(ctas: int, iters: int) -> float:
    return float(lib().mx_calib_mfma_operands_flops(int(ctas), int(iters)))


def mx_calib_mfma_operands_clock(ops, ctas: int, iters: int, sink, clocks, stream=None) -> None:
    """mx_calib_mfma_operands that writes each wave's core-clock and 100 MHz counter ticks over
    its MFMA loop to `clocks` (an int64 device tensor of at least 8 * ctas elements)."""
    _dev(ops, None, "ops")
    _dev(sink, None, "sink")
    _dev(clocks, None, "clocks")
    if sink.numel() * sink.element_size() < 4:
        raise ValueError("sink must hold at least 4 bytes")
    if clocks.numel() * clocks.element_size() < 64 * int(ctas):
        raise ValueError("clocks must hold 8 * ctas uint64 values")
    _check(lib().mx_calib_mfma_operands_clock(ops.data_ptr(), ops.numel() * ops.element_size(), int(ctas),
                                              int(iters), sink.data_ptr(), clocks.data_ptr(), _stream_ptr(stream)),
           "mx_calib_mfma_operands_clock")


__all__ = [
    "LIB_PATH", "MxError", "lib", "status_string", "mx_prepared_layout_version",
    "mx_prepared_weight_bytes", "mx_a4w4_gemm_workspace_bytes", "mx_prepare_weight",
    "mx_prepare_weight_packed", "mx_unprepare_weight", "mx_quant_act", "mx_a4w4_gemm", "mx_a4w4_gemm_grouped",
    "mx_a4w4_gemm_plan", "mx_a16w4_gemm_plan", "mx_a4w4_gemm_grouped_plan", "mx_a4w4_gemm_grouped_act_quant",
    "mx_a4w4_gemm_grouped_act_quant_plan", "mx_a4w4_gemm_grouped_mx", "mx_a4w4_gemm_grouped_mx_plan",
    "mx_moe_combine", "mx_a16w4_gemm", "mx_kv_cache_bytes", "mx_kv_tables", "mx_kv_tables_workspace_bytes",
    "mx_kv_write", "mx_kv_read", "mx_kv_attention", "mx_kv_attention_workspace_bytes", "mx_kv_attention_plan", "mx_kv_append",
    "mx_verify_drafts", "mx_verify_drafts_workspace_bytes", "mx_moe_route", "mx_moe_sort", "mx_moe_sort_workspace_bytes",
    "MX_SCORE_SOFTMAX", "MX_SCORE_SIGMOID", "MX_ROPE_HALVES", "MX_ROPE_PAIRS", "MX_ACT_SILU", "MX_ACT_SWIGLU", "mx_calib_read", "mx_calib_mfma",
    "mx_calib_mfma_flops", "mx_calib_mfma_operands", "mx_calib_mfma_operands_flops",
    "mx_calib_mfma_operands_clock",
]
