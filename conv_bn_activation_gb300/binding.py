"""Thin Python binding over the C ABI in include/cb.h (ctypes).

Argument marshalling only: every step of the computation runs in libcb.so's
CUDA kernels.  torch supplies device memory and streams.  If libcb.so is
missing or cannot be loaded, every call raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import numpy as np

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libcb.so")
_lib = None
_lock = threading.Lock()

# enums (include/cb.h)
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_ALIGNMENT, ERR_CUDA, ERR_TIMEOUT, ERR_WORKSPACE = range(7)
ACT_NONE, ACT_RELU, ACT_SILU = 0, 1, 2
RES_NONE, RES_PRE_ACT, RES_POST_ACT = 0, 1, 2
LAYOUT_NHWC, LAYOUT_NCHW = 0, 1
DTYPE_F32, DTYPE_BF16 = 0, 1
PATH_DIRECT, PATH_DEPTHWISE, PATH_TC_IM2COL, PATH_TC_HALO, PATH_TC_HALO_CM, PATH_POINTWISE, PATH_STEM = range(1, 8)

EXPORTED = (
    "cb_fold_bn", "cb_repack_weights", "cb_conv_bn_act", "cb_dw_separable_block_workspace",
    "cb_dw_separable_block", "cb_avgpool_linear", "cb_preprocess_u8", "cb_preprocess_u8_three_pass",
    "cb_get_device_error", "cb_last_cuda_error", "cb_set_kernel_policy", "cb_status_string", "cb_version",
    "cb_round_weights_tf32", "cb_get_kernel_policy", "cb_layer_uses_tensor_cores",
    "cb_dw_separable_block_static", "cb_conv_path", "cb_debug_timeout_probe", "cb_autotune_conv",
    "cb_autotune_clear", "cb_autotune_entries", "cb_preprocess_stem_u8", "cb_dw_separable_block_fused",
    "cb_set_tuning", "cb_last_launch", "cb_debug_sample_coords", "cb_convert_weights_bf16", "cb_stage_body",
    "cb_attention", "cb_cache_append", "cb_attention_decode", "cb_attention_decode_workspace",
    "cb_norm_rotate", "cb_cache4_append", "cb_cache4_read", "cb_attention_decode4", "cb_attention_decode4_workspace",
)
STATIC_SCRATCH_BYTES = 16 * 1024 * 1024  # CB_STATIC_SCRATCH_BYTES


class CbTensor(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("n", ctypes.c_int), ("h", ctypes.c_int), ("w", ctypes.c_int), ("c", ctypes.c_int),
        ("stride_n", ctypes.c_longlong), ("stride_h", ctypes.c_longlong),
        ("stride_w", ctypes.c_longlong), ("stride_c", ctypes.c_longlong),
        ("layout", ctypes.c_int), ("dtype", ctypes.c_int),
    ]


class CbHeads(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("batch", ctypes.c_int), ("len", ctypes.c_int), ("heads", ctypes.c_int), ("dim", ctypes.c_int),
        ("stride_b", ctypes.c_longlong), ("stride_l", ctypes.c_longlong), ("stride_h", ctypes.c_longlong),
        ("dtype", ctypes.c_int),
    ]


class CbScore(ctypes.Structure):
    _fields_ = [
        ("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p),
        ("causal", ctypes.c_int), ("q_offset", ctypes.c_int),
        ("prefix_len", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
        ("doc_q", ctypes.c_void_p), ("doc_k", ctypes.c_void_p),
    ]


class CbPagedCache(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("heads", ctypes.c_int),
        ("dim_k", ctypes.c_int), ("dim_v", ctypes.c_int),
        ("k_stride_page", ctypes.c_longlong), ("k_stride_slot", ctypes.c_longlong), ("k_stride_head", ctypes.c_longlong),
        ("v_stride_page", ctypes.c_longlong), ("v_stride_slot", ctypes.c_longlong), ("v_stride_head", ctypes.c_longlong),
        ("table", ctypes.c_void_p), ("batch", ctypes.c_int), ("max_pages", ctypes.c_int),
        ("table_stride", ctypes.c_longlong), ("dtype", ctypes.c_int),
    ]


class CbHeadRule(ctypes.Structure):
    _fields_ = [
        ("norm", ctypes.c_int), ("eps", ctypes.c_float), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
        ("rotary", ctypes.c_int), ("adjacent", ctypes.c_int), ("axes", ctypes.c_int),
        ("freq", ctypes.c_void_p), ("axis", ctypes.c_void_p), ("pos", ctypes.c_void_p),
        ("pos_stride_axis", ctypes.c_longlong), ("pos_stride_b", ctypes.c_longlong),
    ]


class CbPagedCache4(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("heads", ctypes.c_int),
        ("dim_k", ctypes.c_int), ("dim_v", ctypes.c_int),
        ("k_stride_page", ctypes.c_longlong), ("k_stride_slot", ctypes.c_longlong), ("k_stride_head", ctypes.c_longlong),
        ("v_stride_page", ctypes.c_longlong), ("v_stride_slot", ctypes.c_longlong), ("v_stride_head", ctypes.c_longlong),
        ("ks_stride_page", ctypes.c_longlong), ("ks_stride_slot", ctypes.c_longlong), ("ks_stride_head", ctypes.c_longlong),
        ("vs_stride_page", ctypes.c_longlong), ("vs_stride_slot", ctypes.c_longlong), ("vs_stride_head", ctypes.c_longlong),
        ("table", ctypes.c_void_p), ("batch", ctypes.c_int), ("max_pages", ctypes.c_int),
        ("table_stride", ctypes.c_longlong),
    ]


class CbLaunchInfo(ctypes.Structure):
    _fields_ = [("grid", ctypes.c_int), ("threads", ctypes.c_int), ("smem_bytes", ctypes.c_size_t),
                ("cluster", ctypes.c_int), ("blocks_per_sm", ctypes.c_int), ("kernel", ctypes.c_char_p)]


class CbError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {status_string(status)}"
        if status == ERR_CUDA:
            msg += f" (cudaError {load().cb_last_cuda_error()})"
        super().__init__(msg)


def load():
    """Load libcb.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(f"libcb.so not built ({_LIB_PATH}); run __graft_entry__.build()")
            lib = ctypes.CDLL(_LIB_PATH)
            P, I, F, LL, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong, ctypes.c_size_t
            T = ctypes.POINTER(CbTensor)
            H = SC = HR = PC = P  # cb_heads, cb_score, cb_head_rule, cb_paged_cache(4): packed bytes, or a pointer to the structure
            sig = {
                "cb_fold_bn": [P, P, P, P, F, I, P, P],
                "cb_repack_weights": [P, I, I, I, I, I, P],
                "cb_conv_bn_act": [T, P, P, P, I, I, I, I, I, I, T, I, T, P],
                "cb_dw_separable_block_workspace": [T, I, I, ctypes.POINTER(S)],
                "cb_dw_separable_block": [T, P, P, P, P, P, P, P, P, P, I, T, P, S, P],
                "cb_dw_separable_block_static": [T, P, P, P, P, P, P, P, P, P, I, T, P],
                "cb_stage_body": [T, P, P, P, P, P, P, P, P, P, I, T, P],
                "cb_avgpool_linear": [T, P, P, I, P, P],
                "cb_preprocess_u8": [P, I, I, I, LL, P, I, I, P],
                "cb_preprocess_u8_three_pass": [P, I, I, I, LL, P, P, P, I, I, P],
                "cb_attention": [H, H, H, SC, H, P],
                "cb_cache_append": [H, H, P, P, PC, P],
                "cb_attention_decode_workspace": [H, PC, ctypes.POINTER(S)],
                "cb_attention_decode": [H, PC, P, P, F, F, P, H, P, S, P],
                "cb_norm_rotate": [H, H, HR, H, H, P],
                "cb_cache4_append": [H, H, P, P, PC, P],
                "cb_cache4_read": [PC, P, P, H, H, P],
                "cb_attention_decode4_workspace": [H, PC, ctypes.POINTER(S)],
                "cb_attention_decode4": [H, PC, P, P, F, F, P, H, P, S, P],
                "cb_get_device_error": [P],
                "cb_last_cuda_error": [],
                "cb_set_kernel_policy": [I],
                "cb_get_kernel_policy": [],
                "cb_round_weights_tf32": [P, LL, P],
                "cb_convert_weights_bf16": [P, LL, P],
                "cb_layer_uses_tensor_cores": [I, I, I, I, I],
                "cb_conv_path": [T, T, I, I, I, I],
                "cb_debug_timeout_probe": [I, P],
                "cb_debug_sample_coords": [I, I, P, P, P, P],
                "cb_autotune_conv": [T, P, P, P, I, I, I, I, I, I, T, I, T, P],
                "cb_autotune_clear": [],
                "cb_preprocess_stem_u8": [P, I, I, I, LL, I, I, P, P, P, I, T, P],
                "cb_dw_separable_block_fused": [T, T, P, P],
                "cb_autotune_entries": [],
                "cb_set_tuning": [ctypes.c_char_p, ctypes.c_char_p],
                "cb_last_launch": [ctypes.POINTER(CbLaunchInfo)],
                "cb_status_string": [I],
                "cb_version": [],
            }
            for name, args in sig.items():
                fn = getattr(lib, name)
                fn.argtypes = args
                fn.restype = ctypes.c_char_p if name == "cb_status_string" else ctypes.c_int
            _lib = lib
    return _lib


def status_string(s: int) -> str:
    return load().cb_status_string(int(s)).decode()


def _check(status: int, where: str):
    if status != OK:
        raise CbError(status, where)


def _stream_ptr(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# ----------------------------------------------------------------- views
def dtype_code(t) -> int:
    """cb_dtype of a torch tensor: float32 -> DTYPE_F32, bfloat16 -> DTYPE_BF16."""
    import torch
    if t.dtype == torch.float32:
        return DTYPE_F32
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise TypeError(f"activation tensors are float32 or bfloat16, got {t.dtype}")


def nhwc(t, n=None, h=None, w=None, c=None) -> CbTensor:
    """View of a torch tensor indexed [N, H, W, C] (any strides, unit channel stride)."""
    N, H, W, C = t.shape
    sn, sh, sw, sc = t.stride()
    return CbTensor(t.data_ptr(), N if n is None else n, H if h is None else h, W if w is None else w,
                    C if c is None else c, sn, sh, sw, sc, LAYOUT_NHWC, dtype_code(t))


def nchw(t) -> CbTensor:
    """View of a torch tensor indexed [N, C, H, W] (unit W stride)."""
    N, C, H, W = t.shape
    sn, sc, sh, sw = t.stride()
    return CbTensor(t.data_ptr(), N, H, W, C, sn, sh, sw, sc, LAYOUT_NCHW, dtype_code(t))


# The attention calls are small (a decode step's kernels take microseconds), so their views are
# packed by struct, in the layout of the ctypes structures: a ctypes structure takes several times
# as long to build.
_HEADS = struct.Struct("P4i3qi4x")   # CbHeads
_SCORE = struct.Struct("2fP2i4P")    # CbScore
_RULE, _RULE_POS = struct.Struct("if2P3i4x2P"), struct.Struct("P2q")  # CbHeadRule: what a Rotation holds, and the positions
_raw_stream = None
_codes = None
_several = False  # more than one CUDA device


def _init_codes():
    global _codes, _raw_stream
    import torch
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda device: torch.cuda.current_stream(device).cuda_stream)
    global _several
    _several = torch.cuda.device_count() > 1
    _codes = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, "i32": torch.int32, "f32": torch.float32}


def _device_of(*tensors):
    """The CUDA device that the tensors of a call lie on, all of them."""
    device = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != device or device < 0:
            raise ValueError("the tensors of a GPU call are on one CUDA device, got " + ", ".join(str(t.device) for t in tensors))
    return device


def _stream_of(device, stream):
    """The stream's handle: `stream`, or the device's current one.  The library launches on the current device."""
    if _several:
        import torch
        if torch.cuda.current_device() != device:
            raise ValueError(f"the call's tensors are on device {device}, the current one is {torch.cuda.current_device()}")
    if stream is not None:
        return stream.cuda_stream
    if _codes is None:
        _init_codes()
    return _raw_stream(device)


def heads(t) -> bytes:
    """cb_heads of a torch tensor indexed [B, L, H, D] (any strides, D contiguous), packed."""
    if _codes is None:
        _init_codes()
    B, L, H, D = t.shape
    sb, sl, sh, sd = t.stride()
    if sd != 1 and D > 1:
        raise ValueError("the last dim of a [B, L, H, D] view is contiguous")
    code = _codes.get(t.dtype)
    if code is None:
        raise TypeError(f"activation tensors are float32 or bfloat16, got {t.dtype}")
    return _HEADS.pack(t.data_ptr(), B, L, H, D, sb, sl, sh, code)


def _heads1(t) -> bytes:
    """cb_heads of a torch tensor indexed [B, H, D], one token per sequence, packed."""
    if _codes is None:
        _init_codes()
    B, H, D = t.shape
    sb, sh, sd = t.stride()
    if sd != 1 and D > 1:
        raise ValueError("the last dim of a [B, H, D] view is contiguous")
    code = _codes.get(t.dtype)
    if code is None:
        raise TypeError(f"activation tensors are float32 or bfloat16, got {t.dtype}")
    return _HEADS.pack(t.data_ptr(), B, 1, H, D, sb, 0, sh, code)


def _device_array(t, name, dtype, shape, device=None):
    """Pointer of a contiguous device tensor ("i32" or "f32") of this shape, on `device` (None: any); None is the
    null pointer."""
    if t is None:
        return 0
    if _codes is None:
        _init_codes()
    at = t.get_device()
    if t.dtype is not _codes[dtype] or t.shape != shape or at < 0 or device not in (None, at) or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {_codes[dtype]} tensor of shape {shape} on the call's device, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


class Score:
    """The score rule of `attention` (cb_score): how q.k becomes a score and which keys a query sees.

    softcap > 0 caps scores by softcap * tanh(s / softcap); slopes: float32 [Hq], the bias
    -slopes[h] * |i + q_offset - j|; causal, with prefix_len (int32 [B]) keys that every query sees;
    kv_len: int32 [B]; doc_q / doc_k: int32 [B, Lq] / [B, Lk], negative = padding.  Keeps the tensors."""

    def __init__(self, scale, softcap=0.0, slopes=None, causal=False, q_offset=0, prefix_len=None, kv_len=None,
                 doc_q=None, doc_k=None):
        self.scale, self.softcap, self.causal, self.q_offset = float(scale), float(softcap), bool(causal), int(q_offset)
        self.slopes, self.prefix_len, self.kv_len, self.doc_q, self.doc_k = slopes, prefix_len, kv_len, doc_q, doc_k

    def view(self, batch, lq, lk, hq, device=None) -> bytes:
        """cb_score for [batch, lq, hq, .] queries over lk keys, packed; checks the arrays' shapes and device."""
        slopes, prefix, kv, dq, dk = self.slopes, self.prefix_len, self.kv_len, self.doc_q, self.doc_k
        return _SCORE.pack(self.scale, self.softcap,
                           0 if slopes is None else _device_array(slopes, "slopes", "f32", (hq,), device),
                           self.causal, self.q_offset,
                           0 if prefix is None else _device_array(prefix, "prefix_len", "i32", (batch,), device),
                           0 if kv is None else _device_array(kv, "kv_len", "i32", (batch,), device),
                           0 if dq is None else _device_array(dq, "doc_q", "i32", (batch, lq), device),
                           0 if dk is None else _device_array(dk, "doc_k", "i32", (batch, lk), device))


class PagedCache:
    """A paged key-value cache (cb_paged_cache): k_pages [P, page, H, Dk] and v_pages [P, page, H, Dv]
    (any strides, the last dim contiguous), table int32 [B, max_pages] (rows contiguous): token j of
    sequence b lies in page table[b, j // page], slot j % page.  Holds the tensors; the table's
    contents may change between calls."""

    def __init__(self, k_pages, v_pages, table):
        if k_pages.shape[:3] != v_pages.shape[:3] or k_pages.dtype != v_pages.dtype:
            raise ValueError("k_pages and v_pages: the same pages, slots, heads and dtype")
        if k_pages.stride(3) != 1 or v_pages.stride(3) != 1:
            raise ValueError("the last dim of the pages is contiguous")
        if str(table.dtype) != "torch.int32" or table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
            raise ValueError("table: an int32 device tensor [B, max_pages] with contiguous rows")
        _device_of(k_pages, v_pages, table)
        self.k_pages, self.v_pages, self.table = k_pages, v_pages, table
        P, page, H, Dk = k_pages.shape
        self.view = CbPagedCache(k_pages.data_ptr(), v_pages.data_ptr(), P, page, H, Dk, v_pages.shape[3],
                                 *k_pages.stride()[:3], *v_pages.stride()[:3], table.data_ptr(), table.shape[0],
                                 table.shape[1], table.stride(0), dtype_code(k_pages))
        self.ref = ctypes.byref(self.view)


class Rotation:
    """How `norm_rotate` treats the heads of a token (cb_head_rule).

    norm: y = x / sqrt(mean x^2 + eps) * weight (q_weight, k_weight: float32 [dim], None: 1).
    freq: float32 [pairs], radians per position (None: nothing turns); pair p is dims (p, p + pairs), or with
    `adjacent` (2p, 2p + 1), and follows axis[p] of the `axes` positions of a token (int32 [pairs], None: the first).
    Keeps the tensors."""

    def __init__(self, freq=None, axis=None, axes=1, adjacent=False, norm=False, eps=1e-6, q_weight=None, k_weight=None):
        if not norm and (q_weight is not None or k_weight is not None):
            raise ValueError("q_weight and k_weight are the norm's")
        if axis is not None and freq is None:
            raise ValueError("axis: the axes of freq's pairs")
        self.freq, self.axis, self.axes, self.adjacent = freq, axis, int(axes), bool(adjacent)
        self.norm, self.eps, self.q_weight, self.k_weight = bool(norm), float(eps), q_weight, k_weight
        tensors = [t for t in (freq, axis, q_weight, k_weight) if t is not None]
        self.device = _device_of(*tensors) if tensors else None
        self.pairs = 0 if freq is None else freq.shape[0]
        weight = next((t for t in (q_weight, k_weight) if t is not None), None)
        self.dim = None if weight is None else weight.shape[0]
        self._head = _RULE.pack(self.norm, self.eps, _device_array(q_weight, "q_weight", "f32", (self.dim,)),
                                _device_array(k_weight, "k_weight", "f32", (self.dim,)), 2 * self.pairs, self.adjacent, self.axes,
                                _device_array(freq, "freq", "f32", (self.pairs,)), _device_array(axis, "axis", "i32", (self.pairs,)))

    def view(self, batch, length, dim, pos=None, device=None) -> bytes:
        """cb_head_rule for [batch, length, ., dim] heads at `pos`, packed; checks the positions."""
        if self.dim not in (None, dim) or (self.device is not None and device not in (None, self.device)):
            raise ValueError(f"heads of {self.dim} dims on device {self.device}, as the rule's tensors are")
        if not self.pairs:
            return self._head + _RULE_POS.pack(0, 0, 0)
        if pos is None or pos.dtype is not _codes["i32"] or pos.shape != (self.axes, batch, length) or \
                pos.get_device() != self.device or (length > 1 and pos.stride(2) != 1):
            raise ValueError(f"pos: an int32 tensor of shape {(self.axes, batch, length)} on the rule's device, its last dim contiguous")
        sa, sb, _ = pos.stride()
        return self._head + _RULE_POS.pack(pos.data_ptr(), sa, sb)


class PagedCache4:
    """A paged key-value cache in 4 bits (cb_paged_cache4): k_codes [P, page, H, (Dk + 1) // 2] uint8, k_scales
    [P, page, H, scales_per_row(Dk)] bfloat16, v_codes and v_scales likewise (any strides, the last dim contiguous),
    table as in PagedCache.  dim_k, dim_v: needed where odd.  Holds the tensors; the table's contents may change
    between calls.  `PagedCache4.empty` makes the pages, each head's slots of a page side by side."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, table, dim_k=None, dim_v=None):
        dim_k = 2 * k_codes.shape[3] if dim_k is None else int(dim_k)
        dim_v = 2 * v_codes.shape[3] if dim_v is None else int(dim_v)
        for codes, scales, dim in ((k_codes, k_scales, dim_k), (v_codes, v_scales, dim_v)):
            if str(codes.dtype) != "torch.uint8" or str(scales.dtype) != "torch.bfloat16":
                raise ValueError("codes: uint8, scales: bfloat16")
            if codes.shape[:3] != k_codes.shape[:3] or scales.shape[:3] != k_codes.shape[:3]:
                raise ValueError("codes and scales of keys and values: the same pages, slots and heads")
            if codes.shape[3] != (dim + 1) // 2 or scales.shape[3] != scales_per_row(dim):
                raise ValueError(f"rows of {dim} dims: {(dim + 1) // 2} bytes of codes and {scales_per_row(dim)} scales")
            if (codes.stride(3) != 1 and codes.shape[3] > 1) or scales.stride(3) != 1:
                raise ValueError("the last dim of the pages is contiguous")
        if str(table.dtype) != "torch.int32" or table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
            raise ValueError("table: an int32 device tensor [B, max_pages] with contiguous rows")
        _device_of(k_codes, k_scales, v_codes, v_scales, table)
        self.k_codes, self.k_scales, self.v_codes, self.v_scales, self.table = k_codes, k_scales, v_codes, v_scales, table
        P, page, H, _ = k_codes.shape
        self.view = CbPagedCache4(k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), P, page, H,
                                  dim_k, dim_v, *k_codes.stride()[:3], *v_codes.stride()[:3], *k_scales.stride()[:3],
                                  *v_scales.stride()[:3], table.data_ptr(), table.shape[0], table.shape[1], table.stride(0))
        self.ref = ctypes.byref(self.view)

    @classmethod
    def empty(cls, num_pages, page, heads, dim_k, dim_v, table):
        """A cache with pages of zeros on the table's device."""
        import torch
        pages = []
        for dim in (dim_k, dim_v):
            for width, dtype in (((dim + 1) // 2, torch.uint8), (scales_per_row(dim), torch.bfloat16)):
                pages.append(torch.zeros(num_pages, heads, page, width, dtype=dtype, device=table.device).transpose(1, 2))
        return cls(*pages, table, dim_k=dim_k, dim_v=dim_v)


def scales_per_row(dim) -> int:
    """Scales that a 4-bit cache keeps for a token's head: one for 32 dims, an even number."""
    return 2 * ((dim + 63) // 64)


# ----------------------------------------------------------- host helpers
def fold_bn(gamma, beta, mean, var, eps=1e-5):
    """cb_fold_bn on host arrays -> (scale, bias) float32 numpy arrays."""
    g, b, m, v = (np.ascontiguousarray(a, dtype=np.float32) for a in (gamma, beta, mean, var))
    C = g.size
    scale = np.empty(C, np.float32)
    bias = np.empty(C, np.float32)
    _check(load().cb_fold_bn(g.ctypes.data, b.ctypes.data, m.ctypes.data, v.ctypes.data, ctypes.c_float(eps), C,
                             scale.ctypes.data, bias.ctypes.data), "cb_fold_bn")
    return scale, bias


def repack_weights(w_oihw, groups=1):
    """cb_repack_weights: OIHW -> OHWI (dense) or [kh, kw, C] (depthwise), host numpy."""
    w = np.ascontiguousarray(w_oihw, dtype=np.float32)
    Co, cig, kh, kw = w.shape
    out = np.empty(w.size, np.float32)
    _check(load().cb_repack_weights(w.ctypes.data, Co, cig, kh, kw, groups, out.ctypes.data), "cb_repack_weights")
    if groups == 1:
        return out.reshape(Co, kh, kw, cig)
    return out.reshape(kh, kw, Co)


def set_kernel_policy(policy: int):
    _check(load().cb_set_kernel_policy(policy), "cb_set_kernel_policy")


def get_kernel_policy() -> int:
    return load().cb_get_kernel_policy()


def set_tuning(name: str, value=None):
    """cb_set_tuning: set a plan override (CB_HALO_FORCE, CB_IGEMM_FORCE, ...); None restores the default."""
    _check(load().cb_set_tuning(name.encode(), None if value is None else str(value).encode()), "cb_set_tuning")


class tuning:
    """Context manager: a plan override for the calls inside the block, restored to the default on exit."""

    def __init__(self, name: str, value):
        self.name, self.value = name, value

    def __enter__(self):
        set_tuning(self.name, self.value)
        return self

    def __exit__(self, *exc):
        set_tuning(self.name, None)
        return False


def last_launch() -> dict:
    """cb_last_launch: launch configuration, occupancy (CTAs per SM) and name of this thread's last kernel."""
    info = CbLaunchInfo()
    _check(load().cb_last_launch(ctypes.byref(info)), "cb_last_launch")
    return {"grid": info.grid, "threads": info.threads, "smem_bytes": int(info.smem_bytes), "cluster": info.cluster,
            "blocks_per_sm": info.blocks_per_sm, "kernel": (info.kernel or b"?").decode()}


def round_weights_tf32(w):
    """cb_round_weights_tf32 on a host array (any shape) -> rounded float32 copy."""
    a = np.ascontiguousarray(w, dtype=np.float32)
    out = np.empty_like(a)
    _check(load().cb_round_weights_tf32(a.ctypes.data, a.size, out.ctypes.data), "cb_round_weights_tf32")
    return out


def convert_weights_bf16(w):
    """cb_convert_weights_bf16 on a host array (any shape) -> torch.bfloat16 CPU tensor of the same shape."""
    import torch
    a = np.ascontiguousarray(w, dtype=np.float32)
    out = np.empty(a.shape, np.uint16)
    _check(load().cb_convert_weights_bf16(a.ctypes.data, a.size, out.ctypes.data), "cb_convert_weights_bf16")
    return torch.from_numpy(out.view(np.int16)).view(torch.bfloat16)


def layer_uses_tensor_cores(ci, co, k, stride=1, groups=1) -> bool:
    """cb_layer_uses_tensor_cores: the layer computes in TF32 on the tensor cores (round its weights)."""
    return bool(load().cb_layer_uses_tensor_cores(ci, co, k, stride, groups))


def conv_path(x, y, k, stride, pad, groups=1, x_layout=LAYOUT_NHWC) -> int:
    """cb_conv_path: which kernel cb_conv_bn_act would run (PATH_*), 0 if unsupported."""
    xv = nchw(x) if x_layout == LAYOUT_NCHW else nhwc(x)
    yv = nhwc(y)
    return load().cb_conv_path(ctypes.byref(xv), ctypes.byref(yv), k, stride, pad, groups)


def version() -> int:
    return load().cb_version()


# ------------------------------------------------------------- GPU calls
def conv_bn_act(x, w, scale, bias, k, stride, pad, groups, act, y, residual=None, res_mode=RES_NONE,
                stream=None, x_layout=LAYOUT_NHWC):
    """cb_conv_bn_act on torch CUDA tensors.  x: [N,H,W,C] (or [N,C,H,W] with
    x_layout=LAYOUT_NCHW); y, residual: [N,OH,OW,Co] views; w, scale, bias:
    device tensors in the cb_repack_weights / cb_fold_bn layouts.  x, y and
    residual are float32, or all bfloat16 for the layers that take bf16
    storage (depthwise 3x3, narrow 1x1); weights, scale and bias stay float32."""
    xv = nchw(x) if x_layout == LAYOUT_NCHW else nhwc(x)
    yv = nhwc(y)
    rv = nhwc(residual) if residual is not None else None
    st = load().cb_conv_bn_act(ctypes.byref(xv), w.data_ptr(), scale.data_ptr(), bias.data_ptr(), k, k, stride, pad,
                               groups, act, ctypes.byref(rv) if rv is not None else None, res_mode,
                               ctypes.byref(yv), _stream_ptr(stream))
    _check(st, "cb_conv_bn_act")
    return y


def autotune_conv(x, w, scale, bias, k, stride, pad, groups, act, y, residual=None, res_mode=RES_NONE,
                  stream=None, x_layout=LAYOUT_NHWC):
    """cb_autotune_conv: time the layer's tile plans on these buffers, keep the fastest for the
    shape; y holds the result.  Synchronises the stream (not inside graph capture)."""
    xv = nchw(x) if x_layout == LAYOUT_NCHW else nhwc(x)
    yv = nhwc(y)
    rv = nhwc(residual) if residual is not None else None
    st = load().cb_autotune_conv(ctypes.byref(xv), w.data_ptr(), scale.data_ptr(), bias.data_ptr(), k, k, stride,
                                 pad, groups, act, ctypes.byref(rv) if rv is not None else None, res_mode,
                                 ctypes.byref(yv), _stream_ptr(stream))
    _check(st, "cb_autotune_conv")
    return y


def autotune_clear():
    load().cb_autotune_clear()


def autotune_entries() -> int:
    return load().cb_autotune_entries()


def dw_separable_block_workspace(x, c_out, stride) -> int:
    xv = nhwc(x)
    n = ctypes.c_size_t(0)
    _check(load().cb_dw_separable_block_workspace(ctypes.byref(xv), c_out, stride, ctypes.byref(n)),
           "cb_dw_separable_block_workspace")
    return n.value


def dw_separable_block(x, p, stride, y, workspace, stream=None):
    """p: dict of device tensors dw_w, dw_scale, dw_bias, pw_w, pw_scale, pw_bias and optionally
    skip_w, skip_scale, skip_bias.  workspace: uint8 device tensor."""
    xv, yv = nhwc(x), nhwc(y)
    sk = p.get("skip_w")
    st = load().cb_dw_separable_block(
        ctypes.byref(xv), p["dw_w"].data_ptr(), p["dw_scale"].data_ptr(), p["dw_bias"].data_ptr(),
        p["pw_w"].data_ptr(), p["pw_scale"].data_ptr(), p["pw_bias"].data_ptr(),
        sk.data_ptr() if sk is not None else None,
        p["skip_scale"].data_ptr() if sk is not None else None,
        p["skip_bias"].data_ptr() if sk is not None else None,
        stride, ctypes.byref(yv), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _stream_ptr(stream))
    _check(st, "cb_dw_separable_block")
    return y


def stage_body(x1, layers, act, y, stream=None):
    """cb_stage_body: the YOLO-style stage body (1x1 C->C/2, 3x3 C/2->C/2, 1x1 on the concat + x1)
    in one kernel, C = 16 or 32.  layers: three objects with HOST float32 arrays .w_host (OHWI),
    .scale_host, .bias_host (ConvBnAct layers keep them): the call reads them and puts them in the
    launch."""
    xv, yv = nhwc(x1), nhwc(y)
    arrs = []
    for L in layers:
        for a in (L.w_host, L.scale_host, L.bias_host):
            a = np.ascontiguousarray(a, dtype=np.float32)
            arrs.append(a)
    st = load().cb_stage_body(ctypes.byref(xv), *[a.ctypes.data for a in arrs], act, ctypes.byref(yv),
                              _stream_ptr(stream))
    _check(st, "cb_stage_body")
    return y


def dw_separable_block_fused(x, p, y) -> bool:
    """cb_dw_separable_block_fused: the block would run as one kernel."""
    xv, yv = nhwc(x), nhwc(y)
    sk = p.get("skip_w")
    return bool(load().cb_dw_separable_block_fused(ctypes.byref(xv), ctypes.byref(yv), p["pw_w"].data_ptr(),
                                                   sk.data_ptr() if sk is not None else None))


def dw_separable_block_static(x, p, stride, y, stream=None):
    """cb_dw_separable_block_static: the same block with the library's fixed scratch array
    (no workspace argument, no allocation).  Returns the cb status without raising."""
    xv, yv = nhwc(x), nhwc(y)
    sk = p.get("skip_w")
    return load().cb_dw_separable_block_static(
        ctypes.byref(xv), p["dw_w"].data_ptr(), p["dw_scale"].data_ptr(), p["dw_bias"].data_ptr(),
        p["pw_w"].data_ptr(), p["pw_scale"].data_ptr(), p["pw_bias"].data_ptr(),
        sk.data_ptr() if sk is not None else None,
        p["skip_scale"].data_ptr() if sk is not None else None,
        p["skip_bias"].data_ptr() if sk is not None else None,
        stride, ctypes.byref(yv), _stream_ptr(stream))


def avgpool_linear(x, fc_w, fc_b, out, stream=None):
    xv = nhwc(x)
    _check(load().cb_avgpool_linear(ctypes.byref(xv), fc_w.data_ptr(), fc_b.data_ptr(), fc_w.shape[0],
                                    out.data_ptr(), _stream_ptr(stream)), "cb_avgpool_linear")
    return out


def attention(q, k, v, out, score, stream=None):
    """cb_attention on torch CUDA tensors: q [B, Lq, Hq, Dk], k [B, Lk, Hkv, Dk], v [B, Lk, Hkv, Dv],
    out [B, Lq, Hq, Dv] (any strides, the last dim contiguous; all float32 or all bfloat16); score: a
    Score.  Slices of a projection's output are read in place."""
    B, lq, hq, _ = q.shape
    device = _device_of(q, k, v, out)
    st = (_lib or load()).cb_attention(heads(q), heads(k), heads(v), score.view(B, lq, k.shape[1], hq, device), heads(out),
                                       _stream_of(device, stream))
    if st:
        _check(st, "cb_attention")
    return out


def cache_append(k_new, v_new, cache, pos, count=None, stream=None):
    """cb_cache_append: tokens t < count[b] of k_new [B, T, H, Dk] and v_new [B, T, H, Dv] become tokens
    pos[b] + t of the cache's sequences.  pos, count: int32 [B] (count None: all T)."""
    kv, vv, B = heads(k_new), heads(v_new), k_new.shape[0]
    device = _device_of(k_new, v_new, cache.table)
    st = (_lib or load()).cb_cache_append(kv, vv, _device_array(pos, "pos", "i32", (B,), device),
                                          _device_array(count, "count", "i32", (B,), device), cache.ref,
                                          _stream_of(device, stream))
    if st:
        _check(st, "cb_cache_append")


def attention_decode_workspace(q, cache) -> int:
    """cb_attention_decode_workspace: bytes of scratch for q [B, Hq, Dk] over this cache."""
    n = ctypes.c_size_t(0)
    _check(load().cb_attention_decode_workspace(_heads1(q), cache.ref, ctypes.byref(n)), "cb_attention_decode_workspace")
    return n.value


def attention_decode(q, cache, length, out, workspace, scale, softcap=0.0, slopes=None, first=None, stream=None):
    """cb_attention_decode: one new token per sequence, q [B, Hq, Dk] and out [B, Hq, Dv], over the cache's
    tokens first[b] <= j < length[b] (int32 [B]; first None: 0), the query at position length[b] - 1.
    workspace: a contiguous uint8 device tensor of attention_decode_workspace bytes."""
    qv, ov = _heads1(q), _heads1(out)
    B, hq, _ = q.shape
    device = _device_of(q, out, cache.table, workspace)
    if not workspace.is_contiguous():
        raise ValueError("workspace: a contiguous device tensor")
    st = (_lib or load()).cb_attention_decode(
        qv, cache.ref, _device_array(length, "length", "i32", (B,), device), _device_array(first, "first", "i32", (B,), device),
        scale, softcap, _device_array(slopes, "slopes", "f32", (hq,), device), ov, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_of(device, stream))
    if st:
        _check(st, "cb_attention_decode")
    return out


def norm_rotate(q, k, pos, rule, q_out=None, k_out=None, stream=None):
    """cb_norm_rotate on torch CUDA tensors: q [B, L, Hq, D] and k [B, L, Hkv, D] (any strides, the last dim contiguous;
    k None: queries alone) normed and turned as `rule` (a Rotation) says, at pos int32 [axes, B, L] (any strides over
    axes and sequences; None where nothing turns).  q_out, k_out: the results, None: in place."""
    q_out = q if q_out is None else q_out
    k_out = k if k_out is None else k_out
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    B, L, _, D = q.shape
    device = _device_of(q, q_out) if k is None else _device_of(q, k, q_out, k_out)
    st = (_lib or load()).cb_norm_rotate(heads(q), None if k is None else heads(k), rule.view(B, L, D, pos, device), heads(q_out),
                                         None if k is None else heads(k_out), _stream_of(device, stream))
    if st:
        _check(st, "cb_norm_rotate")
    return q_out, k_out


def cache4_append(k_new, v_new, cache, pos, count=None, stream=None):
    """cb_cache4_append: `cache_append` for a PagedCache4; k_new and v_new float32 or bfloat16."""
    kv, vv, B = heads(k_new), heads(v_new), k_new.shape[0]
    device = _device_of(k_new, v_new, cache.table)
    st = (_lib or load()).cb_cache4_append(kv, vv, _device_array(pos, "pos", "i32", (B,), device),
                                           _device_array(count, "count", "i32", (B,), device), cache.ref,
                                           _stream_of(device, stream))
    if st:
        _check(st, "cb_cache4_append")


def cache4_read(cache, k_out, v_out, first=None, count=None, stream=None):
    """cb_cache4_read: the values of a PagedCache4's tokens first[b] + t, t < count[b], as rows t of k_out
    [B, T, H, Dk] and v_out [B, T, H, Dv] (both float32 or both bfloat16).  first, count: int32 [B] (None: 0; all T)."""
    kv, vv, B = heads(k_out), heads(v_out), k_out.shape[0]
    device = _device_of(k_out, v_out, cache.table)
    st = (_lib or load()).cb_cache4_read(cache.ref, _device_array(first, "first", "i32", (B,), device),
                                         _device_array(count, "count", "i32", (B,), device), kv, vv, _stream_of(device, stream))
    if st:
        _check(st, "cb_cache4_read")
    return k_out, v_out


def attention_decode4_workspace(q, cache) -> int:
    """cb_attention_decode4_workspace: bytes of scratch for q [B, Hq, Dk] over this PagedCache4."""
    n = ctypes.c_size_t(0)
    _check(load().cb_attention_decode4_workspace(_heads1(q), cache.ref, ctypes.byref(n)), "cb_attention_decode4_workspace")
    return n.value


def attention_decode4(q, cache, length, out, workspace, scale, softcap=0.0, slopes=None, first=None, stream=None):
    """cb_attention_decode4: `attention_decode` over a PagedCache4; q and out both float32 or both bfloat16.
    workspace: a contiguous uint8 device tensor of attention_decode4_workspace bytes."""
    qv, ov = _heads1(q), _heads1(out)
    B, hq, _ = q.shape
    device = _device_of(q, out, cache.table, workspace)
    if not workspace.is_contiguous():
        raise ValueError("workspace: a contiguous device tensor")
    st = (_lib or load()).cb_attention_decode4(
        qv, cache.ref, _device_array(length, "length", "i32", (B,), device), _device_array(first, "first", "i32", (B,), device),
        scale, softcap, _device_array(slopes, "slopes", "f32", (hq,), device), ov, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_of(device, stream))
    if st:
        _check(st, "cb_attention_decode4")
    return out


def preprocess_u8(src, dst, stream=None):
    """src: uint8 [N, Hs, Ws, 3] device tensor (rows may be padded: src.stride(1) is the pitch);
    dst: float32 [N, 3, Hd, Wd] contiguous device tensor."""
    N, Hs, Ws, _ = src.shape
    _, _, Hd, Wd = dst.shape
    assert src.stride(0) == Hs * src.stride(1) and src.stride(2) == 3 and src.stride(3) == 1
    _check(load().cb_preprocess_u8(src.data_ptr(), N, Hs, Ws, src.stride(1), dst.data_ptr(), Hd, Wd,
                                   _stream_ptr(stream)), "cb_preprocess_u8")
    return dst


def preprocess_stem_u8(src, dst_hw, w, scale, bias, act, y, stream=None):
    """cb_preprocess_stem_u8: u8 frames [N, Hs, Ws, 3] (rows may be padded) resized to dst_hw, /255,
    straight into the 3 -> 16 stride-2 stem; y: [N, OH, OW, 16] NHWC view; w, scale, bias: device
    tensors in the cb_repack_weights / cb_fold_bn layouts."""
    N, Hs, Ws, _ = src.shape
    assert src.stride(0) == Hs * src.stride(1) and src.stride(2) == 3 and src.stride(3) == 1
    yv = nhwc(y)
    _check(load().cb_preprocess_stem_u8(src.data_ptr(), N, Hs, Ws, src.stride(1), dst_hw[0], dst_hw[1],
                                        w.data_ptr(), scale.data_ptr(), bias.data_ptr(), act, ctypes.byref(yv),
                                        _stream_ptr(stream)), "cb_preprocess_stem_u8")
    return y


def preprocess_u8_three_pass(src, tmp_u8, tmp_f32, dst, stream=None):
    N, Hs, Ws, _ = src.shape
    _, _, Hd, Wd = dst.shape
    _check(load().cb_preprocess_u8_three_pass(src.data_ptr(), N, Hs, Ws, src.stride(1), tmp_u8.data_ptr(),
                                              tmp_f32.data_ptr(), dst.data_ptr(), Hd, Wd, _stream_ptr(stream)),
           "cb_preprocess_u8_three_pass")
    return dst


def debug_timeout_probe(timeout_ms, stream=None):
    """cb_debug_timeout_probe: a bounded wait that nothing satisfies (tests the timeout report)."""
    _check(load().cb_debug_timeout_probe(int(timeout_ms), _stream_ptr(stream)), "cb_debug_timeout_probe")


def debug_sample_coords(src_extent, dst_extent, device="cuda", stream=None):
    """cb_debug_sample_coords: the (i0, i1, frac) the preprocess kernels use along one axis, as numpy."""
    import torch
    i0 = torch.empty(dst_extent, dtype=torch.int32, device=device)
    i1 = torch.empty(dst_extent, dtype=torch.int32, device=device)
    a = torch.empty(dst_extent, dtype=torch.float32, device=device)
    _check(load().cb_debug_sample_coords(int(src_extent), int(dst_extent), i0.data_ptr(), i1.data_ptr(),
                                         a.data_ptr(), _stream_ptr(stream)), "cb_debug_sample_coords")
    torch.cuda.synchronize()
    return i0.cpu().numpy(), i1.cpu().numpy(), a.cpu().numpy()


def get_device_error(stream=None) -> int:
    return load().cb_get_device_error(_stream_ptr(stream))
