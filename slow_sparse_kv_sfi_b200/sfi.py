"""ctypes binding of libsfi.so, the C ABI declared in include/sfi.h.

Argument marshalling only: every function passes device pointers, sizes and
a CUDA stream to the entry point of the same name and turns a non-zero
sfi_status into SFIError.  PyTorch tensors serve as device memory; nothing
here computes.  The library must be built (``python -m
slow_sparse_kv_sfi_b200.build``); loading fails loudly otherwise.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsfi.so")
_lib = None


class SFIError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib().sfi_status_str(status).decode() if _lib is not None else str(status)
        super().__init__(f"{where}: {msg} (status {status})")


def lib() -> C.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"libsfi.so is not built ({_LIB_PATH}); run "
                               "`python -m slow_sparse_kv_sfi_b200.build`")
        _lib = C.CDLL(_LIB_PATH)
        _declare(_lib)
    return _lib


class Shape(C.Structure):
    _fields_ = [("B", C.c_int32), ("Hq", C.c_int32), ("Hkv", C.c_int32), ("D", C.c_int32),
                ("page_size", C.c_int32), ("max_pages", C.c_int32), ("num_pages", C.c_int32)]


class Params(C.Structure):
    _fields_ = [("n_sink", C.c_int32), ("n_recent", C.c_int32), ("k_fixed", C.c_int32),
                ("budget_frac", C.c_double), ("lam", C.c_float), ("lambda_clip", C.c_float),
                ("alpha_soft", C.c_float), ("alpha_cross", C.c_float),
                ("nms_window", C.c_int32), ("refresh_budget", C.c_int32),
                ("evidence_window", C.c_int32)]


class PagedKV(C.Structure):
    _fields_ = [("k_pool", C.c_void_p), ("v_pool", C.c_void_p), ("page_table", C.c_void_p),
                ("key_norms", C.c_void_p), ("err", C.c_void_p)]


class Packed(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("pos", C.c_void_p),
                ("headmask", C.c_void_p), ("n_rows", C.c_void_p), ("p_max", C.c_int32)]


class DenseExtras(C.Structure):
    _fields_ = [("lse", C.c_void_p), ("logits", C.c_void_p), ("probs", C.c_void_p),
                ("ld", C.c_int64), ("lse_cand", C.c_void_p), ("cand_lo", C.c_int32),
                ("cand_hi", C.c_int32)]


FMT_E4M3, FMT_INT8 = 0, 1


class QuantKV(C.Structure):
    _fields_ = [("k_pool", C.c_void_p), ("v_pool", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("k_tail", C.c_void_p), ("v_tail", C.c_void_p), ("page_table", C.c_void_p), ("err", C.c_void_p),
                ("format", C.c_int32)]


class BlockIndex(C.Structure):
    _fields_ = [("bounds", C.c_void_p), ("scale", C.c_void_p), ("page_table", C.c_void_p), ("err", C.c_void_p)]


def _declare(L):
    P, I32, I64, SZ = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
    sig = {
        "sfi_status_str": (C.c_char_p, [C.c_int]),
        "sfi_version": (C.c_char_p, []),
        "sfi_workspace_size": (C.c_int, [P, P, C.POINTER(SZ)]),
        "sfi_packed_rows": (C.c_int, [P, P, C.POINTER(I32)]),
        "sfi_budget": (C.c_int, [P, I32, C.POINTER(I32)]),
        "sfi_append_kv": (C.c_int, [P, P, I32, P, P, P]),
        "sfi_key_norms": (C.c_int, [P, P, I32, I32, P]),
        "sfi_dense_attn": (C.c_int, [P, P, I32, P, P, P, P, SZ, P]),
        "sfi_dense_attn_append": (C.c_int, [P, P, I32, P, P, P, P, P, P, SZ, P]),
        "sfi_dense_attn_noalloc": (C.c_int, [P, P, I32, P, P, P, P]),
        "sfi_attn_probs": (C.c_int, [P, I32, P, I64, P, P, P]),
        "sfi_fast_attn": (C.c_int, [P, P, P, I32, P, P, P, P, P, SZ, P]),
        "sfi_fast_attn_append": (C.c_int, [P, P, P, I32, P, P, P, P, P, P, P, SZ, P]),
        "sfi_select_scores": (C.c_int, [P, P, P, I32, P, I64, P, P, P, SZ, P]),
        "sfi_topk_workspace_size": (C.c_int, [I32, I32, C.POINTER(SZ)]),
        "sfi_topk": (C.c_int, [I32, I32, P, I64, I32, I32, P, I64, P, SZ, P]),
        "sfi_select": (C.c_int, [P, P, P, I32, P, I64, P, P, I32, C.POINTER(I32), P, SZ, P]),
        "sfi_compact": (C.c_int, [P, P, P, I32, P, I32, I32, P, P, SZ, P]),
        "sfi_compact_incremental": (C.c_int, [P, P, P, I32, P, I32, I32, P, I32, P, SZ, P]),
        "sfi_poll_error": (C.c_int, [P, C.POINTER(I32)]),
        "sfi_quant_store": (C.c_int, [P, P, P, P, I32, I32, P, P]),
        "sfi_quant_append": (C.c_int, [P, P, P, I32, P, P, P, P]),
        "sfi_quant_load": (C.c_int, [P, P, P, I32, I32, P, P]),
        "sfi_quant_attn": (C.c_int, [P, P, I32, P, P, P, P, P, SZ, P]),
        "sfi_quant_poll_error": (C.c_int, [P, C.POINTER(I32)]),
        "sfi_block_build": (C.c_int, [P, P, P, I32, I32, P, P]),
        "sfi_block_workspace_size": (C.c_int, [P, C.POINTER(SZ)]),
        "sfi_block_select": (C.c_int, [P, P, I32, P, P, I32, I32, I32, P, I32, P, SZ, P]),
        "sfi_block_attn": (C.c_int, [P, P, I32, P, P, P, I32, I32, P, P, P, SZ, P]),
        "sfi_quant_block_attn": (C.c_int, [P, P, I32, P, P, P, I32, I32, P, P, P, SZ, P]),
        "sfi_set_wait_limit": (C.c_int, [C.c_int64]),
        "sfi_get_wait_limit": (C.c_int, [C.POINTER(C.c_int64)]),
        "sfi_selftest_wait": (C.c_int, [P, C.c_int64, P]),
        "sfi_ctx_create": (C.c_int, [P, P, I32, I32, C.POINTER(P)]),
        "sfi_ctx_destroy": (C.c_int, [P]),
        "sfi_ctx_workspace_size": (C.c_int, [P, C.POINTER(SZ)]),
        "sfi_ctx_set_workspace": (C.c_int, [P, P, SZ]),
        "sfi_decode_step": (C.c_int, [P, I32, I32, I32, I32, P, P, P, P, P, P, P, C.POINTER(I32)]),
        "sfi_decode_step_rows": (C.c_int, [P, I32, I32, P, I32, P, P, P, P, P, P, P, P]),
        "sfi_ctx_join": (C.c_int, [P, P]),
        "sfi_ctx_set_timing": (C.c_int, [P, I32]),
        "sfi_ctx_set_timing_layers": (C.c_int, [P, I32, I32]),
        "sfi_ctx_set_compaction": (C.c_int, [P, I32]),
        "sfi_ctx_timing": (C.c_int, [P, I32, C.POINTER(C.c_double), C.POINTER(I64), I32]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args


EXPORTED = ["sfi_status_str", "sfi_version", "sfi_workspace_size", "sfi_packed_rows", "sfi_budget",
            "sfi_append_kv", "sfi_key_norms", "sfi_dense_attn", "sfi_dense_attn_append",
            "sfi_dense_attn_noalloc", "sfi_attn_probs", "sfi_fast_attn", "sfi_fast_attn_append",
            "sfi_select_scores", "sfi_topk_workspace_size", "sfi_topk", "sfi_select", "sfi_compact",
            "sfi_compact_incremental", "sfi_poll_error", "sfi_set_wait_limit", "sfi_get_wait_limit",
            "sfi_selftest_wait",
            "sfi_quant_store", "sfi_quant_append", "sfi_quant_load", "sfi_quant_attn", "sfi_quant_poll_error",
            "sfi_block_build", "sfi_block_workspace_size", "sfi_block_select", "sfi_block_attn",
            "sfi_quant_block_attn",
            "sfi_ctx_create", "sfi_ctx_destroy", "sfi_ctx_workspace_size", "sfi_ctx_set_workspace",
            "sfi_decode_step", "sfi_decode_step_rows", "sfi_ctx_join", "sfi_ctx_set_timing", "sfi_ctx_set_timing_layers", "sfi_ctx_set_compaction",
            "sfi_ctx_timing"]


def _check(st: int, where: str):
    if st != 0:
        raise SFIError(st, where)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream) -> C.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def _ref(x):
    return C.byref(x) if x is not None else None


# ---------------------------------------------------------------- structs from tensors
def make_shape(B, Hq, Hkv, D, max_pages, num_pages) -> Shape:
    return Shape(B, Hq, Hkv, D, 16, max_pages, num_pages)


def make_params(n_sink, n_recent, k_fixed, budget_frac, lam, lam_clip, alpha_soft, alpha_cross,
                nms_window, refresh_budget, evidence_window=1) -> Params:
    return Params(n_sink, n_recent, k_fixed, budget_frac, lam, lam_clip, alpha_soft, alpha_cross,
                  nms_window, refresh_budget, evidence_window)


def make_kv(k_pool, v_pool, page_table, key_norms=None, err=None) -> PagedKV:
    kv = PagedKV(k_pool.data_ptr(), v_pool.data_ptr(), page_table.data_ptr(),
                 None if key_norms is None else key_norms.data_ptr(),
                 None if err is None else err.data_ptr())
    # the sizes that the 8-bit and block calls check against their shape: None when the
    # tensors are not pools of bf16 pages and a table of them, which those calls refuse
    kv.dims = None
    if (k_pool.dim() == 4 and k_pool.shape == v_pool.shape and k_pool.shape[2] == 16 and page_table.dim() == 2
            and k_pool.dtype == v_pool.dtype == torch.bfloat16 and page_table.dtype == torch.int32
            and k_pool.is_contiguous() and v_pool.is_contiguous() and page_table.is_contiguous()):
        kv.dims = (page_table.shape[0], k_pool.shape[1], k_pool.shape[3], page_table.shape[1], k_pool.shape[0])
    kv.device = k_pool.get_device()
    return kv


def make_packed(k, v, pos, headmask, n_rows) -> Packed:
    return Packed(k.data_ptr(), v.data_ptr(), pos.data_ptr(), headmask.data_ptr(),
                  n_rows.data_ptr(), k.shape[2])


def _arg(t, name, dtypes, shape=None, dev=None):
    """Checks a tensor argument of the 8-bit and block calls (dev: the current device, where known) and
    returns its address."""
    if (t.dtype in dtypes and (shape is None or t.shape == shape) and t.is_contiguous()
            and (t.get_device() == dev if dev is not None else t.is_cuda and t.get_device() == torch.cuda.current_device())):
        return t.data_ptr()
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    raise ValueError(f"{name}: must be on the current CUDA device, is on {t.device}")


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# (the public call first looks whether CUDA is up, which the tensors of a call already show)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on(stream, dev):
    """The stream handle of a call: the given stream or the current one, read
    without building a Stream object where torch allows it (3 us of a call)."""
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(dev)
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


_BF16, _F32, _I32 = (torch.bfloat16,), (torch.float32,), (torch.int32,)
_CODES = {FMT_E4M3: (torch.uint8, torch.float8_e4m3fn), FMT_INT8: (torch.uint8, torch.int8)}   # by format


def make_quant_kv(k_pool, v_pool, k_scale, v_scale, k_tail, v_tail, page_table, fmt, err=None) -> QuantKV:
    """k_pool, v_pool: uint8 or the format's own type [num_pages, Hkv, 16, D]; scales: fp32 [num_pages, Hkv];
    tails: bf16 [B, Hkv, 16, D]; page_table: int32 [B, max_pages]; fmt: FMT_E4M3 or FMT_INT8.  The caller
    keeps the tensors alive."""
    n, hkv, rows, d = k_pool.shape
    b, max_pages = page_table.shape
    if rows != 16:
        raise ValueError("k_pool: pages have 16 rows")
    codes = _CODES.get(fmt)
    if codes is None:
        raise ValueError(f"fmt: {fmt}, expected FMT_E4M3 or FMT_INT8")
    tail = (b, hkv, 16, d)
    kv = QuantKV(_arg(k_pool, "k_pool", codes), _arg(v_pool, "v_pool", codes, (n, hkv, 16, d)),
                 _arg(k_scale, "k_scale", _F32, (n, hkv)), _arg(v_scale, "v_scale", _F32, (n, hkv)),
                 _arg(k_tail, "k_tail", _BF16, tail), _arg(v_tail, "v_tail", _BF16, tail),
                 _arg(page_table, "page_table", _I32), None if err is None else _arg(err, "err", _I32, (1,)), fmt)
    kv.dims = (b, hkv, d, max_pages, n)
    kv.device = k_pool.get_device()
    return kv


def make_block_index(bounds, scale, page_table, err=None) -> BlockIndex:
    """bounds: int8 [num_pages, Hkv, 2, D]; scale: fp32 [num_pages, Hkv]; page_table: int32 [B, max_pages]."""
    n, hkv, two, d = bounds.shape
    b, max_pages = page_table.shape
    if two != 2:
        raise ValueError("bounds: an upper and a lower bound per page and head")
    ix = BlockIndex(_arg(bounds, "bounds", (torch.int8,)), _arg(scale, "scale", _F32, (n, hkv)),
                    _arg(page_table, "page_table", _I32), None if err is None else _arg(err, "err", _I32, (1,)))
    ix.dims = (b, hkv, d, max_pages, n)
    ix.device = bounds.get_device()
    return ix


def _dims(shape, *parts, dev=None):
    """The layer's sizes are those its caches and block index were made with (a bf16 cache may have more
    sequences and pages), on the device of the call.  Returns B, Hkv, D."""
    B, Hkv, D = shape.B, shape.Hkv, shape.D
    want = (B, Hkv, D, shape.max_pages, shape.num_pages)
    for x in parts:
        if x is None:
            continue
        have = getattr(x, "dims", want)
        if have != want and not (type(x) is PagedKV and have and have[1:4] == want[1:4] and have[0] >= B
                                 and have[4] >= want[4]):
            raise ValueError(f"{type(x).__name__} has (B, Hkv, D, max_pages, num_pages) "
                             f"{have or 'of no pools of contiguous bf16 pages'}, the shape {want}")
        if dev is not None and getattr(x, "device", dev) != dev:
            raise ValueError(f"{type(x).__name__}: must be on the current CUDA device, is on device {x.device}")
    return B, Hkv, D


def _lens(B, lens, dev):
    return None if lens is None else _arg(lens, "lens", _I32, (B,), dev)


def _attn_args(B, Hq, D, q, out, lse, dev):
    qs = (B, Hq, D)
    return (_arg(q, "q", _BF16, qs, dev), _arg(out, "out", _F32, qs, dev),
            None if lse is None else _arg(lse, "lse", _F32, (B, Hq), dev))


def _sel(B, Hkv, sel, dev):
    size = sel.shape
    if len(size) != 3 or size[0] != B or size[1] != Hkv:
        raise ValueError(f"sel: shape {tuple(size)}, expected ({B}, {Hkv}, at least K)")
    return _arg(sel, "sel", _I32, None, dev), size[2]


def _ws(ws, dev):
    if ws.get_device() == dev and ws.is_contiguous():
        return ws.data_ptr(), ws.nbytes
    return _arg(ws, "ws", (ws.dtype,), None, dev), ws.nbytes


# ---------------------------------------------------------------- entry points
def sfi_version() -> str:
    return lib().sfi_version().decode()


def sfi_workspace_size(shape: Shape, params: Params) -> int:
    n = C.c_size_t(0)
    _check(lib().sfi_workspace_size(C.byref(shape), C.byref(params), C.byref(n)), "sfi_workspace_size")
    return n.value


def sfi_packed_rows(shape: Shape, params: Params) -> int:
    n = C.c_int32(0)
    _check(lib().sfi_packed_rows(C.byref(shape), C.byref(params), C.byref(n)), "sfi_packed_rows")
    return n.value


def sfi_budget(params: Params, L: int) -> int:
    k = C.c_int32(0)
    _check(lib().sfi_budget(C.byref(params), L, C.byref(k)), "sfi_budget")
    return k.value


def sfi_append_kv(shape, kv, L, k_new, v_new, stream=None):
    _check(lib().sfi_append_kv(C.byref(shape), C.byref(kv), L, _p(k_new), _p(v_new), _stream(stream)),
           "sfi_append_kv")


def sfi_key_norms(shape, kv, pos_lo, pos_hi, stream=None):
    _check(lib().sfi_key_norms(C.byref(shape), C.byref(kv), pos_lo, pos_hi, _stream(stream)),
           "sfi_key_norms")


def sfi_dense_attn(shape, kv, L, q, out, ws, extras: Optional[DenseExtras] = None, stream=None):
    _check(lib().sfi_dense_attn(C.byref(shape), C.byref(kv), L, _p(q), _p(out), _ref(extras),
                                _p(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "sfi_dense_attn")


def sfi_dense_attn_append(shape, kv, L, k_new, v_new, q, out, ws, extras: Optional[DenseExtras] = None,
                          stream=None):
    """sfi_append_kv + sfi_dense_attn in one launch."""
    _check(lib().sfi_dense_attn_append(C.byref(shape), C.byref(kv), L, _p(k_new), _p(v_new), _p(q), _p(out),
                                       _ref(extras), _p(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "sfi_dense_attn_append")


def sfi_dense_attn_noalloc(shape, kv, L, q, out, extras: Optional[DenseExtras] = None, stream=None):
    """sfi_dense_attn with its scratch in the library's static device array
    (no workspace, nothing allocated)."""
    _check(lib().sfi_dense_attn_noalloc(C.byref(shape), C.byref(kv), L, _p(q), _p(out), _ref(extras),
                                        _stream(stream)), "sfi_dense_attn_noalloc")


def sfi_attn_probs(shape, L, logits, ld, lse, probs, stream=None):
    _check(lib().sfi_attn_probs(C.byref(shape), L, _p(logits), ld, _p(lse), _p(probs), _stream(stream)),
           "sfi_attn_probs")


def sfi_fast_attn(shape, params, kv, L, q, packed, out, ws, lse=None, stream=None):
    _check(lib().sfi_fast_attn(C.byref(shape), C.byref(params), C.byref(kv), L, _p(q), C.byref(packed),
                               _p(out), _p(lse), _p(ws), ws.numel() * ws.element_size(),
                               _stream(stream)), "sfi_fast_attn")


def sfi_fast_attn_append(shape, params, kv, L, k_new, v_new, q, packed, out, ws, lse=None, stream=None):
    """sfi_append_kv + sfi_fast_attn in one launch."""
    _check(lib().sfi_fast_attn_append(C.byref(shape), C.byref(params), C.byref(kv), L, _p(k_new), _p(v_new),
                                      _p(q), C.byref(packed), _p(out), _p(lse), _p(ws),
                                      ws.numel() * ws.element_size(), _stream(stream)), "sfi_fast_attn_append")


def sfi_select_scores(shape, params, kv, L, logits, ld, lse_cand, scores, ws, stream=None):
    _check(lib().sfi_select_scores(C.byref(shape), C.byref(params), C.byref(kv), L, _p(logits), ld,
                                   _p(lse_cand), _p(scores), _p(ws), ws.numel() * ws.element_size(),
                                   _stream(stream)), "sfi_select_scores")


def sfi_topk_workspace_size(rows, n) -> int:
    v = C.c_size_t(0)
    _check(lib().sfi_topk_workspace_size(rows, n, C.byref(v)), "sfi_topk_workspace_size")
    return v.value


def sfi_topk(rows, n, scores, ld_s, K, offset, idx, ld_i, ws, stream=None):
    """ws: scratch of sfi_topk_workspace_size(rows, n) bytes (0: none needed; ws may be None)."""
    _check(lib().sfi_topk(rows, n, _p(scores), ld_s, K, offset, _p(idx), ld_i, _p(ws),
                          0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)), "sfi_topk")


def sfi_select(shape, params, kv, L, logits, ld, lse_cand, sel_idx, sel_ld, ws, stream=None) -> int:
    k = C.c_int32(0)
    _check(lib().sfi_select(C.byref(shape), C.byref(params), C.byref(kv), L, _p(logits), ld,
                            _p(lse_cand), _p(sel_idx), sel_ld, C.byref(k), _p(ws),
                            ws.numel() * ws.element_size(), _stream(stream)), "sfi_select")
    return k.value


def sfi_compact(shape, params, kv, L, sel_idx, sel_ld, K, packed, ws, stream=None):
    _check(lib().sfi_compact(C.byref(shape), C.byref(params), C.byref(kv), L, _p(sel_idx), sel_ld, K,
                             C.byref(packed), _p(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "sfi_compact")


def sfi_compact_incremental(shape, params, kv, L, sel_idx, sel_ld, K, packed, fresh, ws, stream=None):
    _check(lib().sfi_compact_incremental(C.byref(shape), C.byref(params), C.byref(kv), L, _p(sel_idx), sel_ld, K,
                                         C.byref(packed), int(fresh), _p(ws), ws.numel() * ws.element_size(),
                                         _stream(stream)), "sfi_compact_incremental")


def sfi_poll_error(kv) -> int:
    code = C.c_int32(0)
    _check(lib().sfi_poll_error(C.byref(kv), C.byref(code)), "sfi_poll_error")
    return code.value


def sfi_set_wait_limit(ns: int):
    _check(lib().sfi_set_wait_limit(int(ns)), "sfi_set_wait_limit")


def sfi_get_wait_limit() -> int:
    v = C.c_int64(0)
    _check(lib().sfi_get_wait_limit(C.byref(v)), "sfi_get_wait_limit")
    return v.value


def sfi_selftest_wait(kv, limit_ns: int, stream=None):
    _check(lib().sfi_selftest_wait(C.byref(kv), int(limit_ns), _stream(stream)), "sfi_selftest_wait")


# ---------------------------------------------------------------- 8-bit cache, block-sparse attention
def sfi_quant_store(shape, kv, qkv, pos_lo, L, lens=None, index=None, stream=None):
    dev = _current_device()
    B, Hkv, D = _dims(shape, kv, qkv, index, dev=dev)
    _check(lib().sfi_quant_store(C.byref(shape), C.byref(kv), C.byref(qkv), _ref(index), pos_lo, L,
                                 _lens(B, lens, dev), _on(stream, dev)), "sfi_quant_store")


def sfi_quant_append(shape, qkv, L, k_new, v_new, lens=None, index=None, stream=None):
    dev = _current_device()
    B, Hkv, D = _dims(shape, qkv, index, dev=dev)
    tok = (B, Hkv, D)
    _check(lib().sfi_quant_append(C.byref(shape), C.byref(qkv), _ref(index), L, _lens(B, lens, dev),
                                  _arg(k_new, "k_new", _BF16, tok, dev), _arg(v_new, "v_new", _BF16, tok, dev),
                                  _on(stream, dev)), "sfi_quant_append")


def sfi_quant_load(shape, qkv, kv, pos_lo, L, lens=None, stream=None):
    dev = _current_device()
    B, Hkv, D = _dims(shape, qkv, kv, dev=dev)
    _check(lib().sfi_quant_load(C.byref(shape), C.byref(qkv), C.byref(kv), pos_lo, L, _lens(B, lens, dev),
                                _on(stream, dev)), "sfi_quant_load")


def sfi_quant_attn(shape, qkv, L, q, out, ws, lens=None, lse=None, stream=None):
    dev = _current_device()
    B, Hkv, D = _dims(shape, qkv, dev=dev)
    q, out, lse = _attn_args(B, shape.Hq, D, q, out, lse, dev)
    _check(lib().sfi_quant_attn(C.byref(shape), C.byref(qkv), L, _lens(B, lens, dev), q, out, lse,
                                *_ws(ws, dev), _on(stream, dev)), "sfi_quant_attn")


def sfi_quant_poll_error(qkv) -> int:
    code = C.c_int32(0)
    _check(lib().sfi_quant_poll_error(C.byref(qkv), C.byref(code)), "sfi_quant_poll_error")
    return code.value


def sfi_block_build(shape, kv, index, pos_lo, L, lens=None, stream=None):
    dev = _current_device()
    B, Hkv, D = _dims(shape, kv, index, dev=dev)
    _check(lib().sfi_block_build(C.byref(shape), C.byref(kv), C.byref(index), pos_lo, L, _lens(B, lens, dev),
                                 _on(stream, dev)), "sfi_block_build")


def sfi_block_workspace_size(shape: Shape) -> int:
    n = C.c_size_t(0)
    _check(lib().sfi_block_workspace_size(C.byref(shape), C.byref(n)), "sfi_block_workspace_size")
    return n.value


def sfi_block_select(shape, index, L, q, n_sink, n_recent, K, sel, ws, lens=None, stream=None):
    """sel: int32 [B, Hkv, at least K]."""
    dev = _current_device()
    B, Hkv, D = _dims(shape, index, dev=dev)
    _check(lib().sfi_block_select(C.byref(shape), C.byref(index), L, _lens(B, lens, dev),
                                  _arg(q, "q", _BF16, (B, shape.Hq, D), dev), n_sink, n_recent, K,
                                  *_sel(B, Hkv, sel, dev), *_ws(ws, dev), _on(stream, dev)),
           "sfi_block_select")


def sfi_block_attn(shape, kv, L, q, sel, K, out, ws, lens=None, lse=None, stream=None):
    """Attention over blocks sel[:, :, :K] of the bf16 cache."""
    dev = _current_device()
    B, Hkv, D = _dims(shape, kv, dev=dev)
    q, out, lse = _attn_args(B, shape.Hq, D, q, out, lse, dev)
    _check(lib().sfi_block_attn(C.byref(shape), C.byref(kv), L, _lens(B, lens, dev), q,
                                *_sel(B, Hkv, sel, dev), K, out, lse, *_ws(ws, dev), _on(stream, dev)),
           "sfi_block_attn")


def sfi_quant_block_attn(shape, qkv, L, q, sel, K, out, ws, lens=None, lse=None, stream=None):
    """sfi_block_attn on the 8-bit cache."""
    dev = _current_device()
    B, Hkv, D = _dims(shape, qkv, dev=dev)
    q, out, lse = _attn_args(B, shape.Hq, D, q, out, lse, dev)
    _check(lib().sfi_quant_block_attn(C.byref(shape), C.byref(qkv), L, _lens(B, lens, dev), q,
                                      *_sel(B, Hkv, sel, dev), K, out, lse, *_ws(ws, dev),
                                      _on(stream, dev)), "sfi_quant_block_attn")


class Context:
    """Owns an sfi_ctx (side stream, per-layer events) and its workspace tensor."""

    def __init__(self, shape: Shape, params: Params, n_layers: int, overlap: bool = True,
                 device=None, incremental: bool = True):
        self.shape, self.params = shape, params
        h = C.c_void_p()
        _check(lib().sfi_ctx_create(C.byref(shape), C.byref(params), n_layers, int(overlap),
                                    C.byref(h)), "sfi_ctx_create")
        self.h = h
        n = C.c_size_t(0)
        _check(lib().sfi_ctx_workspace_size(h, C.byref(n)), "sfi_ctx_workspace_size")
        self.ws = torch.empty(n.value, dtype=torch.uint8, device=device or "cuda")
        _check(lib().sfi_ctx_set_workspace(h, _p(self.ws), n.value), "sfi_ctx_set_workspace")
        _check(lib().sfi_ctx_set_compaction(h, int(incremental)), "sfi_ctx_set_compaction")
        self._slow = C.c_int32(0)

    def decode_step(self, layer, step, boundary_prev, L, kv, packed, q, k_new, v_new, out,
                    stream=None) -> bool:
        slow = C.c_int32(0)
        _check(lib().sfi_decode_step(self.h, layer, step, int(boundary_prev), L, C.byref(kv),
                                     C.byref(packed), _p(q), _p(k_new), _p(v_new), _p(out),
                                     _stream(stream), C.byref(slow)), "sfi_decode_step")
        return bool(slow.value)

    def decode_step_rows(self, layer, step, boundary_prev, L, kv, packed, q, k_new, v_new, out,
                         stream=None):
        """One layer-step with a trigger per sequence; boundary_prev: B flags
        (or None).  Returns the per-sequence slow decisions."""
        B = self.shape.B
        bnd = None
        if boundary_prev is not None:
            bnd = (C.c_int32 * B)(*[int(x) for x in boundary_prev])
        slow = (C.c_int32 * B)()
        _check(lib().sfi_decode_step_rows(self.h, layer, step, bnd, L, C.byref(kv), C.byref(packed), _p(q),
                                          _p(k_new), _p(v_new), _p(out), _stream(stream), slow),
               "sfi_decode_step_rows")
        return [bool(x) for x in slow]

    def decode_step_ptr(self, layer, step, boundary_prev, L, kv_ref, packed_ref, q, k_new, v_new, out,
                        stream) -> bool:
        """decode_step with raw device addresses (ints), C.byref(...) of the
        cache and packed structs and a raw stream handle: no tensor
        marshalling, for drivers that issue many layer-steps."""
        st = lib().sfi_decode_step(self.h, layer, step, boundary_prev, L, kv_ref, packed_ref, q, k_new, v_new, out,
                                   stream, C.byref(self._slow))
        if st != 0:
            raise SFIError(st, "sfi_decode_step")
        return bool(self._slow.value)

    def join(self, stream=None):
        _check(lib().sfi_ctx_join(self.h, _stream(stream)), "sfi_ctx_join")

    def set_timing(self, layer_stride: int, first_layer: int = 0):
        """Time the attention launches of layers first, first + n, ... (n = layer_stride; 0 = off)."""
        _check(lib().sfi_ctx_set_timing_layers(self.h, int(first_layer), int(layer_stride)),
               "sfi_ctx_set_timing_layers")

    def timing(self, kind: int, reset: bool = True):
        ms = C.c_double(0)
        n = C.c_int64(0)
        _check(lib().sfi_ctx_timing(self.h, kind, C.byref(ms), C.byref(n), int(reset)), "sfi_ctx_timing")
        return ms.value, n.value

    def close(self):
        if getattr(self, "h", None):
            lib().sfi_ctx_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
