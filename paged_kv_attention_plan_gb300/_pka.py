"""ctypes binding of libpka.so — argument marshalling only.

Every function here has the name of the C entry point it calls and does
nothing but check types, pass raw pointers and raise on a non-zero status;
all work happens in the library's host planner and CUDA kernels.  The
binding refuses to run when libpka.so is missing (there is no fallback).
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpka.so")

PKA_NHD, PKA_HND = 0, 1
PKA_MASK_NONE, PKA_MASK_CAUSAL, PKA_MASK_CUSTOM = 0, 1, 2
PKA_SPLIT_OFF, PKA_SPLIT_AUTO, PKA_SPLIT_FIXED = 0, 1, 2
PKA_KV_BF16, PKA_KV_FP8_E4M3 = 0, 1
PKA_ROPE_PLAIN, PKA_ROPE_LINEAR, PKA_ROPE_BY_PARTS = 0, 1, 2

STATUS = {0: "PKA_OK", 1: "PKA_ERR_INVALID_ARG", 2: "PKA_ERR_METADATA", 3: "PKA_ERR_UNSUPPORTED",
          4: "PKA_ERR_WORKSPACE", 5: "PKA_ERR_STALE_PLAN", 6: "PKA_ERR_CUDA",
          7: "PKA_ERR_DEVICE_TIMEOUT"}

EXPORTED = ["pka_status_str", "pka_version", "pka_validate", "pka_plan_create",
            "pka_plan_destroy", "pka_plan", "pka_plan_get_info", "pka_plan_wait", "pka_run",
            "pka_append_paged_kv_cache", "pka_merge_states", "pka_packbits",
            "pka_get_device_error", "pka_last_error", "pka_run_static_scratch",
            "pka_plan_cascade", "pka_selftest_bounded_wait", "pka_check_indices",
            "pka_rope_init", "pka_apply_rope", "pka_rope_append_paged_kv_cache",
            "pka_copy_pages", "pka_alloc_pages", "pka_free_pages", "pka_fork_pages",
            "pka_compact_pages"]


class pka_params(ctypes.Structure):
    _fields_ = [("num_qo_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("mask_mode", ctypes.c_int32),
                ("sm_scale", ctypes.c_float), ("kv_ragged", ctypes.c_int32),
                ("split_mode", ctypes.c_int32), ("fixed_split_pages", ctypes.c_int32),
                ("num_sms", ctypes.c_int32), ("graph_max_batch", ctypes.c_int32),
                ("graph_max_qo_rows", ctypes.c_int32), ("graph_max_kv_tokens", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float), ("decode_on_tensor_cores", ctypes.c_int32),
                ("reserved", ctypes.c_int32 * 1)]


class pka_rope_params(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_len", ctypes.c_double), ("low_rotations", ctypes.c_double),
                ("high_rotations", ctypes.c_double), ("magnitude", ctypes.c_double),
                ("frequencies_h", ctypes.c_void_p)]


class pka_rope(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("magnitude", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("turns", ctypes.c_uint64 * 64)]


class pka_plan_info(ctypes.Structure):
    _fields_ = [("int_ws_bytes", ctypes.c_uint64), ("float_ws_bytes", ctypes.c_uint64),
                ("num_requests", ctypes.c_int32), ("nnz_qo", ctypes.c_int32),
                ("total_kv", ctypes.c_int64), ("num_decode_ctas", ctypes.c_int32),
                ("num_decode_items", ctypes.c_int32), ("num_prefill_ctas", ctypes.c_int32),
                ("num_prefill_items", ctypes.c_int32), ("num_merge_tasks", ctypes.c_int32),
                ("num_partial_records", ctypes.c_int32),
                ("decode_chunk_tokens", ctypes.c_int32), ("num_decode_joins", ctypes.c_int32),
                ("kv_scratch_rows", ctypes.c_int32), ("reserved", ctypes.c_int32 * 3)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_ if f != "reserved"}


class PkaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = ""
        if status == 6:
            try:
                detail = " — " + lib().pka_last_error().decode()
            except Exception:
                pass
        super().__init__(f"{where}: {STATUS.get(status, status)} ({_str(status)}){detail}")


_lib = None


def lib():
    """Load libpka.so once; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libpka.so is missing ({LIB_PATH}); build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        P = ctypes.POINTER
        L.pka_status_str.restype = ctypes.c_char_p
        L.pka_status_str.argtypes = [ctypes.c_int]
        L.pka_version.argtypes = [P(i32), P(i32)]
        L.pka_validate.argtypes = [P(pka_params), i32, vp, vp, vp]
        L.pka_plan_create.argtypes = [P(vp)]
        L.pka_plan_destroy.argtypes = [vp]
        L.pka_plan_destroy.restype = None
        L.pka_plan.argtypes = [vp, P(pka_params), i32, vp, vp, vp, vp, sz, vp, sz, vp]
        L.pka_plan_cascade.argtypes = [vp, P(pka_params), i32, vp, vp, vp, vp, vp, sz, vp, sz,
                                       vp]
        L.pka_plan_get_info.argtypes = [vp, P(pka_plan_info)]
        L.pka_plan_wait.argtypes = [vp]
        L.pka_run.argtypes = [vp, P(pka_params), vp, vp, vp, i64, vp, vp, vp, vp, vp, sz, vp]
        L.pka_run_static_scratch.argtypes = [vp, P(pka_params), vp, vp, vp, i64, vp, vp, vp, vp,
                                             vp]
        L.pka_append_paged_kv_cache.argtypes = [P(pka_params), i32, vp, vp, vp, i64, vp, vp, vp,
                                                vp, vp, i64, vp]
        L.pka_merge_states.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, vp]
        L.pka_packbits.argtypes = [vp, i64, vp, vp]
        L.pka_get_device_error.argtypes = [P(i32), vp]
        L.pka_selftest_bounded_wait.argtypes = [i32, i32, vp]
        L.pka_check_indices.argtypes = [P(pka_params), i32, vp, vp, vp, i64, vp, i64, P(i64)]
        L.pka_rope_init.argtypes = [P(pka_rope_params), P(pka_rope)]
        L.pka_apply_rope.argtypes = [P(pka_rope), i32, i32, i64, vp, vp, i32, i64, vp, i64, vp,
                                     i32, i64, vp, i64, vp]
        L.pka_rope_append_paged_kv_cache.argtypes = [P(pka_params), P(pka_rope), i32, i64, vp,
                                                     i64, vp, vp, i64, vp, i64, vp, vp, vp, vp,
                                                     vp, vp, vp, i64, i64, vp]
        L.pka_copy_pages.argtypes = [P(pka_params), i32, vp, vp, i64, i64, i64, vp, vp, vp, i64,
                                     vp, vp]
        L.pka_alloc_pages.argtypes = [vp, i32, i32, vp, vp]
        L.pka_free_pages.argtypes = [vp, i32, vp, i64, vp]
        L.pka_fork_pages.argtypes = [i32, vp, i32, i32, vp, vp, i32, vp, i32, vp, vp, vp, i32,
                                     vp, vp, vp, vp, vp]
        L.pka_compact_pages.argtypes = [vp, i32, vp, i64, vp, vp, vp, vp, vp, vp, vp]
        L.pka_last_error.argtypes = []
        L.pka_last_error.restype = ctypes.c_char_p
        for name in EXPORTED:
            if name not in ("pka_status_str", "pka_plan_destroy", "pka_last_error"):
                getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _str(status: int) -> str:
    try:
        return lib().pka_status_str(status).decode()
    except Exception:  # library missing while formatting an error
        return "?"


def _check(status: int, where: str):
    if status != 0:
        raise PkaError(status, where)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        return t.data_ptr()
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    raise TypeError(f"unsupported buffer type {type(t)}")


def _int32_host(a, name):
    """Host int32 metadata (numpy or CPU torch); int64 is rejected, not cast."""
    if a is None:
        return None
    if isinstance(a, torch.Tensor):
        if a.dtype != torch.int32:
            raise TypeError(f"{name} must be int32, got {a.dtype}")
        if a.is_cuda:
            raise TypeError(f"{name} must be a host tensor for planning")
        return np.ascontiguousarray(a.numpy())
    a = np.asarray(a)
    if a.dtype != np.int32:
        raise TypeError(f"{name} must be int32, got {a.dtype}")
    return np.ascontiguousarray(a)


def _dev(t, name, dtype):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _dev_pool(t, name, params=None):
    """K/V pool: the last three dims contiguous; pages may be strided (5-D view).
    bf16, or uint8 e4m3 codes when the params say so."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    want = (torch.uint8 if params is not None and params.kv_dtype == PKA_KV_FP8_E4M3
            else torch.bfloat16)
    if t.dtype != want:
        raise TypeError(f"{name} must be {want}, got {t.dtype}")
    if t.dim() >= 3 and (t.stride(-1) != 1 or t.stride(-2) != t.shape[-1]
                         or t.stride(-3) != t.shape[-1] * t.shape[-2]):
        raise ValueError(f"{name}: the last three dims must be contiguous")
    return t.data_ptr()


# The checks of the operators around the cache: their calls are a few
# microseconds long, so each tensor is checked by one expression, and only a
# tensor that fails it is looked at again for what to say.
_BF16, _U8, _I32 = torch.bfloat16, torch.uint8, torch.int32


def _refuse(t, name, dtype, dev, what):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{dev}")
    raise ValueError(f"{name} must be {what}, got {tuple(t.shape)} with strides {t.stride()}")


def _here(t, name, dtype, dev):
    """Pointer of a contiguous tensor of `dtype` on CUDA device `dev` (the
    current one, where the call launches)."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev \
            and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, dtype, dev, "contiguous")


def _here_rows(t, name, dev, rows, heads, dim):
    """(pointer, row stride) of bf16 rows [rows, heads, dim]: the heads of a
    row contiguous, the rows at any stride (slices of a fused projection)."""
    if isinstance(t, torch.Tensor) and t.dtype is _BF16 and t.get_device() == dev \
            and t.shape == (rows, heads, dim):
        s0, s1, s2 = t.stride()
        if s2 == 1 and (s1 == dim or heads == 1):
            return t.data_ptr(), s0 if rows > 1 else heads * dim
    _refuse(t, name, _BF16, dev,
            f"{_shape(rows, heads, dim)} with the heads of a row contiguous")


def _shape(*dims):
    return "[" + ", ".join(map(str, dims)) + "]"


def _here_pools(k, v, params, dev):
    """(pointer of k, of v, their shape, their strides) of K/V pools alike,
    [.., pages, P, Hk, D] or [.., pages, Hk, P, D] of the params' layout, each
    page contiguous."""
    a, b, d = params.page_size, params.num_kv_heads, params.head_dim
    if params.layout != PKA_NHD:
        a, b = b, a
    dtype = _U8 if params.kv_dtype == PKA_KV_FP8_E4M3 else _BF16
    if isinstance(k, torch.Tensor) and isinstance(v, torch.Tensor) and k.dtype is dtype \
            and v.dtype is dtype and k.get_device() == dev and v.get_device() == dev:
        shape, strides = k.shape, k.stride()
        if shape[-3:] == (a, b, d) and strides[-3:] == (b * d, d, 1) and v.shape == shape \
                and v.stride() == strides:
            return k.data_ptr(), v.data_ptr(), shape, strides
    what = f"{_shape('..', a, b, d)} with each page contiguous"
    for t, name in ((k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev \
                or t.shape[-3:] != (a, b, d) or t.stride()[-3:] != (b * d, d, 1):
            _refuse(t, name, dtype, dev, what)
    raise ValueError("k and v must have one shape and the same strides")


def _here_stream(stream, dev) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return _stream(stream)


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def make_params(num_qo_heads, num_kv_heads, head_dim, page_size=1, layout="NHD",
                mask_mode="causal", sm_scale=0.0, kv_ragged=False, split_mode="auto",
                fixed_split_pages=1, num_sms=0, graph_max_batch=0, graph_max_qo_rows=0,
                graph_max_kv_tokens=0, kv_dtype="bf16", k_scale=1.0,
                v_scale=1.0, decode_on_tensor_cores=False) -> pka_params:
    p = pka_params()
    p.num_qo_heads, p.num_kv_heads, p.head_dim = num_qo_heads, num_kv_heads, head_dim
    p.page_size = page_size
    p.layout = {"NHD": PKA_NHD, "HND": PKA_HND}[layout] if isinstance(layout, str) else layout
    p.mask_mode = ({"none": PKA_MASK_NONE, "causal": PKA_MASK_CAUSAL, "custom": PKA_MASK_CUSTOM}
                   [mask_mode] if isinstance(mask_mode, str) else mask_mode)
    p.sm_scale = sm_scale
    p.kv_ragged = int(bool(kv_ragged))
    p.split_mode = ({"off": PKA_SPLIT_OFF, "auto": PKA_SPLIT_AUTO, "fixed": PKA_SPLIT_FIXED}
                    [split_mode] if isinstance(split_mode, str) else split_mode)
    p.fixed_split_pages = fixed_split_pages
    p.num_sms = num_sms
    p.graph_max_batch = graph_max_batch
    p.graph_max_qo_rows = graph_max_qo_rows
    p.graph_max_kv_tokens = graph_max_kv_tokens
    p.kv_dtype = ({"bf16": PKA_KV_BF16, "e4m3": PKA_KV_FP8_E4M3}[kv_dtype]
                  if isinstance(kv_dtype, str) else kv_dtype)
    p.k_scale, p.v_scale = k_scale, v_scale
    p.decode_on_tensor_cores = int(bool(decode_on_tensor_cores))
    return p


_ROPE_SCALING = {"none": PKA_ROPE_PLAIN, "linear": PKA_ROPE_LINEAR, "parts": PKA_ROPE_BY_PARTS}


def make_rope(rotary_dim, base=10000.0, interleaved=False, scaling="none", factor=1.0,
              original_len=0.0, low_rotations=1.0, high_rotations=32.0, magnitude=1.0,
              frequencies=None) -> pka_rope:
    """The rotation that pka_apply_rope and pka_rope_append_paged_kv_cache take
    (see pka_rope_init in include/pka.h).  ``frequencies``: rotary_dim / 2
    radians a position, in place of base and scaling."""
    p = pka_rope_params()
    p.rotary_dim, p.interleaved = rotary_dim, int(bool(interleaved))
    p.scaling = _ROPE_SCALING[scaling] if isinstance(scaling, str) else scaling
    p.base, p.factor, p.original_len = base, factor, original_len
    p.low_rotations, p.high_rotations = low_rotations, high_rotations
    p.magnitude = magnitude
    if frequencies is not None:
        f = np.ascontiguousarray(frequencies, dtype=np.float64)
        if f.shape != (rotary_dim // 2,):
            raise ValueError(f"frequencies: {rotary_dim // 2} values, got shape {f.shape}")
        p.frequencies_h = f.ctypes.data
    return pka_rope_init(p)


# ---------------------------------------------------------------------------
# The C entry points, one Python function each.
# ---------------------------------------------------------------------------

def pka_status_str(status: int) -> str:
    return _str(status)


def pka_version():
    a, b = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().pka_version(ctypes.byref(a), ctypes.byref(b)), "pka_version")
    return a.value, b.value


def pka_validate(params, qo_indptr, kv_indptr, last_page_len) -> int:
    kv = _int32_host(kv_indptr, "kv_indptr")
    qo = _int32_host(qo_indptr, "qo_indptr")
    last = _int32_host(last_page_len, "last_page_len")
    return lib().pka_validate(ctypes.byref(params), len(kv) - 1, _ptr(qo), _ptr(kv), _ptr(last))


def pka_plan_create():
    h = ctypes.c_void_p()
    _check(lib().pka_plan_create(ctypes.byref(h)), "pka_plan_create")
    return h


def pka_plan_destroy(handle):
    if handle:
        lib().pka_plan_destroy(handle)


def pka_plan(handle, params, qo_indptr, kv_indptr, last_page_len, int_ws, pinned,
             stream=None, check=True) -> int:
    kv = _int32_host(kv_indptr, "kv_indptr")
    qo = _int32_host(qo_indptr, "qo_indptr")
    last = _int32_host(last_page_len, "last_page_len")
    ws_ptr = _ptr(int_ws) if int_ws is not None else None
    ws_bytes = int_ws.numel() * int_ws.element_size() if int_ws is not None else 0
    pin_bytes = (pinned.numel() * pinned.element_size() if isinstance(pinned, torch.Tensor)
                 else pinned.nbytes)
    st = _stream(stream) if int_ws is not None else None
    s = lib().pka_plan(handle, ctypes.byref(params), len(kv) - 1, _ptr(qo), _ptr(kv), _ptr(last),
                       ws_ptr, ws_bytes, _ptr(pinned), pin_bytes, st)
    if check:
        _check(s, "pka_plan")
    return s


def pka_plan_cascade(handle, params, levels, int_ws, pinned, stream=None, check=True) -> int:
    """``levels``: list, root first, of (qo_indptr, kv_indptr, last_page_len) host int32."""
    arrs = [tuple(_int32_host(a, n) for a, n in zip(lv, ("qo_indptr", "kv_indptr",
                                                          "last_page_len")))
            for lv in levels]
    n = len(arrs)
    nodes = np.asarray([len(a[1]) - 1 for a in arrs], dtype=np.int32)
    ptrs = [(ctypes.c_void_p * max(n, 1))(*[_ptr(a[i]) for a in arrs]) for i in range(3)]
    ws_ptr = _ptr(int_ws) if int_ws is not None else None
    ws_bytes = int_ws.numel() * int_ws.element_size() if int_ws is not None else 0
    pin_bytes = (pinned.numel() * pinned.element_size() if isinstance(pinned, torch.Tensor)
                 else pinned.nbytes)
    st = _stream(stream) if int_ws is not None else None
    s = lib().pka_plan_cascade(handle, ctypes.byref(params), n, _ptr(nodes),
                               ctypes.cast(ptrs[0], ctypes.c_void_p),
                               ctypes.cast(ptrs[1], ctypes.c_void_p),
                               ctypes.cast(ptrs[2], ctypes.c_void_p), ws_ptr, ws_bytes,
                               _ptr(pinned), pin_bytes, st)
    if check:
        _check(s, "pka_plan_cascade")
    return s


def pka_plan_get_info(handle) -> pka_plan_info:
    info = pka_plan_info()
    _check(lib().pka_plan_get_info(handle, ctypes.byref(info)), "pka_plan_get_info")
    return info


def pka_plan_wait(handle):
    _check(lib().pka_plan_wait(handle), "pka_plan_wait")


def pka_run(handle, params, q, k, v, page_stride, kv_indices, packed_mask, o, lse, float_ws,
            stream=None, check=True) -> int:
    bf16 = torch.bfloat16
    fws = float_ws.numel() * float_ws.element_size() if float_ws is not None else 0
    s = lib().pka_run(handle, ctypes.byref(params), _dev(q, "q", bf16),
                      _dev_pool(k, "k", params), _dev_pool(v, "v", params), int(page_stride),
                      _dev(kv_indices, "kv_indices", torch.int32),
                      _dev(packed_mask, "packed_mask", torch.uint8), _dev(o, "o", bf16),
                      _dev(lse, "lse", torch.float32), _ptr(float_ws), fws, _stream(stream))
    if check:
        _check(s, "pka_run")
    return s


def pka_run_static_scratch(handle, params, q, k, v, page_stride, kv_indices, packed_mask, o,
                           lse, stream=None, check=True) -> int:
    """pka_run with the split-KV scratch in the library's static device array
    (no workspace from the caller; see include/pka.h)."""
    bf16 = torch.bfloat16
    s = lib().pka_run_static_scratch(
        handle, ctypes.byref(params), _dev(q, "q", bf16), _dev_pool(k, "k", params),
        _dev_pool(v, "v", params),
        int(page_stride), _dev(kv_indices, "kv_indices", torch.int32),
        _dev(packed_mask, "packed_mask", torch.uint8), _dev(o, "o", bf16),
        _dev(lse, "lse", torch.float32), _stream(stream))
    if check:
        _check(s, "pka_run_static_scratch")
    return s


def pka_append_paged_kv_cache(params, k_new, v_new, append_indptr, kv_indptr, kv_indices,
                              last_page_len, k, v, page_stride, stream=None, check=True) -> int:
    bf16, i32 = torch.bfloat16, torch.int32
    s = lib().pka_append_paged_kv_cache(
        ctypes.byref(params), append_indptr.numel() - 1, _dev(k_new, "k_new", bf16),
        _dev(v_new, "v_new", bf16), _dev(append_indptr, "append_indptr", i32), k_new.shape[0],
        _dev(kv_indptr, "kv_indptr", i32), _dev(kv_indices, "kv_indices", i32),
        _dev(last_page_len, "last_page_len", i32), _dev_pool(k, "k", params),
        _dev_pool(v, "v", params),
        int(page_stride),
        _stream(stream))
    if check:
        _check(s, "pka_append_paged_kv_cache")
    return s


def pka_rope_init(rope_params) -> pka_rope:
    rope = pka_rope()
    _check(lib().pka_rope_init(ctypes.byref(rope_params), ctypes.byref(rope)), "pka_rope_init")
    return rope


def pka_apply_rope(rope, positions, q=None, q_out=None, k=None, k_out=None, transpose=False,
                   stream=None, check=True) -> int:
    """Rotate q and / or k ([rows, heads, head_dim], rows at any stride) into
    q_out and k_out, which may be q and k themselves.  Autograd does not see the
    call: a backward pass calls it with transpose on the outputs' gradients."""
    some = q if q is not None else k
    if not isinstance(some, torch.Tensor) or some.dim() != 3:
        raise ValueError("q and k must be [rows, heads, head_dim], one of them given")
    dev = torch.cuda.current_device()
    rows, hq, dim = some.shape
    hk = 0
    qp = qo = kp = ko = None
    qs = qos = ks = kos = 0
    if q is not None:
        qp, qs = _here_rows(q, "q", dev, rows, hq, dim)
        qo, qos = (qp, qs) if q_out is q else _here_rows(q_out, "q_out", dev, rows, hq, dim)
    else:
        hq = 0
    if k is not None:
        hk = k.shape[-2]
        kp, ks = _here_rows(k, "k", dev, rows, hk, dim)
        ko, kos = (kp, ks) if k_out is k else _here_rows(k_out, "k_out", dev, rows, hk, dim)
    pos = _here(positions, "positions", _I32, dev)
    if positions.numel() != rows:
        raise ValueError(f"positions: {rows} values, got {positions.numel()}")
    s = lib().pka_apply_rope(ctypes.byref(rope), 1 if transpose else 0, dim, rows, pos, qp, hq, qs,
                             qo, qos, kp, hk, ks, ko, kos, _here_stream(stream, dev))
    if check and s:
        _check(s, "pka_apply_rope")
    return s


def pka_rope_append_paged_kv_cache(params, rope, q, q_out, k_new, v_new, append_indptr, kv_indptr,
                                   kv_indices, last_page_len, k, v, page_stride, positions=None,
                                   stream=None, check=True) -> int:
    """pka_append_paged_kv_cache of rotated rows; q and q_out may be None.  k
    and v are the pools [pages, ...] and page_stride theirs; rows past
    append_indptr[-1] are left."""
    dev = torch.cuda.current_device()
    hk, d, rows = params.num_kv_heads, params.head_dim, k_new.shape[0]
    batch = append_indptr.numel() - 1
    qp = qo = pos = None
    qs = 0
    if q is not None:
        hq = params.num_qo_heads
        qp, qs = _here_rows(q, "q", dev, rows, hq, d)
        qo, qos = (qp, qs) if q_out is q else _here_rows(q_out, "q_out", dev, rows, hq, d)
        if qos != hq * d:
            _refuse(q_out, "q_out", _BF16, dev, "contiguous")
    kp, ks = _here_rows(k_new, "k_new", dev, rows, hk, d)
    vp, vs = _here_rows(v_new, "v_new", dev, rows, hk, d)
    if positions is not None:
        pos = _here(positions, "positions", _I32, dev)
        if positions.numel() != rows:
            raise ValueError(f"positions: {rows} values, got {positions.numel()}")
    app = _here(append_indptr, "append_indptr", _I32, dev)
    ptr = _here(kv_indptr, "kv_indptr", _I32, dev)
    idx = _here(kv_indices, "kv_indices", _I32, dev)
    last = _here(last_page_len, "last_page_len", _I32, dev)
    if kv_indptr.numel() != batch + 1 or last_page_len.numel() != batch:
        raise ValueError("kv_indptr and last_page_len must describe append_indptr's requests")
    kpool, vpool, shape, strides = _here_pools(k, v, params, dev)
    if len(shape) != 4:
        raise ValueError("k and v must be pools [pages, ...]")
    if page_stride != strides[0] and shape[0] > 1:
        raise ValueError(f"page_stride: the pools' is {strides[0]}, got {page_stride}")
    s = lib().pka_rope_append_paged_kv_cache(
        ctypes.byref(params), ctypes.byref(rope), batch, rows, qp, qs, qo, kp, ks, vp, vs, pos,
        app, ptr, idx, last, kpool, vpool,
        int(page_stride), shape[0], _here_stream(stream, dev))
    if check and s:
        _check(s, "pka_rope_append_paged_kv_cache")
    return s


def pka_copy_pages(params, k, v, src, dst, slots=None, num_copies=None, stream=None,
                   check=True) -> int:
    """Copy pages src[i] over dst[i] (their first slots[i] slots) in pools
    [pages, ...] or, for all layers at once, [layers, pages, ...] of any layer
    and page stride.  num_copies: a device count (its first element) of the
    entries that hold, as pka_fork_pages and pka_compact_pages write it."""
    dev, i32 = torch.cuda.current_device(), _I32
    kp, vp, shape, strides = _here_pools(k, v, params, dev)
    if len(shape) not in (4, 5):
        raise ValueError("k and v must be pools [pages, ...] or [layers, pages, ...]")
    layers = shape[0] if len(shape) == 5 else 1
    n = src.numel()
    if dst.numel() != n or (slots is not None and slots.numel() != n):
        raise ValueError("src, dst and slots must have one length")
    s = lib().pka_copy_pages(
        ctypes.byref(params), layers, kp, vp, strides[-4], strides[0] if layers > 1 else 0,
        shape[-4], _here(src, "src", i32, dev), _here(dst, "dst", i32, dev),
        None if slots is None else _here(slots, "slots", i32, dev), n,
        None if num_copies is None else _here(num_copies, "num_copies", i32, dev),
        _here_stream(stream, dev))
    if check and s:
        _check(s, "pka_copy_pages")
    return s


def pka_alloc_pages(page_refs, pages, stream=None, check=True) -> int:
    """Take as many pages as `pages` has room for."""
    dev, i32 = torch.cuda.current_device(), _I32
    s = lib().pka_alloc_pages(_here(page_refs, "page_refs", i32, dev), page_refs.numel(),
                              pages.numel(), _here(pages, "pages", i32, dev),
                              _here_stream(stream, dev))
    if check and s:
        _check(s, "pka_alloc_pages")
    return s


def pka_free_pages(page_refs, pages, stream=None, check=True) -> int:
    dev, i32 = torch.cuda.current_device(), _I32
    s = lib().pka_free_pages(_here(page_refs, "page_refs", i32, dev), page_refs.numel(),
                             _here(pages, "pages", i32, dev), pages.numel(),
                             _here_stream(stream, dev))
    if check and s:
        _check(s, "pka_free_pages")
    return s


def pka_fork_pages(page_size, page_refs, kv_indptr, kv_indices, last_page_len, parent,
                   child_indptr, child_indices, copy_src, copy_dst, copy_slots, counts,
                   stream=None, check=True) -> int:
    """Tables of children that continue parents, whose pages are held; the copy
    lists and counts go to pka_copy_pages.  All arrays are device int32."""
    dev, i32 = torch.cuda.current_device(), _I32
    parents, children = last_page_len.numel(), parent.numel()
    if kv_indptr.numel() != parents + 1 or child_indptr.numel() != children + 1:
        raise ValueError("an indptr has one element more than its requests")
    if min(copy_src.numel(), copy_dst.numel(), copy_slots.numel()) < children:
        raise ValueError("the copy lists hold one element a child")
    if counts.numel() < 2:
        raise ValueError("counts holds two elements")
    s = lib().pka_fork_pages(
        page_size, _here(page_refs, "page_refs", i32, dev), page_refs.numel(), parents,
        _here(kv_indptr, "kv_indptr", i32, dev), _here(kv_indices, "kv_indices", i32, dev),
        kv_indices.numel(), _here(last_page_len, "last_page_len", i32, dev), children,
        _here(parent, "parent", i32, dev), _here(child_indptr, "child_indptr", i32, dev),
        _here(child_indices, "child_indices", i32, dev), child_indices.numel(),
        _here(copy_src, "copy_src", i32, dev), _here(copy_dst, "copy_dst", i32, dev),
        _here(copy_slots, "copy_slots", i32, dev), _here(counts, "counts", i32, dev),
        _here_stream(stream, dev))
    if check and s:
        _check(s, "pka_fork_pages")
    return s


def pka_compact_pages(page_refs, kv_indices, page_refs_out, kv_indices_out, page_map, copy_src,
                      copy_dst, counts, stream=None, check=True) -> int:
    """Move the live pages to the front of the pool: the new references and
    table entries (either may be written in place), the map and the moves."""
    dev, i32 = torch.cuda.current_device(), _I32
    n = page_refs.numel()
    if page_refs_out.numel() != n or page_map.numel() != n:
        raise ValueError("page_refs_out and page_map hold one element a page")
    if kv_indices_out.numel() != kv_indices.numel():
        raise ValueError("kv_indices_out must have kv_indices' length")
    if min(copy_src.numel(), copy_dst.numel()) < n // 2 or counts.numel() < 2:
        raise ValueError("the copy lists hold one element for two pages, counts two")
    s = lib().pka_compact_pages(
        _here(page_refs, "page_refs", i32, dev), n, _here(kv_indices, "kv_indices", i32, dev),
        kv_indices.numel(), _here(page_refs_out, "page_refs_out", i32, dev),
        _here(kv_indices_out, "kv_indices_out", i32, dev), _here(page_map, "page_map", i32, dev),
        _here(copy_src, "copy_src", i32, dev), _here(copy_dst, "copy_dst", i32, dev),
        _here(counts, "counts", i32, dev), _here_stream(stream, dev))
    if check and s:
        _check(s, "pka_compact_pages")
    return s


def pka_merge_states(v, s, indptr, v_out, s_out=None, stream=None):
    rows = indptr.numel() - 1
    _check(lib().pka_merge_states(_dev(v, "v", torch.float32), _dev(s, "s", torch.float32),
                                  _dev(indptr, "indptr", torch.int32), rows, v.shape[1],
                                  v.shape[2], _dev(v_out, "v_out", torch.bfloat16),
                                  _dev(s_out, "s_out", torch.float32), _stream(stream)),
           "pka_merge_states")


def pka_packbits(bools, out, stream=None):
    _check(lib().pka_packbits(_dev(bools, "bools", torch.uint8), bools.numel(),
                              _dev(out, "out", torch.uint8), _stream(stream)), "pka_packbits")


def pka_last_error() -> str:
    return lib().pka_last_error().decode()


def pka_get_device_error(stream=None) -> int:
    code = ctypes.c_int32()
    _check(lib().pka_get_device_error(ctypes.byref(code), _stream(stream)), "pka_get_device_error")
    return code.value


def pka_selftest_bounded_wait(arrive: bool, polls: int, stream=None):
    _check(lib().pka_selftest_bounded_wait(1 if arrive else 0, int(polls), _stream(stream)),
           "pka_selftest_bounded_wait")


def pka_check_indices(params, kv_indptr, kv_indices, last_page_len, num_pool_pages,
                      append_indptr=None):
    """Host check of a page table; returns (status, bad_index) without raising."""
    kv = _int32_host(kv_indptr, "kv_indptr")
    idx = _int32_host(kv_indices, "kv_indices")
    last = _int32_host(last_page_len, "last_page_len")
    app = _int32_host(append_indptr, "append_indptr")
    bad = ctypes.c_int64(-2)
    s = lib().pka_check_indices(ctypes.byref(params), len(kv) - 1, _ptr(app), _ptr(kv),
                                _ptr(idx), len(idx), _ptr(last), int(num_pool_pages),
                                ctypes.byref(bad))
    return s, bad.value
