"""Python binding of libpkc (paged-KV cascade decode attention for GB300).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libpkc.so``.  torch tensors supply device memory and the
current CUDA stream; their data pointers go straight to the C ABI declared
in ``include/pkc.h``.  If the library has not been built, every call raises
-- there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libpkc.so")

PKC_OK = 0
STATUS_NAMES = {0: "PKC_OK", 1: "PKC_ERR_INVALID_ARG", 2: "PKC_ERR_UNSUPPORTED",
                3: "PKC_ERR_WORKSPACE", 4: "PKC_ERR_BLOCK_TABLE", 5: "PKC_ERR_CUDA",
                6: "PKC_ERR_TIMEOUT", 7: "PKC_ERR_PLAN", 8: "PKC_ERR_NO_PAGES"}
F32, F16, BF16, E4M3, MX4 = 0, 1, 2, 3, 4

# Header indices of the plan buffer (include/pkc.h).
PLAN_FIELDS = ["MAGIC", "TOTAL_WORDS", "NUM_CTAS", "TILE_Q", "N_REQ", "KV_CHUNK",
               "N_UNITS", "N_WORK", "N_PARTIALS", "N_SPLIT", "N_EMPTY",
               "OFF_CTA_INDPTR", "OFF_CTA_WORK", "OFF_WORK_UNIT", "OFF_WORK_KV_BEGIN",
               "OFF_WORK_KV_END", "OFF_WORK_PARTIAL", "OFF_UNIT_REQ", "OFF_UNIT_QTILE",
               "OFF_UNIT_KV_LEN", "OFF_UNIT_N_CHUNKS", "OFF_UNIT_PARTIAL_BEGIN",
               "OFF_UNIT_LIST", "OFF_CTA_COST", "OFF_WORK_ORDER", "OFF_ORDER_REC"]
PLAN = {name: i for i, name in enumerate(PLAN_FIELDS)}
PLAN_MAGIC = 0x504B4331

# Every symbol the C ABI exports, with (restype, argtypes).
_c = ctypes
_P, _I, _I64, _SZ, _F, _D = _c.c_void_p, _c.c_int, _c.c_int64, _c.c_size_t, _c.c_float, _c.c_double
SIGNATURES = {
    "pkc_version": (_I, []),
    "pkc_last_error": (_c.c_char_p, []),
    "pkc_merge_state": (_I, [_P, _P, _P, _P, _P, _P, _I64, _I, _I, _I, _P]),
    "pkc_merge_states": (_I, [_P, _P, _P, _P, _I64, _I, _I, _I, _I, _P]),
    "pkc_merge_states_to": (_I, [_P, _P, _P, _P, _I64, _I, _I, _I, _I, _I, _P]),
    "pkc_plan_words": (_I, [_P, _I, _I, _I, _c.POINTER(_SZ)]),
    "pkc_plan": (_I, [_P, _P, _I, _I, _I, _D, _D, _P, _SZ]),
    "pkc_plan_upload": (_I, [_P, _P, _SZ, _P]),
    "pkc_workspace_size": (_I, [_I, _I, _I, _I, _I, _c.POINTER(_SZ)]),
    "pkc_workspace_init": (_I, [_P, _SZ, _P]),
    "pkc_device_status": (_I, [_P, _P, _c.POINTER(_c.c_int32)]),
    "pkc_paged_decode_state": (_I, [_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I64, _F,
                                    _P, _P, _SZ, _P, _P, _I, _P]),
    "pkc_prefix_attention_state": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P, _SZ,
                                        _P, _P, _I, _P]),
    "pkc_paged_decode_state_noalloc": (_I, [_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I64,
                                            _F, _P, _P, _P, _P, _I, _P]),
    "pkc_paged_decode_state_fp8": (_I, [_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I64, _F,
                                        _F, _F, _P, _P, _SZ, _P, _P, _P]),
    "pkc_set_stage_events": (_I, [_c.POINTER(_P), _I]),
    "pkc_set_decode_kernel": (_I, [_I]),
    "pkc_set_decode_schedule": (_I, [_I]),
    "pkc_set_contraction": (_I, [_I]),
    "pkc_set_prefix_ctas": (_I, [_I]),
    "pkc_set_cascade_small": (_I, [_I]),
    "pkc_last_launch_blocks": (_I, [_c.POINTER(_c.c_int), _c.POINTER(_c.c_int)]),
    "pkc_selftest_wait_timeout": (_I, [_P, _SZ, _c.POINTER(_c.c_int32), _P]),
    "pkc_append_kv": (_I, [_P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I64, _I, _P, _SZ, _P]),
    "pkc_cascade_decode_multilevel": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _P, _I, _I, _I,
                                           _I, _I, _I64, _F, _P, _P, _SZ, _P, _P, _I, _P]),
    "pkc_cascade_decode_paged_prefix": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _P, _I, _I,
                                             _I, _I, _I, _I64, _F, _P, _P, _SZ, _P, _P, _I, _P]),
    "pkc_cascade_decode": (_I, [_P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I,
                                _I64, _F, _P, _P, _SZ, _P, _P, _I, _P]),
    "pkc_cascade_decode_state": (_I, [_P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _P, _I, _I, _I, _I,
                                      _I, _I64, _F, _P, _P, _SZ, _P, _P, _I, _P]),
    "pkc_append_kv_mx4": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I64, _I,
                               _P, _SZ, _P]),
    "pkc_gather_kv_mx4": (_I, [_P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I64, _P, _P, _I,
                               _P, _SZ, _P]),
    "pkc_paged_decode_state_mx4": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I64, _F,
                                        _P, _P, _SZ, _P, _P, _I, _P]),
    "pkc_accumulate_weights": (_I, [_P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I64, _F, _F, _F,
                                    _P, _I64, _I, _I, _P, _SZ, _P]),
    "pkc_evict_select": (_I, [_P, _I64, _P, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "pkc_evict_compact": (_I, [_P, _I, _P, _P, _P, _P, _P, _I, _P, _P, _I64, _I, _I, _I, _I, _I64, _I,
                               _P, _SZ, _P]),
    "pkc_release_pages": (_I, [_P, _I, _P, _I, _I, _I64, _P, _P, _SZ, _P]),
    "pkc_assign_pages": (_I, [_P, _I, _P, _P, _I, _I, _I, _I64, _P, _P, _P, _P, _P, _SZ, _P]),
    "pkc_rope_append_kv": (_I, [_P, _I64, _P, _P, _I64, _P, _P, _P, _I, _I, _F, _I, _I, _I, _I, _P, _P, _P,
                                _I, _I64, _F, _F, _I, _I, _P, _SZ, _P]),
    "pkc_chunk_workspace_size": (_I, [_c.POINTER(_SZ)]),
    "pkc_paged_chunk_state": (_I, [_P, _P, _I, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I64, _F, _I, _I,
                                   _P, _SZ, _P, _P, _I, _I, _P]),
}

_lib = None
_lock = threading.Lock()


class PkcError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


def lib():
    """The loaded libpkc.so.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"libpkc.so not found at {LIB_PATH}; build it first "
                    "(python -c 'import __graft_entry__ as g; g.build()')")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def _check(rc):
    if rc != PKC_OK:
        raise PkcError(rc, lib().pkc_last_error().decode())


# A small call's time is the host's: the helpers below run a dozen times per
# call, so they import torch once, compare devices by index and hand plain
# integers to ctypes.
_torch = _get_device = _get_stream = None


def _getters(torch):
    """Functions for the current device's index and for a device's current
    stream (its handle): the ones torch's own wrappers call, which cost a
    fraction of them, or the wrappers in a torch that lacks those."""
    return (getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device,
            getattr(torch._C, "_cuda_getCurrentRawStream", None)
            or (lambda index: torch.cuda.current_stream(index).cuda_stream))


def _t():
    """torch, imported on the first call that takes tensors."""
    global _torch, _get_device, _get_stream
    if _torch is None:
        import torch
        _get_device, _get_stream = _getters(torch)
        _torch = torch
    return _torch


def _dtype_code(t) -> int:
    torch = _torch or _t()
    d = t.dtype
    return F16 if d == torch.float16 else BF16 if d == torch.bfloat16 else {torch.float32: F32}[d]


def _device():
    """The current device's index (tensors on it exist: CUDA is initialised)."""
    if _torch is None:
        _t()
    return _get_device()


def _stream(stream):
    if stream is None:
        index = _device()
        return _get_stream(index)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _host_i32(a):
    return np.ascontiguousarray(np.asarray(a), dtype=np.int32)


def _hptr(a):
    return None if a is None else ctypes.c_void_p(a.ctypes.data)


# ---------------------------------------------------------------------------
# Argument checks.  The C ABI takes raw pointers and sizes, so a tensor of the
# wrong dtype, shape or device would be read past its end; the binding
# checks every tensor against the sizes it passes down.
# ---------------------------------------------------------------------------

def _expect(name, t, dtypes, shape, device=None):
    """t must be a contiguous CUDA tensor of one of `dtypes` whose shape
    matches `shape` (None entries match any size) on `device`."""
    if not isinstance(t, (_torch or _t()).Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape == shape and t.dtype in dtypes and t.is_contiguous() and device is not None and t.device == device:
        return
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {list(dtypes)}")
    if len(t.shape) != len(shape) or any(w is not None and w != g for g, w in zip(t.shape, shape)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)} (None = any)")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be on {device if device is not None else 'a CUDA device'}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_paged(q, k_cache, v_cache, block_table, cache_seqlens, workspace, o, lse, kv_dtypes):
    """The common tensors of the paged-decode and cascade calls."""
    import torch
    _expect("q", q, (torch.float16, torch.bfloat16), (None, None, None))
    B, Hq, D = q.shape
    dev = q.device
    _expect("k_cache", k_cache, kv_dtypes, (None, None, None, D), dev)
    _expect("v_cache", v_cache, (k_cache.dtype,), tuple(k_cache.shape), dev)
    _expect("block_table", block_table, (torch.int32,), (B, None), dev)
    _expect("cache_seqlens", cache_seqlens, (torch.int32,), (B,), dev)
    if workspace is not None:
        _expect("workspace", workspace, (torch.uint8,), (None,), dev)
    if o is not None:
        _expect("o", o, (q.dtype,), (B, Hq, D), dev)
    if lse is not None:
        _expect("lse", lse, (torch.float32,), (B, Hq), dev)


def _check_prefix(q, k_prefix, v_prefix, prefix_kv_indptr):
    """Contiguous shared prefixes [L, Hkv, D] of q's dtype, L >= the last indptr."""
    _expect("k_prefix", k_prefix, (q.dtype,), (None, None, q.shape[2]), q.device)
    _expect("v_prefix", v_prefix, (q.dtype,), tuple(k_prefix.shape), q.device)
    if len(prefix_kv_indptr) and int(prefix_kv_indptr[-1]) > k_prefix.shape[0]:
        raise ValueError("prefix_kv_indptr ends past the prefix tensors")


def version() -> int:
    return lib().pkc_version()


# ---------------------------------------------------------------------------
# Merge operator
# ---------------------------------------------------------------------------

def merge_state(v_a, s_a, v_b, s_b, v_out=None, s_out=None, stream=None):
    """(v_a, s_a) (+) (v_b, s_b); v [T, H, D], s [T, H] float32."""
    import torch
    _expect("v_a", v_a, (torch.float32, torch.float16, torch.bfloat16), (None, None, None))
    T, H, D = v_a.shape
    for name, t, dt, shp in (("s_a", s_a, torch.float32, (T, H)), ("v_b", v_b, v_a.dtype, (T, H, D)),
                             ("s_b", s_b, torch.float32, (T, H)), ("v_out", v_out, v_a.dtype, (T, H, D)),
                             ("s_out", s_out, torch.float32, (T, H))):
        if t is not None:
            _expect(name, t, (dt,), shp, v_a.device)
    v_out = torch.empty_like(v_a) if v_out is None else v_out
    s_out = torch.empty_like(s_a) if s_out is None else s_out
    _check(lib().pkc_merge_state(_ptr(v_a), _ptr(s_a), _ptr(v_b), _ptr(s_b), _ptr(v_out),
                                 _ptr(s_out), T, H, D, _dtype_code(v_a), _stream(stream)))
    return v_out, s_out


def merge_states(v, s, v_out=None, s_out=None, stream=None):
    """n-ary (+) over axis 1: v [T, n, H, D], s [T, n, H] -> [T, H, D], [T, H]."""
    import torch
    _expect("v", v, (torch.float32, torch.float16, torch.bfloat16), (None, None, None, None))
    T, n, H, D = v.shape
    _expect("s", s, (torch.float32,), (T, n, H), v.device)
    if v_out is not None:
        _expect("v_out", v_out, (v.dtype,), (T, H, D), v.device)
    if s_out is not None:
        _expect("s_out", s_out, (torch.float32,), (T, H), v.device)
    v_out = torch.empty((T, H, D), dtype=v.dtype, device=v.device) if v_out is None else v_out
    s_out = torch.empty((T, H), dtype=torch.float32, device=v.device) if s_out is None else s_out
    _check(lib().pkc_merge_states(_ptr(v), _ptr(s), _ptr(v_out), _ptr(s_out), T, n, H, D,
                                  _dtype_code(v), _stream(stream)))
    return v_out, s_out


def merge_states_to(v, s, out_dtype, v_out=None, s_out=None, stream=None):
    """n-ary (+) of float32 states v [T, n, H, D], s [T, n, H] into a result
    of out_dtype (torch.float16 / torch.bfloat16 / torch.float32), rounded
    once."""
    import torch
    _expect("v", v, (torch.float32,), (None, None, None, None))
    T, n, H, D = v.shape
    _expect("s", s, (torch.float32,), (T, n, H), v.device)
    if v_out is not None:
        _expect("v_out", v_out, (out_dtype,), (T, H, D), v.device)
    if s_out is not None:
        _expect("s_out", s_out, (torch.float32,), (T, H), v.device)
    v_out = torch.empty((T, H, D), dtype=out_dtype, device=v.device) if v_out is None else v_out
    s_out = torch.empty((T, H), dtype=torch.float32, device=v.device) if s_out is None else s_out
    _check(lib().pkc_merge_states_to(_ptr(v), _ptr(s), _ptr(v_out), _ptr(s_out), T, n, H, D, F32,
                                     _dtype_code(v_out), _stream(stream)))
    return v_out, s_out


# ---------------------------------------------------------------------------
# Plan and workspace
# ---------------------------------------------------------------------------

def plan_words(n, num_ctas, tile_q=1, qo_len=None) -> int:
    q = None if qo_len is None else _host_i32(qo_len)
    out = ctypes.c_size_t()
    _check(lib().pkc_plan_words(_hptr(q), n, tile_q, num_ctas, ctypes.byref(out)))
    return out.value


def plan(kv_len, num_ctas, tile_q=1, qo_len=None, alpha=1.0, beta=1.0, out=None):
    """Host-side load-balanced plan; returns the int32 plan buffer."""
    kv = _host_i32(kv_len)
    q = None if qo_len is None else _host_i32(qo_len)
    words = plan_words(len(kv), num_ctas, tile_q, q)
    if out is None:
        out = np.zeros(words, np.int32)
    assert out.dtype == np.int32 and out.flags.c_contiguous and out.size >= words
    _check(lib().pkc_plan(_hptr(q), _hptr(kv), len(kv), tile_q, num_ctas, float(alpha),
                          float(beta), _hptr(out), out.size))
    return out


def plan_upload(plan_buf, workspace, stream=None):
    _check(lib().pkc_plan_upload(_hptr(plan_buf), _ptr(workspace), workspace.numel(),
                                 _stream(stream)))


def workspace_size(batch, num_qo_heads, num_ctas=0, prefix_splits=0, head_dim=128) -> int:
    out = ctypes.c_size_t()
    _check(lib().pkc_workspace_size(batch, num_qo_heads, head_dim, num_ctas, prefix_splits,
                                    ctypes.byref(out)))
    return out.value


def workspace_init(workspace, stream=None):
    _check(lib().pkc_workspace_init(_ptr(workspace), workspace.numel(), _stream(stream)))


def device_status(workspace, stream=None) -> int:
    st = ctypes.c_int32()
    _check(lib().pkc_device_status(_ptr(workspace), _stream(stream), ctypes.byref(st)))
    return st.value


# ---------------------------------------------------------------------------
# Attention states
# ---------------------------------------------------------------------------

def paged_decode_state(q, k_cache, v_cache, block_table, cache_seqlens, sm_scale, workspace,
                       plan_buf=None, o=None, lse=None, stream=None):
    """States of q [B, Hq, 128] over each request's paged cache."""
    import torch
    _check_paged(q, k_cache, v_cache, block_table, cache_seqlens, workspace, o, lse, (q.dtype,))
    B, Hq, D = q.shape
    P, ps, Hkv, _ = k_cache.shape
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(lib().pkc_paged_decode_state(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), block_table.shape[1],
        _ptr(cache_seqlens), B, Hq, Hkv, D, ps, P, float(sm_scale), _hptr(plan_buf),
        _ptr(workspace), workspace.numel(), _ptr(o), _ptr(lse), _dtype_code(q), _stream(stream)))
    return o, lse


def paged_decode_state_fp8(q, k_cache, v_cache, block_table, cache_seqlens, sm_scale, workspace,
                           k_scale=1.0, v_scale=1.0, plan_buf=None, o=None, lse=None, stream=None):
    """States of fp16 q [B, Hq, 128] over an e4m3 paged cache (uint8 codes
    [P, page_size, Hkv, 128]); the cached values are k_scale * e4m3(k) and
    v_scale * e4m3(v)."""
    import torch
    B, Hq, D = q.shape
    P, ps, Hkv, _ = k_cache.shape
    if q.dtype != torch.float16 or k_cache.dtype != torch.uint8 or v_cache.dtype != torch.uint8:
        raise TypeError("paged_decode_state_fp8: q must be float16 and the caches uint8 e4m3 codes")
    _check_paged(q, k_cache, v_cache, block_table, cache_seqlens, workspace, o, lse, (torch.uint8,))
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(lib().pkc_paged_decode_state_fp8(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), block_table.shape[1],
        _ptr(cache_seqlens), B, Hq, Hkv, D, ps, P, float(sm_scale), float(k_scale), float(v_scale),
        _hptr(plan_buf), _ptr(workspace), workspace.numel(), _ptr(o), _ptr(lse), _stream(stream)))
    return o, lse


def append_kv(k_new, v_new, k_cache, v_cache, block_table, cache_seqlens, workspace,
              append_mask=None, stream=None):
    """Write one new token per request (k_new / v_new [B, Hkv, 128]) into the
    paged cache at each request's next slot and grow cache_seqlens by one, in
    place; an fp8 cache takes uint8 e4m3 codes."""
    import torch
    _expect("k_cache", k_cache, (torch.float16, torch.bfloat16, torch.uint8), (None, None, None, None))
    P, ps, Hkv, D = k_cache.shape
    dev = k_cache.device
    _expect("v_cache", v_cache, (k_cache.dtype,), tuple(k_cache.shape), dev)
    _expect("k_new", k_new, (k_cache.dtype,), (None, Hkv, D), dev)
    B = k_new.shape[0]
    _expect("v_new", v_new, (k_cache.dtype,), (B, Hkv, D), dev)
    _expect("block_table", block_table, (torch.int32,), (B, None), dev)
    _expect("cache_seqlens", cache_seqlens, (torch.int32,), (B,), dev)
    _expect("workspace", workspace, (torch.uint8,), (None,), dev)
    if append_mask is not None:
        _expect("append_mask", append_mask, (torch.uint8,), (B,), dev)
    if k_cache.dtype == torch.uint8:
        code = E4M3
    else:
        code = _dtype_code(k_cache)
    _check(lib().pkc_append_kv(
        _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
        block_table.shape[1], _ptr(cache_seqlens), _ptr(append_mask), B, Hkv, D, ps, P, code,
        _ptr(workspace), workspace.numel(), _stream(stream)))


# ---------------------------------------------------------------------------
# Microscaled 4-bit (mx4) paged cache
# ---------------------------------------------------------------------------

def _expect_current(t):
    """The library launches on the current device: refuse tensors of another."""
    if t.get_device() != _device():
        raise ValueError(f"tensors are on {t.device}, the current device is cuda:{_device()}")


def _expect_all(device, *specs):
    """_expect for many tensors of known dtype and shape: specs are
    (name, tensor, dtype, shape)."""
    index = device.index
    for name, t, dtype, shape in specs:
        try:
            if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == index:
                continue
        except AttributeError:
            pass  # not a tensor: _expect says so
        _expect(name, t, (dtype,), shape, device)


def _sizes(t, n):
    """t's sizes, with unknown ones to n where there are fewer (for a check)."""
    s = getattr(t, "shape", ())
    return tuple(s) if len(s) == n else (None,) * n


def _leading(name, t, dtypes, n, last=None):
    """Sizes of a call's first tensor, of n dimensions and on the current
    device; all else is left to _expect_all."""
    s = _sizes(t, n)
    if s[0] is None or t.dtype not in dtypes or not t.is_cuda or t.get_device() != _device():
        _expect(name, t, dtypes, (None,) * (n - 1) + (last,))
        _expect_current(t)
    return s


def _check_mx4(k_codes, k_scales, v_codes, v_scales, block_table, workspace):
    """The four pools of an mx4 cache, its table and the workspace."""
    torch = _torch or _t()
    u8 = torch.uint8
    P, ps, Hkv, _ = _leading("k_codes", k_codes, (u8,), 4, 64)
    B, n_pages = _sizes(block_table, 2)
    dev = k_codes.device
    _expect_all(dev, ("k_codes", k_codes, u8, (P, ps, Hkv, 64)), ("k_scales", k_scales, u8, (P, ps, Hkv, 4)),
                ("v_codes", v_codes, u8, (P, ps, Hkv, 64)), ("v_scales", v_scales, u8, (P, ps, Hkv, 4)),
                ("block_table", block_table, torch.int32, (B, n_pages)),
                ("workspace", workspace, u8, _sizes(workspace, 1)))
    return P, ps, Hkv, B, dev


def append_kv_mx4(k_new, v_new, new_indptr, k_codes, k_scales, v_codes, v_scales, block_table,
                  cache_seqlens, workspace, stream=None):
    """Quantise new tokens (k_new / v_new [T, Hkv, 128], rows new_indptr[b] ..
    new_indptr[b+1]-1 for request b, device int32) to the end of every
    request's mx4 cache and grow cache_seqlens, in place."""
    torch = _torch or _t()
    P, ps, Hkv, B, dev = _check_mx4(k_codes, k_scales, v_codes, v_scales, block_table, workspace)
    T = _sizes(k_new, 3)[0]
    _expect("k_new", k_new, (torch.float16, torch.bfloat16), (T, Hkv, 128), dev)
    _expect_all(dev, ("v_new", v_new, k_new.dtype, (T, Hkv, 128)),
                ("new_indptr", new_indptr, torch.int32, (B + 1,)),
                ("cache_seqlens", cache_seqlens, torch.int32, (B,)))
    _check(lib().pkc_append_kv_mx4(
        _ptr(k_new), _ptr(v_new), _ptr(new_indptr), k_new.shape[0], _ptr(k_codes), _ptr(k_scales),
        _ptr(v_codes), _ptr(v_scales), _ptr(block_table), block_table.shape[1], _ptr(cache_seqlens),
        B, Hkv, 128, ps, P, _dtype_code(k_new), _ptr(workspace), workspace.numel(), _stream(stream)))


def gather_kv_mx4(k_codes, k_scales, v_codes, v_scales, block_table, first, out_indptr, total,
                  workspace, dtype=None, k=None, v=None, stream=None):
    """Tokens of an mx4 cache as 16-bit rows [total, Hkv, 128] of dtype
    (default torch.float16): row t of out_indptr[b] .. out_indptr[b+1]-1 is
    token first[b] + t - out_indptr[b] of request b.  Rows of no request stay
    as they were in given k and v (and are undefined in new ones)."""
    torch = _torch or _t()
    P, ps, Hkv, B, dev = _check_mx4(k_codes, k_scales, v_codes, v_scales, block_table, workspace)
    _expect_all(dev, ("first", first, torch.int32, (B,)), ("out_indptr", out_indptr, torch.int32, (B + 1,)))
    if dtype is None:
        dtype = torch.float16 if k is None else k.dtype
    if dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"gather_kv_mx4: dtype must be torch.float16 or torch.bfloat16 (got {dtype})")
    total = int(total)
    if total < 0:
        raise ValueError(f"gather_kv_mx4: total must be >= 0 (got {total})")
    for name, t in (("k", k), ("v", v)):
        if t is not None:
            _expect(name, t, (dtype,), (total, Hkv, 128), dev)
    k = torch.empty((total, Hkv, 128), dtype=dtype, device=dev) if k is None else k
    v = torch.empty_like(k) if v is None else v
    _check(lib().pkc_gather_kv_mx4(
        _ptr(k_codes), _ptr(k_scales), _ptr(v_codes), _ptr(v_scales), _ptr(block_table),
        block_table.shape[1], _ptr(first), _ptr(out_indptr), total, B, Hkv, 128, ps, P, _ptr(k),
        _ptr(v), _dtype_code(k), _ptr(workspace), workspace.numel(), _stream(stream)))
    return k, v


def paged_decode_state_mx4(q, k_codes, k_scales, v_codes, v_scales, block_table, cache_seqlens,
                           sm_scale, workspace, plan_buf=None, o=None, lse=None, stream=None):
    """States of fp16 / bf16 q [B, Hq, 128] over each request's mx4 cache."""
    torch = _torch or _t()
    P, ps, Hkv, B, dev = _check_mx4(k_codes, k_scales, v_codes, v_scales, block_table, workspace)
    Hq = _sizes(q, 3)[1]
    _expect("q", q, (torch.float16, torch.bfloat16), (B, Hq, 128), dev)
    _expect_all(dev, ("cache_seqlens", cache_seqlens, torch.int32, (B,)))
    if o is not None:
        _expect("o", o, (q.dtype,), (B, Hq, 128), dev)
    if lse is not None:
        _expect("lse", lse, (torch.float32,), (B, Hq), dev)
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, Hq), dtype=torch.float32, device=dev) if lse is None else lse
    _check(lib().pkc_paged_decode_state_mx4(
        _ptr(q), _ptr(k_codes), _ptr(k_scales), _ptr(v_codes), _ptr(v_scales), _ptr(block_table),
        block_table.shape[1], _ptr(cache_seqlens), B, Hq, Hkv, 128, ps, P, float(sm_scale),
        _hptr(plan_buf), _ptr(workspace), workspace.numel(), _ptr(o), _ptr(lse), _dtype_code(q),
        _stream(stream)))
    return o, lse


# ---------------------------------------------------------------------------
# Eviction by accumulated attention weight
# ---------------------------------------------------------------------------

def _kv_kind(cache, scales):
    """(kv_dtype code, row length) of a cache: 16-bit, e4m3 codes, or mx4
    codes (given with their scales)."""
    torch = _torch or _t()
    if scales is not None:
        return MX4, 64
    if cache.dtype == torch.uint8:
        return E4M3, 128
    return _dtype_code(cache), 128


def accumulate_weights(q, lse, k_cache, block_table, cache_seqlens, sm_scale, weights, workspace,
                       decay=1.0, k_scale=1.0, k_scales=None, stream=None):
    """weights[b, h, t] = decay * weights[b, h, t] + the attention weights that
    q [B, Hq, 128] with LSE lse [B, Hq] gives cached token t, summed over KV
    head h's query heads; weights [B, Hkv, W] float32, in place.  k_cache:
    16-bit of q's dtype, e4m3 codes (fp16 q, k_scale), or mx4 codes with
    k_scales."""
    torch = _torch or _t()
    P, ps, Hkv, _ = _leading("k_cache", k_cache, (torch.float16, torch.bfloat16, torch.uint8), 4)
    kind, row = _kv_kind(k_cache, k_scales)
    dev = k_cache.device
    kv_dtype = torch.uint8 if k_scales is not None else k_cache.dtype
    B, Hq, _ = _sizes(q, 3)
    _expect("q", q, (torch.float16, torch.bfloat16), (B, Hq, 128), dev)
    _expect_all(dev, ("k_cache", k_cache, kv_dtype, (P, ps, Hkv, row)),
                ("lse", lse, torch.float32, (B, Hq)),
                ("block_table", block_table, torch.int32, (B, _sizes(block_table, 2)[1])),
                ("cache_seqlens", cache_seqlens, torch.int32, (B,)),
                ("weights", weights, torch.float32, (B, Hkv, _sizes(weights, 3)[2])),
                ("workspace", workspace, torch.uint8, _sizes(workspace, 1)))
    if k_scales is not None:
        _expect("k_scales", k_scales, (torch.uint8,), (P, ps, Hkv, 4), dev)
    _check(lib().pkc_accumulate_weights(
        _ptr(q), _ptr(lse), _ptr(k_cache), _ptr(k_scales), _ptr(block_table), block_table.shape[1],
        _ptr(cache_seqlens), B, Hq, Hkv, 128, ps, P, float(sm_scale), float(k_scale), float(decay),
        _ptr(weights), weights.shape[2], _dtype_code(q), kind, _ptr(workspace), workspace.numel(),
        _stream(stream)))
    return weights


def evict_select(weights, cache_seqlens, budget, sinks, recent, workspace, keep=None, stream=None):
    """The slots that each (request, KV head) keeps, [B, Hkv, budget] int32 in
    ascending order: the first `sinks`, the last `recent`, and the largest of
    weights [B, Hkv, W] between them (all, then -1, of a request within the
    budget)."""
    torch = _torch or _t()
    B, Hkv, W = _leading("weights", weights, (torch.float32,), 3)
    dev = weights.device
    budget, sinks, recent = int(budget), int(sinks), int(recent)
    if budget < 1 or sinks < 0 or recent < 0 or sinks + recent > budget:
        raise ValueError("evict_select: budget must be >= 1, sinks and recent >= 0 and together at most the "
                         f"budget (got {budget}, {sinks}, {recent})")
    _expect_all(dev, ("weights", weights, torch.float32, (B, Hkv, W)),
                ("cache_seqlens", cache_seqlens, torch.int32, (B,)),
                ("workspace", workspace, torch.uint8, _sizes(workspace, 1)))
    if keep is not None:
        _expect("keep", keep, (torch.int32,), (B, Hkv, budget), dev)
    keep = torch.empty((B, Hkv, budget), dtype=torch.int32, device=dev) if keep is None else keep
    _check(lib().pkc_evict_select(_ptr(weights), W, _ptr(cache_seqlens), B, Hkv, budget, sinks, recent,
                                  _ptr(keep), _ptr(workspace), workspace.numel(), _stream(stream)))
    return keep


def evict_compact(keep, k_cache, v_cache, block_table, cache_seqlens, workspace, weights=None,
                  k_scales=None, v_scales=None, stream=None):
    """Move the slots keep [B, Hkv, budget] of every request longer than the
    budget to its first slots and cut its length, in place: K and V (16-bit,
    e4m3 codes, or mx4 codes with their scales) and, given, the accumulated
    weights [B, Hkv, W]."""
    torch = _torch or _t()
    P, ps, Hkv, _ = _leading("k_cache", k_cache, (torch.float16, torch.bfloat16, torch.uint8), 4)
    if (k_scales is None) != (v_scales is None):
        raise ValueError("evict_compact: k_scales and v_scales are given together")
    kind, row = _kv_kind(k_cache, k_scales)
    dev = k_cache.device
    kv_dtype = torch.uint8 if k_scales is not None else k_cache.dtype
    B, _, budget = _sizes(keep, 3)
    _expect_all(dev, ("k_cache", k_cache, kv_dtype, (P, ps, Hkv, row)), ("v_cache", v_cache, kv_dtype, (P, ps, Hkv, row)),
                ("keep", keep, torch.int32, (B, Hkv, budget)),
                ("block_table", block_table, torch.int32, (B, _sizes(block_table, 2)[1])),
                ("cache_seqlens", cache_seqlens, torch.int32, (B,)),
                ("workspace", workspace, torch.uint8, _sizes(workspace, 1)))
    if k_scales is not None:
        _expect_all(dev, ("k_scales", k_scales, torch.uint8, (P, ps, Hkv, 4)),
                    ("v_scales", v_scales, torch.uint8, (P, ps, Hkv, 4)))
    if weights is not None:
        _expect_all(dev, ("weights", weights, torch.float32, (B, Hkv, _sizes(weights, 3)[2])))
    _check(lib().pkc_evict_compact(
        _ptr(keep), budget, _ptr(k_cache), _ptr(v_cache), _ptr(k_scales), _ptr(v_scales),
        _ptr(block_table), block_table.shape[1], _ptr(cache_seqlens), _ptr(weights),
        0 if weights is None else weights.shape[2], B, Hkv, 128, ps, P, kind, _ptr(workspace),
        workspace.numel(), _stream(stream)))


# ---------------------------------------------------------------------------
# A prompt's way into the cache: pages, rotary positions, chunk attention
# ---------------------------------------------------------------------------

def page_pool(num_pages, device="cuda"):
    """The map of a pool whose pages are all free: int32 words, bit p % 32 of
    word p / 32 for page p (release_pages and assign_pages keep it)."""
    torch = _torch or _t()
    num_pages = int(num_pages)
    if num_pages < 0:
        raise ValueError(f"page_pool: num_pages must be >= 0 (got {num_pages})")
    words = np.full((num_pages + 31) // 32, 0xFFFFFFFF, np.uint32)
    if num_pages % 32:
        words[-1] = (1 << num_pages % 32) - 1
    return torch.from_numpy(words.view(np.int32)).to(device)


def _c_int(name, x):
    """x as the C int that ctypes would cut it to."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} must fit in 32 bits (got {x})")
    return x


# The calls of a step pass their tensors through one expression: all as they
# should be, or _expect says what is not (a check after another costs 2 us more
# of a call's 16).

def _check_pages(block_table, cache_seqlens, free_pages, num_pages, workspace):
    torch = _torch or _t()
    try:
        B, n_pages = block_table.shape
        i32, at = torch.int32, block_table.get_device()
        if (at >= 0 and at == _get_device() and num_pages >= 0 and type(num_pages) is int
                and block_table.dtype is i32 and cache_seqlens.dtype is i32 and free_pages.dtype is i32 and workspace.dtype is torch.uint8
                and cache_seqlens.shape == (B,) and free_pages.shape == ((num_pages + 31) // 32,) and workspace.dim() == 1
                and block_table.is_contiguous() and cache_seqlens.is_contiguous() and free_pages.is_contiguous() and workspace.is_contiguous()
                and cache_seqlens.get_device() == at and free_pages.get_device() == at and workspace.get_device() == at):
            return B, n_pages, num_pages, block_table.device
    except (AttributeError, TypeError, ValueError):
        pass
    B, n_pages = _leading("block_table", block_table, (torch.int32,), 2)
    dev = block_table.device
    num_pages = int(num_pages)
    if num_pages < 0:
        raise ValueError(f"num_pages must be >= 0 (got {num_pages})")
    _expect_all(dev, ("block_table", block_table, torch.int32, (B, n_pages)),
                ("cache_seqlens", cache_seqlens, torch.int32, (B,)),
                ("free_pages", free_pages, torch.int32, ((num_pages + 31) // 32,)),
                ("workspace", workspace, torch.uint8, _sizes(workspace, 1)))
    return B, n_pages, num_pages, dev


def release_pages(block_table, cache_seqlens, free_pages, page_size, num_pages, workspace, stream=None):
    """Give the pages behind every request's length back to the pool
    free_pages (of page_pool), in place: their table entries become -1."""
    B, stride, num_pages, _ = _check_pages(block_table, cache_seqlens, free_pages, num_pages, workspace)
    _check(lib().pkc_release_pages(
        block_table.data_ptr(), stride, cache_seqlens.data_ptr(), B, _c_int("page_size", page_size), num_pages, free_pages.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _stream(stream)))


def assign_pages(block_table, cache_seqlens, new_indptr, total_new, free_pages, page_size, num_pages, workspace,
                 slots=None, positions=None, seqlens_out=None, stream=None):
    """Pages for total_new new tokens (request b's are new_indptr[b] ..
    new_indptr[b+1]-1, device int32) taken from free_pages into block_table, in
    place.  Returns (slots [total_new] int64: page * page_size + slot, or -1;
    positions [total_new] int32; the lengths with the new tokens [B] int32,
    a new tensor unless seqlens_out is given -- cache_seqlens itself may be)."""
    torch = _torch or _t()
    B, stride, num_pages, dev = _check_pages(block_table, cache_seqlens, free_pages, num_pages, workspace)
    total = _c_int("total_new", total_new)
    if total < 0:
        raise ValueError(f"assign_pages: total_new must be >= 0 (got {total})")
    _expect_all(dev, ("new_indptr", new_indptr, torch.int32, (B + 1,)))
    if slots is None:
        slots = torch.empty(total, dtype=torch.int64, device=dev)
    else:
        _expect("slots", slots, (torch.int64,), (total,), dev)
    if positions is None:
        positions = torch.empty(total, dtype=torch.int32, device=dev)
    else:
        _expect("positions", positions, (torch.int32,), (total,), dev)
    if seqlens_out is None:
        seqlens_out = torch.empty_like(cache_seqlens)
    else:
        _expect("seqlens_out", seqlens_out, (torch.int32,), (B,), dev)
    _check(lib().pkc_assign_pages(
        block_table.data_ptr(), stride, cache_seqlens.data_ptr(), new_indptr.data_ptr(), total, B, _c_int("page_size", page_size), num_pages,
        free_pages.data_ptr(), slots.data_ptr(), positions.data_ptr(), seqlens_out.data_ptr(), workspace.data_ptr(), workspace.numel(),
        _stream(stream)))
    return slots, positions, seqlens_out


def rope_frequencies(rotary_dim=128, base=10000.0, factor=1.0, context=None, slow=1.0, fast=32.0, device="cuda"):
    """(inv_freq [rotary_dim / 2] float64, amplitude) for rope_append_kv: base
    ** (-2 i / rotary_dim) radians per token.  factor > 1 stretches positions
    that many times: all pairs alike without `context` (amplitude 1), else by
    parts -- pairs that turn `fast` times or more within `context` tokens keep
    their frequency, those that turn `slow` times or less are slowed by the
    factor, with a linear blend between (amplitude 0.1 ln factor + 1)."""
    torch = _torch or _t()
    rotary_dim, base, factor = int(rotary_dim), float(base), float(factor)
    if rotary_dim < 2 or rotary_dim % 2 or not base > 0 or not factor >= 1:
        raise ValueError("rope_frequencies: rotary_dim must be even and >= 2, base > 0, factor >= 1 "
                         f"(got {rotary_dim}, {base}, {factor})")
    f = base ** (-np.arange(0, rotary_dim, 2, dtype=np.float64) / rotary_dim)
    amplitude = 1.0
    if factor > 1 and context is None:
        f = f / factor
    elif factor > 1:
        if not (float(context) > 0 and fast > slow):
            raise ValueError("rope_frequencies: context must be > 0 and fast > slow")
        keep = np.clip((float(context) * f / (2 * np.pi) - slow) / (fast - slow), 0.0, 1.0)
        f = f * (keep + (1 - keep) / factor)
        amplitude = 0.1 * float(np.log(factor)) + 1.0
    return torch.from_numpy(f).to(device), amplitude


def _expect_rows(name, t, dtype, shape, device):
    """t [T, H, 128] with dense heads: the tokens may lie apart, as in a part
    of a larger projection.  Returns the distance of two tokens in elements."""
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != device.index:
        raise ValueError(f"{name} must be on {device}")
    st = t.stride()
    if st[2] != 1 or (st[1] != 128 and shape[1] != 1):
        raise ValueError(f"{name} must have dense heads (strides {st})")
    return st[0] if shape[0] > 1 else shape[1] * 128


def rope_append_kv(q, k_new, v_new, positions, slots, inv_freq, k_cache, v_cache, workspace, interleaved=False,
                   amplitude=1.0, k_scale=1.0, v_scale=1.0, q_out=None, stream=None):
    """Turn q [T, Hq, 128] and k_new [T, Hkv, 128] by their positions [T] int32
    (pairs of the first 2 * len(inv_freq) elements; inv_freq float64 as of
    rope_frequencies), write k and v_new [T, Hkv, 128] to slots [T] int64 of the
    paged pools (of q's dtype, or uint8 e4m3 codes with scales) and return the
    turned q (dense).  q, k_new and v_new may be slices of one projection."""
    torch = _torch or _t()
    try:
        pool, (T, Hq, D), (half,) = k_cache.shape, q.shape, inv_freq.shape
        P, ps, Hkv, row = pool
        rows, dtype, kv_dtype, at = (T, Hkv, 128), q.dtype, k_cache.dtype, k_cache.get_device()
        (q_stride, q_head, q_one), kv_strides = q.stride(), k_new.stride()
        kv_stride, kv_head, kv_one = kv_strides
        plain = (at >= 0 and at == _get_device() and T > 1 and D == 128 and row == 128
                 and (dtype is torch.float16 or dtype is torch.bfloat16) and (kv_dtype is dtype or kv_dtype is torch.uint8)
                 and k_new.dtype is dtype and v_new.dtype is dtype and v_cache.dtype is kv_dtype and positions.dtype is torch.int32
                 and slots.dtype is torch.int64 and inv_freq.dtype is torch.float64 and workspace.dtype is torch.uint8
                 and k_new.shape == rows and v_new.shape == rows and v_cache.shape == pool and positions.shape == (T,)
                 and slots.shape == (T,) and workspace.dim() == 1
                 and q_head == 128 and q_one == 1 and kv_head == 128 and kv_one == 1 and v_new.stride() == kv_strides
                 and k_cache.is_contiguous() and v_cache.is_contiguous() and positions.is_contiguous() and slots.is_contiguous()
                 and inv_freq.is_contiguous() and workspace.is_contiguous()
                 and q.get_device() == at and k_new.get_device() == at and v_new.get_device() == at and v_cache.get_device() == at
                 and positions.get_device() == at and slots.get_device() == at and inv_freq.get_device() == at
                 and workspace.get_device() == at)
    except (AttributeError, TypeError, ValueError):
        plain = False
    if not plain:
        P, ps, Hkv, _ = _leading("k_cache", k_cache, (torch.float16, torch.bfloat16, torch.uint8), 4, 128)
        dev = k_cache.device
        T, Hq, _ = _sizes(q, 3)
        if T is None or q.dtype not in (torch.float16, torch.bfloat16):
            _expect("q", q, (torch.float16, torch.bfloat16), (None, None, 128), dev)
        dtype = q.dtype
        q_stride = _expect_rows("q", q, dtype, (T, Hq, 128), dev)
        kv_stride = _expect_rows("k_new", k_new, dtype, (T, Hkv, 128), dev)
        if _expect_rows("v_new", v_new, dtype, (T, Hkv, 128), dev) != kv_stride:
            raise ValueError("k_new and v_new must have the same strides")
        kv_dtype = torch.uint8 if k_cache.dtype == torch.uint8 else dtype
        half = _sizes(inv_freq, 1)[0]
        _expect_all(dev, ("k_cache", k_cache, kv_dtype, (P, ps, Hkv, 128)), ("v_cache", v_cache, kv_dtype, (P, ps, Hkv, 128)),
                    ("positions", positions, torch.int32, (T,)), ("slots", slots, torch.int64, (T,)),
                    ("inv_freq", inv_freq, torch.float64, (half,)),
                    ("workspace", workspace, torch.uint8, _sizes(workspace, 1)))
    dev = k_cache.device
    if q_out is None:
        q_out = torch.empty((T, Hq, 128), dtype=dtype, device=dev)
    else:
        _expect("q_out", q_out, (dtype,), (T, Hq, 128), dev)
    code = F16 if dtype is torch.float16 else BF16
    _check(lib().pkc_rope_append_kv(
        q.data_ptr(), q_stride, k_new.data_ptr(), v_new.data_ptr(), kv_stride, positions.data_ptr(), slots.data_ptr(), inv_freq.data_ptr(),
        2 * half, 1 if interleaved else 0, float(amplitude), T, Hq, Hkv, 128, q_out.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), ps, P, float(k_scale), float(v_scale), code, E4M3 if kv_dtype is torch.uint8 else code,
        workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return q_out


def chunk_workspace_size() -> int:
    """Bytes of workspace that paged_chunk_state needs, for any problem (added
    to workspace_size(...) where one workspace serves other calls too)."""
    out = ctypes.c_size_t()
    _check(lib().pkc_chunk_workspace_size(ctypes.byref(out)))
    return out.value


def paged_chunk_state(q, q_indptr, k_cache, v_cache, block_table, cache_seqlens, sm_scale, workspace, causal=True,
                      window=0, out_dtype=None, o=None, lse=None, stream=None):
    """States of a chunk of new tokens per request over its paged cache, which
    holds them already: q [T, Hq, 128], rows q_indptr[b] .. q_indptr[b+1]-1
    (device int32) are the last of request b's cache_seqlens[b] tokens.  A row
    attends to the tokens up to its own (all, if not causal), at most the last
    `window` of them (0: no limit).  o has q's dtype, or float32 (out_dtype)
    for states merged further."""
    torch = _torch or _t()
    try:
        pool, (T, Hq, D), (B, stride) = k_cache.shape, q.shape, block_table.shape
        P, ps, Hkv, row = pool
        dtype, i32, at = k_cache.dtype, torch.int32, k_cache.get_device()
        plain = (at >= 0 and at == _get_device() and D == 128 and row == 128
                 and (dtype is torch.float16 or dtype is torch.bfloat16) and q.dtype is dtype and v_cache.dtype is dtype
                 and block_table.dtype is i32 and q_indptr.dtype is i32 and cache_seqlens.dtype is i32 and workspace.dtype is torch.uint8
                 and v_cache.shape == pool and q_indptr.shape == (B + 1,) and cache_seqlens.shape == (B,) and workspace.dim() == 1
                 and q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous() and block_table.is_contiguous()
                 and q_indptr.is_contiguous() and cache_seqlens.is_contiguous() and workspace.is_contiguous()
                 and q.get_device() == at and v_cache.get_device() == at and block_table.get_device() == at
                 and q_indptr.get_device() == at and cache_seqlens.get_device() == at and workspace.get_device() == at)
    except (AttributeError, TypeError, ValueError):
        plain = False
    if not plain:
        P, ps, Hkv, _ = _leading("k_cache", k_cache, (torch.float16, torch.bfloat16), 4, 128)
        dtype = k_cache.dtype
        T, Hq, _ = _sizes(q, 3)
        B, stride = _sizes(block_table, 2)
        _expect_all(k_cache.device, ("q", q, dtype, (T, Hq, 128)), ("k_cache", k_cache, dtype, (P, ps, Hkv, 128)),
                    ("v_cache", v_cache, dtype, (P, ps, Hkv, 128)), ("block_table", block_table, torch.int32, (B, stride)),
                    ("q_indptr", q_indptr, torch.int32, (None if B is None else B + 1,)),
                    ("cache_seqlens", cache_seqlens, torch.int32, (B,)),
                    ("workspace", workspace, torch.uint8, _sizes(workspace, 1)))
    dev = k_cache.device
    if out_dtype is None:
        out_dtype = dtype if o is None else o.dtype
    if out_dtype is not dtype and out_dtype is not torch.float32:
        raise TypeError(f"paged_chunk_state: out_dtype must be {dtype} or torch.float32 (got {out_dtype})")
    if o is None:
        o = torch.empty_like(q, dtype=out_dtype)
    else:
        _expect("o", o, (out_dtype,), (T, Hq, 128), dev)
    if lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    else:
        _expect("lse", lse, (torch.float32,), (T, Hq), dev)
    code = F16 if dtype is torch.float16 else BF16
    _check(lib().pkc_paged_chunk_state(
        q.data_ptr(), q_indptr.data_ptr(), T, k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), stride, cache_seqlens.data_ptr(), B,
        Hq, Hkv, 128, ps, P, float(sm_scale), 1 if causal else 0, _c_int("window", window), workspace.data_ptr(), workspace.numel(),
        o.data_ptr(), lse.data_ptr(), code, F32 if out_dtype is torch.float32 else code, _stream(stream)))
    return o, lse


DECODE_KERNELS = {"auto": 0, "simt": 1, "mma": 2}


def set_decode_kernel(which):
    """Kernel for 16-bit paged decode: "auto", "simt" (CUDA cores) or "mma"
    (tensor cores); process-wide."""
    _check(lib().pkc_set_decode_kernel(DECODE_KERNELS[which]))


DECODE_SCHEDULES = {"dynamic": 1, "static": 0}


def set_decode_schedule(which):
    """Schedule of a planned decode: "dynamic" (blocks take the plan's chunks
    from a shared longest-first queue; default) or "static" (each block runs
    its CTA's list of the plan); process-wide."""
    _check(lib().pkc_set_decode_schedule(DECODE_SCHEDULES[which]))


def set_contraction(which):
    """'separate' (default): a standalone contraction kernel, launched as the
    suffix decode's programmatic dependent; 'separate_plain': the same kernel
    launched plainly; 'fused': the attention kernels contract split states
    themselves (one launch fewer).  All give the same bits."""
    _check(lib().pkc_set_contraction({"separate": 0, "fused": 1, "separate_plain": 2}[which]))


def set_cascade_small(max_rows):
    """Largest query rows per KV head of a prefix group for which an unplanned
    cascade reads its prefixes through the decode kernel (one launch); 0 never."""
    _check(lib().pkc_set_cascade_small(int(max_rows)))


def set_prefix_ctas(n):
    """Thread blocks of the prefix stage: n > 0 caps them at n; 0 (default)
    is automatic: every SM, or, in a planned cascade call whose prefix is
    bound by the tensor pipe, a quarter of the SMs next to a dynamically
    scheduled decode on the rest (pkc.h, pkc_set_prefix_ctas); process-wide."""
    n = int(n)
    if n < 0:
        raise ValueError(f"set_prefix_ctas: n must be >= 0 (got {n})")
    _check(lib().pkc_set_prefix_ctas(n))


def last_launch_blocks():
    """(prefix blocks, decode blocks) of this thread's last cascade call."""
    pb, db = _c.c_int(0), _c.c_int(0)
    _check(lib().pkc_last_launch_blocks(_c.byref(pb), _c.byref(db)))
    return pb.value, db.value


def paged_decode_state_noalloc(q, k_cache, v_cache, block_table, cache_seqlens, sm_scale,
                               plan_buf=None, o=None, lse=None, device_status=None, stream=None):
    """paged_decode_state without a caller workspace, for callers that
    cannot allocate device memory: the library's own fixed 8 MiB device
    array holds the scratch.  Calls that overlap on the GPU race on it."""
    import torch
    _check_paged(q, k_cache, v_cache, block_table, cache_seqlens, None, o, lse, (q.dtype,))
    B, Hq, D = q.shape
    P, ps, Hkv, _ = k_cache.shape
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(lib().pkc_paged_decode_state_noalloc(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), block_table.shape[1],
        _ptr(cache_seqlens), B, Hq, Hkv, D, ps, P, float(sm_scale), _hptr(plan_buf), _ptr(o),
        _ptr(lse), _ptr(device_status), _dtype_code(q), _stream(stream)))
    return o, lse


def prefix_attention_state(q, k_prefix, v_prefix, prefix_kv_indptr, prefix_req_indptr, sm_scale,
                           workspace, o=None, lse=None, stream=None):
    """States of q [B, Hq, 128] over each request's shared prefix (fp32 O)."""
    import torch
    _expect("q", q, (torch.float16, torch.bfloat16), (None, None, None))
    _check_prefix(q, k_prefix, v_prefix, _host_i32(prefix_kv_indptr))
    _expect("workspace", workspace, (torch.uint8,), (None,), q.device)
    if o is not None:
        _expect("o", o, (torch.float32,), tuple(q.shape), q.device)
    if lse is not None:
        _expect("lse", lse, (torch.float32,), tuple(q.shape[:2]), q.device)
    B, Hq, D = q.shape
    Hkv = k_prefix.shape[1]
    kv_ptr, req_ptr = _host_i32(prefix_kv_indptr), _host_i32(prefix_req_indptr)
    o = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device) if o is None else o
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(lib().pkc_prefix_attention_state(
        _ptr(q), _ptr(k_prefix), _ptr(v_prefix), _hptr(kv_ptr), _hptr(req_ptr), len(kv_ptr) - 1,
        B, Hq, Hkv, D, float(sm_scale), _ptr(workspace), workspace.numel(), _ptr(o), _ptr(lse),
        _dtype_code(q), _stream(stream)))
    return o, lse


def cascade_decode(q, k_prefix, v_prefix, prefix_kv_indptr, prefix_req_indptr, k_cache, v_cache,
                   block_table, cache_seqlens, sm_scale, workspace, plan_buf=None, o=None,
                   lse=None, stream=None):
    """Final O [B, Hq, 128] and LSE [B, Hq] over shared prefix + paged suffix."""
    import torch
    _check_paged(q, k_cache, v_cache, block_table, cache_seqlens, workspace, o, lse, (q.dtype,))
    _check_prefix(q, k_prefix, v_prefix, _host_i32(prefix_kv_indptr))
    B, Hq, D = q.shape
    P, ps, Hkv, _ = k_cache.shape
    kv_ptr, req_ptr = _host_i32(prefix_kv_indptr), _host_i32(prefix_req_indptr)
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(lib().pkc_cascade_decode(
        _ptr(q), _ptr(k_prefix), _ptr(v_prefix), _hptr(kv_ptr), _hptr(req_ptr), len(kv_ptr) - 1,
        _ptr(k_cache), _ptr(v_cache), _ptr(block_table), block_table.shape[1], _ptr(cache_seqlens),
        B, Hq, Hkv, D, ps, P, float(sm_scale), _hptr(plan_buf), _ptr(workspace),
        workspace.numel(), _ptr(o), _ptr(lse), _dtype_code(q), _stream(stream)))
    return o, lse


def cascade_decode_state(q, k_prefix, v_prefix, prefix_kv_indptr, prefix_req_indptr, k_cache,
                         v_cache, block_table, cache_seqlens, sm_scale, workspace, plan_buf=None,
                         o=None, lse=None, stream=None):
    """cascade_decode returning the unrounded state: O [B, Hq, 128] float32 and
    LSE [B, Hq], for states merged further (KV sharding)."""
    import torch
    B, Hq, D = q.shape
    _check_paged(q, k_cache, v_cache, block_table, cache_seqlens, workspace, None, lse, (q.dtype,))
    _check_prefix(q, k_prefix, v_prefix, _host_i32(prefix_kv_indptr))
    if o is not None:
        _expect("o", o, (torch.float32,), (B, Hq, D), q.device)
    P, ps, Hkv, _ = k_cache.shape
    kv_ptr, req_ptr = _host_i32(prefix_kv_indptr), _host_i32(prefix_req_indptr)
    o = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device) if o is None else o
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(lib().pkc_cascade_decode_state(
        _ptr(q), _ptr(k_prefix), _ptr(v_prefix), _hptr(kv_ptr), _hptr(req_ptr), len(kv_ptr) - 1,
        _ptr(k_cache), _ptr(v_cache), _ptr(block_table), block_table.shape[1], _ptr(cache_seqlens),
        B, Hq, Hkv, D, ps, P, float(sm_scale), _hptr(plan_buf), _ptr(workspace),
        workspace.numel(), _ptr(o), _ptr(lse), _dtype_code(q), _stream(stream)))
    return o, lse


def cascade_decode_multilevel(q, k_prefix, v_prefix, prefix_kv_indptr, prefix_req_ranges, k_cache,
                              v_cache, block_table, cache_seqlens, sm_scale, workspace, plan_buf=None,
                              o=None, lse=None, stream=None):
    """The cascade with prefix groups as request ranges [(begin, end)] that may
    overlap: each request attends to every group's prefix that holds it."""
    import torch
    _check_paged(q, k_cache, v_cache, block_table, cache_seqlens, workspace, o, lse, (q.dtype,))
    _check_prefix(q, k_prefix, v_prefix, _host_i32(prefix_kv_indptr))
    B, Hq, D = q.shape
    P, ps, Hkv, _ = k_cache.shape
    kv_ptr = _host_i32(prefix_kv_indptr)
    rr = _host_i32(prefix_req_ranges).reshape(-1, 2)
    rb, re = np.ascontiguousarray(rr[:, 0]), np.ascontiguousarray(rr[:, 1])
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(lib().pkc_cascade_decode_multilevel(
        _ptr(q), _ptr(k_prefix), _ptr(v_prefix), _hptr(kv_ptr), _hptr(rb), _hptr(re), len(kv_ptr) - 1,
        _ptr(k_cache), _ptr(v_cache), _ptr(block_table), block_table.shape[1], _ptr(cache_seqlens),
        B, Hq, Hkv, D, ps, P, float(sm_scale), _hptr(plan_buf), _ptr(workspace),
        workspace.numel(), _ptr(o), _ptr(lse), _dtype_code(q), _stream(stream)))
    return o, lse


def cascade_decode_paged_prefix(q, prefix_pages, prefix_page_indptr, prefix_kv_indptr,
                                prefix_req_ranges, k_cache, v_cache, block_table, cache_seqlens,
                                sm_scale, workspace, plan_buf=None, o=None, lse=None, stream=None):
    """The multi-level cascade with each group's prefix read in place from the
    page pool: prefix_pages (device int32) lists group j's pages at
    prefix_page_indptr[j] .. prefix_page_indptr[j+1]-1."""
    import torch
    _check_paged(q, k_cache, v_cache, block_table, cache_seqlens, workspace, o, lse, (q.dtype,))
    _expect("prefix_pages", prefix_pages, (torch.int32,), (None,), q.device)
    if len(prefix_page_indptr) and int(_host_i32(prefix_page_indptr)[-1]) > prefix_pages.shape[0]:
        raise ValueError("prefix_page_indptr ends past prefix_pages")
    B, Hq, D = q.shape
    P, ps, Hkv, _ = k_cache.shape
    kv_ptr, pg_ptr = _host_i32(prefix_kv_indptr), _host_i32(prefix_page_indptr)
    rr = _host_i32(prefix_req_ranges).reshape(-1, 2)
    rb, re = np.ascontiguousarray(rr[:, 0]), np.ascontiguousarray(rr[:, 1])
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(lib().pkc_cascade_decode_paged_prefix(
        _ptr(q), _ptr(prefix_pages), _hptr(pg_ptr), _hptr(kv_ptr), _hptr(rb), _hptr(re), len(kv_ptr) - 1,
        _ptr(k_cache), _ptr(v_cache), _ptr(block_table), block_table.shape[1], _ptr(cache_seqlens),
        B, Hq, Hkv, D, ps, P, float(sm_scale), _hptr(plan_buf), _ptr(workspace),
        workspace.numel(), _ptr(o), _ptr(lse), _dtype_code(q), _stream(stream)))
    return o, lse


def selftest_wait_timeout(workspace, stream=None) -> bool:
    """Run the bounded-wait failure path on the GPU (about 2 s): True if the
    wait gave up and returned as designed; the status word then holds
    PKC_ERR_TIMEOUT (read it with device_status)."""
    import torch
    _expect("workspace", workspace, (torch.uint8,), (None,))
    out = ctypes.c_int32(0)
    _check(lib().pkc_selftest_wait_timeout(_ptr(workspace), workspace.numel(), ctypes.byref(out),
                                           _stream(stream)))
    return out.value == 1


def set_stage_events(events):
    """Record 4 torch.cuda.Event objects around the stages of the next
    cascade_decode call on this thread (None clears)."""
    if events is None:
        _check(lib().pkc_set_stage_events(None, 0))
        return
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check(lib().pkc_set_stage_events(arr, len(events)))


def plan_dict(buf):
    """Decode a plan buffer into Python lists (for inspection and tests)."""
    h = {k: int(buf[v]) for k, v in PLAN.items()}
    nc, nw, nu = h["NUM_CTAS"], h["N_WORK"], h["N_UNITS"]

    def arr(off, n):
        return buf[h[off]:h[off] + n].tolist()
    indptr = arr("OFF_CTA_INDPTR", nc + 1)
    cta_work_flat = arr("OFF_CTA_WORK", nw)
    return {
        "header": h,
        "kv_chunk": h["KV_CHUNK"],
        "cta_work": [cta_work_flat[indptr[c]:indptr[c + 1]] for c in range(nc)],
        "work": list(zip(arr("OFF_WORK_UNIT", nw), arr("OFF_WORK_KV_BEGIN", nw),
                         arr("OFF_WORK_KV_END", nw))),
        "partial": arr("OFF_WORK_PARTIAL", nw),
        "unit_req": arr("OFF_UNIT_REQ", nu),
        "unit_qtile": arr("OFF_UNIT_QTILE", nu),
        "unit_kv_len": arr("OFF_UNIT_KV_LEN", nu),
        "unit_n_chunks": arr("OFF_UNIT_N_CHUNKS", nu),
        "unit_partial_begin": arr("OFF_UNIT_PARTIAL_BEGIN", nu),
        "split_units": arr("OFF_UNIT_LIST", h["N_SPLIT"]),
        "empty_units": buf[h["OFF_UNIT_LIST"] + h["N_SPLIT"]:
                           h["OFF_UNIT_LIST"] + h["N_SPLIT"] + h["N_EMPTY"]].tolist(),
        "cta_cost": buf[h["OFF_CTA_COST"]:h["OFF_CTA_COST"] + 2 * nc].view(np.float64).tolist(),
        "n_partials": h["N_PARTIALS"],
        "order": arr("OFF_WORK_ORDER", nw),
        "order_rec": [tuple(buf[h["OFF_ORDER_REC"] + 4 * i:h["OFF_ORDER_REC"] + 4 * i + 4].tolist())
                      for i in range(nw)],
    }
