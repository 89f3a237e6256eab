"""Thin ctypes binding of libfa_gb300.so.

The functions carry the C entry points' names and only marshal arguments
(tensor pointers, sizes, the current CUDA stream); every step of the attention
path runs in the library's kernels.  There is no fallback: if the library is
missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfa_gb300.so")

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_CUDA = 3
FA_ERR_DEVICE_TIMEOUT = 4
FA_ERR_DEVICE_VALUE = 5

FA_CACHE_BF16 = 0
FA_CACHE_E4M3 = 1

# Every symbol include/fa.h declares, with (restype, argtypes).
_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
_F = ctypes.c_float
SIGNATURES = {
    "fa_fwd": (_I, [_P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _P]),
    "fa_bwd_workspace_size": (ctypes.c_size_t, [_I, _I, _I, _I, _I, _I]),
    "fa_fwd_splitkv": (_I, [_P, _P, _P, _P, _P, _I, _P, _P, _I, _P, ctypes.c_size_t,
                            _I, _I, _I, _I, _I, _I, _P]),
    "fa_fwd_splitkv_workspace_size": (ctypes.c_size_t, [_I, _I, _I, _I, _I, _I, _I]),
    "fa_fwd_splitkv_default_splits": (_I, [_I, _I, _I, _I, _I, _I]),
    "fa_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P, ctypes.c_size_t,
                    _I, _I, _I, _I, _I, _I, _P]),
    "fa_bwd_stage": (_I, [_I, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P,
                          ctypes.c_size_t, _I, _I, _I, _I, _I, _I, _P]),
    "fa_bwd_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P,
                            _I, _I, _I, _I, _I, _I, _P]),
    "fa_fwd_masked": (_I, [_P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _P, _P,
                           _I, _I, _I, _I, _I, _I, _P]),
    "fa_bwd_masked": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _P, _P, _P, _P,
                           ctypes.c_size_t, _I, _I, _I, _I, _I, _I, _P]),
    "fa_block_mask_build": (_I, [_P, _I, _I, _I, _P, _P, _P, ctypes.c_int64,
                                 ctypes.POINTER(ctypes.c_int64)]),
    "fa_paged_tables": (_I, [_P, _P, _P, _I, _P, _P, _I, _P, _P, _P, _P, _I, _P, _I, _I, _I, _P]),
    "fa_paged_append": (_I, [_P, _P, _L, _L, _L, _L, _P, _P, _P, _I, _P, _P, _L, _L, _L,
                             _I, _I, _I, _I, _I, _P]),
    "fa_paged_decode": (_I, [_P, _P, _P, _I, _P, _P, _L, _L, _L, _P, _P, _I, _P, _P, _P,
                             ctypes.c_size_t, _I, _I, _I, _I, _I, _I, _I, _I, _P]),
    "fa_paged_decode_workspace_size": (ctypes.c_size_t, [_I, _I, _I, _I, _I]),
    "fa_paged_tables_packed": (_I, [ctypes.c_char_p]),
    "fa_paged_append_packed": (_I, [ctypes.c_char_p]),
    "fa_paged_decode_packed": (_I, [ctypes.c_char_p]),
    "fa_paged_decode_shared": (_I, [_P, _P, _P, _I, _P, _P, _L, _L, _L, _P, _P, _P, _I, _P, _P, _I, _P,
                                    _P, _P, ctypes.c_size_t, _I, _I, _I, _I, _I, _I, _I, _I, _P]),
    "fa_paged_decode_shared_workspace_size": (ctypes.c_size_t, [_I] * 7),
    "fa_rotary": (_I, [_P, _L, _L, _L, _P, _L, _L, _L, _P, _L, _L, _L, _P, _L, _L, _L, _P, _L, _L, _L,
                       _P, _P, _I, _I, _I, _I, _F, _I, _I, _I, _I, _I, _P]),
    "fa_paged_rotary_append": (_I, [_P, _L, _L, _P, _L, _L, _L, _P, _L, _L, _P, _L, _L, _P, _L, _L, _P,
                                    _P, _I, _I, _I, _F, _P, _P, _P, _I, _P, _P, _L, _L, _L, _I, _I, _I,
                                    _I, _I, _I, _I, _P]),
    "fa_paged_free": (_I, [_P, _P, _I, _P, _P, _I, _P, _P, _I, _P, _P, _P, _I, _I, _I, _P]),
    "fa_paged_fork": (_I, [_P, _P, _P, _I, _P, _P, _I, _P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _P]),
    "fa_paged_compact": (_I, [_P, _P, _I, _P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "fa_paged_copy": (_I, [_P, _I, _P, _P, _I, _L, _L, _L, _L, _I, _I, _I, _I, _I, _P]),
    **{f"fa_{n}_packed": (_I, [ctypes.c_char_p]) for n in (
        "paged_decode_shared", "rotary", "paged_rotary_append", "paged_free", "paged_fork", "paged_compact", "paged_copy")},
    "fa_check_status": (_I, [_P]),
    "fa_status_string": (ctypes.c_char_p, [_I]),
    "fa_set_wait_limit_ns": (_I, [ctypes.c_uint64]),
    "fa_set_bwd_kv_rows": (_I, [ctypes.c_int]),
    "fa_set_bwd_q_splits": (_I, [ctypes.c_int]),
    "fa_bwd_plan": (_I, [ctypes.c_int] * 9 + [ctypes.POINTER(ctypes.c_int)] * 2),
    "fa_set_fwd_schedule": (_I, [ctypes.c_int]),
    "fa_selftest_wait_timeout": (_I, [_P]),
    "fa_device_sm_count": (_I, []),
}

_lib = None


class FAError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed: {msg} (status {code})")
        self.code = code


def load(path: str = LIB_PATH):
    """Load the shared library (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load().fa_status_string(code).decode()


def _check(fn: str, code: int):
    if code != FA_OK:
        raise FAError(fn, code, status_string(code))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _need(t: torch.Tensor, dtype, name: str):
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")


# ---------------------------------------------------------------- C names

def fa_fwd(q, k, v, seg_q, seg_kv, causal, o, lse, stream=None, check=True) -> int:
    """Enqueue the forward pass on tensors already in device memory."""
    B, K, G, T, H = q.shape
    S = k.shape[2]
    rc = load().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(seg_q), _ptr(seg_kv), int(bool(causal)),
                       _ptr(o), _ptr(lse), B, K, G, T, S, H, _stream(stream))
    if check:
        _check("fa_fwd", rc)
    return rc


def fa_fwd_splitkv(q, k, v, seg_q, seg_kv, causal, o, lse, n_splits, workspace, stream=None,
                   check=True) -> int:
    B, K, G, T, H = q.shape
    S = k.shape[2]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().fa_fwd_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(seg_q), _ptr(seg_kv),
                               int(bool(causal)), _ptr(o), _ptr(lse), int(n_splits),
                               _ptr(workspace), ws_bytes, B, K, G, T, S, H, _stream(stream))
    if check:
        _check("fa_fwd_splitkv", rc)
    return rc


def fa_fwd_splitkv_workspace_size(B, K, G, T, S, H, n_splits) -> int:
    return int(load().fa_fwd_splitkv_workspace_size(B, K, G, T, S, H, n_splits))


def fa_fwd_splitkv_default_splits(B, K, G, T, S, H) -> int:
    return int(load().fa_fwd_splitkv_default_splits(B, K, G, T, S, H))


def fa_bwd_workspace_size(B, K, G, T, S, H) -> int:
    return int(load().fa_bwd_workspace_size(B, K, G, T, S, H))


def fa_bwd(q, k, v, o, lse, dO, seg_q, seg_kv, causal, dq, dk, dv, workspace,
           stream=None, check=True) -> int:
    B, K, G, T, H = q.shape
    S = k.shape[2]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(seg_q),
                       _ptr(seg_kv), int(bool(causal)), _ptr(dq), _ptr(dk), _ptr(dv),
                       _ptr(workspace), ws_bytes, B, K, G, T, S, H, _stream(stream))
    if check:
        _check("fa_bwd", rc)
    return rc


def fa_bwd_stage(stage, q, k, v, o, lse, dO, seg_q, seg_kv, causal, dq, dk, dv, workspace,
                 stream=None, check=True) -> int:
    B, K, G, T, H = q.shape
    S = k.shape[2]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().fa_bwd_stage(int(stage), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO),
                             _ptr(seg_q), _ptr(seg_kv), int(bool(causal)), _ptr(dq), _ptr(dk),
                             _ptr(dv), _ptr(workspace), ws_bytes, B, K, G, T, S, H,
                             _stream(stream))
    if check:
        _check("fa_bwd_stage", rc)
    return rc


def fa_bwd_noalloc(q, k, v, o, lse, dO, seg_q, seg_kv, causal, dq, dk, dv, stream=None,
                   check=True) -> int:
    """fa_bwd with the library's fixed scratch instead of a caller workspace."""
    B, K, G, T, H = q.shape
    S = k.shape[2]
    rc = load().fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO),
                               _ptr(seg_q), _ptr(seg_kv), int(bool(causal)), _ptr(dq), _ptr(dk),
                               _ptr(dv), B, K, G, T, S, H, _stream(stream))
    if check:
        _check("fa_bwd_noalloc", rc)
    return rc


def fa_check_status(stream=None) -> int:
    return int(load().fa_check_status(_stream(stream)))


def fa_set_wait_limit_ns(ns: int) -> int:
    return int(load().fa_set_wait_limit_ns(int(ns)))


def fa_set_fwd_schedule(mode: int) -> int:
    """Forward grid: 0 chooses, 1 one CTA per Q tile, 2 persistent (H <= 128, no split-KV)."""
    return int(load().fa_set_fwd_schedule(int(mode)))


def fa_set_bwd_kv_rows(rows: int) -> int:
    """Backward KV tile size for H = 128: 0 chooses per call, 64 / 128 force it."""
    return int(load().fa_set_bwd_kv_rows(int(rows)))


def fa_set_bwd_q_splits(n: int) -> int:
    """dK/dV Q-range split on grids smaller than the GPU: 0 chooses per call, 1..4 force it."""
    return int(load().fa_set_bwd_q_splits(int(n)))


def fa_bwd_plan(B, K, G, T, S, H, causal, masked, sm_count):
    """(status, kv_rows, q_splits) the backward would choose with the default knobs."""
    kv, qs = ctypes.c_int(0), ctypes.c_int(0)
    rc = int(load().fa_bwd_plan(B, K, G, T, S, H, int(bool(causal)), int(bool(masked)), sm_count,
                                ctypes.byref(kv), ctypes.byref(qs)))
    return rc, kv.value, qs.value


def fa_selftest_wait_timeout(stream=None) -> int:
    return int(load().fa_selftest_wait_timeout(_stream(stream)))


def fa_device_sm_count() -> int:
    return int(load().fa_device_sm_count())


def fa_block_mask_build(dense, heads, T, S, block_class, partial_index, partial_bits,
                        partial_capacity) -> tuple:
    """Host arrays in, (status, n_partial) out."""
    n = ctypes.c_int64(0)
    ptr = lambda a: None if a is None else ctypes.c_void_p(a.ctypes.data)
    rc = load().fa_block_mask_build(ptr(dense), heads, T, S, ptr(block_class), ptr(partial_index),
                                    ptr(partial_bits), int(partial_capacity), ctypes.byref(n))
    return rc, int(n.value)


def fa_fwd_masked(q, k, v, seg_q, seg_kv, causal, mask, o, lse, stream=None, check=True) -> int:
    """`mask` = (block_class, partial_index, partial_bits, mask_heads), device tensors."""
    B, K, G, T, H = q.shape
    S = k.shape[2]
    cls, idx, bits, heads = mask
    rc = load().fa_fwd_masked(_ptr(q), _ptr(k), _ptr(v), _ptr(seg_q), _ptr(seg_kv),
                              int(bool(causal)), _ptr(cls), _ptr(idx), _ptr(bits), int(heads),
                              _ptr(o), _ptr(lse), B, K, G, T, S, H, _stream(stream))
    if check:
        _check("fa_fwd_masked", rc)
    return rc


def fa_bwd_masked(q, k, v, o, lse, dO, seg_q, seg_kv, causal, mask, dq, dk, dv, workspace,
                  stream=None, check=True) -> int:
    B, K, G, T, H = q.shape
    S = k.shape[2]
    cls, idx, bits, heads = mask
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().fa_bwd_masked(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO),
                              _ptr(seg_q), _ptr(seg_kv), int(bool(causal)), _ptr(cls), _ptr(idx),
                              _ptr(bits), int(heads), _ptr(dq), _ptr(dk), _ptr(dv),
                              _ptr(workspace), ws_bytes, B, K, G, T, S, H, _stream(stream))
    if check:
        _check("fa_bwd_masked", rc)
    return rc


# ----------------------------------------------------- paged cache, C names
#
# The caches are tensors [n_pages, K, page_size, H] (bf16 or float8_e4m3fn) with any
# strides whose innermost is 1; [n_pages, page_size, K, H] memory is passed as its
# transpose(1, 2).  Work goes to the tensors' own device.

# These calls are a few microseconds of GPU work, so their checks are written for
# few Python operations: all in one condition, sizes by numel of contiguous tensors, types
# by identity.  Where it fails, _dense names the tensor that is wrong.

# What torch.cuda's functions call, 2 us cheaper without the objects around it.  A torch without
# CUDA lacks both, and runs the host-only parts of this module all the same.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)
# The packed calls' records: ctypes takes 2 us for two dozen arguments, and a sixth of it here.
_TABLES, _APPEND, _DECODE = (struct.Struct(f"{n}q").pack for n in (17, 21, 25))
_ROTARY, _ROTARY_APPEND, _FREE, _FORK, _COMPACT, _COPY, _SHARED = (
    struct.Struct(f"{n}q").pack for n in (33, 39, 16, 18, 16, 15, 29))
_BF16, _I32, _I64, _F32, _E4M3 = (torch.bfloat16, torch.int32, torch.int64, torch.float32,
                                  torch.float8_e4m3fn)


def _dense(t: torch.Tensor, dtype, n: int, index: int, name: str) -> int:
    """Address of a contiguous tensor of n values of `dtype` on CUDA device `index`."""
    if (t.dtype is not dtype or t.numel() != n or t.get_device() != index
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} values on "
                         f"cuda:{index}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _paged_cache(k_cache, v_cache, k_scale, v_scale, K: int, H: int, index: int):
    """(cache type, shape, strides, k_scale and v_scale addresses) of a checked cache pair."""
    shape, stride, dtype = k_cache.shape, k_cache.stride(), k_cache.dtype
    if len(shape) != 4 or shape[1] != K or shape[3] != H or v_cache.shape != shape:
        raise ValueError(f"k_cache and v_cache must be [n_pages, {K}, page_size, {H}], "
                         f"got {tuple(shape)} and {tuple(v_cache.shape)}")
    # (of dims of one, no stride is used)
    if (stride[3] != 1 or v_cache.stride() != stride) and k_cache.numel() and any(
            n > 1 and (x != y or i == 3 and x != 1)
            for i, (n, x, y) in enumerate(zip(shape, stride, v_cache.stride()))):
        raise ValueError("k_cache and v_cache must have the same strides, innermost 1")
    if k_cache.get_device() != index or v_cache.get_device() != index or index < 0:
        raise ValueError("k_cache and v_cache must be on the CUDA device of the other tensors")
    if v_cache.dtype is not dtype:
        raise ValueError("k_cache and v_cache must have one type")
    if dtype is _BF16:
        if k_scale is not None or v_scale is not None:
            raise ValueError("a bfloat16 cache takes no scales")
        return FA_CACHE_BF16, shape, stride, 0, 0
    if dtype is not _E4M3:
        raise ValueError(f"the cache must be bfloat16 or float8_e4m3fn, got {dtype}")
    return (FA_CACHE_E4M3, shape, stride,
            0 if k_scale is None else _dense(k_scale, _F32, K, index, "k_scale"),
            0 if v_scale is None else _dense(v_scale, _F32, K, index, "v_scale"))


def _raw_stream(stream) -> int:
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def fa_paged_tables(cached_lens, new_lens, free_pages, free_used, block_table, total_lens,
                    token_starts, slots, positions, free_used_out, n_pages, page_size,
                    stream=None, check=True) -> int:
    """Pages and slots of a step's new tokens (see fa.h).  total_lens may be cached_lens and
    free_used_out may be free_used; positions may be None."""
    dev = cached_lens.get_device()
    if dev < 0:
        raise ValueError("cached_lens must be a CUDA tensor")
    if dev != _current_device():
        with torch.cuda.device(dev):
            return fa_paged_tables(cached_lens, new_lens, free_pages, free_used, block_table,
                                   total_lens, token_starts, slots, positions, free_used_out,
                                   n_pages, page_size, stream, check)
    B, tokens, n_free = cached_lens.numel(), slots.numel(), free_pages.numel()
    rows, max_pages = block_table.shape
    if rows != B:
        raise ValueError(f"block_table must have {B} rows, got {rows}")
    if not (_I32 is cached_lens.dtype is new_lens.dtype is free_pages.dtype is free_used.dtype
            is block_table.dtype is total_lens.dtype is token_starts.dtype is free_used_out.dtype
            and slots.dtype is _I64
            and dev == new_lens.get_device() == free_pages.get_device() == free_used.get_device()
            == block_table.get_device() == total_lens.get_device() == token_starts.get_device()
            == slots.get_device() == free_used_out.get_device()
            and B == new_lens.numel() == total_lens.numel() == token_starts.numel() - 1
            and 1 == free_used.numel() == free_used_out.numel()
            and cached_lens.is_contiguous() and new_lens.is_contiguous()
            and free_pages.is_contiguous() and block_table.is_contiguous()
            and total_lens.is_contiguous() and token_starts.is_contiguous()
            and slots.is_contiguous()):
        for t, dtype, n, name in (
                (cached_lens, _I32, B, "cached_lens"), (new_lens, _I32, B, "new_lens"),
                (free_pages, _I32, n_free, "free_pages"), (free_used, _I32, 1, "free_used"),
                (block_table, _I32, B * max_pages, "block_table"),
                (total_lens, _I32, B, "total_lens"),
                (token_starts, _I32, B + 1, "token_starts"), (slots, _I64, tokens, "slots"),
                (free_used_out, _I32, 1, "free_used_out")):
            _dense(t, dtype, n, dev, name)
    rc = (_lib or load()).fa_paged_tables_packed(_TABLES(
        cached_lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(), n_free,
        free_used.data_ptr(), block_table.data_ptr(), max_pages, total_lens.data_ptr(),
        token_starts.data_ptr(), slots.data_ptr(),
        0 if positions is None else _dense(positions, _I32, tokens, dev, "positions"), tokens,
        free_used_out.data_ptr(), B, n_pages, page_size,
        _current_stream(dev) if stream is None else _raw_stream(stream)))
    if rc and check:
        _check("fa_paged_tables", rc)
    return rc


def fa_paged_append(k, v, slots, k_cache, v_cache, k_scale=None, v_scale=None, stream=None,
                    check=True) -> int:
    """Write k, v [N, K, H] (bf16, any token and head strides) into the pages of `slots`."""
    dev = k.get_device()
    if dev >= 0 and dev != _current_device():
        with torch.cuda.device(dev):
            return fa_paged_append(k, v, slots, k_cache, v_cache, k_scale, v_scale, stream, check)
    N, K, H = shape = k.shape
    sk, sv = k.stride(), v.stride()
    if (k.dtype is not _BF16 or v.dtype is not _BF16 or v.shape != shape or v.get_device() != dev
            or ((sk[2] != 1 or sv[2] != 1) and k.numel())):
        raise ValueError("k and v must be bfloat16 tensors of one shape [N, K, H] on one device, "
                         "innermost stride 1")
    kind, cs, st, ks, vs = _paged_cache(k_cache, v_cache, k_scale, v_scale, K, H, dev)
    rc = (_lib or load()).fa_paged_append_packed(_APPEND(
        k.data_ptr(), v.data_ptr(), sk[0], sk[1], sv[0], sv[1],
        _dense(slots, _I64, N, dev, "slots"), k_cache.data_ptr(), v_cache.data_ptr(), kind, ks, vs,
        st[0], st[1], st[2], N, K, H, cs[0], cs[2],
        _current_stream(dev) if stream is None else _raw_stream(stream)))
    if rc and check:
        _check("fa_paged_append", rc)
    return rc


def fa_paged_decode(q, k_cache, v_cache, block_table, lens, o, lse, workspace, k_scale=None,
                    v_scale=None, window=0, stream=None, check=True) -> int:
    """Attention of q [B, K, G, T, H], each request's T newest tokens, over its pages."""
    dev = q.get_device()
    if dev >= 0 and dev != _current_device():
        with torch.cuda.device(dev):
            return fa_paged_decode(q, k_cache, v_cache, block_table, lens, o, lse, workspace,
                                   k_scale, v_scale, window, stream, check)
    B, K, G, T, H = q.shape
    rows = B * K * G * T
    kind, cs, st, ks, vs = _paged_cache(k_cache, v_cache, k_scale, v_scale, K, H, dev)
    requests, max_pages = block_table.shape
    if requests != B:
        raise ValueError(f"block_table must have {B} rows, got {requests}")
    ws = ws_bytes = 0
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
        ws, ws_bytes = workspace.data_ptr(), workspace.nbytes
    if not (_BF16 is q.dtype is o.dtype and _I32 is block_table.dtype is lens.dtype
            and lse.dtype is _F32
            and dev == o.get_device() == lse.get_device() == block_table.get_device()
            == lens.get_device()
            and rows * H == o.numel() and rows == lse.numel() and B == lens.numel()
            and q.is_contiguous() and o.is_contiguous() and lse.is_contiguous()
            and block_table.is_contiguous() and lens.is_contiguous()):
        for t, dtype, n, name in (
                (q, _BF16, rows * H, "q"), (block_table, _I32, B * max_pages, "block_table"),
                (lens, _I32, B, "lens"), (o, _BF16, rows * H, "o"), (lse, _F32, rows, "lse")):
            _dense(t, dtype, n, dev, name)
    rc = (_lib or load()).fa_paged_decode_packed(_DECODE(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), kind, ks, vs, st[0], st[1], st[2],
        block_table.data_ptr(), lens.data_ptr(), window, o.data_ptr(), lse.data_ptr(), ws, ws_bytes,
        B, K, G, T, H, cs[0], cs[2], max_pages,
        _current_stream(dev) if stream is None else _raw_stream(stream)))
    if rc and check:
        _check("fa_paged_decode", rc)
    return rc


def fa_paged_decode_workspace_size(B, K, G, T, H) -> int:
    return int(load().fa_paged_decode_workspace_size(B, K, G, T, H))


def fa_paged_decode_shared(q, k_cache, v_cache, block_table, lens, members, group_starts, prefix_lens, o,
                           lse, workspace, k_scale=None, v_scale=None, stream=None, check=True) -> int:
    """fa_paged_decode of requests that share prefixes: group g is the requests
    members[group_starts[g]:group_starts[g + 1]], their first prefix_lens[g] tokens the same."""
    dev = q.get_device()
    if dev >= 0 and dev != _current_device():
        with torch.cuda.device(dev):
            return fa_paged_decode_shared(q, k_cache, v_cache, block_table, lens, members, group_starts,
                                          prefix_lens, o, lse, workspace, k_scale, v_scale, stream, check)
    B, K, G, T, H = q.shape
    rows, n_groups, n_members = B * K * G * T, prefix_lens.numel(), members.numel()
    kind, cs, st, ks, vs = _paged_cache(k_cache, v_cache, k_scale, v_scale, K, H, dev)
    requests, max_pages = block_table.shape
    if requests != B:
        raise ValueError(f"block_table must have {B} rows, got {requests}")
    ws = ws_bytes = 0
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
        ws, ws_bytes = workspace.data_ptr(), workspace.nbytes
    if not (_BF16 is q.dtype is o.dtype and lse.dtype is _F32
            and _I32 is block_table.dtype is lens.dtype is members.dtype is group_starts.dtype
            is prefix_lens.dtype
            and dev == o.get_device() == lse.get_device() == block_table.get_device()
            == lens.get_device() == members.get_device() == group_starts.get_device()
            == prefix_lens.get_device()
            and rows * H == o.numel() and rows == lse.numel() and B == lens.numel()
            and n_groups + 1 == group_starts.numel()
            and q.is_contiguous() and o.is_contiguous() and lse.is_contiguous()
            and block_table.is_contiguous() and lens.is_contiguous() and members.is_contiguous()
            and group_starts.is_contiguous() and prefix_lens.is_contiguous()):
        for t, dtype, n, name in (
                (q, _BF16, rows * H, "q"), (block_table, _I32, B * max_pages, "block_table"),
                (lens, _I32, B, "lens"), (members, _I32, n_members, "members"),
                (group_starts, _I32, n_groups + 1, "group_starts"),
                (prefix_lens, _I32, n_groups, "prefix_lens"), (o, _BF16, rows * H, "o"),
                (lse, _F32, rows, "lse")):
            _dense(t, dtype, n, dev, name)
    rc = (_lib or load()).fa_paged_decode_shared_packed(_SHARED(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), kind, ks, vs, st[0], st[1], st[2],
        block_table.data_ptr(), lens.data_ptr(), members.data_ptr(), n_members, group_starts.data_ptr(),
        prefix_lens.data_ptr(), n_groups, o.data_ptr(), lse.data_ptr(), ws, ws_bytes, B, K, G, T, H,
        cs[0], cs[2], max_pages, _current_stream(dev) if stream is None else _raw_stream(stream)))
    if rc and check:
        _check("fa_paged_decode_shared", rc)
    return rc


def fa_paged_decode_shared_workspace_size(B, K, G, T, H, n_groups, n_members) -> int:
    return int(load().fa_paged_decode_shared_workspace_size(B, K, G, T, H, n_groups, n_members))


# ------------------------------------------- rotary positions, pages: C names

def _float_bits(x: float) -> int:
    return struct.unpack("i", struct.pack("f", x))[0]


def _turning(positions, inv_freq, axes, tokens: tuple, dev: int):
    """(positions' strides, number of axes, pairs, axes' address) of checked positions [n_axes, *tokens]
    or, of one axis, [*tokens]."""
    shape, st = positions.shape, positions.stride()
    n_axes = 1
    if len(shape) == len(tokens):
        st = (0, *st)
    elif len(shape) == len(tokens) + 1:
        n_axes, shape = shape[0], shape[1:]
    if shape != tokens or positions.dtype is not _I32 or positions.get_device() != dev:
        raise ValueError(f"positions must be an int32 tensor {list(tokens)}, or the axes before them, on "
                         f"cuda:{dev}, got {positions.dtype} {tuple(positions.shape)}")
    pairs = inv_freq.numel()
    _dense(inv_freq, _F32, pairs, dev, "inv_freq")
    return st, n_axes, pairs, 0 if axes is None else _dense(axes, _I32, pairs, dev, "axes")


def _pair_rows(x, out, dev: int, name: str):
    """Checks bfloat16 tensors of one shape on the device, innermost stride 1; returns their strides."""
    sx, so = x.stride(), out.stride()
    if (x.dtype is not _BF16 or out.dtype is not _BF16 or x.shape != out.shape or len(sx) != 4
            or x.get_device() != dev or out.get_device() != dev
            or ((sx[3] != 1 or so[3] != 1) and x.numel())):
        raise ValueError(f"{name} and {name}_out must be bfloat16 tensors of one shape [B, T, heads, H] on "
                         f"cuda:{dev}, innermost stride 1")
    return sx, so


def fa_rotary(q, q_out, k, k_out, positions, inv_freq, axes=None, *, q_scale=1.0, adjacent=False,
              inverse=False, stream=None, check=True) -> int:
    """Turn q [B, T, heads, H] and k (or None) by positions [n_axes, B, T] or [B, T] into q_out and
    k_out, any strides (see fa.h).  q_out may be q, and k_out k."""
    dev = q.get_device()
    if dev < 0:
        raise ValueError("q must be a CUDA tensor")
    if dev != _current_device():
        with torch.cuda.device(dev):
            return fa_rotary(q, q_out, k, k_out, positions, inv_freq, axes, q_scale=q_scale,
                             adjacent=adjacent, inverse=inverse, stream=stream, check=check)
    sq, sqo = _pair_rows(q, q_out, dev, "q")
    B, T, heads, H = q.shape
    if k is None:
        kp = kop = kh = 0
        sk = sko = (0, 0, 0)
    else:
        sk, sko = _pair_rows(k, k_out, dev, "k")
        if k.shape[0] != B or k.shape[1] != T or k.shape[3] != H:
            raise ValueError(f"k must be [{B}, {T}, heads, {H}], got {tuple(k.shape)}")
        kp, kop, kh = k.data_ptr(), k_out.data_ptr(), k.shape[2]
    sp, n_axes, pairs, ax = _turning(positions, inv_freq, axes, (B, T), dev)
    rc = (_lib or load()).fa_rotary_packed(_ROTARY(
        q.data_ptr(), sq[0], sq[1], sq[2], q_out.data_ptr(), sqo[0], sqo[1], sqo[2],
        kp, sk[0], sk[1], sk[2], kop, sko[0], sko[1], sko[2],
        positions.data_ptr(), sp[0], sp[1], sp[2], inv_freq.data_ptr(), ax, pairs, n_axes,
        1 if adjacent else 0, 1 if inverse else 0, _float_bits(q_scale), B, T, heads, kh, H,
        _current_stream(dev) if stream is None else _raw_stream(stream)))
    if rc and check:
        _check("fa_rotary", rc)
    return rc


def fa_paged_rotary_append(q, k, v, positions, inv_freq, slots, q_out, k_cache, v_cache, axes=None,
                           k_scale=None, v_scale=None, *, q_scale=1.0, adjacent=False, stream=None,
                           check=True) -> int:
    """Turn q [N, heads, H] into q_out, [B, K, G, T, H] with B * T = N or [N, heads, H], and write the
    turned k and v [N, K, H] into the pages of `slots`.  positions [n_axes, N] or [N]."""
    dev = q.get_device()
    if dev < 0:
        raise ValueError("q must be a CUDA tensor")
    if dev != _current_device():
        with torch.cuda.device(dev):
            return fa_paged_rotary_append(q, k, v, positions, inv_freq, slots, q_out, k_cache, v_cache,
                                          axes, k_scale, v_scale, q_scale=q_scale, adjacent=adjacent,
                                          stream=stream, check=check)
    N, heads, H = shape = q.shape
    kv, out = k.shape, q_out.shape
    sq, sk, sv, so = q.stride(), k.stride(), v.stride(), q_out.stride()
    if (not _BF16 is q.dtype is k.dtype is v.dtype is q_out.dtype or kv != v.shape
            or len(kv) != 3 or kv[0] != N or kv[2] != H
            or not dev == k.get_device() == v.get_device() == q_out.get_device()
            or (sk[2] != 1 or sv[2] != 1) and k.numel()
            or (sq[2] != 1 or so[-1] != 1) and q.numel()):
        raise ValueError("q, k and v must be bfloat16 tensors [N, heads, H] (k and v of one shape) and "
                         "q_out one on their device, innermost stride 1")
    K = kv[1]
    if len(out) == 5:
        B, Kq, G, T, Ho = out
        if B * T != N or Kq * G != heads or Ho != H or (Kq > 1 and G > 1 and so[1] != G * so[2]):
            raise ValueError(f"q_out must be [B, K, G, T, {H}] with B * T = {N} and K * G = {heads}, one "
                             f"stride for all heads, got {tuple(out)}")
        ob, ot, oh = so[0], so[3], so[2] if G > 1 else so[1]
    else:
        if out != shape:
            raise ValueError(f"q_out must be [B, K, G, T, {H}] or {tuple(shape)}, got {tuple(out)}")
        B, T, (ob, ot, oh) = 1, N, (0, so[0], so[1])
    sp, n_axes, pairs, ax = _turning(positions, inv_freq, axes, (N,), dev)
    kind, cs, st, ks, vs = _paged_cache(k_cache, v_cache, k_scale, v_scale, K, H, dev)
    rc = (_lib or load()).fa_paged_rotary_append_packed(_ROTARY_APPEND(
        q.data_ptr(), sq[0], sq[1], q_out.data_ptr(), ob, ot, oh, k.data_ptr(), sk[0], sk[1],
        v.data_ptr(), sv[0], sv[1], positions.data_ptr(), sp[0], sp[1], inv_freq.data_ptr(), ax, pairs,
        n_axes, 1 if adjacent else 0, _float_bits(q_scale), _dense(slots, _I64, N, dev, "slots"),
        k_cache.data_ptr(), v_cache.data_ptr(), kind, ks, vs, st[0], st[1], st[2], B, T, heads, K, H,
        cs[0], cs[2], _current_stream(dev) if stream is None else _raw_stream(stream)))
    if rc and check:
        _check("fa_paged_rotary_append", rc)
    return rc


def _pool(lens, block_table, shares, free_pages, free_used, lens_out, free_used_out):
    """(device, B, max_pages, n_pages, n_free) of the checked tensors of a pool."""
    dev = lens.get_device()
    if dev < 0:
        raise ValueError("lens must be a CUDA tensor")
    B, n_pages, n_free = lens.numel(), shares.numel(), free_pages.numel()
    table = block_table.shape
    if len(table) != 2 or table[0] != B:
        raise ValueError(f"block_table must have {B} rows, got {tuple(table)}")
    max_pages = table[1]
    if not (_I32 is lens.dtype is block_table.dtype is shares.dtype is free_pages.dtype is free_used.dtype
            and dev == block_table.get_device() == shares.get_device() == free_pages.get_device()
            == free_used.get_device() and 1 == free_used.numel()
            and lens.is_contiguous() and block_table.is_contiguous() and shares.is_contiguous()
            and free_pages.is_contiguous()
            and (lens_out is lens or _I32 is lens_out.dtype and dev == lens_out.get_device()
                 and B == lens_out.numel() and lens_out.is_contiguous())
            and (free_used_out is free_used or _I32 is free_used_out.dtype
                 and dev == free_used_out.get_device() and 1 == free_used_out.numel())):
        for t, n, name in ((lens, B, "lens"), (block_table, B * max_pages, "block_table"),
                           (shares, n_pages, "shares"), (free_pages, n_free, "free_pages"),
                           (free_used, 1, "free_used"), (lens_out, B, "lens_out"),
                           (free_used_out, 1, "free_used_out")):
            _dense(t, _I32, n, dev, name)
    return dev, B, max_pages, n_pages, n_free


def fa_paged_free(rows, lens, block_table, shares, free_pages, free_used, lens_out, free_used_out,
                  page_size, keep=None, stream=None, check=True) -> int:
    """Requests rows keep their first `keep` tokens (None: none) and give their other pages back
    (see fa.h).  lens_out may be lens and free_used_out may be free_used."""
    dev, B, max_pages, n_pages, n_free = _pool(lens, block_table, shares, free_pages, free_used, lens_out,
                                               free_used_out)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return fa_paged_free(rows, lens, block_table, shares, free_pages, free_used, lens_out,
                                 free_used_out, page_size, keep, stream, check)
    N = rows.numel()
    rc = (_lib or load()).fa_paged_free_packed(_FREE(
        _dense(rows, _I32, N, dev, "rows"), 0 if keep is None else _dense(keep, _I32, N, dev, "keep"), N,
        lens.data_ptr(), block_table.data_ptr(), max_pages, shares.data_ptr(), free_pages.data_ptr(),
        n_free, free_used.data_ptr(), lens_out.data_ptr(), free_used_out.data_ptr(), B, n_pages, page_size,
        _current_stream(dev) if stream is None else _raw_stream(stream)))
    if rc and check:
        _check("fa_paged_free", rc)
    return rc


def fa_paged_fork(parents, children, lens, block_table, shares, free_pages, free_used, lens_out, copies,
                  free_used_out, page_size, fork_lens=None, stream=None, check=True) -> int:
    """Requests children go on with the first fork_lens tokens (None: all) of parents, whose full pages
    they share; copies [N, 3] is for fa_paged_copy (see fa.h)."""
    dev, B, max_pages, n_pages, n_free = _pool(lens, block_table, shares, free_pages, free_used, lens_out,
                                               free_used_out)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return fa_paged_fork(parents, children, lens, block_table, shares, free_pages, free_used,
                                 lens_out, copies, free_used_out, page_size, fork_lens, stream, check)
    N = parents.numel()
    rc = (_lib or load()).fa_paged_fork_packed(_FORK(
        _dense(parents, _I32, N, dev, "parents"), _dense(children, _I32, N, dev, "children"),
        0 if fork_lens is None else _dense(fork_lens, _I32, N, dev, "fork_lens"), N, lens.data_ptr(),
        block_table.data_ptr(), max_pages, shares.data_ptr(), free_pages.data_ptr(), n_free,
        free_used.data_ptr(), lens_out.data_ptr(), _dense(copies, _I32, 3 * N, dev, "copies"),
        free_used_out.data_ptr(), B, n_pages, page_size,
        _current_stream(dev) if stream is None else _raw_stream(stream)))
    if rc and check:
        _check("fa_paged_fork", rc)
    return rc


def fa_paged_compact(lens, block_table, shares, free_pages, free_used, block_table_out, shares_out,
                     free_pages_out, moves, page_size, stream=None, check=True) -> int:
    """Tables, share counts and free list of the pool made dense by at most len(moves) moves, which
    fa_paged_copy carries out (see fa.h).  The first three outputs may be their inputs."""
    dev, B, max_pages, n_pages, n_free = _pool(lens, block_table, shares, free_pages, free_used, lens, free_used)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return fa_paged_compact(lens, block_table, shares, free_pages, free_used, block_table_out,
                                    shares_out, free_pages_out, moves, page_size, stream, check)
    n = moves.numel() // 3
    rc = (_lib or load()).fa_paged_compact_packed(_COMPACT(
        lens.data_ptr(), block_table.data_ptr(), max_pages, shares.data_ptr(), free_pages.data_ptr(),
        n_free, free_used.data_ptr(), _dense(block_table_out, _I32, B * max_pages, dev, "block_table_out"),
        _dense(shares_out, _I32, n_pages, dev, "shares_out"),
        _dense(free_pages_out, _I32, n_free, dev, "free_pages_out"), _dense(moves, _I32, 3 * n, dev, "moves"),
        n, B, n_pages, page_size, _current_stream(dev) if stream is None else _raw_stream(stream)))
    if rc and check:
        _check("fa_paged_compact", rc)
    return rc


def fa_paged_copy(moves, k_cache, v_cache, stream=None, check=True) -> int:
    """Carry out moves [N, 3] (page, page, tokens) in caches [n_pages, K, page_size, H], or of several
    layers [layers, n_pages, K, page_size, H]."""
    dev = moves.get_device()
    if dev < 0:
        raise ValueError("moves must be a CUDA tensor")
    if dev != _current_device():
        with torch.cuda.device(dev):
            return fa_paged_copy(moves, k_cache, v_cache, stream, check)
    shape, st, dtype = k_cache.shape, k_cache.stride(), k_cache.dtype
    if len(shape) == 4:
        shape, st = (1, *shape), (0, *st)
    elif len(shape) != 5:
        raise ValueError(f"k_cache must have 4 or 5 dims, got {tuple(k_cache.shape)}")
    if (v_cache.shape != k_cache.shape or v_cache.dtype is not dtype or k_cache.get_device() != dev
            or v_cache.get_device() != dev):
        raise ValueError("k_cache and v_cache must have one type and shape, on the moves' device")
    sv = v_cache.stride()
    # (of dims of one, no stride is used)
    if (st[4] != 1 or sv != st[-len(sv):]) and k_cache.numel() and any(
            n > 1 and (x != y or i == 4 and x != 1)
            for i, (n, x, y) in enumerate(zip(shape, st, (0, *sv)[-5:]))):
        raise ValueError("k_cache and v_cache must have the same strides, innermost 1")
    if dtype is not _BF16 and dtype is not _E4M3:
        raise ValueError(f"the cache must be bfloat16 or float8_e4m3fn, got {dtype}")
    N = moves.numel() // 3
    rc = (_lib or load()).fa_paged_copy_packed(_COPY(
        _dense(moves, _I32, 3 * N, dev, "moves"), N, k_cache.data_ptr(), v_cache.data_ptr(),
        FA_CACHE_BF16 if dtype is _BF16 else FA_CACHE_E4M3, st[0], st[1], st[2], st[3], shape[0], shape[2],
        shape[4], shape[1], shape[3], _current_stream(dev) if stream is None else _raw_stream(stream)))
    if rc and check:
        _check("fa_paged_copy", rc)
    return rc


# ------------------------------------------------------- tensor helpers

def block_mask_from_dense(mask, device=None):
    """Dense boolean mask [heads, T, S] -> (block_class, partial_index,
    partial_bits, heads) built by fa_block_mask_build, as tensors on `device`."""
    import numpy as np
    dense = np.ascontiguousarray(np.asarray(mask, dtype=np.uint8))
    heads, T, S = dense.shape
    nqb, nkb = (T + 127) // 128, (S + 127) // 128
    cls = np.zeros((heads, nqb, nkb), dtype=np.uint8)
    idx = np.zeros((heads, nqb, nkb), dtype=np.int32)
    rc, n = fa_block_mask_build(dense, heads, T, S, cls, idx, None, 0)
    _check("fa_block_mask_build", rc)
    bits = np.zeros((max(n, 1), 128, 4), dtype=np.uint32)
    rc, n2 = fa_block_mask_build(dense, heads, T, S, cls, idx, bits, n)
    _check("fa_block_mask_build", rc)
    out = [torch.from_numpy(cls), torch.from_numpy(idx), torch.from_numpy(bits.view(np.int32))]
    if device is not None:
        out = [t.to(device) for t in out]
    return out[0], out[1], out[2], heads

def attention_forward(q, k, v, *, causal=False, seg_q=None, seg_kv=None, stream=None):
    """Allocate o / lse with torch and run fa_fwd.  Returns (o, lse)."""
    _need(q, torch.bfloat16, "q"); _need(k, torch.bfloat16, "k"); _need(v, torch.bfloat16, "v")
    B, K, G, T, H = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((B, K, G, T), dtype=torch.float32, device=q.device)
    fa_fwd(q, k, v, seg_q, seg_kv, causal, o, lse, stream)
    return o, lse


def attention_forward_splitkv(q, k, v, *, causal=False, seg_q=None, seg_kv=None, n_splits=None,
                              stream=None):
    """fa_fwd_splitkv with torch-allocated outputs and workspace."""
    B, K, G, T, H = q.shape
    S = k.shape[2]
    if n_splits is None:
        n_splits = fa_fwd_splitkv_default_splits(B, K, G, T, S, H)
    o = torch.empty_like(q)
    lse = torch.empty((B, K, G, T), dtype=torch.float32, device=q.device)
    n = fa_fwd_splitkv_workspace_size(B, K, G, T, S, H, n_splits)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
    fa_fwd_splitkv(q, k, v, seg_q, seg_kv, causal, o, lse, n_splits, ws, stream)
    return o, lse


def attention_backward(q, k, v, o, lse, dO, *, causal=False, seg_q=None, seg_kv=None,
                       stream=None, workspace=None):
    """Allocate dq / dk / dv (and the workspace unless given) and run fa_bwd."""
    B, K, G, T, H = q.shape
    S = k.shape[2]
    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dv = torch.empty_like(v)
    if workspace is None:
        n = fa_bwd_workspace_size(B, K, G, T, S, H)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
    fa_bwd(q, k, v, o, lse, dO, seg_q, seg_kv, causal, dq, dk, dv, workspace, stream)
    return dq, dk, dv


def _allocating_on(stream, device):
    """Scope in which torch allocates from the memory of `stream` (None: the current one): memory of
    another stream could be given out again before this one's work is over."""
    if stream is None:
        return torch.cuda.device(device)
    if not hasattr(stream, "cuda_stream"):
        stream = (torch.cuda.ExternalStream(int(stream), device=device) if stream
                  else torch.cuda.default_stream(device))
    return torch.cuda.stream(stream)


def paged_tables(cached_lens, new_lens, free_pages, free_used, block_table, *, n_pages, page_size,
                 max_tokens, stream=None):
    """Allocate a step's outputs with torch and run fa_paged_tables, which also writes the
    newly opened pages into block_table.  Returns (total_lens, token_starts, slots, positions,
    free_used) tensors, the last for the next step."""
    new = lambda n, dtype=torch.int32: torch.empty(n, dtype=dtype, device=cached_lens.device)
    B = cached_lens.shape[0]
    with _allocating_on(stream, cached_lens.device):
        total, starts, used = new(B), new(B + 1), new(1)
        slots, positions = new(max_tokens, torch.int64), new(max_tokens)
    fa_paged_tables(cached_lens, new_lens, free_pages, free_used, block_table, total, starts, slots,
                    positions, used, n_pages, page_size, stream)
    return total, starts, slots, positions, used


def paged_attention_decode(q, k_cache, v_cache, block_table, lens, *, k_scale=None, v_scale=None,
                           window=0, stream=None, workspace=None):
    """Allocate o / lse (and the workspace unless given) and run fa_paged_decode."""
    B, K, G, T, H = q.shape
    with _allocating_on(stream, q.device):
        o = torch.empty_like(q)
        lse = torch.empty((B, K, G, T), dtype=torch.float32, device=q.device)
        if workspace is None:
            n = fa_paged_decode_workspace_size(B, K, G, T, H)
            workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
    fa_paged_decode(q, k_cache, v_cache, block_table, lens, o, lse, workspace, k_scale, v_scale,
                    window, stream)
    return o, lse


def paged_attention_decode_shared(q, k_cache, v_cache, block_table, lens, members, group_starts,
                                  prefix_lens, *, k_scale=None, v_scale=None, stream=None,
                                  workspace=None):
    """Allocate o / lse (and the workspace unless given) and run fa_paged_decode_shared."""
    B, K, G, T, H = q.shape
    with _allocating_on(stream, q.device):
        o = torch.empty_like(q)
        lse = torch.empty((B, K, G, T), dtype=torch.float32, device=q.device)
        if workspace is None:
            n = fa_paged_decode_shared_workspace_size(B, K, G, T, H, prefix_lens.numel(), members.numel())
            workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
    fa_paged_decode_shared(q, k_cache, v_cache, block_table, lens, members, group_starts, prefix_lens, o, lse,
                           workspace, k_scale, v_scale, stream)
    return o, lse


def _rotary_pair(q, k, positions, inv_freq, axes, adjacent, q_scale, inverse, stream):
    """Shared by the two helpers below: outputs laid out the other way round."""
    def laid(x):
        B, T, heads, H = x.shape
        if inverse:
            return torch.empty((B, T, heads, H), dtype=x.dtype, device=x.device)
        return torch.empty((B, heads, T, H), dtype=x.dtype, device=x.device).transpose(1, 2)

    with _allocating_on(stream, q.device):
        q_out, k_out = laid(q), None if k is None else laid(k)
    fa_rotary(q, q_out, k, k_out, positions, inv_freq, axes, q_scale=q_scale, adjacent=adjacent,
              inverse=inverse, stream=stream)
    return q_out, k_out


def rotary_forward(q, k, positions, inv_freq, axes=None, *, q_scale=None, adjacent=False, stream=None):
    """Turn a projection's q [B, T, K * G, H] and k [B, T, K, H] and lay them out for the attention:
    returns q [B, K, G, T, H], multiplied by q_scale (None: H**-0.5), and k [B, K, T, H]."""
    B, T, heads, H = q.shape
    K = k.shape[2]
    if K == 0 or heads % K:
        raise ValueError(f"q's heads must be a multiple of k's, got {heads} and {K}")
    q, k = _rotary_pair(q, k, positions, inv_freq, axes, adjacent,
                        H ** -0.5 if q_scale is None else q_scale, False, stream)
    return q.transpose(1, 2).unflatten(1, (K, heads // K)), k.transpose(1, 2)


def rotary_backward(dq, dk, positions, inv_freq, axes=None, *, q_scale=None, adjacent=False, stream=None):
    """Gradients of rotary_forward's q [B, T, K * G, H] and k [B, T, K, H] from the attention's dq
    [B, K, G, T, H] and dk [B, K, T, H] (contiguous, as attention_backward gives them)."""
    _need(dq, torch.bfloat16, "dq"); _need(dk, torch.bfloat16, "dk")
    H = dq.shape[-1]
    return _rotary_pair(dq.flatten(1, 2).transpose(1, 2), dk.transpose(1, 2), positions, inv_freq, axes,
                        adjacent, H ** -0.5 if q_scale is None else q_scale, True, stream)


def paged_free(rows, lens, block_table, shares, free_pages, free_used, *, page_size, keep=None, stream=None):
    """Run fa_paged_free in place: lens, shares, free_pages and free_used are updated."""
    fa_paged_free(rows, lens, block_table, shares, free_pages, free_used, lens, free_used, page_size, keep,
                  stream)


def paged_fork(parents, children, lens, block_table, shares, free_pages, free_used, *, page_size,
               fork_lens=None, stream=None):
    """Run fa_paged_fork in place: lens, block_table, shares and free_used are updated.  Returns the
    copies [N, 3] that fa_paged_copy has to carry out."""
    with _allocating_on(stream, lens.device):
        copies = torch.empty((parents.numel(), 3), dtype=torch.int32, device=lens.device)
    fa_paged_fork(parents, children, lens, block_table, shares, free_pages, free_used, lens, copies, free_used,
                  page_size, fork_lens, stream)
    return copies


def paged_compact(lens, block_table, shares, free_pages, free_used, *, page_size, max_moves, stream=None):
    """Run fa_paged_compact in place: block_table, shares and free_pages are updated.  Returns the
    moves [max_moves, 3] that fa_paged_copy has to carry out."""
    with _allocating_on(stream, lens.device):
        moves = torch.empty((max_moves, 3), dtype=torch.int32, device=lens.device)
    fa_paged_compact(lens, block_table, shares, free_pages, free_used, block_table, shares, free_pages, moves,
                     page_size, stream)
    return moves
