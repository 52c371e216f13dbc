"""ctypes binding of libattn.so (the C ABI in include/attn.h).

Argument marshalling only: every step of the computation runs in the CUDA
library.  PyTorch owns the device memory and the stream; tensors are passed by
``data_ptr()`` and the current stream by handle.  If the compiled library is
missing this module raises immediately -- there is no fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
import fractions
import math
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY_PATH = os.path.join(_PKG, "libattn.so")

ATTN_OK = 0
STATUS_NAMES = {0: "ATTN_OK", 1: "ATTN_ERR_INVALID_ARG", 2: "ATTN_ERR_UNSUPPORTED", 3: "ATTN_ERR_CUDA",
                4: "ATTN_ERR_TIMEOUT", 5: "ATTN_ERR_WORKSPACE", 6: "ATTN_ERR_DEVICE_BOUNDS"}
LAYOUTS = {"bshd": 0, "bhsd": 1}

_lock = threading.Lock()
_lib = None

_p = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_sz = ctypes.c_size_t
_u64 = ctypes.c_uint64


class AttnError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {STATUS_NAMES.get(code, code)}")


def load():
    """Load libattn.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIBRARY_PATH):
                raise RuntimeError(
                    f"{LIBRARY_PATH} is missing: build the CUDA library first "
                    "(python -c 'import __graft_entry__ as g; g.build()')")
            lib = ctypes.CDLL(LIBRARY_PATH)
            fwd_args = [_p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _f, _p]
            lib.attn_fwd.argtypes = fwd_args
            lib.attn_fwd_simple.argtypes = fwd_args
            lib.attn_fwd_rounded.argtypes = fwd_args[:-1] + [_i, _p]
            lib.attn_fwd_host.argtypes = fwd_args[:-1] + [_i, _p, _sz, _p]
            lib.attn_fwd_host.restype = _i
            lib.attn_fwd_host_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i]
            lib.attn_fwd_host_workspace_bytes.restype = _sz
            lib.attn_fwd_varlen.argtypes = [_p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _i, _f,
                                            _i, _p]
            lib.attn_fwd_paged.argtypes = [_p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i,
                                           _f, _i, _p]
            lib.attn_fwd_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i, _i]
            lib.attn_fwd_workspace_bytes.restype = _sz
            lib.attn_set_workspace.argtypes = [_p, _sz]
            lib.attn_set_workspace.restype = _i
            lib.attn_decode_workspace_bytes.argtypes = [_i, _i, _i, _i]
            lib.attn_decode_workspace_bytes.restype = _sz
            lib.attn_decode_paged.argtypes = [_p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _f, _p,
                                              _sz, _p]
            lib.attn_decode_paged_append.argtypes = [_p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i,
                                                     _i, _f, _p, _sz, _p]
            lib.attn_decode_paged_append.restype = _i
            lib.attn_decode_paged_noalloc.argtypes = [_p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i,
                                                      _f, _p]
            lib.attn_decode_paged_noalloc.restype = _i
            lib.attn_lse_merge.argtypes = [_p, _p, _p, _p, _i, _i, _i, _i, _p]
            lib.attn_get_device_status.argtypes = [_p, ctypes.POINTER(_i)]
            lib.attn_set_wait_budget_ns.argtypes = [_u64]
            lib.attn_debug_inject.argtypes = [_i]
            lib.attn_selftest_umma.argtypes = [_p, _p, _p, _i, _p]
            rotate_args = [_p, _p, _f, _p, _i, _p, _i, _i]
            append_args = [_p, _p, _p] + rotate_args + [_i] * 8 + [_sz, _sz, _sz, _p]
            lib.attn_qk_norm_rope.argtypes = [_p, _p, _p, _p] + rotate_args + [_i] * 6 + [_sz] * 6 + [_p]
            lib.attn_append_paged.argtypes = [_p] * 6 + append_args
            lib.attn_append_paged_q4.argtypes = [_p] * 5 + append_args
            lib.attn_gather_paged_q4.argtypes = [_p] * 6 + [_i] * 7 + [_p]
            lib.attn_decode_q4_workspace_bytes.argtypes = [_i] * 5
            lib.attn_decode_q4_workspace_bytes.restype = _sz
            lib.attn_decode_paged_q4.argtypes = [_p] * 6 + [_i] * 7 + [_f, _p, _sz, _p]
            lib.attn_fwd_paged_q4_workspace_bytes.argtypes = [_i] * 4
            lib.attn_fwd_paged_q4_workspace_bytes.restype = _sz
            lib.attn_fwd_paged_q4.argtypes = [_p] * 7 + [_i] * 11 + [_f, _i, _p, _sz, _p]
            lib.attn_status_string.argtypes = [_i]
            lib.attn_status_string.restype = ctypes.c_char_p
            lib.attn_version.restype = _i
            for name in ("attn_fwd", "attn_fwd_simple", "attn_fwd_rounded", "attn_fwd_varlen", "attn_fwd_paged",
                         "attn_decode_paged",
                         "attn_lse_merge",
                         "attn_get_device_status", "attn_set_wait_budget_ns", "attn_debug_inject",
                         "attn_selftest_umma", "attn_qk_norm_rope", "attn_append_paged", "attn_append_paged_q4",
                         "attn_gather_paged_q4", "attn_decode_paged_q4", "attn_fwd_paged_q4"):
                getattr(lib, name).restype = _i
            _lib = lib
    return _lib


def _check(rc: int, what: str):
    if rc != ATTN_OK:
        raise AttnError(rc, what)


def _stream(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _dev_tensor(t: torch.Tensor, name: str, dtype):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _dims(q, k, layout):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k, v must be 4-D")
    if layout == "bshd":
        B, Sq, Hq, d = q.shape
        _, Sk, Hkv, _ = k.shape
    elif layout == "bhsd":
        B, Hq, Sq, d = q.shape
        _, Hkv, Sk, _ = k.shape
    else:
        raise ValueError(f"layout must be 'bshd' or 'bhsd', got {layout!r}")
    return B, Hq, Hkv, Sq, Sk, d


ROUNDING = {"rtne": 0, "rtna": 1, "rtz": 2}


def _fwd_call(fn_name, q, k, v, causal, scale, layout, out, lse, stream, rounding="rtne"):
    lib = load()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _dev_tensor(t, n, torch.bfloat16)
    if k.shape != v.shape:
        raise ValueError("k and v must have the same shape")
    B, Hq, Hkv, Sq, Sk, d = _dims(q, k, layout)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, Sq), device=q.device, dtype=torch.float32)
    elif lse is not False:
        _dev_tensor(lse, "lse", torch.float32)
    lse_ptr = None if lse is False else lse.data_ptr()
    args = [q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse_ptr, B, Hq, Hkv, Sq, Sk, d, LAYOUTS[layout],
            int(bool(causal)), float(scale)]
    if rounding != "rtne":
        if fn_name != "attn_fwd":
            raise ValueError(f"{fn_name} rounds its output to nearest even only")
        fn_name = "attn_fwd_rounded"
        args.append(ROUNDING[rounding])
    rc = getattr(lib, fn_name)(*args, _stream(stream))
    _check(rc, fn_name)
    return out, (None if lse is False else lse)


def fwd(q, k, v, *, causal=False, scale=None, layout="bshd", out=None, lse=None, stream=None, rounding="rtne"):
    """Fused exact attention forward: returns (out bf16 in q's layout, lse fp32 [B, Hq, Sq]).

    Pass ``lse=False`` to skip the log-sum-exp output.  ``rounding`` selects how
    the fp32 result is rounded to the bf16 output: "rtne" (nearest, ties to
    even; C entry point attn_fwd), "rtna" (nearest, ties away from zero) or
    "rtz" (toward zero), the latter two through attn_fwd_rounded.
    """
    if rounding not in ROUNDING:
        raise ValueError(f"rounding must be one of {sorted(ROUNDING)}, got {rounding!r}")
    return _fwd_call("attn_fwd", q, k, v, causal, scale, layout, out, lse, stream, rounding)


def fwd_host_workspace_bytes(B: int, Hq: int, Hkv: int, Sq: int, Sk: int, d: int = 128) -> int:
    """Device workspace bytes fwd_host needs for this shape."""
    return int(load().attn_fwd_host_workspace_bytes(B, Hq, Hkv, Sq, Sk, d))


def fwd_host(q, k, v, *, causal=False, scale=None, layout="bshd", out=None, lse=None, workspace=None, stream=None,
             rounding="rtne"):
    """The forward pass from and to host memory (C entry point attn_fwd_host).

    q, k, v: CPU bf16 tensors (pin them for asynchronous copies); out/lse: CPU
    tensors to write (allocated pinned when omitted; ``lse=False`` skips it).
    workspace: a CUDA uint8 tensor of at least fwd_host_workspace_bytes(...)
    bytes (allocated when omitted).  Returns (out, lse); they are complete once
    ``stream`` (default: the current stream) has reached this point.
    """
    lib = load()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        if t.device.type != "cpu" or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous CPU bfloat16 tensor")
    if rounding not in ROUNDING:
        raise ValueError(f"rounding must be one of {sorted(ROUNDING)}, got {rounding!r}")
    if k.shape != v.shape:
        raise ValueError("k and v must have the same shape")
    B, Hq, Hkv, Sq, Sk, d = _dims(q, k, layout)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16).pin_memory()
    if lse is None:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32).pin_memory()
    need = fwd_host_workspace_bytes(B, Hq, Hkv, Sq, Sk, d)
    if workspace is None:
        workspace = torch.empty(max(need, 1), device="cuda", dtype=torch.uint8)
    _dev_tensor(workspace, "workspace", torch.uint8)
    lse_ptr = None if lse is False else lse.data_ptr()
    rc = lib.attn_fwd_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse_ptr, B, Hq, Hkv, Sq, Sk, d,
                           LAYOUTS[layout], int(bool(causal)), float(scale), ROUNDING[rounding], workspace.data_ptr(),
                           workspace.numel(), _stream(stream))
    _check(rc, "attn_fwd_host")
    return out, (None if lse is False else lse)


def fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, *, max_seqlen_q=None, max_seqlen_k=None, causal=False,
               scale=None, out=None, lse=None, stream=None, rounding="rtne"):
    """Attention over a packed batch of variable-length sequences.

    q [total_q, Hq, d], k and v [total_k, Hkv, d] bf16; cu_seqlens_q/k int32 [B+1]
    on the device.  Returns (out [total_q, Hq, d] bf16, lse [Hq, total_q] fp32).
    max_seqlen_q/k bound the sequence lengths; when omitted they are read from
    the offsets, which copies them to the host (a synchronisation).  Rows of
    ``out``/``lse`` outside every sequence are left as given.
    """
    lib = load()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _dev_tensor(t, n, torch.bfloat16)
    _dev_tensor(cu_seqlens_q, "cu_seqlens_q", torch.int32)
    _dev_tensor(cu_seqlens_k, "cu_seqlens_k", torch.int32)
    if rounding not in ROUNDING:
        raise ValueError(f"rounding must be one of {sorted(ROUNDING)}, got {rounding!r}")
    if q.dim() != 3 or k.dim() != 3 or k.shape != v.shape:
        raise ValueError("q must be [total_q, Hq, d] and k, v [total_k, Hkv, d]")
    total_q, Hq, d = q.shape
    total_k, Hkv, _ = k.shape
    B = cu_seqlens_q.numel() - 1
    if cu_seqlens_k.numel() != B + 1 or B < 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must both have B + 1 entries, B >= 1")
    if max_seqlen_q is None:
        max_seqlen_q = max(1, int(torch.diff(cu_seqlens_q).max()))
    if max_seqlen_k is None:
        max_seqlen_k = max(1, int(torch.diff(cu_seqlens_k).max()))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((Hq, total_q), device=q.device, dtype=torch.float32)
    elif lse is not False:
        _dev_tensor(lse, "lse", torch.float32)
    lse_ptr = None if lse is False else lse.data_ptr()
    rc = lib.attn_fwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse_ptr,
                             cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), B, Hq, Hkv, total_q, total_k,
                             int(max_seqlen_q), int(max_seqlen_k), d, int(bool(causal)), float(scale),
                             ROUNDING[rounding], _stream(stream))
    _check(rc, "attn_fwd_varlen")
    return out, (None if lse is False else lse)


def fwd_paged(q, k_pages, v_pages, block_table, seqlens_k, cu_seqlens_q, *, max_seqlen_q=None, causal=True,
              scale=None, out=None, lse=None, stream=None, rounding="rtne"):
    """Prefill of packed query chunks against a paged KV cache (chunked prefill).

    q [total_q, Hq, d] bf16; k_pages, v_pages [num_pages, 16, Hkv, d] bf16; block_table [B, max_blocks]
    int32; seqlens_k [B] int32 (cache lengths, chunk included); cu_seqlens_q [B+1] int32 -- all on the
    device.  Returns (out [total_q, Hq, d] bf16, lse [Hq, total_q] fp32).  max_seqlen_q, when omitted,
    is read from the offsets (a synchronisation).
    """
    lib = load()
    for t, n in ((q, "q"), (k_pages, "k_pages"), (v_pages, "v_pages")):
        _dev_tensor(t, n, torch.bfloat16)
    for t, n in ((block_table, "block_table"), (seqlens_k, "seqlens_k"), (cu_seqlens_q, "cu_seqlens_q")):
        _dev_tensor(t, n, torch.int32)
    if rounding not in ROUNDING:
        raise ValueError(f"rounding must be one of {sorted(ROUNDING)}, got {rounding!r}")
    if q.dim() != 3 or k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
        raise ValueError("q must be [total_q, Hq, d] and the pools [num_pages, 16, Hkv, d]")
    total_q, Hq, d = q.shape
    num_pages, page_size, Hkv, _ = k_pages.shape
    B = seqlens_k.numel()
    if cu_seqlens_q.numel() != B + 1 or block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("cu_seqlens_q must have B + 1 entries and block_table B rows")
    if max_seqlen_q is None:
        max_seqlen_q = max(1, int(torch.diff(cu_seqlens_q).max()))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((Hq, total_q), device=q.device, dtype=torch.float32)
    elif lse is not False:
        _dev_tensor(lse, "lse", torch.float32)
    lse_ptr = None if lse is False else lse.data_ptr()
    rc = lib.attn_fwd_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
                            seqlens_k.data_ptr(), cu_seqlens_q.data_ptr(), out.data_ptr(), lse_ptr, B, Hq, Hkv,
                            total_q, int(max_seqlen_q), d, page_size, num_pages, block_table.shape[1],
                            int(bool(causal)), float(scale), ROUNDING[rounding], _stream(stream))
    _check(rc, "attn_fwd_paged")
    return out, (None if lse is False else lse)


def fwd_simple(q, k, v, *, causal=False, scale=None, layout="bshd", out=None, lse=None, stream=None):
    """The same operation through the plain SIMT kernel (debugging cross-check; slow)."""
    return _fwd_call("attn_fwd_simple", q, k, v, causal, scale, layout, out, lse, stream)


def fwd_workspace_bytes(B: int, Hq: int, Hkv: int, Sq: int, Sk: int, d: int = 128, causal: bool = False) -> int:
    """Workspace bytes that let attn_fwd split its last wave of work for this shape (current device)."""
    return int(load().attn_fwd_workspace_bytes(B, Hq, Hkv, Sq, Sk, d, int(bool(causal))))


def set_workspace(buf=None):
    """Register a CUDA uint8 tensor (or None to clear) as the current device's attn_fwd workspace.

    The caller keeps ownership and must keep the tensor alive while it is registered.
    """
    if buf is None:
        _check(load().attn_set_workspace(None, 0), "attn_set_workspace")
        return
    _dev_tensor(buf, "workspace", torch.uint8)
    _check(load().attn_set_workspace(buf.data_ptr(), buf.numel()), "attn_set_workspace")


def decode_workspace_bytes(B: int, Hq: int, d: int, max_blocks_per_seq: int) -> int:
    return int(load().attn_decode_workspace_bytes(B, Hq, d, max_blocks_per_seq))


def decode_paged(q, k_pages, v_pages, block_table, seqlens, *, scale=None, out=None, lse=None, workspace=None,
                 stream=None):
    """One decode step over a paged KV cache.

    q [B, Hq, d] bf16; k_pages/v_pages [num_pages, 16, Hkv, d] bf16; block_table [B, max_blocks] int32;
    seqlens [B] int32 (device).  Returns (out [B, Hq, d] bf16, lse [B, Hq] fp32).
    """
    lib = load()
    _dev_tensor(q, "q", torch.bfloat16)
    _dev_tensor(k_pages, "k_pages", torch.bfloat16)
    _dev_tensor(v_pages, "v_pages", torch.bfloat16)
    _dev_tensor(block_table, "block_table", torch.int32)
    _dev_tensor(seqlens, "seqlens", torch.int32)
    B, Hq, d = q.shape
    num_pages, page_size, Hkv, _ = k_pages.shape
    max_blocks = block_table.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq), device=q.device, dtype=torch.float32)
    need = decode_workspace_bytes(B, Hq, d, max_blocks)
    if workspace is None:
        workspace = torch.empty(max(need, 1), device=q.device, dtype=torch.uint8)
    lse_ptr = None if lse is False else lse.data_ptr()
    rc = lib.attn_decode_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
                               seqlens.data_ptr(), out.data_ptr(), lse_ptr, B, Hq, Hkv, d, page_size, num_pages,
                               max_blocks, float(scale), workspace.data_ptr(), workspace.numel(),
                               _stream(stream))
    _check(rc, "attn_decode_paged")
    return out, (None if lse is False else lse)


def decode_paged_append(q, k_new, v_new, k_pages, v_pages, block_table, seqlens, *, scale=None, out=None, lse=None,
                        workspace=None, stream=None):
    """Append k_new/v_new [B, Hkv, d] at position seqlens[b] of each sequence's pages and decode over the
    seqlens[b] + 1 keys, in one launch.  seqlens (the lengths before the append) is not modified.
    Returns (out [B, Hq, d] bf16, lse [B, Hq] fp32); k_pages and v_pages are updated in place."""
    lib = load()
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new"), (k_pages, "k_pages"), (v_pages, "v_pages")):
        _dev_tensor(t, n, torch.bfloat16)
    _dev_tensor(block_table, "block_table", torch.int32)
    _dev_tensor(seqlens, "seqlens", torch.int32)
    B, Hq, d = q.shape
    num_pages, page_size, Hkv, _ = k_pages.shape
    if k_new.shape != (B, Hkv, d) or v_new.shape != (B, Hkv, d):
        raise ValueError("k_new and v_new must be [B, Hkv, d]")
    max_blocks = block_table.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq), device=q.device, dtype=torch.float32)
    need = decode_workspace_bytes(B, Hq, d, max_blocks)
    if workspace is None:
        workspace = torch.empty(max(need, 1), device=q.device, dtype=torch.uint8)
    lse_ptr = None if lse is False else lse.data_ptr()
    rc = lib.attn_decode_paged_append(q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), k_pages.data_ptr(),
                                      v_pages.data_ptr(), block_table.data_ptr(), seqlens.data_ptr(), out.data_ptr(),
                                      lse_ptr, B, Hq, Hkv, d, page_size, num_pages, max_blocks, float(scale),
                                      workspace.data_ptr(), workspace.numel(), _stream(stream))
    _check(rc, "attn_decode_paged_append")
    return out, (None if lse is False else lse)


def decode_paged_noalloc(q, k_pages, v_pages, block_table, seqlens, *, scale=None, out=None, lse=None,
                         stream=None):
    """decode_paged for callers that cannot allocate device memory.

    Same arguments and results as ``decode_paged`` minus the workspace: the
    split partials live in a fixed 16 MiB device array owned by the library
    (shared by every call, so calls must not overlap on the GPU).  ``out`` and
    ``lse`` must be passed by a caller that cannot allocate; when they are
    omitted this wrapper allocates them with torch for convenience.
    """
    lib = load()
    _dev_tensor(q, "q", torch.bfloat16)
    _dev_tensor(k_pages, "k_pages", torch.bfloat16)
    _dev_tensor(v_pages, "v_pages", torch.bfloat16)
    _dev_tensor(block_table, "block_table", torch.int32)
    _dev_tensor(seqlens, "seqlens", torch.int32)
    B, Hq, d = q.shape
    num_pages, page_size, Hkv, _ = k_pages.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq), device=q.device, dtype=torch.float32)
    lse_ptr = None if lse is False else lse.data_ptr()
    rc = lib.attn_decode_paged_noalloc(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                       block_table.data_ptr(), seqlens.data_ptr(), out.data_ptr(), lse_ptr, B, Hq,
                                       Hkv, d, page_size, num_pages, block_table.shape[1], float(scale),
                                       _stream(stream))
    _check(rc, "attn_decode_paged_noalloc")
    return out, (None if lse is False else lse)


Q4_BLOCK_BYTES = 2560  # one page of one KV head in the 4-bit cache (ATTN_Q4_BLOCK_BYTES)
_PI = fractions.Fraction("3.14159265358979323846264338327950288419716939937510582")


def _on_current_device(*tensors):
    """The library launches on the current device: every tensor must live there."""
    want = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.device.index != want:
            raise ValueError(f"tensor on {t.device}, but the current device is cuda:{want}")


def _on_stream(stream):
    """Outputs and workspaces made here belong to the stream that writes them."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _strided(t, name):
    """A CUDA bf16 tensor whose last dimension is contiguous (the others may be strided)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() < 2 or t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _step(t, dim):
    # the stride of a dimension of length one is never used, whatever it says
    return 0 if t.shape[dim] == 1 else t.stride(dim)


def _ptr(t):
    return None if t is None else t.data_ptr()


def rope_table(inv_freq, axes=None, *, device="cuda"):
    """The plan of a position rotation (attn_rope_pair_t entries), made once and kept by the caller.

    inv_freq: the radians per position of each of the rotary_dim / 2 pairs (floats, or a 1-D tensor; any
    frequencies, e.g. ``base ** (-2 i / rotary_dim)`` or a rescaled form of it); axes: the position axis of each
    pair (default: all 0).  Returns an int64 [rotary_dim / 2, 2] tensor on ``device``: each pair's turns per
    position in units of 2**-64, and its axis.
    """
    freq = inv_freq.tolist() if isinstance(inv_freq, torch.Tensor) else [float(f) for f in inv_freq]
    axis = [0] * len(freq) if axes is None else [int(a) for a in axes]
    if not freq or len(axis) != len(freq):
        raise ValueError("inv_freq must not be empty, and axes must have one entry per frequency")
    if not all(math.isfinite(f) for f in freq):
        raise ValueError("inv_freq must be finite")
    if not all(0 <= a < 4 for a in axis):
        raise ValueError("axes must be 0 .. 3")
    rows = []
    for f, a in zip(freq, axis):
        turns = round(fractions.Fraction(f) * 2**63 / _PI) % 2**64
        rows.append([turns - 2**64 if turns >= 2**63 else turns, a])
    return torch.tensor(rows, dtype=torch.int64).to(device)


def _rotate_args(q_weight, k_weight, eps, positions, pos_shape, rope, interleaved):
    """The norm and rotation arguments of a call, checked, in the C order."""
    for w, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _dev_tensor(w, n, torch.bfloat16)
            if w.shape != (128,):
                raise ValueError(f"{n} must have 128 elements")
    n_axes = 1
    if positions is not None:
        _dev_tensor(positions, "positions", torch.int32)
        if tuple(positions.shape) == pos_shape:
            pass
        elif positions.dim() == len(pos_shape) + 1 and tuple(positions.shape[1:]) == pos_shape:
            n_axes = positions.shape[0]
        else:
            raise ValueError(f"positions must be {list(pos_shape)} or [axes, {', '.join(map(str, pos_shape))}], "
                             f"got {list(positions.shape)}")
    rotary_dim = 0
    if rope is not None:
        _dev_tensor(rope, "rope", torch.int64)
        if rope.dim() != 2 or rope.shape[1] != 2:
            raise ValueError("rope must be a table made by rope_table")
        rotary_dim = 2 * rope.shape[0]
        if positions is None:
            n_axes = 4  # the default position is the same on every axis
    _on_current_device(q_weight, k_weight, positions, rope)
    return [_ptr(q_weight), _ptr(k_weight), float(eps), _ptr(positions), n_axes, _ptr(rope), rotary_dim,
            int(bool(interleaved))]


def qk_norm_rope(q, k=None, *, rope=None, positions=None, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                 layout="bshd", q_out=None, k_out=None, stream=None):
    """Root-mean-square norm of every query and key head and the position rotation, in one pass.

    q [B, S, Hq, 128] and k [B, S, Hkv, 128] bf16 (``layout="bshd"``), [B, H, S, 128] ("bhsd"), or packed
    [total, H, 128]; they may be strided views of a fused projection (k may be None).  rope: a plan of rope_table;
    positions: int32 [B, S] or [axes, B, S] ([total], [axes, total] for packed tensors), default 0 .. S-1 on every
    axis; q_weight, k_weight: bf16 [128], None for no norm.  Returns (q_out, k_out), dense in the layout (k_out None
    without k); q_out may be q itself when it is dense.
    """
    lib = load()
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be 'bshd' or 'bhsd', got {layout!r}")
    _strided(q, "q")
    if k is not None:
        _strided(k, "k")
    packed = q.dim() == 3
    if packed and layout != "bshd":
        raise ValueError("packed tensors are [total, H, 128] (layout 'bshd')")
    if q.dim() not in (3, 4) or (k is not None and k.dim() != q.dim()):
        raise ValueError("q and k must be 4-D, or both packed 3-D")
    q4, k4 = (q.unsqueeze(0), None if k is None else k.unsqueeze(0)) if packed else (q, k)
    s_dim, h_dim = (1, 2) if layout == "bshd" else (2, 1)
    B, S, Hq, d = q4.shape[0], q4.shape[s_dim], q4.shape[h_dim], q4.shape[3]
    Hkv = 0 if k is None else k4.shape[h_dim]
    if k is not None and (k4.shape[0] != B or k4.shape[s_dim] != S or k4.shape[3] != d):
        raise ValueError("q and k must have the same batch, positions and head dimension")
    for o, x, n in ((q_out, q, "q_out"), (k_out, k, "k_out")):
        if o is not None:
            _dev_tensor(o, n, torch.bfloat16)
            if x is None or o.shape != x.shape:
                raise ValueError(f"{n} must have its input's shape")
    args = _rotate_args(q_weight, k_weight, eps, positions, (S,) if packed else (B, S), rope, interleaved)
    _on_current_device(q, k, q_out, k_out)
    with _on_stream(stream):
        if q_out is None:
            q_out = torch.empty(q.shape, device=q.device, dtype=torch.bfloat16)
        if k_out is None and k is not None:
            k_out = torch.empty(k.shape, device=k.device, dtype=torch.bfloat16)
    steps = [_step(q4, i) for i in (0, s_dim, h_dim)] + ([0] * 3 if k is None else
                                                         [_step(k4, i) for i in (0, s_dim, h_dim)])
    rc = lib.attn_qk_norm_rope(q.data_ptr(), _ptr(k), q_out.data_ptr(), _ptr(k_out), *args, B, S, Hq, Hkv, d,
                               LAYOUTS[layout], *steps, _stream(stream))
    _check(rc, "attn_qk_norm_rope")
    return q_out, k_out


def _append(fn_name, q, k, v, pools, Hkv_pool, num_pages, page_size, block_table, seqlens, cu_seqlens, rope, positions,
            q_weight, k_weight, eps, interleaved, q_out, stream):
    lib = load()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        if t is None and n == "q":
            continue
        _strided(t, n)
        if t.dim() != 3 or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
            raise ValueError(f"{n} must be [tokens, H, 128] with the heads of a token contiguous")
    for t, n in ((block_table, "block_table"), (seqlens, "seqlens")):
        _dev_tensor(t, n, torch.int32)
    if cu_seqlens is not None:
        _dev_tensor(cu_seqlens, "cu_seqlens", torch.int32)
    total, Hkv, d = k.shape
    B = seqlens.numel()
    if v.shape != k.shape or (q is not None and (q.shape[0] != total or q.shape[2] != d)):
        raise ValueError("q, k, v must have the same tokens and head dimension, k and v the same heads")
    if Hkv != Hkv_pool:
        raise ValueError(f"the cache has {Hkv_pool} KV heads, k and v have {Hkv}")
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must have one row per sequence")
    if cu_seqlens is None and total != B:
        raise ValueError("without cu_seqlens there is one new token per sequence")
    if cu_seqlens is not None and cu_seqlens.numel() != B + 1:
        raise ValueError("cu_seqlens must have B + 1 entries")
    if q_out is not None:
        _dev_tensor(q_out, "q_out", torch.bfloat16)
        if q is None or q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
    args = _rotate_args(q_weight, k_weight, eps, positions, (total,), rope, interleaved)
    _on_current_device(q, k, v, *pools, block_table, seqlens, cu_seqlens, q_out)
    if q is not None and q_out is None:
        with _on_stream(stream):
            q_out = torch.empty(q.shape, device=q.device, dtype=torch.bfloat16)
    steps = [0 if t is None else (t.shape[1] * d if total == 1 else t.stride(0)) for t in (q, k, v)]
    rc = getattr(lib, fn_name)(_ptr(q), k.data_ptr(), v.data_ptr(), _ptr(q_out), *[t.data_ptr() for t in pools],
                               block_table.data_ptr(), seqlens.data_ptr(), _ptr(cu_seqlens), *args, B, total,
                               0 if q is None else q.shape[1], Hkv, d, page_size, num_pages, block_table.shape[1],
                               *steps, _stream(stream))
    _check(rc, fn_name)
    return q_out


def append_paged(q, k, v, k_pages, v_pages, block_table, seqlens, cu_seqlens=None, *, rope=None, positions=None,
                 q_weight=None, k_weight=None, eps=1e-6, interleaved=False, q_out=None, stream=None):
    """Write new tokens' keys and values into the paged cache, with the norm and rotation of qk_norm_rope on the way.

    q [total, Hq, 128] (or None), k and v [total, Hkv, 128] bf16, the sequences' new tokens back to back (views of a
    fused projection need no copy); k_pages, v_pages [num_pages, 16, Hkv, 128] bf16, updated in place; block_table
    [B, max_blocks], seqlens [B] (the lengths WITH the new tokens) and cu_seqlens [B + 1] int32 (None: one token per
    sequence).  positions: int32 [total] or [axes, total], default: each token's position in its cache.  Returns
    q_out [total, Hq, 128] (None without q): the q of fwd_paged or decode_paged over the same arrays.
    """
    for t, n in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        _dev_tensor(t, n, torch.bfloat16)
    if k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
        raise ValueError("k_pages and v_pages must be [num_pages, 16, Hkv, 128]")
    num_pages, page_size, Hkv, d = k_pages.shape
    if isinstance(k, torch.Tensor) and k.shape[-1] != d:
        raise ValueError("k and the pages must have the same head dimension")
    return _append("attn_append_paged", q, k, v, (k_pages, v_pages), Hkv, num_pages, page_size, block_table, seqlens,
                   cu_seqlens, rope, positions, q_weight, k_weight, eps, interleaved, q_out, stream)


def _q4_cache(cache):
    _dev_tensor(cache, "cache", torch.uint8)
    if cache.dim() != 3 or cache.shape[2] != Q4_BLOCK_BYTES:
        raise ValueError(f"cache must be [num_pages, Hkv, {Q4_BLOCK_BYTES}]")
    return cache.shape[0], cache.shape[1]


def append_paged_q4(q, k, v, cache, block_table, seqlens, cu_seqlens=None, *, rope=None, positions=None,
                    q_weight=None, k_weight=None, eps=1e-6, interleaved=False, q_out=None, stream=None):
    """append_paged into a cache held in 4 bits: cache [num_pages, Hkv, Q4_BLOCK_BYTES] uint8, updated in place."""
    num_pages, Hkv = _q4_cache(cache)
    return _append("attn_append_paged_q4", q, k, v, (cache,), Hkv, num_pages, 16, block_table, seqlens, cu_seqlens,
                   rope, positions, q_weight, k_weight, eps, interleaved, q_out, stream)


def gather_paged_q4(cache, block_table, seqlens, cu_seqlens_k, *, total_k=None, k_out=None, v_out=None, stream=None):
    """Read sequences back from a 4-bit cache: (k, v) bf16 [total_k, Hkv, 128], sequence b's seqlens[b] tokens from row
    cu_seqlens_k[b] on -- the k and v of fwd_varlen.  total_k, when omitted, is read from the outputs given or the
    offsets (a synchronisation)."""
    lib = load()
    num_pages, Hkv = _q4_cache(cache)
    for t, n in ((block_table, "block_table"), (seqlens, "seqlens"), (cu_seqlens_k, "cu_seqlens_k")):
        _dev_tensor(t, n, torch.int32)
    B = seqlens.numel()
    if block_table.dim() != 2 or block_table.shape[0] != B or cu_seqlens_k.numel() != B + 1:
        raise ValueError("block_table must have B rows and cu_seqlens_k B + 1 entries")
    for o, n in ((k_out, "k_out"), (v_out, "v_out")):
        if o is not None:
            _dev_tensor(o, n, torch.bfloat16)
            if o.dim() != 3 or o.shape[1:] != (Hkv, 128) or (total_k is not None and o.shape[0] != total_k):
                raise ValueError(f"{n} must be [total_k, Hkv, 128]")
            total_k = o.shape[0]
    _on_current_device(cache, block_table, seqlens, cu_seqlens_k, k_out, v_out)
    if total_k is None:
        total_k = max(1, int(cu_seqlens_k[-1]))
    with _on_stream(stream):
        if k_out is None:
            k_out = torch.empty((total_k, Hkv, 128), device=cache.device, dtype=torch.bfloat16)
        if v_out is None:
            v_out = torch.empty((total_k, Hkv, 128), device=cache.device, dtype=torch.bfloat16)
    rc = lib.attn_gather_paged_q4(cache.data_ptr(), block_table.data_ptr(), seqlens.data_ptr(),
                                  cu_seqlens_k.data_ptr(), k_out.data_ptr(), v_out.data_ptr(), B, Hkv, int(total_k),
                                  128, 16, num_pages, block_table.shape[1], _stream(stream))
    _check(rc, "attn_gather_paged_q4")
    return k_out, v_out


def decode_q4_workspace_bytes(B: int, Hq: int, Hkv: int, d: int, max_blocks_per_seq: int) -> int:
    """Device workspace bytes decode_paged_q4 needs for this shape."""
    return int(load().attn_decode_q4_workspace_bytes(B, Hq, Hkv, d, max_blocks_per_seq))


def decode_paged_q4(q, cache, block_table, seqlens, *, scale=None, out=None, lse=None, workspace=None, stream=None):
    """One decode step over a cache held in 4 bits (the arguments of decode_paged, with one cache tensor
    [num_pages, Hkv, Q4_BLOCK_BYTES] uint8).  Returns (out [B, Hq, 128] bf16, lse [B, Hq] fp32)."""
    lib = load()
    num_pages, Hkv = _q4_cache(cache)
    _dev_tensor(q, "q", torch.bfloat16)
    for t, n in ((block_table, "block_table"), (seqlens, "seqlens")):
        _dev_tensor(t, n, torch.int32)
    if q.dim() != 3 or block_table.dim() != 2 or block_table.shape[0] != q.shape[0] or seqlens.numel() != q.shape[0]:
        raise ValueError("q must be [B, Hq, 128], block_table [B, max_blocks] and seqlens [B]")
    B, Hq, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _attn_out(out, lse, q.shape, (B, Hq))
    _on_current_device(q, cache, block_table, seqlens, out, workspace, None if lse is False else lse)
    need = decode_q4_workspace_bytes(B, Hq, Hkv, d, block_table.shape[1])
    if workspace is not None:
        _dev_tensor(workspace, "workspace", torch.uint8)
    with _on_stream(stream):
        if out is None:
            out = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((B, Hq), device=q.device, dtype=torch.float32)
        if workspace is None:
            workspace = torch.empty(max(need, 1), device=q.device, dtype=torch.uint8)
        rc = lib.attn_decode_paged_q4(q.data_ptr(), cache.data_ptr(), block_table.data_ptr(), seqlens.data_ptr(),
                                      out.data_ptr(), None if lse is False else lse.data_ptr(), B, Hq, Hkv, d, 16,
                                      num_pages, block_table.shape[1], float(scale), workspace.data_ptr(),
                                      workspace.numel(), _stream(stream))
    _check(rc, "attn_decode_paged_q4")
    return out, (None if lse is False else lse)


def _attn_out(out, lse, out_shape, lse_shape):
    if out is not None:
        _dev_tensor(out, "out", torch.bfloat16)
        if out.shape != out_shape:
            raise ValueError(f"out must be {list(out_shape)}")
    if lse is not None and lse is not False:
        _dev_tensor(lse, "lse", torch.float32)
        if tuple(lse.shape) != lse_shape:
            raise ValueError(f"lse must be {list(lse_shape)}")


def fwd_paged_q4_workspace_bytes(B: int, Hkv: int, d: int, max_total_k: int) -> int:
    """Device workspace bytes fwd_paged_q4 needs for caches of max_total_k tokens in all."""
    return int(load().attn_fwd_paged_q4_workspace_bytes(B, Hkv, d, max_total_k))


def fwd_paged_q4(q, cache, block_table, seqlens_k, cu_seqlens_q, *, max_seqlen_q=None, max_total_k=None, causal=True,
                 scale=None, out=None, lse=None, workspace=None, stream=None, rounding="rtne"):
    """Prefill of packed query chunks against a cache held in 4 bits (the arguments of fwd_paged, with one cache tensor
    [num_pages, Hkv, Q4_BLOCK_BYTES] uint8).  max_total_k bounds the sum of seqlens_k; it and max_seqlen_q, when
    omitted, are read from the device (a synchronisation).  Returns (out [total_q, Hq, 128] bf16, lse [Hq, total_q])."""
    lib = load()
    num_pages, Hkv = _q4_cache(cache)
    _dev_tensor(q, "q", torch.bfloat16)
    for t, n in ((block_table, "block_table"), (seqlens_k, "seqlens_k"), (cu_seqlens_q, "cu_seqlens_q")):
        _dev_tensor(t, n, torch.int32)
    if rounding not in ROUNDING:
        raise ValueError(f"rounding must be one of {sorted(ROUNDING)}, got {rounding!r}")
    if q.dim() != 3:
        raise ValueError("q must be [total_q, Hq, 128]")
    total_q, Hq, d = q.shape
    B = seqlens_k.numel()
    if cu_seqlens_q.numel() != B + 1 or block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("cu_seqlens_q must have B + 1 entries and block_table B rows")
    _attn_out(out, lse, q.shape, (Hq, total_q))
    if workspace is not None:
        _dev_tensor(workspace, "workspace", torch.uint8)
    _on_current_device(q, cache, block_table, seqlens_k, cu_seqlens_q, out, workspace, None if lse is False else lse)
    if max_seqlen_q is None:
        max_seqlen_q = max(1, int(torch.diff(cu_seqlens_q).max()))
    if max_total_k is None:
        max_total_k = max(1, int(seqlens_k.sum()))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = fwd_paged_q4_workspace_bytes(B, Hkv, d, int(max_total_k))
    with _on_stream(stream):
        if out is None:
            out = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((Hq, total_q), device=q.device, dtype=torch.float32)
        if workspace is None:
            workspace = torch.empty(max(need, 1), device=q.device, dtype=torch.uint8)
        rc = lib.attn_fwd_paged_q4(q.data_ptr(), cache.data_ptr(), block_table.data_ptr(), seqlens_k.data_ptr(),
                                   cu_seqlens_q.data_ptr(), out.data_ptr(), None if lse is False else lse.data_ptr(),
                                   B, Hq, Hkv, total_q, int(max_seqlen_q), d, 16, num_pages, block_table.shape[1],
                                   int(max_total_k), int(bool(causal)), float(scale), ROUNDING[rounding],
                                   workspace.data_ptr(), workspace.numel(), _stream(stream))
    _check(rc, "attn_fwd_paged_q4")
    return out, (None if lse is False else lse)


def lse_merge(o_parts, lse_parts, *, out=None, lse=None, stream=None, rounding="rtne"):
    """Merge key-range partials: o_parts [rows, nsplit, d] fp32, lse_parts [rows, nsplit] fp32.

    ``rounding`` ("rtne", "rtna" or "rtz") selects the fp32 -> bf16 rounding of out.
    """
    if rounding not in ROUNDING:
        raise ValueError(f"rounding must be one of {sorted(ROUNDING)}, got {rounding!r}")
    lib = load()
    _dev_tensor(o_parts, "o_parts", torch.float32)
    _dev_tensor(lse_parts, "lse_parts", torch.float32)
    rows, nsplit, d = o_parts.shape
    if out is None:
        out = torch.empty((rows, d), device=o_parts.device, dtype=torch.bfloat16)
    if lse is None:
        lse = torch.empty((rows,), device=o_parts.device, dtype=torch.float32)
    rc = lib.attn_lse_merge(o_parts.data_ptr(), lse_parts.data_ptr(), out.data_ptr(), lse.data_ptr(), rows, nsplit,
                            d, ROUNDING[rounding], _stream(stream))
    _check(rc, "attn_lse_merge")
    return out, lse


def device_status(stream=None):
    """Synchronise the stream, read and clear the device status word: (code, site)."""
    site = _i(0)
    rc = load().attn_get_device_status(_stream(stream), ctypes.byref(site))
    return rc, site.value


def set_wait_budget_ns(ns: int):
    _check(load().attn_set_wait_budget_ns(int(ns)), "attn_set_wait_budget_ns")


def debug_inject(mode: int):
    _check(load().attn_debug_inject(int(mode)), "attn_debug_inject")


def selftest_umma(a, b, mode: int, stream=None):
    """128x128x128 tensor-core layout check: mode 0 -> a @ b.T, mode 1 -> a @ b (fp32 [128, 128])."""
    _dev_tensor(a, "a", torch.bfloat16)
    _dev_tensor(b, "b", torch.bfloat16)
    c = torch.empty((128, 128), device=a.device, dtype=torch.float32)
    _check(load().attn_selftest_umma(a.data_ptr(), b.data_ptr(), c.data_ptr(), int(mode), _stream(stream)),
           "attn_selftest_umma")
    return c


def status_string(code: int) -> str:
    return load().attn_status_string(int(code)).decode()


def version() -> int:
    return int(load().attn_version())
