"""ctypes binding of libattn.so (the C ABI in include/attn.h), with a quicker
way (_quick.so, csrc/binding.cpp) for the operators whose calls take a few
microseconds.

Argument marshalling only: every step of the computation runs in the CUDA
library.  PyTorch owns the device memory and the stream; tensors are passed by
``data_ptr()`` and the current stream by handle.  If the library is missing
this module raises immediately -- there is no fallback path.  _quick.so is bound
to the torch that it was built against; where it is missing or was built for
another one, load() says so and its operators take the way through ctypes, a few
microseconds a call longer.
"""
from __future__ import annotations

import ctypes
import fractions
import importlib
import math
import os
import threading
import warnings

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY_PATH = os.path.join(_PKG, "libattn.so")

ATTN_OK = 0
STATUS_NAMES = {0: "ATTN_OK", 1: "ATTN_ERR_INVALID_ARG", 2: "ATTN_ERR_UNSUPPORTED", 3: "ATTN_ERR_CUDA",
                4: "ATTN_ERR_TIMEOUT", 5: "ATTN_ERR_WORKSPACE", 6: "ATTN_ERR_DEVICE_BOUNDS"}
LAYOUTS = {"bshd": 0, "bhsd": 1}

_lock = threading.Lock()
_lib = None
_quick = None  # _quick.so: the quick way into the operators around the paged cache

_p = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_sz = ctypes.c_size_t
_u64 = ctypes.c_uint64


class AttnError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {STATUS_NAMES.get(code, code)}")


class _NoQuick:
    """In the place of _quick where it cannot be used: every call goes the long way."""
    qk_norm_rope = append = gather = decode = fwd = tree = verify = compact = staticmethod(lambda *args: None)


def _load_quick():
    """_quick, or (with a warning) what stands in for it."""
    from . import build
    built, here = build.built_abi(), build.abi_tag()
    if not os.path.exists(build.QUICK) or built is None:
        why = "is missing"
    elif built != here:
        why = f"was built for {built}; this is {here}"
    else:
        try:
            return importlib.import_module("._quick", __package__)
        except ImportError as e:
            why = f"cannot be imported ({e})"
    warnings.warn(f"{build.QUICK} {why}: the operators around the paged cache are called through ctypes, which takes "
                  "about 10 us more a call (python -c 'import __graft_entry__ as g; g.build()' builds it)",
                  RuntimeWarning, stacklevel=3)
    return _NoQuick()


def load():
    """Load libattn.so (raises if it has not been built)."""
    global _lib, _quick
    with _lock:
        if _lib is None:
            if not os.path.exists(LIBRARY_PATH):
                raise RuntimeError(
                    f"{LIBRARY_PATH} is missing: build the CUDA library first "
                    "(python -c 'import __graft_entry__ as g; g.build()')")
            lib = ctypes.CDLL(LIBRARY_PATH)
            _quick = _load_quick()
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
            lib.attn_fwd_tree_paged_workspace_bytes.argtypes = [_i] * 5
            lib.attn_fwd_tree_paged_workspace_bytes.restype = _sz
            lib.attn_fwd_tree_paged.argtypes = [_p] * 9 + [_i] * 9 + [_f, _i, _p, _sz, _p]
            lib.attn_verify_tree_workspace_bytes.argtypes = [_i] * 6
            lib.attn_verify_tree_workspace_bytes.restype = _sz
            lib.attn_verify_tree.argtypes = [_p, _p, _i] + [_p] * 9 + [_i] * 4 + [_sz] * 3 + [_p, _sz, _p]
            lib.attn_compact_paged.argtypes = [_p] * 8 + [_i] * 9 + [_p]
            lib.attn_status_string.argtypes = [_i]
            lib.attn_status_string.restype = ctypes.c_char_p
            lib.attn_version.restype = _i
            for name in ("attn_fwd", "attn_fwd_simple", "attn_fwd_rounded", "attn_fwd_varlen", "attn_fwd_paged",
                         "attn_decode_paged",
                         "attn_lse_merge",
                         "attn_get_device_status", "attn_set_wait_budget_ns", "attn_debug_inject",
                         "attn_selftest_umma", "attn_qk_norm_rope", "attn_append_paged", "attn_append_paged_q4",
                         "attn_gather_paged_q4", "attn_decode_paged_q4", "attn_fwd_paged_q4",
                         "attn_fwd_tree_paged", "attn_verify_tree", "attn_compact_paged"):
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


# The operators below run in a few microseconds on small calls, less than Python
# takes to look at their tensors.  So a call first goes to _quick (csrc/binding.cpp),
# which checks, makes the outputs and launches, and which returns None when anything
# is not plainly in order, or a launch failed.  Then, and on a stream of the caller's, the function's own body runs: it checks one thing after the other and
# says what is wrong.  _in gives a tensor's address, and anything out of order
# goes to _refuse.
_raw_stream = torch._C._cuda_getCurrentRawStream
_device = torch._C._cuda_getDevice
_bf16 = torch.bfloat16
_i32 = torch.int32
_i64 = torch.int64


def _refuse(t, name, dtype, dev, contiguous=True):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not contiguous and (t.dim() < 2 or t.stride(-1) != 1):
        raise ValueError(f"{name} must be contiguous in its last dimension")
    raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{dev}")


def _in(t, name, dtype, dev):
    """The address of a contiguous tensor of dtype on the current device dev."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass  # not a tensor
    _refuse(t, name, dtype, dev)


def _in_strided(t, name, dev):
    """The address of a bf16 tensor that is contiguous in its last dimension (the others may be strided)."""
    try:
        if t.dtype is _bf16 and t.get_device() == dev and t.dim() >= 2 and t.stride(-1) == 1:
            return t.data_ptr()
    except AttributeError:
        pass  # not a tensor
    _refuse(t, name, _bf16, dev, contiguous=False)


def _current():
    """The device that the library launches on: the current one (-2, which no tensor is on: there is none)."""
    try:
        return _device()
    except RuntimeError:
        return -2


def _empty(shape, dtype, device, stream):
    """An output or workspace, which belongs to the stream that writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


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


def _rotate_args(q_weight, k_weight, eps, positions, pos_shape, rope, interleaved, dev):
    """The norm and rotation arguments of a call, checked, in the C order."""
    wq = wk = pos = None
    n_axes = 1
    if q_weight is not None:
        wq = _in(q_weight, "q_weight", _bf16, dev)
        if q_weight.shape != (128,):
            raise ValueError("q_weight must have 128 elements")
    if k_weight is not None:
        wk = _in(k_weight, "k_weight", _bf16, dev)
        if k_weight.shape != (128,):
            raise ValueError("k_weight must have 128 elements")
    if positions is not None:
        pos = _in(positions, "positions", _i32, dev)
        shape = positions.shape
        if shape != pos_shape:
            if len(shape) != len(pos_shape) + 1 or shape[1:] != pos_shape:
                raise ValueError(f"positions must be {list(pos_shape)} or [axes, {', '.join(map(str, pos_shape))}], "
                                 f"got {list(shape)}")
            n_axes = shape[0]
    if rope is None:
        return wq, wk, eps, pos, n_axes, None, 0, interleaved
    plan = _in(rope, "rope", _i64, dev)
    shape = rope.shape
    if len(shape) != 2 or shape[1] != 2:
        raise ValueError("rope must be a table made by rope_table")
    # the default position is the same on every axis
    return wq, wk, eps, pos, n_axes if pos else 4, plan, 2 * shape[0], interleaved


def qk_norm_rope(q, k=None, *, rope=None, positions=None, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                 layout="bshd", q_out=None, k_out=None, stream=None):
    """Root-mean-square norm of every query and key head and the position rotation, in one pass.

    q [B, S, Hq, 128] and k [B, S, Hkv, 128] bf16 (``layout="bshd"``), [B, H, S, 128] ("bhsd"), or packed
    [total, H, 128]; they may be strided views of a fused projection (k may be None).  rope: a plan of rope_table;
    positions: int32 [B, S] or [axes, B, S] ([total], [axes, total] for packed tensors), default 0 .. S-1 on every
    axis; q_weight, k_weight: bf16 [128], None for no norm.  Returns (q_out, k_out), dense in the layout (k_out None
    without k); q_out may be q itself when it is dense.
    """
    lib = _lib or load()
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be 'bshd' or 'bhsd', got {layout!r}")
    if stream is None:
        done = _quick.qk_norm_rope(q, k, q_weight, k_weight, eps, positions, rope, interleaved, LAYOUTS[layout], q_out,
                                   k_out)
        if done is not None:
            return done
    dev = _current()
    qp = _in_strided(q, "q", dev)
    kp = None if k is None else _in_strided(k, "k", dev)
    shape = q.shape
    k_shape = None if k is None else k.shape
    if len(shape) == 4:
        b_dim, s_dim, h_dim = (0, 1, 2) if layout == "bshd" else (0, 2, 1)
        B = shape[0]
        pos_shape = (B, shape[s_dim])
    elif len(shape) == 3 and layout == "bshd":
        b_dim, s_dim, h_dim = None, 0, 1
        B = 1
        pos_shape = (shape[0],)
    else:
        raise ValueError("q and k must be 4-D, or both packed [total, H, 128] (layout 'bshd')")
    S, Hq, d = shape[s_dim], shape[h_dim], shape[-1]
    Hkv = 0
    if k is not None:
        if len(k_shape) != len(shape) or k_shape[s_dim] != S or k_shape[-1] != d or (b_dim == 0 and k_shape[0] != B):
            raise ValueError("q and k must have the same batch, positions and head dimension")
        Hkv = k_shape[h_dim]
    args = _rotate_args(q_weight, k_weight, eps, positions, pos_shape, rope, interleaved, dev)
    if q_out is None:
        q_out = _empty(shape, _bf16, q.device, stream)
        qo = q_out.data_ptr()
    else:
        qo = _in(q_out, "q_out", _bf16, dev)
        if q_out.shape != shape:
            raise ValueError("q_out must have q's shape")
    ko = None
    if k_out is not None:
        ko = _in(k_out, "k_out", _bf16, dev)
        if k is None or k_out.shape != k_shape:
            raise ValueError("k_out must have k's shape")
    elif k is not None:
        k_out = _empty(k_shape, _bf16, q.device, stream)
        ko = k_out.data_ptr()
    # the stride of a dimension of length one is never used, whatever it says
    qs = q.stride()
    ks = (0,) * len(qs) if k is None else k.stride()
    many, long = b_dim == 0 and B > 1, S > 1
    rc = lib.attn_qk_norm_rope(
        qp, kp, qo, ko, *args, B, S, Hq, Hkv, d, LAYOUTS[layout], qs[0] if many else 0, qs[s_dim] if long else 0,
        qs[h_dim] if Hq > 1 else 0, ks[0] if many else 0, ks[s_dim] if long else 0, ks[h_dim] if Hkv > 1 else 0,
        _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "attn_qk_norm_rope")
    return q_out, k_out


def _append(fn, q, k, v, pools, Hkv_pool, num_pages, page_size, block_table, seqlens, cu_seqlens, rope, positions,
            q_weight, k_weight, eps, interleaved, q_out, stream, dev):
    qp = None if q is None else _in_strided(q, "q", dev)
    kp, vp = _in_strided(k, "k", dev), _in_strided(v, "v", dev)
    table, lens = _in(block_table, "block_table", _i32, dev), _in(seqlens, "seqlens", _i32, dev)
    cu = None if cu_seqlens is None else _in(cu_seqlens, "cu_seqlens", _i32, dev)
    shape, table_shape = k.shape, block_table.shape
    if len(shape) != 3 or v.shape != shape:
        raise ValueError("k and v must be [tokens, Hkv, 128], of the same shape")
    total, Hkv, d = shape
    B = seqlens.numel()
    ks, vs = k.stride(), v.stride()
    qs, Hq = None, 0
    if q is not None:
        q_shape, qs = q.shape, q.stride()
        if len(q_shape) != 3 or q_shape[0] != total or q_shape[2] != d:
            raise ValueError("q must be [tokens, Hq, 128], of the tokens and head dimension of k")
        Hq = q_shape[1]
    if (Hq > 1 and qs[1] != d) or (Hkv > 1 and (ks[1] != d or vs[1] != d)):
        raise ValueError("q, k and v must have the heads of a token contiguous")
    if Hkv != Hkv_pool:
        raise ValueError(f"the cache has {Hkv_pool} KV heads, k and v have {Hkv}")
    if len(table_shape) != 2 or table_shape[0] != B:
        raise ValueError("block_table must have one row per sequence")
    if cu is None:
        if total != B:
            raise ValueError("without cu_seqlens there is one new token per sequence")
    elif cu_seqlens.numel() != B + 1:
        raise ValueError("cu_seqlens must have B + 1 entries")
    qo = None
    if q_out is not None:
        qo = _in(q_out, "q_out", _bf16, dev)
        if q is None or q_out.shape != q_shape:
            raise ValueError("q_out must have q's shape")
    args = _rotate_args(q_weight, k_weight, eps, positions, (total,), rope, interleaved, dev)
    if q is not None and q_out is None:
        q_out = _empty(q_shape, _bf16, q.device, stream)
        qo = q_out.data_ptr()
    rc = fn(qp, kp, vp, qo, *pools, table, lens, cu, *args, B, total, Hq, Hkv, d, page_size, num_pages,
            table_shape[1], *((0 if q is None else qs[0], ks[0], vs[0]) if total > 1 else (Hq * d, Hkv * d, Hkv * d)),
            _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, fn.__name__)
    return q_out


def append_paged(q, k, v, k_pages, v_pages, block_table, seqlens, cu_seqlens=None, *, rope=None, positions=None,
                 q_weight=None, k_weight=None, eps=1e-6, interleaved=False, q_out=None, stream=None):
    """Write new tokens' keys and values into the paged cache, with the norm and rotation of qk_norm_rope on the way.

    q [total, Hq, 128] (or None), k and v [total, Hkv, 128] bf16, the sequences' new tokens back to back (views of a
    fused projection need no copy); k_pages, v_pages [num_pages, 16, Hkv, 128] bf16, updated in place; block_table
    [B, max_blocks], seqlens [B] (the lengths WITH the new tokens) and cu_seqlens [B + 1] int32 (None: one token per
    sequence, none where the length is 0).  positions: int32 [total] or [axes, total], default: each token's position in its cache.  Returns
    q_out [total, Hq, 128] (None without q): the q of fwd_paged or decode_paged over the same arrays.
    """
    lib = _lib or load()
    if stream is None:
        done = _quick.append(q, k, v, k_pages, v_pages, block_table, seqlens, cu_seqlens, q_weight, k_weight, eps,
                             positions, rope, interleaved, q_out) if v_pages is not None else None
        if done is not None:
            return done[0]
    dev = _current()
    pools = _in(k_pages, "k_pages", _bf16, dev), _in(v_pages, "v_pages", _bf16, dev)
    shape = k_pages.shape
    if len(shape) != 4 or v_pages.shape != shape:
        raise ValueError("k_pages and v_pages must be [num_pages, 16, Hkv, 128]")
    num_pages, page_size, Hkv, d = shape
    if d != 128:
        raise ValueError("k_pages and v_pages must be [num_pages, 16, Hkv, 128]")
    return _append(lib.attn_append_paged, q, k, v, pools, Hkv, num_pages, page_size, block_table, seqlens, cu_seqlens,
                   rope, positions, q_weight, k_weight, eps, interleaved, q_out, stream, dev)


def _q4_cache(cache, dev):
    """Address, pages and KV heads of a 4-bit cache."""
    ptr = _in(cache, "cache", torch.uint8, dev)
    shape = cache.shape
    if len(shape) != 3 or shape[2] != Q4_BLOCK_BYTES:
        raise ValueError(f"cache must be [num_pages, Hkv, {Q4_BLOCK_BYTES}]")
    return ptr, shape[0], shape[1]


def append_paged_q4(q, k, v, cache, block_table, seqlens, cu_seqlens=None, *, rope=None, positions=None,
                    q_weight=None, k_weight=None, eps=1e-6, interleaved=False, q_out=None, stream=None):
    """append_paged into a cache held in 4 bits: cache [num_pages, Hkv, Q4_BLOCK_BYTES] uint8, updated in place."""
    lib = _lib or load()
    if stream is None:
        done = _quick.append(q, k, v, cache, None, block_table, seqlens, cu_seqlens, q_weight, k_weight, eps, positions,
                             rope, interleaved, q_out)
        if done is not None:
            return done[0]
    dev = _current()
    ptr, num_pages, Hkv = _q4_cache(cache, dev)
    return _append(lib.attn_append_paged_q4, q, k, v, (ptr,), Hkv, num_pages, 16, block_table, seqlens, cu_seqlens,
                   rope, positions, q_weight, k_weight, eps, interleaved, q_out, stream, dev)


def gather_paged_q4(cache, block_table, seqlens, cu_seqlens_k, *, total_k=None, k_out=None, v_out=None, stream=None):
    """Read sequences back from a 4-bit cache: (k, v) bf16 [total_k, Hkv, 128], sequence b's seqlens[b] tokens from row
    cu_seqlens_k[b] on -- the k and v of fwd_varlen.  total_k, when omitted, is read from the outputs given or the
    offsets (a synchronisation)."""
    lib = _lib or load()
    if stream is None:
        done = _quick.gather(cache, block_table, seqlens, cu_seqlens_k, total_k, k_out, v_out)
        if done is not None:
            return done
    dev = _current()
    ptr, num_pages, Hkv = _q4_cache(cache, dev)
    table, lens = _in(block_table, "block_table", _i32, dev), _in(seqlens, "seqlens", _i32, dev)
    cu = _in(cu_seqlens_k, "cu_seqlens_k", _i32, dev)
    table_shape = block_table.shape
    B = seqlens.numel()
    if len(table_shape) != 2 or table_shape[0] != B or cu_seqlens_k.numel() != B + 1:
        raise ValueError("block_table must have B rows and cu_seqlens_k B + 1 entries")
    for o, n in ((k_out, "k_out"), (v_out, "v_out")):
        if o is not None:
            _in(o, n, _bf16, dev)
            if o.dim() != 3 or o.shape[1:] != (Hkv, 128) or (total_k is not None and o.shape[0] != total_k):
                raise ValueError(f"{n} must be [total_k, Hkv, 128]")
            total_k = o.shape[0]
    if total_k is None:
        total_k = max(1, int(cu_seqlens_k[-1]))
    if k_out is None:
        k_out = _empty((total_k, Hkv, 128), _bf16, cache.device, stream)
    if v_out is None:
        v_out = _empty((total_k, Hkv, 128), _bf16, cache.device, stream)
    rc = lib.attn_gather_paged_q4(ptr, table, lens, cu, k_out.data_ptr(), v_out.data_ptr(), B, Hkv, total_k, 128, 16,
                                  num_pages, table_shape[1], _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "attn_gather_paged_q4")
    return k_out, v_out


def decode_q4_workspace_bytes(B: int, Hq: int, Hkv: int, d: int, max_blocks_per_seq: int) -> int:
    """Device workspace bytes decode_paged_q4 needs for this shape."""
    return int(load().attn_decode_q4_workspace_bytes(B, Hq, Hkv, d, max_blocks_per_seq))


def _attn_out(out, lse, shape, lse_shape, device, stream, dev):
    """out and lse as given (checked) or made, and their addresses."""
    if out is None:
        out = _empty(shape, _bf16, device, stream)
        op = out.data_ptr()
    else:
        op = _in(out, "out", _bf16, dev)
        if out.shape != shape:
            raise ValueError(f"out must be {list(shape)}")
    if lse is None:
        lse = _empty(lse_shape, torch.float32, device, stream)
        return out, lse, op, lse.data_ptr()
    if lse is False:
        return out, None, op, None
    lp = _in(lse, "lse", torch.float32, dev)
    if lse.shape != lse_shape:
        raise ValueError(f"lse must be {list(lse_shape)}")
    return out, lse, op, lp


def decode_paged_q4(q, cache, block_table, seqlens, *, scale=None, out=None, lse=None, workspace=None, stream=None):
    """One decode step over a cache held in 4 bits (the arguments of decode_paged, with one cache tensor
    [num_pages, Hkv, Q4_BLOCK_BYTES] uint8).  Returns (out [B, Hq, 128] bf16, lse [B, Hq] fp32)."""
    lib = _lib or load()
    if stream is None:
        done = _quick.decode(q, scale, out, lse, cache, block_table, seqlens, workspace)
        if done is not None:
            return done
    dev = _current()
    ptr, num_pages, Hkv = _q4_cache(cache, dev)
    qp = _in(q, "q", _bf16, dev)
    table, lens = _in(block_table, "block_table", _i32, dev), _in(seqlens, "seqlens", _i32, dev)
    shape, table_shape = q.shape, block_table.shape
    if len(shape) != 3 or len(table_shape) != 2 or table_shape[0] != shape[0] or seqlens.numel() != shape[0]:
        raise ValueError("q must be [B, Hq, 128], block_table [B, max_blocks] and seqlens [B]")
    B, Hq, d = shape
    out, lse, op, lp = _attn_out(out, lse, shape, (B, Hq), q.device, stream, dev)
    if workspace is None:
        need = lib.attn_decode_q4_workspace_bytes(B, Hq, Hkv, d, table_shape[1])
        workspace = _empty(max(need, 1), torch.uint8, q.device, stream)
        wp = workspace.data_ptr()
    else:
        wp = _in(workspace, "workspace", torch.uint8, dev)
    rc = lib.attn_decode_paged_q4(qp, ptr, table, lens, op, lp, B, Hq, Hkv, d, 16, num_pages, table_shape[1],
                                  1.0 / math.sqrt(d) if scale is None else scale, wp, workspace.numel(),
                                  _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "attn_decode_paged_q4")
    return out, lse


def fwd_paged_q4_workspace_bytes(B: int, Hkv: int, d: int, max_total_k: int) -> int:
    """Device workspace bytes fwd_paged_q4 needs for caches of max_total_k tokens in all."""
    return int(load().attn_fwd_paged_q4_workspace_bytes(B, Hkv, d, max_total_k))


def fwd_paged_q4(q, cache, block_table, seqlens_k, cu_seqlens_q, *, max_seqlen_q=None, max_total_k=None, causal=True,
                 scale=None, out=None, lse=None, workspace=None, stream=None, rounding="rtne"):
    """Prefill of packed query chunks against a cache held in 4 bits (the arguments of fwd_paged, with one cache tensor
    [num_pages, Hkv, Q4_BLOCK_BYTES] uint8).  max_total_k bounds the sum of seqlens_k; it and max_seqlen_q, when
    omitted, are read from the device (a synchronisation).  Returns (out [total_q, Hq, 128] bf16, lse [Hq, total_q])."""
    lib = _lib or load()
    if rounding not in ROUNDING:
        raise ValueError(f"rounding must be one of {sorted(ROUNDING)}, got {rounding!r}")
    if stream is None:
        done = _quick.fwd(q, scale, out, lse, cache, block_table, seqlens_k, workspace, cu_seqlens_q, max_seqlen_q,
                          max_total_k, causal, ROUNDING[rounding])
        if done is not None:
            return done
    dev = _current()
    ptr, num_pages, Hkv = _q4_cache(cache, dev)
    qp = _in(q, "q", _bf16, dev)
    table, lens = _in(block_table, "block_table", _i32, dev), _in(seqlens_k, "seqlens_k", _i32, dev)
    cu = _in(cu_seqlens_q, "cu_seqlens_q", _i32, dev)
    shape, table_shape = q.shape, block_table.shape
    B = seqlens_k.numel()
    if len(shape) != 3:
        raise ValueError("q must be [total_q, Hq, 128]")
    if cu_seqlens_q.numel() != B + 1 or len(table_shape) != 2 or table_shape[0] != B:
        raise ValueError("cu_seqlens_q must have B + 1 entries and block_table B rows")
    total_q, Hq, d = shape
    if max_seqlen_q is None:
        max_seqlen_q = max(1, int(torch.diff(cu_seqlens_q).max()))
    if max_total_k is None:
        max_total_k = max(1, int(seqlens_k.sum()))
    out, lse, op, lp = _attn_out(out, lse, shape, (Hq, total_q), q.device, stream, dev)
    if workspace is None:
        need = lib.attn_fwd_paged_q4_workspace_bytes(B, Hkv, d, max_total_k)
        workspace = _empty(max(need, 1), torch.uint8, q.device, stream)
        wp = workspace.data_ptr()
    else:
        wp = _in(workspace, "workspace", torch.uint8, dev)
    rc = lib.attn_fwd_paged_q4(qp, ptr, table, lens, cu, op, lp, B, Hq, Hkv, total_q, max_seqlen_q, d, 16, num_pages,
                               table_shape[1], max_total_k, bool(causal), 1.0 / math.sqrt(d) if scale is None else scale,
                               ROUNDING[rounding], wp, workspace.numel(),
                               _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "attn_fwd_paged_q4")
    return out, lse


TREE_MAX = 256  # tokens of a sequence's tree (ATTN_TREE_MAX)


def fwd_tree_paged_workspace_bytes(B: int, Hq: int, Hkv: int, d: int, max_seqlen_q: int) -> int:
    """Device workspace bytes fwd_tree_paged needs for this shape."""
    return int(load().attn_fwd_tree_paged_workspace_bytes(B, Hq, Hkv, d, max_seqlen_q))


def fwd_tree_paged(q, k_pages, v_pages, block_table, seqlens_k, cu_seqlens_q, parents, *, max_seqlen_q=None, scale=None,
                   out=None, lse=None, workspace=None, stream=None, rounding="rtne"):
    """Attention of trees of drafted tokens against a paged KV cache (the tensors of fwd_paged; a sequence's tree is the
    last tokens of its cache).

    parents [total_q] int32: each token's parent by its place in its own sequence's tree, before its own, or -1.  A token
    sees the keys before the tree, itself and its ancestors.  A tree has at most TREE_MAX tokens; max_seqlen_q, when
    omitted, is read from the offsets (a synchronisation).  Returns (out [total_q, Hq, 128] bf16, lse [Hq, total_q]).
    """
    lib = _lib or load()
    if rounding not in ROUNDING:
        raise ValueError(f"rounding must be one of {sorted(ROUNDING)}, got {rounding!r}")
    if stream is None:
        done = _quick.tree(q, scale, out, lse, k_pages, v_pages, block_table, seqlens_k, cu_seqlens_q, parents,
                           max_seqlen_q, workspace, ROUNDING[rounding])
        if done is not None:
            return done
    dev = _current()
    qp, kp, vp = _in(q, "q", _bf16, dev), _in(k_pages, "k_pages", _bf16, dev), _in(v_pages, "v_pages", _bf16, dev)
    table, lens = _in(block_table, "block_table", _i32, dev), _in(seqlens_k, "seqlens_k", _i32, dev)
    cu, par = _in(cu_seqlens_q, "cu_seqlens_q", _i32, dev), _in(parents, "parents", _i32, dev)
    shape, pool, table_shape = q.shape, k_pages.shape, block_table.shape
    B = seqlens_k.numel()
    if len(shape) != 3 or len(pool) != 4 or v_pages.shape != pool or pool[3] != shape[2]:
        raise ValueError("q must be [total_q, Hq, 128] and the pools [num_pages, 16, Hkv, 128]")
    total_q, Hq, d = shape
    num_pages, page_size, Hkv, _ = pool
    if cu_seqlens_q.numel() != B + 1 or len(table_shape) != 2 or table_shape[0] != B:
        raise ValueError("cu_seqlens_q must have B + 1 entries and block_table B rows")
    if parents.numel() != total_q:
        raise ValueError("parents must have one entry per row of q")
    if max_seqlen_q is None:
        max_seqlen_q = max(1, int(torch.diff(cu_seqlens_q).max()))
    out, lse, op, lp = _attn_out(out, lse, shape, (Hq, total_q), q.device, stream, dev)
    if workspace is None:
        need = lib.attn_fwd_tree_paged_workspace_bytes(B, Hq, Hkv, d, max_seqlen_q)
        workspace = _empty(max(need, 1), torch.uint8, q.device, stream)
        wp = workspace.data_ptr()
    else:
        wp = _in(workspace, "workspace", torch.uint8, dev)
    rc = lib.attn_fwd_tree_paged(qp, kp, vp, table, lens, cu, par, op, lp, B, Hq, Hkv, total_q, max_seqlen_q, d,
                                 page_size, num_pages, table_shape[1], 1.0 / math.sqrt(d) if scale is None else scale,
                                 ROUNDING[rounding], wp, workspace.numel(),
                                 _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "attn_fwd_tree_paged")
    return out, lse


_DTYPES = {torch.bfloat16: 0, torch.float32: 1}


def _rows(t, name, dtype, dev, shape):
    """Address and row stride of a [rows, vocab] tensor whose rows are contiguous."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.dim() == 2 and t.stride(1) == 1:
            if t.shape != shape:
                raise ValueError(f"{name} must be {list(shape)}")
            return t.data_ptr(), t.stride(0) if shape[0] > 1 else shape[1]
    except AttributeError:
        pass  # not a tensor
    _refuse(t, name, dtype, dev, contiguous=False)


def _out_i32(t, name, shape, like, stream, dev):
    """An int32 output as given (checked) or made, and its address."""
    if t is None:
        t = _empty(shape, _i32, like.device, stream)
        return t, t.data_ptr()
    ptr = _in(t, name, _i32, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    return t, ptr


def verify_tree_workspace_bytes(B: int, total: int, vocab: int, max_seqlen: int, dtype=torch.bfloat16,
                                with_draft: bool = False) -> int:
    """Device workspace bytes verify_tree needs for this shape."""
    return int(load().attn_verify_tree_workspace_bytes(B, total, vocab, max_seqlen, _DTYPES[dtype], int(with_draft)))


def verify_tree(logits, tokens, parents, cu_seqlens, *, draft_logits=None, temperature=None, uniforms=None, noise=None,
                max_seqlen=None, path=None, out_tokens=None, counts=None, workspace=None, stream=None):
    """Which drafted tokens of each sequence's tree are kept, and the token that follows them, from given random numbers.

    logits [total, vocab] bf16 or fp32 (rows may be strided): the target's at every node; tokens, parents [total] and
    cu_seqlens [B + 1] int32: the trees, each root first (the token emitted last) and every node behind its parent.
    draft_logits: the distributions that every node's children were drawn from, like logits; None where they were chosen
    in another way.  temperature [B] fp32 (<= 0: the largest logit), uniforms [total] fp32 in [0, 1) and noise
    [B, vocab] fp32, exponential numbers; without temperature every sequence takes its largest logits and there are no
    draft_logits, uniforms or noise.  max_seqlen (at most TREE_MAX), when omitted, is read from the offsets (a
    synchronisation).

    Returns (path, out_tokens, counts): int32 [B, max_seqlen] with counts[b] entries each and -1 behind, the kept nodes
    (the root first) and the emitted tokens (those of the kept nodes after the root, and the last one).  Outputs that are
    given must not overlap an input or one another.
    """
    lib = _lib or load()
    if stream is None:
        done = _quick.verify(logits, tokens, parents, cu_seqlens, draft_logits, temperature, uniforms, noise, max_seqlen,
                             path, out_tokens, counts, workspace)
        if done is not None:
            return done
    dev = _current()
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda or logits.dtype not in _DTYPES:
        raise TypeError("logits must be a CUDA tensor of bfloat16 or float32")
    dtype, shape = logits.dtype, logits.shape
    if len(shape) != 2:
        raise ValueError("logits must be [total, vocab]")
    total, vocab = shape
    lp, ls = _rows(logits, "logits", dtype, dev, shape)
    tok, par = _in(tokens, "tokens", _i32, dev), _in(parents, "parents", _i32, dev)
    cu = _in(cu_seqlens, "cu_seqlens", _i32, dev)
    B = cu_seqlens.numel() - 1
    if tokens.numel() != total or parents.numel() != total or B < 1:
        raise ValueError("tokens and parents must have one entry per row of logits, cu_seqlens B + 1")
    dp = tp = up = np_ = None
    ds = ns = 0
    if temperature is None:
        if draft_logits is not None or uniforms is not None or noise is not None:
            raise ValueError("draft_logits, uniforms and noise go with a temperature")
    else:
        tp = _in(temperature, "temperature", torch.float32, dev)
        if uniforms is None or noise is None:
            raise ValueError("drawing (temperature) needs uniforms and noise")
        up = _in(uniforms, "uniforms", torch.float32, dev)
        np_, ns = _rows(noise, "noise", torch.float32, dev, (B, vocab))
        if temperature.numel() != B or uniforms.numel() != total:
            raise ValueError("temperature must have B entries and uniforms one per row of logits")
        if draft_logits is not None:
            dp, ds = _rows(draft_logits, "draft_logits", dtype, dev, shape)
    if max_seqlen is None:
        max_seqlen = max(1, int(torch.diff(cu_seqlens).max()))
    path, pp = _out_i32(path, "path", (B, max_seqlen), logits, stream, dev)
    out_tokens, op = _out_i32(out_tokens, "out_tokens", (B, max_seqlen), logits, stream, dev)
    counts, cp = _out_i32(counts, "counts", (B,), logits, stream, dev)
    if workspace is None:
        need = lib.attn_verify_tree_workspace_bytes(B, total, vocab, max_seqlen, _DTYPES[dtype], dp is not None)
        workspace = _empty(max(need, 1), torch.uint8, logits.device, stream)
        wp = workspace.data_ptr()
    else:
        wp = _in(workspace, "workspace", torch.uint8, dev)
    rc = lib.attn_verify_tree(lp, dp, _DTYPES[dtype], tok, par, cu, tp, up, np_, pp, op, cp, B, total, vocab, max_seqlen,
                              ls, ds, ns, wp, workspace.numel(), _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "attn_verify_tree")
    return path, out_tokens, counts


def compact_paged(k_pages, v_pages, block_table, seqlens_k, cu_seqlens, path, counts, *, total=None, seqlens_out=None,
                  stream=None):
    """Cut a paged cache down to the accepted path of each sequence's tree (path and counts of verify_tree).

    k_pages, v_pages [num_pages, 16, Hkv, 128] or [layers, num_pages, 16, Hkv, 128] bf16, updated in place; block_table,
    seqlens_k (with the trees) and cu_seqlens as for fwd_tree_paged.  The kept nodes' keys and values move to the tree's
    first places.  total bounds the offsets (default: B times path's width).  Returns the new lengths, int32 [B]
    (seqlens_out, which must not overlap an input).
    """
    lib = _lib or load()
    if stream is None:
        done = _quick.compact(k_pages, v_pages, block_table, seqlens_k, cu_seqlens, path, counts, total, seqlens_out)
        if done is not None:
            return done[0]
    dev = _current()
    kp, vp = _in(k_pages, "k_pages", _bf16, dev), _in(v_pages, "v_pages", _bf16, dev)
    table, lens = _in(block_table, "block_table", _i32, dev), _in(seqlens_k, "seqlens_k", _i32, dev)
    cu, pt, ct = _in(cu_seqlens, "cu_seqlens", _i32, dev), _in(path, "path", _i32, dev), _in(counts, "counts", _i32, dev)
    pool, table_shape, path_shape = k_pages.shape, block_table.shape, path.shape
    B = seqlens_k.numel()
    if len(pool) not in (4, 5) or v_pages.shape != pool:
        raise ValueError("k_pages and v_pages must be [num_pages, 16, Hkv, 128] or [layers, num_pages, 16, Hkv, 128]")
    layers = 1 if len(pool) == 4 else pool[0]
    num_pages, page_size, Hkv, d = pool[-4:]
    if len(table_shape) != 2 or table_shape[0] != B or cu_seqlens.numel() != B + 1:
        raise ValueError("block_table must have B rows and cu_seqlens B + 1 entries")
    if len(path_shape) != 2 or path_shape[0] != B or counts.numel() != B:
        raise ValueError("path must be [B, max_seqlen] and counts [B]")
    if total is None:
        total = max(1, B * path_shape[1])
    seqlens_out, sp = _out_i32(seqlens_out, "seqlens_out", (B,), k_pages, stream, dev)
    rc = lib.attn_compact_paged(kp, vp, table, lens, cu, pt, ct, sp, B, layers, Hkv, total, path_shape[1], d, page_size,
                                num_pages, table_shape[1], _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "attn_compact_paged")
    return seqlens_out


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
