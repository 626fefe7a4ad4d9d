"""ctypes binding of libpgd (include/pgd.h).  Argument marshalling only: every
step of the path runs in the library's CUDA kernels; there is no fallback.
The library is loaded on first use and a missing build is an error."""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading
from typing import Optional, Sequence, Tuple

import torch

from . import build as _build

_lock = threading.Lock()
_lib: Optional[ctypes.CDLL] = None

HEAD_DIM = 128

# status codes (pgd_status)
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_OUT_OF_BLOCKS, ERR_WORKSPACE, ERR_CUDA, \
    ERR_BLOCK_STATE = range(7)
# device error bits (PGD_DEVERR_*)
DEVERR_BAD_BLOCK_ID, DEVERR_BAD_CONTEXT, DEVERR_BAD_POSITION, DEVERR_TIMEOUT = 1, 2, 4, 8

#: every symbol include/pgd.h declares, with (argtypes, restype)
_P, _I, _F, _Z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
_D = ctypes.c_double
SIGNATURES = {
    "pgd_status_string": ([_I], ctypes.c_char_p),
    "pgd_last_error_detail": ([], ctypes.c_char_p),
    "pgd_version": ([], _I),
    "pgd_kv_append": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P], _I),
    "pgd_attention_workspace_size": ([_I, _I, _I, _I, _I], _Z),
    "pgd_paged_decode_attention": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I,
                                    _P, _Z, _P], _I),
    "pgd_attention_grid": ([_I, _I, _I, _I, _I], _I),
    "pgd_paged_decode_attention_noalloc": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I,
                                            _F, _I, _P], _I),
    "pgd_append_decode_attention": ([_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I,
                                     _F, _I, _P, _Z, _P], _I),
    "pgd_kv_append_tokens": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P], _I),
    "pgd_verify_workspace_size": ([_I, _I, _I, _I, _I, _I], _Z),
    "pgd_paged_verify_attention": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F,
                                    _I, _P, _Z, _P], _I),
    "pgd_append_verify_attention": ([_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I,
                                     _I, _F, _I, _P, _Z, _P], _I),
    "pgd_verify_step": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I,
                         _I, _I, _I, _F, _I, _P, _Z, _P], _I),
    "pgd_mla_workspace_size": ([_I, _I, _I], _Z),
    "pgd_mla_append": ([_P, _P, _P, _P, _I, _I, _I, _I, _I, _P], _I),
    "pgd_mla_decode_attention": ([_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P, _Z,
                                  _P], _I),
    "pgd_mla_append_decode_attention": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F,
                                         _I, _P, _Z, _P], _I),
    "pgd_mla_step": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I,
                      _P, _Z, _P], _I),
    "pgd_cascade_workspace_size": ([_I, _I, _I, _I, _I, _I, _I, _I], _Z),
    "pgd_cascade_decode_attention": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I,
                                      _I, _I, _I, _I, _I, _F, _I, _P, _Z, _P], _I),
    "pgd_kv_append_fp8": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P], _I),
    "pgd_paged_decode_attention_fp8": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F,
                                        _I, _P, _Z, _P], _I),
    "pgd_append_decode_attention_fp8": ([_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I,
                                         _I, _F, _I, _P, _Z, _P], _I),
    "pgd_decode_step": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I,
                         _I, _I, _F, _I, _P, _Z, _P], _I),
    "pgd_decode_step_fp8": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I,
                             _I, _I, _I, _F, _I, _P, _Z, _P], _I),
    "pgd_block_workspace_size": ([_I, _I, _I, _I, _I], _Z),
    "pgd_kv_append_fp8b": ([_P] * 9 + [_I] * 8 + [_P], _I),
    "pgd_kv_read_fp8b": ([_P] * 9 + [_I] * 8 + [_P], _I),
    "pgd_paged_decode_attention_fp8b": ([_P] * 8 + [_I] * 7 + [_F, _I, _P, _Z, _P], _I),
    "pgd_append_decode_attention_fp8b": ([_P] * 10 + [_I] * 7 + [_F, _I, _P, _Z, _P], _I),
    "pgd_block_bounds": ([_P] * 7 + [_I] * 7 + [_P], _I),
    "pgd_select_blocks": ([_P] * 7 + [_I] * 10 + [_P], _I),
    "pgd_selected_decode_attention": ([_P] * 8 + [_I] * 7 + [_F, _I, _P, _Z, _P], _I),
    "pgd_sparse_decode_attention": ([_P] * 12 + [_I] * 10 + [_F, _I, _P, _Z, _P], _I),
    "pgd_fp4_workspace_size": ([_I, _I, _I, _I, _I], _Z),
    "pgd_kv_append_fp4": ([_P] * 7 + [_I] * 8 + [_F, _F, _P], _I),
    "pgd_kv_read_fp4": ([_P] * 7 + [_I] * 8 + [_F, _F, _P], _I),
    "pgd_paged_decode_attention_fp4": ([_P] * 6 + [_I] * 7 + [_F, _F, _F, _I, _P, _Z, _P], _I),
    "pgd_append_decode_attention_fp4": ([_P] * 8 + [_I] * 7 + [_F, _F, _F, _I, _P, _Z, _P], _I),
    "pgd_rope_frequencies": ([_P, _I, _D, _I, _D, _D, _D, _D], _I),
    "pgd_rope": ([_P] * 6 + [_I] * 7 + [_F, _P, _P], _I),
    "pgd_rope_append": ([_P] * 9 + [_I] * 9 + [_F, _P, _P], _I),
    "pgd_grow_tables": ([_P] * 12 + [_I] * 5 + [_P], _I),
    "pgd_trim_tables": ([_P] * 5 + [_I] * 4 + [_P], _I),
    "pgd_copy_blocks_fp4": ([_P, _P, _P, _P, _I, _I, _I, _I, _I, _P], _I),
    "pgd_copy_blocks": ([_P, _P, _P, _P, _I, _I, _I, _I, _I, _P], _I),
    "pgd_device_errors": ([_P, _I, _P], _I),
    "pgd_read_stream": ([_P, _Z, _I, _P], _I),
    "pgd_set_wait_limit_ns": ([ctypes.c_uint64], None),
    "pgd_wait_limit_ns": ([], ctypes.c_uint64),
    "pgd_set_short_context_tokens": ([_I], _I),
    "pgd_short_path": ([_I, _I, _I, _I, _I], _I),
    "pgd_alloc_create": ([_I, _P], _I),
    "pgd_alloc_destroy": ([_P], None),
    "pgd_alloc_allocate": ([_P, _I, _P], _I),
    "pgd_alloc_share": ([_P, _P, _I], _I),
    "pgd_alloc_release": ([_P, _P, _I], _I),
    "pgd_alloc_refcount": ([_P, _I], _I),
    "pgd_alloc_num_free": ([_P], _I),
    "pgd_alloc_num_blocks": ([_P], _I),
    "pgd_alloc_append_slot": ([_P, _P, _I, _I, _I, _P, _P], _I),
    "pgd_alloc_fork": ([_P, _P, _I, _I, _P, _I], _I),
    "pgd_validate_tables": ([_P, _P, _I, _I, _I, _I], _I),
}


class PGDError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__("pgd status %d: %s" % (status, detail))
        self.status = status
        self.detail = detail


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """The loaded libpgd.  Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    "libpgd.so is not built (%s); run paged_gqa_decode_kv_gb300.build.build() "
                    "or __graft_entry__.build()" % path)
            L = ctypes.CDLL(path)
            for name, (args, res) in SIGNATURES.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = res
            _lib = L
        return _lib


def _check(status: int) -> None:
    if status != OK:
        L = lib()
        raise PGDError(status, "%s: %s" % (L.pgd_status_string(status).decode(),
                                           L.pgd_last_error_detail().decode()))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _made_for(stream, make, result: bool = False) -> torch.Tensor:
    """A buffer that a call on `stream` makes itself: allocated and filled on
    that stream, so that the call finds it filled and its memory is not given
    to other work before the call is done.  result: the caller keeps it, and
    reads it on the current stream."""
    if stream is None:
        return make()
    current = torch.cuda.current_stream()
    if stream.cuda_stream == current.cuda_stream:
        return make()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    with torch.cuda.stream(stream):
        t = make()
    if result and t.is_cuda:
        t.record_stream(current)
    return t


def _need(t: torch.Tensor, dtype: torch.dtype, name: str, cuda: bool = True) -> None:
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if cuda and not t.is_cuda:
        raise ValueError("%s must be on a CUDA device" % name)


def _cache_dims(k_cache: torch.Tensor) -> Tuple[int, int, int, int]:
    """(NB, n_kv, bs, d) of a pool [NB][n_kv][bs/8][d/8][8][8] (each (block,
    head) tile stored as 8x8 core matrices)."""
    if k_cache.dim() != 6 or tuple(k_cache.shape[4:]) != (8, 8):
        raise ValueError("cache must be [NB][n_kv][bs/8][d/8][8][8]")
    NB, n_kv, rg, nc = k_cache.shape[:4]
    return NB, n_kv, rg * 8, nc * 8


# --------------------------------------------------------------------- GPU ops
def kv_append(k_new, v_new, k_cache, v_cache, block_tables, positions, stream=None) -> None:
    """Write k_new/v_new [B][n_kv][d] at logical positions[b] of every sequence."""
    for t, n in ((k_new, "k_new"), (v_new, "v_new"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, torch.bfloat16, n)
    _need(block_tables, torch.int32, "block_tables")
    _need(positions, torch.int32, "positions")
    NB, n_kv, bs, d = _cache_dims(k_cache)
    B, MB = block_tables.shape
    _check(lib().pgd_kv_append(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                               _ptr(block_tables), _ptr(positions), B, n_kv, d, bs, MB, NB,
                               _stream(stream)))


def workspace_size(B: int, n_q: int, n_kv: int, num_splits: int = 0, d: int = HEAD_DIM) -> int:
    return int(lib().pgd_attention_workspace_size(B, n_q, n_kv, d, num_splits))


def make_workspace(B: int, n_q: int, n_kv: int, num_splits: int = 0, device=None) -> torch.Tensor:
    """A zero-filled workspace for these shapes (torch allocations are
    256-byte aligned)."""
    n = max(1, workspace_size(B, n_q, n_kv, num_splits))
    return torch.zeros(n, dtype=torch.uint8, device=device or torch.device("cuda"))


def attention_grid(B: int, n_q: int, n_kv: int, bs: int, num_splits: int = 0) -> int:
    return int(lib().pgd_attention_grid(B, n_q, n_kv, bs, num_splits))


def _attention_call(fp8, out, q, k_cache, v_cache, block_tables, context_lens, scale,
                    num_splits=0, workspace=None, stream=None):
    _need(q, torch.bfloat16, "q")
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, torch.uint8 if fp8 else torch.bfloat16, n)
    _need(block_tables, torch.int32, "block_tables")
    _need(context_lens, torch.int32, "context_lens")
    B, n_q, d = q.shape
    NB, n_kv, bs, _ = _cache8_dims(k_cache) if fp8 else _cache_dims(k_cache)
    if out is None:
        out = _made_for(stream, lambda: torch.empty_like(q), result=True)
    _need(out, torch.bfloat16, "out")
    if workspace is None:
        workspace = _made_for(stream, lambda: make_workspace(B, n_q, n_kv, num_splits, q.device))
    MB = block_tables.shape[1]
    name = "pgd_paged_decode_attention_fp8" if fp8 else "pgd_paged_decode_attention"
    return name, (
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
        B, n_q, n_kv, d, bs, MB, NB, float(scale), int(num_splits), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)), out, workspace


def paged_decode_attention(out, q, k_cache, v_cache, block_tables, context_lens, scale: float,
                           num_splits: int = 0, workspace: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """out[B][n_q][d] (bf16) = paged decode attention of q over the cache."""
    name, args, out, workspace = _attention_call(False, out, q, k_cache, v_cache, block_tables,
                                                 context_lens, scale, num_splits, workspace,
                                                 stream)
    _check(getattr(lib(), name)(*args))
    return out


def paged_decode_attention_noalloc(out, q, k_cache, v_cache, block_tables, context_lens,
                                   scale: float, num_splits: int = 0, stream=None) -> torch.Tensor:
    """paged_decode_attention without a workspace argument, for callers that
    cannot allocate device memory: the library keeps the scratch in its own
    fixed device array (shared by every call on a device; calls that overlap
    on one GPU race).  `out` must be given -- this call allocates nothing."""
    for t, n in ((out, "out"), (q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, torch.bfloat16, n)
    _need(block_tables, torch.int32, "block_tables")
    _need(context_lens, torch.int32, "context_lens")
    B, n_q, d = q.shape
    NB, n_kv, bs, _ = _cache_dims(k_cache)
    MB = block_tables.shape[1]
    _check(lib().pgd_paged_decode_attention_noalloc(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
        B, n_q, n_kv, d, bs, MB, NB, float(scale), int(num_splits), _stream(stream)))
    return out


def _append_attention_call(fp8, out, q, k_new, v_new, k_cache, v_cache, block_tables,
                           context_lens, scale, num_splits=0, workspace=None, stream=None):
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new")):
        _need(t, torch.bfloat16, n)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, torch.uint8 if fp8 else torch.bfloat16, n)
    _need(block_tables, torch.int32, "block_tables")
    _need(context_lens, torch.int32, "context_lens")
    B, n_q, d = q.shape
    NB, n_kv, bs, _ = _cache8_dims(k_cache) if fp8 else _cache_dims(k_cache)
    if out is None:
        out = _made_for(stream, lambda: torch.empty_like(q), result=True)
    _need(out, torch.bfloat16, "out")
    if workspace is None:
        workspace = _made_for(stream, lambda: make_workspace(B, n_q, n_kv, num_splits, q.device))
    MB = block_tables.shape[1]
    name = "pgd_append_decode_attention_fp8" if fp8 else "pgd_append_decode_attention"
    return name, (
        _ptr(out), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
        _ptr(block_tables), _ptr(context_lens), B, n_q, n_kv, d, bs, MB, NB, float(scale),
        int(num_splits), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)), out, workspace


def append_decode_attention(out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens,
                            scale: float, num_splits: int = 0,
                            workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """kv_append of k_new/v_new at context_lens - 1, then paged decode
    attention over the updated cache (one call; two kernels, the attention
    prologue overlapping the append, or one short-context kernel that
    appends itself)."""
    name, args, out, workspace = _append_attention_call(
        False, out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, scale,
        num_splits, workspace, stream)
    _check(getattr(lib(), name)(*args))
    return out


def _decode_step_call(out_h, q_h, k_new_h, v_new_h, context_lens_h, out_d, q_d, k_new_d,
                      v_new_d, context_lens_d, k_cache, v_cache, block_tables, scale, num_splits,
                      workspace, stream=None):
    for t, n in ((out_h, "out_h"), (q_h, "q_h"), (k_new_h, "k_new_h"), (v_new_h, "v_new_h")):
        _need(t, torch.bfloat16, n, cuda=False)
    _need(context_lens_h, torch.int32, "context_lens_h", cuda=False)
    B, n_q, d = q_h.shape
    fp8 = k_cache.dtype == torch.uint8
    NB, n_kv, bs, _ = _cache8_dims(k_cache) if fp8 else _cache_dims(k_cache)
    MB = block_tables.shape[1]
    name = "pgd_decode_step_fp8" if fp8 else "pgd_decode_step"
    return name, (
        _ptr(out_h), _ptr(q_h), _ptr(k_new_h), _ptr(v_new_h), _ptr(context_lens_h), _ptr(out_d),
        _ptr(q_d), _ptr(k_new_d), _ptr(v_new_d), _ptr(context_lens_d), _ptr(k_cache),
        _ptr(v_cache), _ptr(block_tables), B, n_q, n_kv, d, bs, MB, NB, float(scale),
        int(num_splits), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)), None, workspace


def decode_step(out_h, q_h, k_new_h, v_new_h, context_lens_h, out_d, q_d, k_new_d, v_new_d,
                context_lens_d, k_cache, v_cache, block_tables, scale: float, num_splits: int,
                workspace: torch.Tensor, stream=None) -> None:
    """One decode step with host inputs/outputs: append at context_lens - 1,
    then attention, all on `stream`.  Page-locked (pinned) host tensors are
    read and written in place by the kernels; pageable ones go through the
    given device tensors and a copy each.  An 8-bit pool (uint8) selects the
    FP8 path."""
    name, args, _, _ = _decode_step_call(out_h, q_h, k_new_h, v_new_h, context_lens_h, out_d, q_d,
                                         k_new_d, v_new_d, context_lens_d, k_cache, v_cache,
                                         block_tables, scale, num_splits, workspace, stream)
    _check(getattr(lib(), name)(*args))


class PreparedCall:
    """One C-ABI call whose arguments were checked and marshalled once;
    calling the object enqueues the same call again (same buffers, same
    stream) and returns its output tensor.  The Python side of a regular
    binding call -- a dozen tensor checks and pointer conversions -- takes
    about 10 us, longer than a short-context decode step on the GPU; a
    prepared call leaves only the C call (a few us).  The caller's buffers must
    stay alive and unchanged in shape while the object is used; the output and
    the workspace, which the call may have made itself, are held by it."""
    __slots__ = ("name", "_fn", "_args", "out", "workspace")

    def __init__(self, name: str, args: tuple, out=None, workspace=None):
        self.name = name
        self._fn = getattr(lib(), name)
        self._args = args
        self.out = out
        self.workspace = workspace

    def __call__(self):
        s = self._fn(*self._args)
        if s != OK:
            _check(s)
        return self.out


def prepare(op: str, *args, **kwargs) -> PreparedCall:
    """A PreparedCall of one of the step calls, with the arguments that call
    takes: "paged_decode_attention", "paged_decode_attention_fp8",
    "append_decode_attention", "append_decode_attention_fp8", "decode_step",
    "append_verify_attention", "verify_step", "paged_decode_attention_fp8b",
    "append_decode_attention_fp8b", "sparse_decode_attention",
    "paged_decode_attention_fp4" or "append_decode_attention_fp4"."""
    if op == "paged_decode_attention":
        return PreparedCall(*_attention_call(False, *args, **kwargs))
    if op == "paged_decode_attention_fp8":
        return PreparedCall(*_attention_call(True, *args, **kwargs))
    if op == "append_decode_attention":
        return PreparedCall(*_append_attention_call(False, *args, **kwargs))
    if op == "append_decode_attention_fp8":
        return PreparedCall(*_append_attention_call(True, *args, **kwargs))
    if op == "decode_step":
        return PreparedCall(*_decode_step_call(*args, **kwargs))
    if op == "append_verify_attention":
        return PreparedCall(*_append_verify_call(*args, **kwargs))
    if op == "verify_step":
        return PreparedCall(*_verify_step_call(*args, **kwargs))
    if op == "paged_decode_attention_fp8b":
        return PreparedCall(*_prepared8b(*args, **kwargs))
    if op == "append_decode_attention_fp8b":
        return PreparedCall(*_prepared_append8b(*args, **kwargs))
    if op == "sparse_decode_attention":
        return PreparedCall(*_prepared_sparse(*args, **kwargs))
    if op == "paged_decode_attention_fp4":
        return PreparedCall(*_prepared4(*args, **kwargs))
    if op == "append_decode_attention_fp4":
        return PreparedCall(*_prepared_append4(*args, **kwargs))
    raise ValueError("no prepared form of %r" % op)


# ---------------------------------------------------------------- cascade
def kv_append_tokens(k_new, v_new, k_cache, v_cache, block_tables, positions,
                     stream=None) -> None:
    """Write k_new/v_new [B][T][n_kv][d]: token j of sequence b at logical
    position positions[b] + j."""
    for t, n in ((k_new, "k_new"), (v_new, "v_new"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, torch.bfloat16, n)
    _need(block_tables, torch.int32, "block_tables")
    _need(positions, torch.int32, "positions")
    NB, n_kv, bs, d = _cache_dims(k_cache)
    B, MB = block_tables.shape
    T = k_new.shape[1]
    _check(lib().pgd_kv_append_tokens(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                      _ptr(block_tables), _ptr(positions), B, T, n_kv, d, bs, MB,
                                      NB, _stream(stream)))


def verify_workspace_size(B: int, T: int, n_q: int, n_kv: int, num_splits: int = 0,
                          d: int = HEAD_DIM) -> int:
    return int(lib().pgd_verify_workspace_size(B, T, n_q, n_kv, d, num_splits))


def paged_verify_attention(out, q, k_cache, v_cache, block_tables, context_lens, scale: float,
                           num_splits: int = 0, workspace: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """out[B][T][n_q][d] (bf16): each of the T new query tokens of a sequence
    attends to its cached context up to and including its own position."""
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, torch.bfloat16, n)
    _need(block_tables, torch.int32, "block_tables")
    _need(context_lens, torch.int32, "context_lens")
    B, T, n_q, d = q.shape
    NB, n_kv, bs, d2 = _cache_dims(k_cache)
    if out is None:
        out = _made_for(stream, lambda: torch.empty_like(q), result=True)
    _need(out, torch.bfloat16, "out")
    if workspace is None:
        n = max(1, verify_workspace_size(B, T, n_q, n_kv, num_splits))
        workspace = _made_for(stream, lambda: torch.zeros(n, dtype=torch.uint8, device=q.device))
    MB = block_tables.shape[1]
    _check(lib().pgd_paged_verify_attention(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
        B, T, n_q, n_kv, d, bs, MB, NB, float(scale), int(num_splits), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def _verify_workspace(workspace, B, T, n_q, n_kv, num_splits, device, stream):
    if workspace is None:
        n = max(1, verify_workspace_size(B, T, n_q, n_kv, num_splits))
        workspace = _made_for(stream, lambda: torch.zeros(n, dtype=torch.uint8, device=device))
    return workspace


def _append_verify_call(out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens,
                        scale, num_splits=0, workspace=None, stream=None):
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new"), (k_cache, "k_cache"),
                 (v_cache, "v_cache")):
        _need(t, torch.bfloat16, n)
    _need(block_tables, torch.int32, "block_tables")
    _need(context_lens, torch.int32, "context_lens")
    B, T, n_q, d = q.shape
    NB, n_kv, bs, _ = _cache_dims(k_cache)
    if out is None:
        out = _made_for(stream, lambda: torch.empty_like(q), result=True)
    _need(out, torch.bfloat16, "out")
    workspace = _verify_workspace(workspace, B, T, n_q, n_kv, num_splits, q.device, stream)
    MB = block_tables.shape[1]
    return "pgd_append_verify_attention", (
        _ptr(out), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
        _ptr(block_tables), _ptr(context_lens), B, T, n_q, n_kv, d, bs, MB, NB, float(scale),
        int(num_splits), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)), out, workspace


def append_verify_attention(out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens,
                            scale: float, num_splits: int = 0,
                            workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One verify step in one call: the T new tokens of every sequence
    (k_new/v_new [B][T][n_kv][d]) appended at context_lens - T + j, then
    paged_verify_attention over the updated caches (its prologue overlapping
    the append)."""
    name, args, out, workspace = _append_verify_call(
        out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, scale, num_splits,
        workspace, stream)
    _check(getattr(lib(), name)(*args))
    return out


def _verify_step_call(out_h, q_h, k_new_h, v_new_h, context_lens_h, out_d, q_d, k_new_d,
                      v_new_d, context_lens_d, k_cache, v_cache, block_tables, scale, num_splits,
                      workspace, stream=None):
    for t, n in ((out_h, "out_h"), (q_h, "q_h"), (k_new_h, "k_new_h"), (v_new_h, "v_new_h")):
        _need(t, torch.bfloat16, n, cuda=False)
    _need(context_lens_h, torch.int32, "context_lens_h", cuda=False)
    _need(k_cache, torch.bfloat16, "k_cache")
    B, T, n_q, d = q_h.shape
    NB, n_kv, bs, _ = _cache_dims(k_cache)
    MB = block_tables.shape[1]
    return "pgd_verify_step", (
        _ptr(out_h), _ptr(q_h), _ptr(k_new_h), _ptr(v_new_h), _ptr(context_lens_h), _ptr(out_d),
        _ptr(q_d), _ptr(k_new_d), _ptr(v_new_d), _ptr(context_lens_d), _ptr(k_cache),
        _ptr(v_cache), _ptr(block_tables), B, T, n_q, n_kv, d, bs, MB, NB, float(scale),
        int(num_splits), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)), None, workspace


def verify_step(out_h, q_h, k_new_h, v_new_h, context_lens_h, out_d, q_d, k_new_d, v_new_d,
                context_lens_d, k_cache, v_cache, block_tables, scale: float, num_splits: int,
                workspace: torch.Tensor, stream=None) -> None:
    """One verify step with host inputs/outputs (q and out [B][T][n_q][d],
    k_new/v_new [B][T][n_kv][d]): append at context_lens - T + j, then verify
    attention, all on `stream`.  Page-locked (pinned) host tensors are read
    and written in place by the kernels; pageable ones go through the given
    device tensors and a copy each."""
    name, args, _, _ = _verify_step_call(out_h, q_h, k_new_h, v_new_h, context_lens_h, out_d, q_d,
                                         k_new_d, v_new_d, context_lens_d, k_cache, v_cache,
                                         block_tables, scale, num_splits, workspace, stream)
    _check(getattr(lib(), name)(*args))


def _mla_pool_dims(pool: torch.Tensor) -> Tuple[int, int, int]:
    """(NB, bs, D) of a latent pool bf16 [NB][bs/8][D/8][8][8]."""
    if pool.dim() != 5 or tuple(pool.shape[3:]) != (8, 8):
        raise ValueError("latent pool must be [NB][bs/8][D/8][8][8]")
    return pool.shape[0], pool.shape[1] * 8, pool.shape[2] * 8


def mla_append(c_new, cache, block_tables, positions, stream=None) -> None:
    """Write c_new[b] ([B][576] bf16) at logical position positions[b]."""
    _need(c_new, torch.bfloat16, "c_new")
    _need(cache, torch.bfloat16, "cache")
    _need(block_tables, torch.int32, "block_tables")
    _need(positions, torch.int32, "positions")
    NB, bs, D = _mla_pool_dims(cache)
    B, MB = block_tables.shape
    _check(lib().pgd_mla_append(_ptr(c_new), _ptr(cache), _ptr(block_tables), _ptr(positions),
                                B, D, bs, MB, NB, _stream(stream)))


def mla_workspace_size(B: int, H: int, num_splits: int = 0) -> int:
    return int(lib().pgd_mla_workspace_size(B, H, num_splits))


def _mla_out(q, stream):
    make = lambda: torch.empty((*q.shape[:2], 512), dtype=torch.bfloat16, device=q.device)
    return _made_for(stream, make, result=True)


def _mla_workspace(q, num_splits, stream):
    n = max(256, mla_workspace_size(*q.shape[:2], num_splits))
    return _made_for(stream, lambda: torch.empty(n, dtype=torch.uint8, device=q.device))


def mla_decode_attention(out, q, cache, block_tables, context_lens, scale: float,
                         num_splits: int = 0, workspace: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """out[B][H][512] (bf16) = decode attention of the absorbed queries q
    ([B][H][576]) over the latent cache."""
    _need(q, torch.bfloat16, "q")
    _need(cache, torch.bfloat16, "cache")
    _need(block_tables, torch.int32, "block_tables")
    _need(context_lens, torch.int32, "context_lens")
    B, H, D = q.shape
    NB, bs, D2 = _mla_pool_dims(cache)
    if out is None:
        out = _mla_out(q, stream)
    _need(out, torch.bfloat16, "out")
    if workspace is None:
        workspace = _mla_workspace(q, num_splits, stream)
    MB = block_tables.shape[1]
    _check(lib().pgd_mla_decode_attention(
        _ptr(out), _ptr(q), _ptr(cache), _ptr(block_tables), _ptr(context_lens), B, H, D, 512,
        bs, MB, NB, float(scale), int(num_splits), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def mla_append_decode_attention(out, q, c_new, cache, block_tables, context_lens, scale: float,
                                num_splits: int = 0, workspace: Optional[torch.Tensor] = None,
                                stream=None) -> torch.Tensor:
    """mla_append of c_new at context_lens - 1, then mla_decode_attention over
    the updated cache (one call, two kernels and the merge; the attention
    prologue overlaps the append)."""
    _need(q, torch.bfloat16, "q")
    _need(c_new, torch.bfloat16, "c_new")
    _need(cache, torch.bfloat16, "cache")
    _need(block_tables, torch.int32, "block_tables")
    _need(context_lens, torch.int32, "context_lens")
    B, H, D = q.shape
    NB, bs, D2 = _mla_pool_dims(cache)
    if out is None:
        out = _mla_out(q, stream)
    _need(out, torch.bfloat16, "out")
    if workspace is None:
        workspace = _mla_workspace(q, num_splits, stream)
    MB = block_tables.shape[1]
    _check(lib().pgd_mla_append_decode_attention(
        _ptr(out), _ptr(q), _ptr(c_new), _ptr(cache), _ptr(block_tables), _ptr(context_lens), B,
        H, D, 512, bs, MB, NB, float(scale), int(num_splits), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def mla_step(out_h, q_h, c_new_h, context_lens_h, out_d, q_d, c_new_d, context_lens_d, cache,
             block_tables, scale: float, num_splits: int, workspace: torch.Tensor,
             stream=None) -> None:
    """One MLA decode step with host inputs/outputs (q [B][H][576], c_new
    [B][576], out [B][H][512]): q copied to q_d, page-locked c_new, context
    lengths and out read and written in place (pageable ones through the
    given device tensors and a copy), then mla_append_decode_attention, all
    on `stream`."""
    for t, n in ((out_h, "out_h"), (q_h, "q_h"), (c_new_h, "c_new_h")):
        _need(t, torch.bfloat16, n, cuda=False)
    _need(context_lens_h, torch.int32, "context_lens_h", cuda=False)
    _need(cache, torch.bfloat16, "cache")
    B, H, D = q_h.shape
    NB, bs, _ = _mla_pool_dims(cache)
    MB = block_tables.shape[1]
    _check(lib().pgd_mla_step(
        _ptr(out_h), _ptr(q_h), _ptr(c_new_h), _ptr(context_lens_h), _ptr(out_d), _ptr(q_d),
        _ptr(c_new_d), _ptr(context_lens_d), _ptr(cache), _ptr(block_tables), B, H, D, 512, bs,
        MB, NB, float(scale), int(num_splits), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def cascade_workspace_size(B: int, n_q: int, n_kv: int, bs: int, max_group_size: int,
                           max_group_blocks: int, num_splits: int = 0, d: int = HEAD_DIM) -> int:
    return int(lib().pgd_cascade_workspace_size(B, n_q, n_kv, d, bs, num_splits, max_group_size,
                                                max_group_blocks))


def cascade_decode_attention(out, q, k_cache, v_cache, block_tables, context_lens,
                             seq_prefix_blocks, group_first, group_size, group_blocks,
                             max_group_size: int, max_group_blocks: int, scale: float,
                             num_splits: int = 0, workspace: Optional[torch.Tensor] = None,
                             stream=None) -> torch.Tensor:
    """Paged decode attention with shared prefixes read once per group (see
    pgd_cascade_decode_attention); group arrays are device int32."""
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, torch.bfloat16, n)
    for t, n in ((block_tables, "block_tables"), (context_lens, "context_lens"),
                 (seq_prefix_blocks, "seq_prefix_blocks"), (group_first, "group_first"),
                 (group_size, "group_size"), (group_blocks, "group_blocks")):
        _need(t, torch.int32, n)
    B, n_q, d = q.shape
    NB, n_kv, bs, _ = _cache_dims(k_cache)
    if out is None:
        out = _made_for(stream, lambda: torch.empty_like(q), result=True)
    _need(out, torch.bfloat16, "out")
    if workspace is None:
        n = cascade_workspace_size(B, n_q, n_kv, bs, max_group_size, max_group_blocks, num_splits)
        n = max(1, n)
        workspace = _made_for(stream, lambda: torch.zeros(n, dtype=torch.uint8, device=q.device))
    MB = block_tables.shape[1]
    _check(lib().pgd_cascade_decode_attention(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
        _ptr(seq_prefix_blocks), _ptr(group_first), _ptr(group_size), _ptr(group_blocks),
        group_first.numel(), int(max_group_size), int(max_group_blocks), B, n_q, n_kv, d, bs, MB,
        NB, float(scale), int(num_splits), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


# ------------------------------------------------------------ 8-bit KV cache
def _cache8_dims(pool: torch.Tensor) -> Tuple[int, int, int, int]:
    """(NB, n_kv, bs, d) of an 8-bit pool uint8 [NB][n_kv][bs/8][8*d + 32]."""
    if pool.dim() != 4 or pool.dtype != torch.uint8 or (pool.shape[3] - 32) % 8:
        raise ValueError("8-bit cache must be uint8 [NB][n_kv][bs/8][8*d + 32]")
    NB, n_kv, ng, gb = pool.shape
    return NB, n_kv, ng * 8, (gb - 32) // 8


def kv_append_fp8(k_new, v_new, k_cache, v_cache, block_tables, positions, stream=None) -> None:
    """Quantise k_new/v_new [B][n_kv][d] (bf16) per (token, head) and write
    codes and scales at logical positions[b] of the 8-bit pools."""
    _need(k_new, torch.bfloat16, "k_new")
    _need(v_new, torch.bfloat16, "v_new")
    _need(k_cache, torch.uint8, "k_cache")
    _need(v_cache, torch.uint8, "v_cache")
    _need(block_tables, torch.int32, "block_tables")
    _need(positions, torch.int32, "positions")
    NB, n_kv, bs, d = _cache8_dims(k_cache)
    B, MB = block_tables.shape
    _check(lib().pgd_kv_append_fp8(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                   _ptr(block_tables), _ptr(positions), B, n_kv, d, bs, MB, NB,
                                   _stream(stream)))


def paged_decode_attention_fp8(out, q, k_cache, v_cache, block_tables, context_lens,
                               scale: float, num_splits: int = 0,
                               workspace: Optional[torch.Tensor] = None,
                               stream=None) -> torch.Tensor:
    """out[B][n_q][d] (bf16) = paged decode attention of q over the 8-bit cache."""
    name, args, out, workspace = _attention_call(True, out, q, k_cache, v_cache, block_tables,
                                                 context_lens, scale, num_splits, workspace,
                                                 stream)
    _check(getattr(lib(), name)(*args))
    return out


def append_decode_attention_fp8(out, q, k_new, v_new, k_cache, v_cache, block_tables,
                                context_lens, scale: float, num_splits: int = 0,
                                workspace: Optional[torch.Tensor] = None,
                                stream=None) -> torch.Tensor:
    """kv_append_fp8 at context_lens - 1, then attention over the 8-bit cache."""
    name, args, out, workspace = _append_attention_call(
        True, out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, scale,
        num_splits, workspace, stream)
    _check(getattr(lib(), name)(*args))
    return out


# ------------------------------------------------- block-scaled 8-bit KV cache
# The calls of this section and the next check and convert their tensors in
# binding/tensors.cpp: they run for a few microseconds on the GPU, and a dozen
# tensors took longer than that in Python.
_tensor_side = None


def _tensors():
    """The binding's tensor extension.  Raises if it has not been built."""
    global _tensor_side
    if _tensor_side is None:
        lib()  # (a missing build says so)
        path = _build.tensors_path()
        if not os.path.exists(path):
            raise RuntimeError("%s is not built; run paged_gqa_decode_kv_gb300.build.build()" % path)
        loader = importlib.machinery.ExtensionFileLoader("_pgd_tensors", path)
        spec = importlib.util.spec_from_file_location("_pgd_tensors", path, loader=loader)
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
        _tensor_side = module
    return _tensor_side


def block_workspace_size(B: int, n_q: int, n_kv: int, num_splits: int = 0,
                         d: int = HEAD_DIM) -> int:
    return int(lib().pgd_block_workspace_size(B, n_q, n_kv, d, num_splits))


def make_block_workspace(B: int, n_q: int, n_kv: int, num_splits: int = 0,
                         device=None) -> torch.Tensor:
    """A zero-filled workspace of the block-scaled and selected attention
    calls; one serves calls of any sizes up to these, in stream order."""
    n = max(1, block_workspace_size(B, n_q, n_kv, num_splits))
    return torch.zeros(n, dtype=torch.uint8, device=device or torch.device("cuda"))


def kv_append_fp8b(k_new, v_new, k_cache, v_cache, k_scales, v_scales, block_tables, positions,
                   token_starts=None, max_tokens: Optional[int] = None, stream=None) -> None:
    """Quantise new tokens into the block-scaled pools (uint8
    [NB][n_kv][bs/8][8][8][16], scales fp32 [NB][n_kv]) at positions[b] on:
    rows token_starts[b] .. token_starts[b + 1] - 1 of k_new/v_new
    ([N][n_kv][d] bf16; at most max_tokens each), or without token_starts the
    same number of tokens for every sequence ([B][n_kv][d] or
    [B][T][n_kv][d])."""
    s = (_tensor_side or _tensors()).range(
        False, k_new, v_new, k_cache, v_cache, k_scales, v_scales, block_tables, positions,
        token_starts, max_tokens, stream)
    if s:
        _check(s)


def kv_read_fp8b(k_out, v_out, k_cache, v_cache, k_scales, v_scales, block_tables, positions,
                 token_starts=None, max_tokens: Optional[int] = None, stream=None) -> None:
    """Read ranges of positions back into rows of k_out/v_out (bf16): the
    arguments of kv_append_fp8b, the other way."""
    s = (_tensor_side or _tensors()).range(
        True, k_out, v_out, k_cache, v_cache, k_scales, v_scales, block_tables, positions,
        token_starts, max_tokens, stream)
    if s:
        _check(s)


def _out_and_scratch(out, q, n_kv, num_splits, workspace, stream):
    """The output and the workspace of a decode call, made where not given."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [B][n_q][d]")
    if out is None:
        out = _made_for(stream, lambda: torch.empty_like(q), result=True)
    if workspace is None:
        if not q.is_cuda:
            raise ValueError("q must be on a CUDA device")
        workspace = _made_for(stream, lambda: make_block_workspace(q.shape[0], q.shape[1], n_kv,
                                                                   num_splits, q.device))
    return out, workspace


def _pool_heads(k_cache) -> int:
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 6:
        raise ValueError("k_cache must be a pool of 6 dims")
    return k_cache.shape[1]


def _attention8b(pack, out, q, k_new, v_new, k_cache, v_cache, k_scales, v_scales, block_tables,
                 context_lens, scale, num_splits, workspace, stream):
    if out is None or workspace is None:
        if isinstance(k_cache, torch.Tensor) and k_cache.dtype != torch.uint8:
            raise TypeError("k_cache must be torch.uint8, got %s" % k_cache.dtype)
        out, workspace = _out_and_scratch(out, q, _pool_heads(k_cache), num_splits, workspace,
                                          stream)
    return out, workspace, (_tensor_side or _tensors()).attention(
        out, q, k_new, v_new, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens,
        scale, num_splits, workspace, stream, pack)


def paged_decode_attention_fp8b(out, q, k_cache, v_cache, k_scales, v_scales, block_tables,
                                context_lens, scale: float, num_splits: int = 0,
                                workspace: Optional[torch.Tensor] = None,
                                stream=None) -> torch.Tensor:
    """out[B][n_q][d] (bf16) = paged decode attention of q over the
    block-scaled 8-bit cache."""
    out, _, s = _attention8b(False, out, q, None, None, k_cache, v_cache, k_scales, v_scales,
                             block_tables, context_lens, scale, num_splits, workspace, stream)
    if s:
        _check(s)
    return out


def append_decode_attention_fp8b(out, q, k_new, v_new, k_cache, v_cache, k_scales, v_scales,
                                 block_tables, context_lens, scale: float, num_splits: int = 0,
                                 workspace: Optional[torch.Tensor] = None,
                                 stream=None) -> torch.Tensor:
    """kv_append_fp8b of one token per sequence at context_lens - 1, then
    attention over the block-scaled cache."""
    out, _, s = _attention8b(False, out, q, k_new, v_new, k_cache, v_cache, k_scales, v_scales,
                             block_tables, context_lens, scale, num_splits, workspace, stream)
    if s:
        _check(s)
    return out


# ------------------------------------------------------------- 4-bit KV cache
GROUP_BYTES4 = 1152  # 16 tokens of a tile: 1024 of codes, 128 of scales


def pool_shape4(num_blocks: int, n_kv: int, block_size: int) -> Tuple[int, int, int, int]:
    """Shape of a 4-bit pool (uint8)."""
    return num_blocks, n_kv, block_size // 16, GROUP_BYTES4


def _cache4_dims(pool: torch.Tensor) -> Tuple[int, int, int, int]:
    """(NB, n_kv, bs, d) of a 4-bit pool uint8 [NB][n_kv][bs/16][1152]."""
    if pool.dim() != 4 or pool.shape[3] != GROUP_BYTES4:
        raise ValueError("4-bit cache must be uint8 [NB][n_kv][bs/16][%d]" % GROUP_BYTES4)
    NB, n_kv, ng, _ = pool.shape
    return NB, n_kv, ng * 16, HEAD_DIM


def fp4_workspace_size(B: int, n_q: int, n_kv: int, num_splits: int = 0,
                       d: int = HEAD_DIM) -> int:
    return int(lib().pgd_fp4_workspace_size(B, n_q, n_kv, d, num_splits))


def make_fp4_workspace(B: int, n_q: int, n_kv: int, num_splits: int = 0,
                       device=None) -> torch.Tensor:
    """A zero-filled workspace of the 4-bit attention calls; one serves calls of
    any sizes up to these, in stream order."""
    n = max(1, fp4_workspace_size(B, n_q, n_kv, num_splits))
    return torch.zeros(n, dtype=torch.uint8, device=device or torch.device("cuda"))


def kv_append_fp4(k_new, v_new, k_cache, v_cache, block_tables, positions, token_starts=None,
                  max_tokens: Optional[int] = None, k_scale: float = 1.0, v_scale: float = 1.0,
                  stream=None) -> None:
    """Quantise new tokens into the 4-bit pools (uint8 [NB][n_kv][bs/16][1152])
    at positions[b] on: rows token_starts[b] .. token_starts[b + 1] - 1 of
    k_new/v_new ([N][n_kv][d] bf16; at most max_tokens each), or without
    token_starts the same number of tokens for every sequence ([B][n_kv][d] or
    [B][T][n_kv][d]).  k_scale, v_scale: powers of two, the cache's own."""
    s = (_tensor_side or _tensors()).range4(False, k_new, v_new, k_cache, v_cache, block_tables,
                                            positions, token_starts, max_tokens, k_scale, v_scale,
                                            stream)
    if s:
        _check(s)


def kv_read_fp4(k_out, v_out, k_cache, v_cache, block_tables, positions, token_starts=None,
                max_tokens: Optional[int] = None, k_scale: float = 1.0, v_scale: float = 1.0,
                stream=None) -> None:
    """Read ranges of positions back into rows of k_out/v_out (bf16): the
    arguments of kv_append_fp4, the other way."""
    s = (_tensor_side or _tensors()).range4(True, k_out, v_out, k_cache, v_cache, block_tables,
                                            positions, token_starts, max_tokens, k_scale, v_scale,
                                            stream)
    if s:
        _check(s)


def _attention4(pack, out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, scale,
                k_scale, v_scale, num_splits, workspace, stream):
    if out is None or workspace is None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be [B][n_q][d]")
        if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
            raise ValueError("k_cache must be a 4-bit pool")
        if not q.is_cuda:
            raise ValueError("q must be on a CUDA device")
        if out is None:
            out = _made_for(stream, lambda: torch.empty_like(q), result=True)
        if workspace is None:
            workspace = _made_for(stream, lambda: make_fp4_workspace(
                q.shape[0], q.shape[1], k_cache.shape[1], num_splits, q.device))
    return out, workspace, (_tensor_side or _tensors()).attention4(
        out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, scale, k_scale,
        v_scale, num_splits, workspace, stream, pack)


def paged_decode_attention_fp4(out, q, k_cache, v_cache, block_tables, context_lens, scale: float,
                               k_scale: float = 1.0, v_scale: float = 1.0, num_splits: int = 0,
                               workspace: Optional[torch.Tensor] = None,
                               stream=None) -> torch.Tensor:
    """out[B][n_q][d] (bf16) = paged decode attention of q over the 4-bit
    cache."""
    out, _, s = _attention4(False, out, q, None, None, k_cache, v_cache, block_tables,
                            context_lens, scale, k_scale, v_scale, num_splits, workspace, stream)
    if s:
        _check(s)
    return out


def append_decode_attention_fp4(out, q, k_new, v_new, k_cache, v_cache, block_tables,
                                context_lens, scale: float, k_scale: float = 1.0,
                                v_scale: float = 1.0, num_splits: int = 0,
                                workspace: Optional[torch.Tensor] = None,
                                stream=None) -> torch.Tensor:
    """kv_append_fp4 of one token per sequence at context_lens - 1, then
    attention over the 4-bit cache."""
    if k_new is None or v_new is None:
        raise TypeError("k_new and v_new must be tensors")
    out, _, s = _attention4(False, out, q, k_new, v_new, k_cache, v_cache, block_tables,
                            context_lens, scale, k_scale, v_scale, num_splits, workspace, stream)
    if s:
        _check(s)
    return out


def _prepared4(out, q, k_cache, v_cache, block_tables, context_lens, scale, k_scale=1.0,
               v_scale=1.0, num_splits=0, workspace=None, stream=None):
    out, workspace, args = _attention4(True, out, q, None, None, k_cache, v_cache, block_tables,
                                       context_lens, scale, k_scale, v_scale, num_splits,
                                       workspace, stream)
    return "pgd_paged_decode_attention_fp4", args, out, workspace


def _prepared_append4(out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, scale,
                      k_scale=1.0, v_scale=1.0, num_splits=0, workspace=None, stream=None):
    if k_new is None or v_new is None:
        raise TypeError("k_new and v_new must be tensors")
    out, workspace, args = _attention4(True, out, q, k_new, v_new, k_cache, v_cache, block_tables,
                                       context_lens, scale, k_scale, v_scale, num_splits,
                                       workspace, stream)
    return "pgd_append_decode_attention_fp4", args, out, workspace


# ------------------------------------------------------------ rotary positions
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "ramp_dim": 3, "ramp_wavelength": 4}


def rope_frequencies(rotary: int, base: float = 10000.0, scaling: str = "none",
                     factor: float = 1.0, original_context: float = 0.0, slow_turns: float = 1.0,
                     fast_turns: float = 32.0, device=None) -> torch.Tensor:
    """The frequencies of `rotary` rotated dims as rope and rope_append take
    them (int64 [rotary / 2], turns a position in units of 2^-64), scaled for
    long contexts by "linear", "base", "ramp_dim" or "ramp_wavelength" (see
    pgd_rope_frequencies).  device None: the current CUDA device."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError("scaling must be one of %s, got %r" % (sorted(ROPE_SCALINGS), scaling))
    buf = (ctypes.c_int64 * max(1, int(rotary) // 2))()
    _check(lib().pgd_rope_frequencies(ctypes.addressof(buf), int(rotary), float(base),
                                      ROPE_SCALINGS[scaling], float(factor),
                                      float(original_context), float(slow_turns),
                                      float(fast_turns)))
    t = torch.tensor(list(buf), dtype=torch.int64)
    return t.to(device if device is not None else torch.device("cuda"))


def rope(q_out, k_out, q, k, positions, frequencies, interleaved: bool = False, first: int = 0,
         factor: float = 1.0, stream=None):
    """Rotary positions: rows q [T][n_q][d] to q_out and k [T][n_kv][d] to k_out
    (bf16; strided over tokens and heads as views of one projection's output
    are; an output may be its input, None makes it; k None: q alone), positions
    int32 [T], the rotated dims first .. first + 2 * len(frequencies) - 1 as
    halves or as interleaved pairs, cosine and sine times `factor`.  Returns
    q_out, k_out."""
    if q_out is None:
        q_out = _made_for(stream, lambda: torch.empty(q.shape, dtype=q.dtype, device=q.device),
                          result=True)
    if k is not None and k_out is None:
        k_out = _made_for(stream, lambda: torch.empty(k.shape, dtype=k.dtype, device=k.device),
                          result=True)
    s = (_tensor_side or _tensors()).rope(q_out, k_out, q, k, positions, frequencies,
                                          bool(interleaved), first, factor, stream)
    if s:
        _check(s)
    return q_out, k_out


def rope_append(q_out, q, k, v, k_cache, v_cache, slots, positions, frequencies,
                interleaved: bool = False, first: int = 0, factor: float = 1.0, stream=None):
    """rope with K written into the paged bf16 cache, and V beside it, at
    slots[t] = block * block size + slot (int64 [T]; negative: the token is left
    out).  Returns q_out (None makes it)."""
    if q_out is None:
        q_out = _made_for(stream, lambda: torch.empty(q.shape, dtype=q.dtype, device=q.device),
                          result=True)
    s = (_tensor_side or _tensors()).rope_append(q_out, q, k, v, k_cache, v_cache, slots,
                                                 positions, frequencies, bool(interleaved), first,
                                                 factor, stream)
    if s:
        _check(s)
    return q_out


# ------------------------------------------------ block tables grown on the GPU
def make_block_pool(num_blocks: int, device=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(refs, free_bits) of a pool whose blocks are all free."""
    if num_blocks < 1:
        raise ValueError("num_blocks must be positive")
    device = device if device is not None else torch.device("cuda")
    bits = torch.full(((num_blocks + 31) // 32,), -1, dtype=torch.int32, device=device)
    if num_blocks % 32:
        bits[-1] = (1 << (num_blocks % 32)) - 1
    return torch.zeros(num_blocks, dtype=torch.int32, device=device), bits


def grow_tables(block_tables, context_lens, new_tokens, refs, free_bits, block_size: int,
                positions, token_starts, slots, token_positions, copy_src, copy_dst, result,
                stream=None) -> None:
    """Add new_tokens[b] tokens to every row of block_tables [B][MB]: blocks
    from the pool (refs, free_bits), lengths, and the step's positions [B],
    token_starts [B + 1], slots and token_positions [N], copies [B] and result
    [4] (int32, slots int64; see pgd_grow_tables)."""
    s = (_tensor_side or _tensors()).grow(block_tables, context_lens, new_tokens, refs, free_bits,
                                          block_size, positions, token_starts, slots,
                                          token_positions, copy_src, copy_dst, result, stream)
    if s:
        _check(s)


def trim_tables(block_tables, context_lens, keep_lens, refs, free_bits, block_size: int,
                stream=None) -> None:
    """Cut row b to keep_lens[b] tokens and give the blocks behind them back
    (0: release the request)."""
    s = (_tensor_side or _tensors()).trim(block_tables, context_lens, keep_lens, refs, free_bits,
                                          block_size, stream)
    if s:
        _check(s)


# ------------------------------------------------------ block-sparse attention
def block_bounds(bounds, bound_scales, k_cache, block_tables, context_lens, positions=None,
                 max_tokens: Optional[int] = None, k_scales=None, stream=None) -> None:
    """Recompute the key bounds (int8 [NB][n_kv][2][d], fp32 [NB][n_kv]) of
    the blocks that hold positions[b] .. context_lens[b] - 1 (positions None:
    the whole contexts) of a bf16 cache, or of a block-scaled one with its
    k_scales.  max_tokens: the most tokens of a sequence (default: the table
    width)."""
    s = (_tensor_side or _tensors()).bounds(bounds, bound_scales, k_cache, block_tables,
                                            context_lens, positions, max_tokens, k_scales, stream)
    if s:
        _check(s)


def select_blocks(tiles, tile_tokens, q, bounds, bound_scales, block_tables, context_lens,
                  keep_first: int, keep_last: int, block_size: int, stream=None) -> None:
    """tiles [B][n_kv][W] and tile_tokens [B][n_kv] (int32): for every
    sequence and KV head the first keep_first blocks, the last keep_last and
    the others of the largest score, W in all."""
    s = (_tensor_side or _tensors()).select(tiles, tile_tokens, q, bounds, bound_scales,
                                            block_tables, context_lens, keep_first, keep_last,
                                            block_size, stream)
    if s:
        _check(s)


def _need_bounds(bounds) -> None:
    """(None would make the extension take the tiles as given.)"""
    if bounds is None:
        raise TypeError("bounds must be a tensor")


def _tiles_attention(pack, out, q, k_cache, v_cache, k_scales, v_scales, bounds, bound_scales,
                     block_tables, context_lens, tiles, tile_tokens, keep_first, keep_last, scale,
                     num_splits, workspace, stream):
    if out is None or workspace is None:
        if (k_scales is None) != (v_scales is None):
            raise ValueError("a block-scaled cache needs both scales")
        out, workspace = _out_and_scratch(out, q, _pool_heads(k_cache), num_splits, workspace,
                                          stream)
    return out, workspace, (_tensor_side or _tensors()).tiles(
        out, q, k_cache, v_cache, k_scales, v_scales, bounds, bound_scales, block_tables,
        context_lens, tiles, tile_tokens, keep_first, keep_last, scale, num_splits, workspace,
        stream, pack)


def selected_decode_attention(out, q, k_cache, v_cache, tiles, tile_tokens, scale: float,
                              k_scales=None, v_scales=None, num_splits: int = 0,
                              workspace: Optional[torch.Tensor] = None,
                              stream=None) -> torch.Tensor:
    """out[B][n_q][d] (bf16) = decode attention of q over the tiles (block *
    n_kv + head, [B][n_kv][W]) of a bf16 cache, or of a block-scaled one with
    its scales."""
    out, _, s = _tiles_attention(False, out, q, k_cache, v_cache, k_scales, v_scales, None, None,
                                 None, None, tiles, tile_tokens, 0, 0, scale, num_splits,
                                 workspace, stream)
    if s:
        _check(s)
    return out


def sparse_decode_attention(out, q, k_cache, v_cache, bounds, bound_scales, block_tables,
                            context_lens, tiles, tile_tokens, keep_first: int, keep_last: int,
                            scale: float, k_scales=None, v_scales=None, num_splits: int = 0,
                            workspace: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """select_blocks into tiles and tile_tokens, then
    selected_decode_attention over them, in one call."""
    _need_bounds(bounds)
    out, _, s = _tiles_attention(False, out, q, k_cache, v_cache, k_scales, v_scales, bounds,
                                 bound_scales, block_tables, context_lens, tiles, tile_tokens,
                                 keep_first, keep_last, scale, num_splits, workspace, stream)
    if s:
        _check(s)
    return out


def _prepared8b(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, scale,
                num_splits=0, workspace=None, stream=None):
    out, workspace, args = _attention8b(True, out, q, None, None, k_cache, v_cache, k_scales,
                                        v_scales, block_tables, context_lens, scale, num_splits,
                                        workspace, stream)
    return "pgd_paged_decode_attention_fp8b", args, out, workspace


def _prepared_append8b(out, q, k_new, v_new, k_cache, v_cache, k_scales, v_scales, block_tables,
                       context_lens, scale, num_splits=0, workspace=None, stream=None):
    out, workspace, args = _attention8b(True, out, q, k_new, v_new, k_cache, v_cache, k_scales,
                                        v_scales, block_tables, context_lens, scale, num_splits,
                                        workspace, stream)
    return "pgd_append_decode_attention_fp8b", args, out, workspace


def _prepared_sparse(out, q, k_cache, v_cache, bounds, bound_scales, block_tables, context_lens,
                     tiles, tile_tokens, keep_first, keep_last, scale, k_scales=None,
                     v_scales=None, num_splits=0, workspace=None, stream=None):
    _need_bounds(bounds)
    out, workspace, args = _tiles_attention(True, out, q, k_cache, v_cache, k_scales, v_scales,
                                            bounds, bound_scales, block_tables, context_lens,
                                            tiles, tile_tokens, keep_first, keep_last, scale,
                                            num_splits, workspace, stream)
    return "pgd_sparse_decode_attention", args, out, workspace


def copy_blocks(k_cache, v_cache, src_ids, dst_ids, stream=None) -> None:
    """Copy whole physical blocks src_ids[i] -> dst_ids[i] (device int32; a
    pair -1, -1 is none) of bf16 pools, or of 4-bit ones (uint8)."""
    fp4 = getattr(k_cache, "dtype", None) == torch.uint8
    _need(k_cache, torch.uint8 if fp4 else torch.bfloat16, "k_cache")
    _need(v_cache, torch.uint8 if fp4 else torch.bfloat16, "v_cache")
    _need(src_ids, torch.int32, "src_ids")
    _need(dst_ids, torch.int32, "dst_ids")
    NB, n_kv, bs, d = _cache4_dims(k_cache) if fp4 else _cache_dims(k_cache)
    if fp4 and (v_cache.shape != k_cache.shape or dst_ids.shape != src_ids.shape):
        raise ValueError("k_cache and v_cache, src_ids and dst_ids must have one shape")
    fn = lib().pgd_copy_blocks_fp4 if fp4 else lib().pgd_copy_blocks
    _check(fn(_ptr(k_cache), _ptr(v_cache), _ptr(src_ids), _ptr(dst_ids), src_ids.numel(), n_kv,
              d, bs, NB, _stream(stream)))


def device_errors(clear: bool = True, stream=None) -> int:
    """Wait for `stream` and return (then clear) the device error bits."""
    v = ctypes.c_int32(0)
    _check(lib().pgd_device_errors(ctypes.addressof(v), 1 if clear else 0, _stream(stream)))
    return int(v.value)


def read_stream(src: torch.Tensor, mode: int = 0, stream=None) -> None:
    """Read every byte of the CUDA tensor `src` once and discard it (the
    read-only streaming calibration pass; mode 0: 16-byte loads, mode 1:
    4 KiB bulk copies into shared memory)."""
    if not src.is_cuda or not src.is_contiguous():
        raise ValueError("src must be a contiguous CUDA tensor")
    _check(lib().pgd_read_stream(_ptr(src), src.numel() * src.element_size(), int(mode),
                                 _stream(stream)))


def set_wait_limit_ns(ns: int) -> None:
    """Limit of the kernels' bounded waits for launches made after this call
    (0 restores the 4 s default).  A short limit makes waits run out on
    purpose: for tests of the timeout exit only."""
    lib().pgd_set_wait_limit_ns(int(ns))


def wait_limit_ns() -> int:
    return int(lib().pgd_wait_limit_ns())


def set_short_context_tokens(max_tokens: int) -> int:
    """Largest MB * bs (at most 1024) for which an automatic single-query
    call may run the short-context kernel (0: never; negative: the default
    1024).  Returns the previous limit."""
    return int(lib().pgd_set_short_context_tokens(int(max_tokens)))


def uses_short_path(B: int, n_kv: int, bs: int, MB: int, num_splits: int = 0) -> bool:
    """Whether a call with these sizes (B sequences, n_kv KV heads, block size
    bs, table width MB) runs the short-context kernel now (pgd_short_path)."""
    return bool(lib().pgd_short_path(int(B), int(n_kv), int(bs), int(MB), int(num_splits)))


# ------------------------------------------------------------ host allocator
class BlockAllocator:
    """Host pool of physical block ids with reference counts (pgd_alloc_*)."""

    def __init__(self, num_blocks: int):
        h = ctypes.c_void_p()
        _check(lib().pgd_alloc_create(int(num_blocks), ctypes.addressof(h)))
        self._h = h

    def close(self) -> None:
        if self._h:
            lib().pgd_alloc_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @staticmethod
    def _arr(ids: Sequence[int]):
        return (ctypes.c_int32 * max(1, len(ids)))(*ids)

    def allocate(self, n: int) -> list:
        buf = (ctypes.c_int32 * max(1, n))()
        _check(lib().pgd_alloc_allocate(self._h, int(n), buf))
        return list(buf[:n])

    def share(self, ids: Sequence[int]) -> None:
        _check(lib().pgd_alloc_share(self._h, self._arr(ids), len(ids)))

    def release(self, ids: Sequence[int]) -> None:
        _check(lib().pgd_alloc_release(self._h, self._arr(ids), len(ids)))

    def refcount(self, i: int) -> int:
        return int(lib().pgd_alloc_refcount(self._h, int(i)))

    @property
    def num_free(self) -> int:
        return int(lib().pgd_alloc_num_free(self._h))

    @property
    def num_blocks(self) -> int:
        return int(lib().pgd_alloc_num_blocks(self._h))

    def append_slot(self, row: list, pos: int, block_size: int) -> Tuple[int, int]:
        """Make position `pos` of table `row` writable (row updated in place);
        returns the (src, dst) copy-on-write pair or (-1, -1)."""
        buf = (ctypes.c_int32 * len(row))(*row)
        src, dst = ctypes.c_int32(-1), ctypes.c_int32(-1)
        _check(lib().pgd_alloc_append_slot(self._h, buf, len(row), int(block_size), int(pos),
                                           ctypes.addressof(src), ctypes.addressof(dst)))
        row[:] = list(buf)
        return int(src.value), int(dst.value)

    def fork(self, src_row: Sequence[int], n_tokens: int, block_size: int, dst_row: list) -> None:
        s = (ctypes.c_int32 * len(src_row))(*src_row)
        d = (ctypes.c_int32 * len(dst_row))(*dst_row)
        _check(lib().pgd_alloc_fork(self._h, s, int(n_tokens), int(block_size), d, len(dst_row)))
        dst_row[:] = list(d)


def validate_tables(block_tables_h: torch.Tensor, context_lens_h: torch.Tensor, num_blocks: int,
                    block_size: int) -> None:
    """Host check of host copies of the tables and lengths (raises PGDError)."""
    t = block_tables_h.contiguous().to(torch.int32).cpu()
    c = context_lens_h.contiguous().to(torch.int32).cpu()
    B, MB = t.shape
    _check(lib().pgd_validate_tables(_ptr(t), _ptr(c), B, MB, int(num_blocks), int(block_size)))
