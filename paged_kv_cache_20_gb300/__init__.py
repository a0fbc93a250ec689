"""Python binding of libpagedattn.so (paged decode attention for GB300, sm_103a).

Argument marshalling only: every function below checks shapes and dtypes, takes
raw device pointers and the current CUDA stream from PyTorch tensors, and calls
the C function of the same name.  All arithmetic runs in the library's CUDA
kernels; there is no fallback.  If the library has not been built the first call
raises ``RuntimeError``.

Layouts match ``include/pagedattn.h``:
  k_cache, v_cache  [num_blocks, num_kv_heads, block_size, head_dim]  fp16 | bf16
  q, out            [num_seqs, q_len, num_q_heads, head_dim]
  k_new, v_new      [n_tokens, num_kv_heads, head_dim]
  block_tables      int32 [num_seqs, max_blocks_per_seq]
  context_lens      int32 [num_seqs]       (count this step's new tokens)
  slot_mapping      int64 [n_tokens]
  scores, row_pos   fp32, int32 [num_seqs, num_kv_heads, max_blocks_per_seq * block_size]

Streams: a call runs on the current stream, or on the one named by ``stream`` (a
``torch.cuda.Stream`` or a raw handle; ordering it after the work that makes the
arguments is the caller's).  Workspaces and outputs that are not given are made from that
stream's memory pool, as under ``torch.cuda.stream(stream)``: an output that is then used
on another stream wants ``record_stream`` before it is dropped.
"""
from __future__ import annotations

import ctypes
import importlib
import math
import os
import threading
import warnings

import torch

from . import _build

LIBRARY = _build.LIBRARY

PA_OK = 0
PA_ERR_INVALID_ARG = -1
PA_ERR_UNSUPPORTED = -2
PA_ERR_CUDA = -3
PA_ERR_DEVICE_CHECK = -4
PA_ERR_DEVICE_TIMEOUT = -5

PA_FP16, PA_BF16 = 0, 1
_DTYPE = {torch.float16: PA_FP16, torch.bfloat16: PA_BF16}

_c_int, _c_float, _c_size, _c_vp = ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_void_p
_c_i64 = ctypes.c_int64

# name -> (restype, argtypes): mirrors include/pagedattn.h
_SIGNATURES = {
    "pa_status_string": (ctypes.c_char_p, [_c_int]),
    "pa_version": (_c_int, []),
    "pa_slot_mapping": (_c_int, [_c_vp, _c_vp, _c_vp, _c_int, _c_int, _c_int, _c_int, _c_vp]),
    "pa_append_kv": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_int, _c_int, _c_int,
                              _c_int, _c_int, _c_vp]),
    "pa_decode": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_int, _c_int,
                           _c_int, _c_int, _c_float, _c_vp, _c_int, _c_int, _c_int, _c_int]),
    "pa_decode_workspace_size": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int]),
    "pa_decode_partial": (_c_int, [_c_vp, _c_size, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int,
                                   _c_int, _c_int, _c_int, _c_int, _c_float, _c_int, _c_int,
                                   _c_int, _c_int, _c_int, _c_vp]),
    "pa_decode_combine": (_c_int, [_c_vp, _c_vp, _c_size, _c_int, _c_int, _c_int, _c_int,
                                   _c_int, _c_int, _c_vp]),
    "pa_device_error": (_c_int, [_c_vp, _c_int]),
    "pa_selftest_wait_timeout": (_c_int, [_c_vp]),
    "pa_copy_blocks": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_int, _c_int, _c_int,
                                _c_int, _c_int, _c_vp]),
    "pa_append_kv_fp8": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_int, _c_int,
                                  _c_int, _c_int, _c_int, _c_vp, _c_vp, _c_vp]),
    "pa_decode_fp8": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp,
                               _c_vp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_float, _c_int,
                               _c_int, _c_int, _c_int, _c_int, _c_vp, _c_size, _c_vp]),
    "pa_append_decode": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int,
                                  _c_int, _c_int, _c_int, _c_int, _c_float, _c_int, _c_int,
                                  _c_int, _c_int, _c_int, _c_vp, _c_size, _c_vp]),
    "pa_decode_cascade": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int,
                                   _c_int, _c_int, _c_int, _c_int, _c_float, _c_int, _c_int,
                                   _c_int, _c_int, _c_int, _c_int, _c_vp, _c_size, _c_vp]),
    "pa_decode_split_noalloc": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_int,
                                         _c_int, _c_int, _c_int, _c_float, _c_int, _c_int,
                                         _c_int, _c_int, _c_int, _c_vp]),
    "pa_rope_append": (_c_int, [_c_vp] * 10 + [_c_int] * 7 + [_c_i64] * 4 +
                       [_c_int] * 3 + [_c_vp] * 3),
    "pa_decode_scored_workspace_size": (_c_size, [_c_int] * 7),
    "pa_decode_scored": (_c_int, [_c_vp] * 11 + [_c_int] * 5 + [_c_float] + [_c_int] * 5 +
                         [_c_vp, _c_size, _c_vp]),
    "pa_evict_workspace_size": (_c_size, [_c_int] * 3),
    "pa_evict": (_c_int, [_c_vp] * 10 + [_c_int] * 10 + [_c_vp, _c_size, _c_vp]),
    "pa_verify_drafts": (_c_int, [_c_vp] * 10 + [_c_int] * 3 + [_c_i64, _c_i64, _c_vp]),
}

NOALLOC_SCRATCH_BYTES = 8 << 20   # PA_NOALLOC_SCRATCH_BYTES

_lock = threading.Lock()
_lib = None
_fast = None   # the checked calls of csrc/pa_calls.cpp, once the library is loaded


class PagedAttnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")
        self.status = status


def _checked_calls():
    """csrc/pa_calls.cpp (links the same library), or None where it is missing or was built
    for another torch: the binding then makes every check and call itself."""
    try:
        calls = importlib.import_module("._calls", __package__)
        version = getattr(calls, "torch_version", "?")
        if version == torch.__version__:
            return calls
        why = f"built for torch {version}, this is {torch.__version__}"
    except ImportError as e:
        why = str(e)
    warnings.warn(f"{__package__}._calls is not used ({why}): short calls take a few microseconds longer; "
                  "paged_kv_cache_20_gb300._build.build() makes it", RuntimeWarning, stacklevel=3)
    return None


def load(path: str = LIBRARY) -> ctypes.CDLL:
    """Load the library (once).  Raises RuntimeError when it has not been built."""
    global _lib, _fast
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: build it with paged_kv_cache_20_gb300."
                                   "_build.build() (or __graft_entry__.build())")
            lib = ctypes.CDLL(path)
            for name, (res, args) in _SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            if path == LIBRARY:
                _fast = _checked_calls()
            _lib = lib
        return _lib


def status_string(status: int) -> str:
    return load().pa_status_string(status).decode()


def _check(fn: str, status: int) -> None:
    if status != PA_OK:
        raise PagedAttnError(fn, status)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _made(shape, dtype, device, stream) -> torch.Tensor:
    """A workspace or output that the caller did not give, from the memory pool of the
    stream that the call runs on: memory of another stream's pool may be given out again
    once the call has returned, with its kernels still to come."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    handle = _stream(stream)
    if handle == 2:  # cudaStreamPerThread: one handle, a stream in every thread
        raise ValueError("on the per-thread default stream give every workspace and output")
    if not (hasattr(stream, "cuda_stream") and hasattr(stream, "device")):
        # (handles 0 and 1 both name the legacy default stream)
        stream = (torch.cuda.default_stream(device) if handle in (0, 1)
                  else torch.cuda.ExternalStream(handle, device=device))
    elif stream.device != device:
        raise ValueError(f"the stream is of {stream.device}, the tensors are on {device}")
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _cuda(t: torch.Tensor, name: str, dtype=None) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _elt(t: torch.Tensor, name: str) -> int:
    if t.dtype not in _DTYPE:
        raise TypeError(f"{name} must be float16 or bfloat16, got {t.dtype}")
    return _DTYPE[t.dtype]


def _cache_dims(k_cache: torch.Tensor):
    if k_cache.dim() != 4:
        raise ValueError("caches must be [num_blocks, num_kv_heads, block_size, head_dim]")
    return tuple(int(x) for x in k_cache.shape)


# ---------------------------------------------------------------------------- API
def pa_slot_mapping(block_tables: torch.Tensor, context_lens: torch.Tensor, block_size: int,
                    q_len: int = 1, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Slots of each sequence's last q_len positions -> int64 [num_seqs * q_len]."""
    n, maxb = (int(x) for x in block_tables.shape)
    if out is None:
        out = _made((n * q_len,), torch.int64, block_tables.device, stream)
    _check("pa_slot_mapping", load().pa_slot_mapping(
        _cuda(out, "out", torch.int64), _cuda(block_tables, "block_tables", torch.int32),
        _cuda(context_lens, "context_lens", torch.int32), n, maxb, block_size, q_len,
        _stream(stream)))
    return out


def pa_append_kv(k_cache: torch.Tensor, v_cache: torch.Tensor, k_new: torch.Tensor,
                 v_new: torch.Tensor, slot_mapping: torch.Tensor, stream=None) -> None:
    """Copy rows k_new[t], v_new[t] into slot slot_mapping[t] of the caches."""
    num_blocks, h_kv, block_size, head_dim = _cache_dims(k_cache)
    dt = _elt(k_cache, "k_cache")
    for t, nm in ((v_cache, "v_cache"), (k_new, "k_new"), (v_new, "v_new")):
        if t.dtype != k_cache.dtype:
            raise TypeError(f"{nm} must have the cache dtype {k_cache.dtype}")
    n_tokens = int(slot_mapping.shape[0])
    if k_new.shape != (n_tokens, h_kv, head_dim) or v_new.shape != k_new.shape:
        raise ValueError("k_new/v_new must be [n_tokens, num_kv_heads, head_dim]")
    _check("pa_append_kv", load().pa_append_kv(
        _cuda(k_cache, "k_cache"), _cuda(v_cache, "v_cache"), _cuda(k_new, "k_new"),
        _cuda(v_new, "v_new"), _cuda(slot_mapping, "slot_mapping", torch.int64), n_tokens, h_kv,
        head_dim, block_size, num_blocks, dt, _stream(stream)))


def pa_copy_blocks(k_cache: torch.Tensor, v_cache: torch.Tensor, src_blocks: torch.Tensor,
                   dst_blocks: torch.Tensor, stream=None) -> None:
    """Copy whole blocks src_blocks[i] -> dst_blocks[i] in both caches (copy-on-write)."""
    num_blocks, h_kv, block_size, head_dim = _cache_dims(k_cache)
    if v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype:
        raise ValueError("v_cache must match k_cache")
    n = int(src_blocks.shape[0])
    if int(dst_blocks.shape[0]) != n:
        raise ValueError("src_blocks and dst_blocks must have the same length")
    _check("pa_copy_blocks", load().pa_copy_blocks(
        _cuda(k_cache, "k_cache"), _cuda(v_cache, "v_cache"),
        _cuda(src_blocks, "src_blocks", torch.int32), _cuda(dst_blocks, "dst_blocks", torch.int32),
        n, h_kv, head_dim, block_size, num_blocks, _elt(k_cache, "k_cache"), _stream(stream)))


_FP8_CACHE = (torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8))


def _fp8_cache(t: torch.Tensor, name: str) -> int:
    if t.dtype not in _FP8_CACHE:
        raise TypeError(f"{name} must hold e4m3 codes (uint8 or float8_e4m3fn), got {t.dtype}")
    return _cuda(t, name)


def pa_append_kv_fp8(k_cache: torch.Tensor, v_cache: torch.Tensor, k_new: torch.Tensor,
                     v_new: torch.Tensor, slot_mapping: torch.Tensor, k_scale: torch.Tensor,
                     v_scale: torch.Tensor, stream=None) -> None:
    """Quantise 16-bit rows k_new[t], v_new[t] into slot slot_mapping[t] of FP8 caches."""
    num_blocks, h_kv, block_size, head_dim = _cache_dims(k_cache)
    n_tokens = int(slot_mapping.shape[0])
    if k_new.shape != (n_tokens, h_kv, head_dim) or v_new.shape != k_new.shape:
        raise ValueError("k_new/v_new must be [n_tokens, num_kv_heads, head_dim]")
    _check("pa_append_kv_fp8", load().pa_append_kv_fp8(
        _fp8_cache(k_cache, "k_cache"), _fp8_cache(v_cache, "v_cache"), _cuda(k_new, "k_new"),
        _cuda(v_new, "v_new"), _cuda(slot_mapping, "slot_mapping", torch.int64), n_tokens, h_kv,
        head_dim, block_size, num_blocks, _elt(k_new, "k_new"),
        _cuda(k_scale, "k_scale", torch.float32), _cuda(v_scale, "v_scale", torch.float32),
        _stream(stream)))


def pa_decode_fp8(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                  v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                  block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                  q_len: int = 1, num_splits: int = 1, workspace: torch.Tensor | None = None,
                  k_new: torch.Tensor | None = None, v_new: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """Attention over FP8 caches; with k_new/v_new the new rows are appended first
    (quantised, same launch).  num_splits > 1 uses the split-KV pair."""
    num_blocks, h_kv, block_size, head_dim, num_seqs, h_q, maxb = _decode_dims(
        q, k_cache, block_tables, context_lens, q_len)
    if out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must match q")
    kn = vn = None
    if k_new is not None or v_new is not None:
        if k_new is None or v_new is None or k_new.shape != (num_seqs * q_len, h_kv, head_dim) \
                or v_new.shape != k_new.shape or k_new.dtype != q.dtype:
            raise ValueError("k_new/v_new must both be [num_seqs * q_len, num_kv_heads, head_dim]"
                             " of q's dtype")
        kn, vn = _cuda(k_new, "k_new"), _cuda(v_new, "v_new")
    ws_ptr, ws_bytes = None, 0
    if num_splits > 1:
        if workspace is None:
            nbytes = pa_decode_workspace_size(num_seqs, h_q, q_len, head_dim, num_splits)
            workspace = _made((nbytes,), torch.uint8, q.device, stream)
        ws_ptr, ws_bytes = _cuda(workspace, "workspace"), workspace.numel() * workspace.element_size()
    _check("pa_decode_fp8", load().pa_decode_fp8(
        _cuda(out, "out"), _cuda(q, "q"), kn, vn, _fp8_cache(k_cache, "k_cache"),
        _fp8_cache(v_cache, "v_cache"), _cuda(k_scale, "k_scale", torch.float32),
        _cuda(v_scale, "v_scale", torch.float32), _cuda(block_tables, "block_tables", torch.int32),
        _cuda(context_lens, "context_lens", torch.int32), num_seqs, h_q, h_kv, head_dim,
        block_size, float(scale), maxb, num_blocks, q_len, _elt(q, "q"), num_splits, ws_ptr,
        ws_bytes, _stream(stream)))
    return out


def _decode_dims(q, k_cache, block_tables, context_lens, q_len):
    num_blocks, h_kv, block_size, head_dim = _cache_dims(k_cache)
    num_seqs = int(context_lens.shape[0])
    if q.dim() == 3:  # [num_seqs, num_q_heads, head_dim] with q_len == 1
        q_len_t, h_q = 1, int(q.shape[1])
    else:
        q_len_t, h_q = int(q.shape[1]), int(q.shape[2])
    if q_len_t != q_len or int(q.shape[0]) != num_seqs or int(q.shape[-1]) != head_dim:
        raise ValueError("q must be [num_seqs, q_len, num_q_heads, head_dim]")
    if block_tables.dim() != 2 or int(block_tables.shape[0]) != num_seqs:
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq]")
    return num_blocks, h_kv, block_size, head_dim, num_seqs, h_q, int(block_tables.shape[1])


def pa_decode(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
              q_len: int = 1, stream=None) -> torch.Tensor:
    """Single-pass paged attention; writes and returns ``out`` (shape of q)."""
    num_blocks, h_kv, block_size, head_dim, num_seqs, h_q, maxb = _decode_dims(
        q, k_cache, block_tables, context_lens, q_len)
    if out.shape != q.shape or out.dtype != q.dtype or q.dtype != k_cache.dtype:
        raise ValueError("out must match q; q must have the cache dtype")
    _check("pa_decode", load().pa_decode(
        _cuda(out, "out"), _cuda(q, "q"), _cuda(k_cache, "k_cache"), _cuda(v_cache, "v_cache"),
        _cuda(block_tables, "block_tables", torch.int32),
        _cuda(context_lens, "context_lens", torch.int32), num_seqs, h_q, h_kv, head_dim,
        block_size, float(scale), _stream(stream), maxb, num_blocks, q_len,
        _elt(k_cache, "k_cache")))
    return out


def pa_decode_workspace_size(num_seqs: int, num_q_heads: int, q_len: int, head_dim: int,
                             num_splits: int) -> int:
    """Bytes of the split-KV workspace for these sizes (0 for invalid ones)."""
    return int(load().pa_decode_workspace_size(num_seqs, num_q_heads, q_len, head_dim, num_splits))


def workspace_views(workspace: torch.Tensor, num_seqs: int, num_q_heads: int, q_len: int,
                    head_dim: int, num_splits: int):
    """fp32 views (acc, m, l) of a split-KV workspace, per the header's layout."""
    rows = q_len * num_q_heads
    n = num_seqs * num_splits * rows
    align = lambda x: (x + 255) // 256 * 256  # noqa: E731
    acc_b, m_b = align(n * head_dim * 4), align(n * 4)
    raw = workspace.view(torch.uint8)
    acc = raw[:n * head_dim * 4].view(torch.float32).view(num_seqs, num_splits, rows, head_dim)
    m = raw[acc_b:acc_b + n * 4].view(torch.float32).view(num_seqs, num_splits, rows)
    l = raw[acc_b + m_b:acc_b + m_b + n * 4].view(torch.float32).view(num_seqs, num_splits, rows)
    return acc, m, l


def pa_decode_partial(workspace: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, block_tables: torch.Tensor,
                      context_lens: torch.Tensor, scale: float, num_splits: int,
                      q_len: int = 1, stream=None) -> torch.Tensor:
    """Split-KV pass: each of num_splits partitions of every sequence's blocks writes
    its (m, l, unnormalised acc) into the workspace; returns the workspace."""
    num_blocks, h_kv, block_size, head_dim, num_seqs, h_q, maxb = _decode_dims(
        q, k_cache, block_tables, context_lens, q_len)
    nbytes = workspace.numel() * workspace.element_size()
    _check("pa_decode_partial", load().pa_decode_partial(
        _cuda(workspace, "workspace"), nbytes, _cuda(q, "q"), _cuda(k_cache, "k_cache"),
        _cuda(v_cache, "v_cache"), _cuda(block_tables, "block_tables", torch.int32),
        _cuda(context_lens, "context_lens", torch.int32), num_seqs, h_q, h_kv, head_dim,
        block_size, float(scale), num_splits, maxb, num_blocks, q_len, _elt(k_cache, "k_cache"),
        _stream(stream)))
    return workspace


def pa_decode_combine(out: torch.Tensor, workspace: torch.Tensor, num_splits: int,
                      stream=None) -> torch.Tensor:
    """out: [num_seqs, q_len, num_q_heads, head_dim] (or 3-D with q_len 1)."""
    if out.dim() == 3:
        num_seqs, q_len, h_q, head_dim = int(out.shape[0]), 1, int(out.shape[1]), int(out.shape[2])
    else:
        num_seqs, q_len, h_q, head_dim = (int(x) for x in out.shape)
    nbytes = workspace.numel() * workspace.element_size()
    _check("pa_decode_combine", load().pa_decode_combine(
        _cuda(out, "out"), _cuda(workspace, "workspace"), nbytes, num_seqs, h_q, head_dim, q_len,
        num_splits, _elt(out, "out"), _stream(stream)))
    return out


def pa_selftest_wait_timeout(stream=None) -> None:
    """Launch the bounded-wait self-test (sets PA_ERR_DEVICE_TIMEOUT after ~2 s)."""
    _check("pa_selftest_wait_timeout", load().pa_selftest_wait_timeout(_stream(stream)))


def pa_device_error(stream=None, clear: bool = True) -> int:
    """Synchronise the stream; return the device error status (PA_OK == 0)."""
    return int(load().pa_device_error(_stream(stream), 1 if clear else 0))


def pa_append_decode(out: torch.Tensor, q: torch.Tensor, k_new: torch.Tensor,
                     v_new: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                     q_len: int = 1, num_splits: int = 1, workspace: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Fused step: slot mapping + append of k_new/v_new + attention (one launch)."""
    num_blocks, h_kv, block_size, head_dim, num_seqs, h_q, maxb = _decode_dims(
        q, k_cache, block_tables, context_lens, q_len)
    if out.shape != q.shape or out.dtype != q.dtype or q.dtype != k_cache.dtype:
        raise ValueError("out must match q; q must have the cache dtype")
    if k_new.shape != (num_seqs * q_len, h_kv, head_dim) or v_new.shape != k_new.shape:
        raise ValueError("k_new/v_new must be [num_seqs * q_len, num_kv_heads, head_dim]")
    for t, nm in ((k_new, "k_new"), (v_new, "v_new"), (v_cache, "v_cache")):
        if t.dtype != k_cache.dtype:
            raise TypeError(f"{nm} must have the cache dtype {k_cache.dtype}")
    ws_ptr, ws_bytes = None, 0
    if num_splits > 1:
        if workspace is None:
            nbytes = pa_decode_workspace_size(num_seqs, h_q, q_len, head_dim, num_splits)
            workspace = _made((nbytes,), torch.uint8, q.device, stream)
        ws_ptr, ws_bytes = _cuda(workspace, "workspace"), workspace.numel() * workspace.element_size()
    _check("pa_append_decode", load().pa_append_decode(
        _cuda(out, "out"), _cuda(q, "q"), _cuda(k_new, "k_new"), _cuda(v_new, "v_new"),
        _cuda(k_cache, "k_cache"), _cuda(v_cache, "v_cache"),
        _cuda(block_tables, "block_tables", torch.int32),
        _cuda(context_lens, "context_lens", torch.int32), num_seqs, h_q, h_kv, head_dim,
        block_size, float(scale), maxb, num_blocks, q_len, _elt(k_cache, "k_cache"), num_splits,
        ws_ptr, ws_bytes, _stream(stream)))
    return out


def pa_decode_cascade(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, block_tables: torch.Tensor,
                      context_lens: torch.Tensor, scale: float, prefix_blocks: int,
                      q_len: int = 1, tail_splits: int = 1, k_new: torch.Tensor | None = None,
                      v_new: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """Attention of a batch sharing its first ``prefix_blocks`` blocks (block-table row
    0): one pass over the shared prefix for all rows, one over each sequence's own
    blocks (with the append of k_new/v_new when given), then the combine."""
    num_blocks, h_kv, block_size, head_dim, num_seqs, h_q, maxb = _decode_dims(
        q, k_cache, block_tables, context_lens, q_len)
    if out.shape != q.shape or out.dtype != q.dtype or q.dtype != k_cache.dtype:
        raise ValueError("out must match q; q must have the cache dtype")
    if (k_new is None) != (v_new is None):
        raise ValueError("give both k_new and v_new, or neither")
    if k_new is not None:
        if k_new.shape != (num_seqs * q_len, h_kv, head_dim) or v_new.shape != k_new.shape:
            raise ValueError("k_new/v_new must be [num_seqs * q_len, num_kv_heads, head_dim]")
        for t, nm in ((k_new, "k_new"), (v_new, "v_new")):
            if t.dtype != k_cache.dtype:
                raise TypeError(f"{nm} must have the cache dtype {k_cache.dtype}")
    if workspace is None:
        nbytes = pa_decode_workspace_size(num_seqs, h_q, q_len, head_dim, 1 + tail_splits)
        workspace = _made((nbytes,), torch.uint8, q.device, stream)
    _check("pa_decode_cascade", load().pa_decode_cascade(
        _cuda(out, "out"), _cuda(q, "q"),
        None if k_new is None else _cuda(k_new, "k_new"),
        None if v_new is None else _cuda(v_new, "v_new"),
        _cuda(k_cache, "k_cache"), _cuda(v_cache, "v_cache"),
        _cuda(block_tables, "block_tables", torch.int32),
        _cuda(context_lens, "context_lens", torch.int32), num_seqs, h_q, h_kv, head_dim,
        block_size, float(scale), maxb, num_blocks, q_len, _elt(k_cache, "k_cache"),
        int(prefix_blocks), int(tail_splits), _cuda(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def paged_decode_step(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                      k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                      context_lens: torch.Tensor, scale: float, q_len: int = 1,
                      num_splits: int = 1, out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None,
                      slot_mapping: torch.Tensor | None = None, stream=None,
                      fused: bool = False) -> torch.Tensor:
    """One decode step: slot mapping, KV append, then attention.

    fused=False runs pa_slot_mapping -> pa_append_kv -> pa_decode (num_splits == 1)
    or pa_decode_partial + pa_decode_combine (num_splits > 1) on one stream;
    fused=True runs the same step as pa_append_decode (one launch, two with splits).
    Optional ``out``, ``workspace`` and ``slot_mapping`` buffers are reused when
    given (no allocation on the hot path).
    """
    if fused:
        if out is None:
            out = _made(q.shape, q.dtype, q.device, stream)
        return pa_append_decode(out, q, k_new, v_new, k_cache, v_cache, block_tables,
                                context_lens, scale, q_len, num_splits, workspace, stream)
    block_size = int(k_cache.shape[2])
    slot_mapping = pa_slot_mapping(block_tables, context_lens, block_size, q_len,
                                   out=slot_mapping, stream=stream)
    pa_append_kv(k_cache, v_cache, k_new, v_new, slot_mapping, stream=stream)
    if out is None:
        out = _made(q.shape, q.dtype, q.device, stream)
    if num_splits <= 1:
        return pa_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale, q_len,
                         stream=stream)
    if workspace is None:
        num_seqs, h_q, head_dim = int(q.shape[0]), int(q.shape[-2]), int(q.shape[-1])
        nbytes = pa_decode_workspace_size(num_seqs, h_q, q_len, head_dim, num_splits)
        workspace = _made((nbytes,), torch.uint8, q.device, stream)
    pa_decode_partial(workspace, q, k_cache, v_cache, block_tables, context_lens, scale,
                      num_splits, q_len, stream=stream)
    return pa_decode_combine(out, workspace, num_splits, stream=stream)


def pa_decode_split_noalloc(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                            v_cache: torch.Tensor, block_tables: torch.Tensor,
                            context_lens: torch.Tensor, scale: float, num_splits: int,
                            q_len: int = 1, stream=None) -> torch.Tensor:
    """Split-KV attention whose workspace is the library's fixed device array.

    For callers that may not allocate device memory at this point; no tensor is
    allocated here either.  Raises PagedAttnError (PA_ERR_INVALID_ARG) when the
    workspace this call needs exceeds NOALLOC_SCRATCH_BYTES.  Calls that can run
    concurrently on one GPU share the array and must be ordered by the caller.
    """
    num_blocks, h_kv, block_size, head_dim, num_seqs, h_q, maxb = _decode_dims(
        q, k_cache, block_tables, context_lens, q_len)
    if out.shape != q.shape or out.dtype != q.dtype or q.dtype != k_cache.dtype:
        raise ValueError("out must match q; q must have the cache dtype")
    _check("pa_decode_split_noalloc", load().pa_decode_split_noalloc(
        _cuda(out, "out"), _cuda(q, "q"), _cuda(k_cache, "k_cache"), _cuda(v_cache, "v_cache"),
        _cuda(block_tables, "block_tables", torch.int32),
        _cuda(context_lens, "context_lens", torch.int32), num_seqs, h_q, h_kv, head_dim,
        block_size, float(scale), num_splits, maxb, num_blocks, q_len, _elt(k_cache, "k_cache"),
        _stream(stream)))
    return out


# ------------------------------------------------- rotary append, scored decode, eviction
# These calls are short on the GPU (a few microseconds for a decode step's tokens), so a
# call on the current stream goes through csrc/pa_calls.cpp, which makes the checks below
# in compiled code and answers None where one fails.  What it does not take (another
# stream, buffers to be made, padded vocabularies, anything wrong) comes here; the checks
# too are written for the host's time, with the reason worked out only where one fails.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _device_of(t) -> int:
    """Device of the call's first tensor: the calls launch on the current device, so
    tensors of another one are refused."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("tensors must be CUDA tensors")
    dev = t.get_device()
    if dev != _raw_device():
        raise ValueError(f"tensors are on cuda:{dev}, the current device is cuda:{_raw_device()}")
    return dev


def _stream_on(stream, dev: int) -> int:
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream(stream)


def _refuse(t, name: str, dtype, dev: int):
    _cuda(t, name, dtype)
    raise ValueError(f"{name} is on cuda:{t.get_device()}, the others on cuda:{dev}")


def _ptr(t, name: str, dtype, dev: int) -> int:
    """Pointer of a contiguous tensor of this type on this device."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:  # not a tensor
        pass
    _refuse(t, name, dtype, dev)


def _cache_shape(k_cache) -> tuple:
    shape = k_cache.shape
    if len(shape) != 4:
        raise ValueError("caches must be [num_blocks, num_kv_heads, block_size, head_dim]")
    return shape


def _shape(t, name: str, want: tuple) -> None:
    if t.shape != want:
        raise ValueError(f"{name} must be {list(want)}, got {list(t.shape)}")


def _cache_pair(k_cache, v_cache, k_scale, v_scale, elt, shape, dev: int):
    """Pointers of the caches and their scales (None, None: 16-bit caches of type elt)."""
    if (k_scale is None) != (v_scale is None):
        raise ValueError("give both k_scale and v_scale, or neither")
    _shape(v_cache, "v_cache", shape)
    if k_scale is None:
        return _ptr(k_cache, "k_cache", elt, dev), _ptr(v_cache, "v_cache", elt, dev), None, None
    dt = k_cache.dtype
    if dt not in _FP8_CACHE:
        raise TypeError(f"k_cache must hold e4m3 codes (uint8 or float8_e4m3fn), got {dt}")
    _shape(k_scale, "k_scale", (shape[1],))
    _shape(v_scale, "v_scale", (shape[1],))
    return (_ptr(k_cache, "k_cache", dt, dev), _ptr(v_cache, "v_cache", dt, dev),
            _ptr(k_scale, "k_scale", torch.float32, dev), _ptr(v_scale, "v_scale", torch.float32, dev))


def _tokens3(t, name: str, dtype, dev: int, shape) -> tuple[int, int]:
    """Pointer and token stride of [n_tokens, heads, head_dim] with dense heads (a slice
    of a fused projection's output is fine)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev:
        _cuda(t, name, dtype)
        raise ValueError(f"{name} must be on cuda:{dev}")
    _shape(t, name, shape)
    n, h, d = shape
    if t.is_contiguous():
        return t.data_ptr(), h * d
    sn, sh, sd = t.stride()
    if (sd != 1 and d > 1) or (sh != d and h > 1):
        raise ValueError(f"{name}: the heads of a token must be dense")
    return t.data_ptr(), sn if n > 1 else h * d


def rope_table(head_dim: int, rotary_dim: int | None = None, base: float = 10000.0,
               sections=None, inv_freq=None, device="cuda"):
    """(turns, pair_axis) of pa_rope_append, made once per model.

    inv_freq: rotary_dim / 2 angles per position (floats; default base ** (-2i /
    rotary_dim)).  sections: how many consecutive pairs each position axis turns, in
    order (default: one axis turns all).
    """
    rotary_dim = head_dim if rotary_dim is None else rotary_dim
    half = rotary_dim // 2
    if inv_freq is None:
        inv_freq = [base ** (-2.0 * i / rotary_dim) for i in range(half)]
    inv_freq = [float(f) for f in inv_freq]
    sections = [half] if sections is None else [int(n) for n in sections]
    if len(inv_freq) != half or sum(sections) != half or min(sections) < 0:
        raise ValueError("inv_freq and sections must cover rotary_dim / 2 pairs")
    turns = [round(f / (2 * math.pi) * 2.0 ** 64) % (1 << 64) for f in inv_freq]
    turns = [x - (1 << 64) if x >= 1 << 63 else x for x in turns]
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    return (torch.tensor(turns, dtype=torch.int64, device=device),
            torch.tensor(axis, dtype=torch.int32, device=device))


def pa_rope_append(q_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                   k_cache: torch.Tensor, v_cache: torch.Tensor, positions: torch.Tensor,
                   slot_mapping: torch.Tensor, turns: torch.Tensor, pair_axis: torch.Tensor,
                   interleaved: bool = False, k_scale: torch.Tensor | None = None,
                   v_scale: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rotate q into q_out (which may be q) and k on its way into the cache, with v.

    q, q_out [n_tokens, num_q_heads, head_dim]; k, v [n_tokens, num_kv_heads, head_dim];
    tokens may be strided.  positions int32 [num_axes, n_tokens] (or [n_tokens] for one
    axis); turns, pair_axis from rope_table.  k_scale, v_scale: FP8 caches.
    """
    if stream is None and _fast is not None:
        st = _fast.rope_append(q_out, q, k, v, k_cache, v_cache, positions, slot_mapping, turns,
                                pair_axis, interleaved, k_scale, v_scale)
        if st == PA_OK:
            return q_out
        if st is not None:
            raise PagedAttnError("pa_rope_append", st)
    dev = _device_of(q)
    num_blocks, h_kv, block_size, head_dim = cache = _cache_shape(k_cache)
    elt = q.dtype
    dt = _elt(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [n_tokens, num_q_heads, head_dim]")
    q_shape = q.shape
    n_tokens, h_q, q_dim = q_shape
    if q_dim != head_dim:
        raise ValueError("q must have the cache's head_dim")
    kv_shape = (n_tokens, h_kv, head_dim)
    q_ptr, q_st = _tokens3(q, "q", elt, dev, q_shape)
    o_ptr, o_st = _tokens3(q_out, "q_out", elt, dev, q_shape)
    k_ptr, k_st = _tokens3(k, "k", elt, dev, kv_shape)
    v_ptr, v_st = _tokens3(v, "v", elt, dev, kv_shape)
    kc, vc, ks, vs = _cache_pair(k_cache, v_cache, k_scale, v_scale, elt, cache, dev)
    axes = positions.shape[0] if positions.dim() == 2 else 1
    if positions.numel() != axes * n_tokens:
        raise ValueError("positions must be [num_axes, n_tokens]")
    _shape(slot_mapping, "slot_mapping", (n_tokens,))
    if turns.dim() != 1:
        raise ValueError("turns must be [rotary_dim / 2]")
    half = turns.shape[0]
    _shape(pair_axis, "pair_axis", (half,))
    args = (_ptr(positions, "positions", torch.int32, dev),
            _ptr(slot_mapping, "slot_mapping", torch.int64, dev),
            _ptr(turns, "turns", torch.int64, dev), _ptr(pair_axis, "pair_axis", torch.int32, dev))
    if n_tokens == 0:
        return q_out
    st = (_lib or load()).pa_rope_append(
        o_ptr, q_ptr, k_ptr, v_ptr, kc, vc, *args, n_tokens, h_q, h_kv, head_dim, 2 * half, axes,
        interleaved, o_st, q_st, k_st, v_st, block_size, num_blocks, dt, ks, vs,
        _stream_on(stream, dev))
    if st != PA_OK:
        raise PagedAttnError("pa_rope_append", st)
    return q_out


def pa_decode_scored_workspace_size(num_seqs: int, num_q_heads: int, q_len: int, head_dim: int,
                                    num_splits: int, max_blocks_per_seq: int,
                                    block_size: int) -> int:
    """Bytes of pa_decode_scored's workspace (0 for invalid sizes)."""
    return int(load().pa_decode_scored_workspace_size(num_seqs, num_q_heads, q_len, head_dim,
                                                      num_splits, max_blocks_per_seq, block_size))


def pa_decode_scored(out: torch.Tensor, scores: torch.Tensor, q: torch.Tensor,
                     k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                     context_lens: torch.Tensor, scale: float, q_len: int = 1, num_splits: int = 1,
                     workspace: torch.Tensor | None = None, row_pos: torch.Tensor | None = None,
                     seq_lens: torch.Tensor | None = None, k_scale: torch.Tensor | None = None,
                     v_scale: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Paged attention that also adds every cached row's attention weight to scores
    (and notes the positions of this step's rows in row_pos).  FP8 caches with scales."""
    if stream is None and _fast is not None:
        st = _fast.decode_scored(out, scores, q, k_cache, v_cache, block_tables, context_lens, scale,
                                  q_len, num_splits, workspace, row_pos, seq_lens, k_scale, v_scale)
        if st == PA_OK:
            return out
        if st is not None:
            raise PagedAttnError("pa_decode_scored", st)
    dev = _device_of(q)
    num_blocks, h_kv, block_size, head_dim = cache = _cache_shape(k_cache)
    elt = q.dtype
    dt = _elt(q, "q")
    q_shape, tables = q.shape, block_tables.shape
    if len(tables) != 2:
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq]")
    num_seqs, maxb = tables
    h_q = q_shape[-2]
    if q_shape != (num_seqs, q_len, h_q, head_dim) and (q_len != 1 or q_shape != (num_seqs, h_q, head_dim)):
        raise ValueError("q must be [num_seqs, q_len, num_q_heads, head_dim]")
    _shape(context_lens, "context_lens", (num_seqs,))
    _shape(out, "out", q_shape)
    ledger = (num_seqs, h_kv, maxb * block_size)
    _shape(scores, "scores", ledger)
    if (row_pos is None) != (seq_lens is None):
        raise ValueError("give both row_pos and seq_lens, or neither")
    rp = sl = None
    if row_pos is not None:
        _shape(row_pos, "row_pos", ledger)
        _shape(seq_lens, "seq_lens", (num_seqs,))
        rp, sl = _ptr(row_pos, "row_pos", torch.int32, dev), _ptr(seq_lens, "seq_lens", torch.int32, dev)
    kc, vc, ks, vs = _cache_pair(k_cache, v_cache, k_scale, v_scale, elt, cache, dev)
    if workspace is None:
        nbytes = pa_decode_scored_workspace_size(num_seqs, h_q, q_len, head_dim, num_splits, maxb,
                                                 block_size)
        workspace = _made((nbytes,), torch.uint8, q.device, stream)
    st = (_lib or load()).pa_decode_scored(
        _ptr(out, "out", elt, dev), _ptr(scores, "scores", torch.float32, dev), rp,
        _ptr(q, "q", elt, dev), kc, vc, ks, vs, _ptr(block_tables, "block_tables", torch.int32, dev),
        _ptr(context_lens, "context_lens", torch.int32, dev), sl, num_seqs, h_q, h_kv, head_dim,
        block_size, scale, maxb, num_blocks, q_len, dt, num_splits,
        _ptr(workspace, "workspace", workspace.dtype, dev), workspace.nbytes,
        _stream_on(stream, dev))
    if st != PA_OK:
        raise PagedAttnError("pa_decode_scored", st)
    return out


def pa_evict_workspace_size(num_seqs: int, num_kv_heads: int, budget: int) -> int:
    """Bytes of pa_evict's workspace (0 for invalid sizes)."""
    return int(load().pa_evict_workspace_size(num_seqs, num_kv_heads, budget))


def pa_evict(k_cache: torch.Tensor, v_cache: torch.Tensor, scores: torch.Tensor,
             row_pos: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
             seq_lens: torch.Tensor, budget: int, sinks: int = 0, recent: int = 0,
             scores_out: torch.Tensor | None = None, row_pos_out: torch.Tensor | None = None,
             new_lens: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
    """Shorten every sequence longer than ``budget`` rows to it, each KV head keeping its
    first ``sinks`` and last ``recent`` positions and its highest scores.  The ledgers are
    updated in place unless both outputs are given.  Returns the new context lengths."""
    if stream is None and _fast is not None:
        st = _fast.evict(k_cache, v_cache, scores, row_pos, block_tables, context_lens, seq_lens, budget,
                          sinks, recent, scores_out, row_pos_out, new_lens, workspace)
        if st == PA_OK:
            return new_lens
        if st is not None:
            raise PagedAttnError("pa_evict", st)
    dev = _device_of(k_cache)
    num_blocks, h_kv, block_size, head_dim = cache = _cache_shape(k_cache)
    elt = k_cache.dtype
    if elt not in _DTYPE and elt not in _FP8_CACHE:
        raise TypeError(f"k_cache must be 16-bit or hold e4m3 codes, got {elt}")
    _shape(v_cache, "v_cache", cache)
    if block_tables.dim() != 2 or context_lens.dim() != 1:
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq], context_lens [num_seqs]")
    num_seqs, maxb = block_tables.shape
    per_seq, ledger = (num_seqs,), (num_seqs, h_kv, maxb * block_size)
    _shape(context_lens, "context_lens", per_seq)
    _shape(seq_lens, "seq_lens", per_seq)
    _shape(scores, "scores", ledger)
    _shape(row_pos, "row_pos", ledger)
    sc, rp = _ptr(scores, "scores", torch.float32, dev), _ptr(row_pos, "row_pos", torch.int32, dev)
    so, po = sc, rp
    if (scores_out is None) != (row_pos_out is None):
        raise ValueError("give both scores_out and row_pos_out, or neither")
    if scores_out is not None:
        _shape(scores_out, "scores_out", ledger)
        _shape(row_pos_out, "row_pos_out", ledger)
        so = _ptr(scores_out, "scores_out", torch.float32, dev)
        po = _ptr(row_pos_out, "row_pos_out", torch.int32, dev)
    if new_lens is None:
        new_lens = _made(per_seq, torch.int32, context_lens.device, stream)
    _shape(new_lens, "new_lens", per_seq)
    if workspace is None:
        nbytes = pa_evict_workspace_size(num_seqs, h_kv, budget)
        workspace = _made((nbytes,), torch.uint8, k_cache.device, stream)
    st = (_lib or load()).pa_evict(
        _ptr(k_cache, "k_cache", elt, dev), _ptr(v_cache, "v_cache", elt, dev), so, po,
        _ptr(new_lens, "new_lens", torch.int32, dev), sc, rp,
        _ptr(block_tables, "block_tables", torch.int32, dev),
        _ptr(context_lens, "context_lens", torch.int32, dev),
        _ptr(seq_lens, "seq_lens", torch.int32, dev), num_seqs, h_kv, head_dim, block_size, maxb,
        num_blocks, budget, sinks, recent, 2 if elt in _DTYPE else 1,
        _ptr(workspace, "workspace", workspace.dtype, dev), workspace.nbytes,
        _stream_on(stream, dev))
    if st != PA_OK:
        raise PagedAttnError("pa_evict", st)
    return new_lens


def _prob_rows(t, name: str, n: int, r: int, dev: int) -> tuple[int, int]:
    """Pointer and row stride of fp32 [n, r, vocab], rows dense and evenly spaced (a
    slice of a padded vocabulary is fine)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or t.get_device() != dev:
        raise TypeError(f"{name} must be a float32 tensor on cuda:{dev}")
    if t.dim() != 3 or t.shape[0] != n or t.shape[1] != r:
        raise ValueError(f"{name} must be [{n}, {r}, vocab]")
    vocab = t.shape[2]
    if t.is_contiguous():
        return t.data_ptr(), vocab
    s0, s1, s2 = t.stride()
    row = s1 if r > 1 else s0 if n > 1 else vocab
    if (vocab > 1 and s2 != 1) or (n > 1 and s0 != r * row):
        raise ValueError(f"{name}: rows must be dense and evenly spaced")
    return t.data_ptr(), row


def pa_verify_drafts(target_probs: torch.Tensor, draft_probs: torch.Tensor | None,
                     draft_tokens: torch.Tensor, accept_u: torch.Tensor, sample_u: torch.Tensor,
                     draft_lens: torch.Tensor | None = None,
                     context_lens: torch.Tensor | None = None,
                     out_tokens: torch.Tensor | None = None,
                     num_accepted: torch.Tensor | None = None,
                     new_lens: torch.Tensor | None = None, stream=None):
    """Accept drafted tokens and sample the one after them, from given uniforms.

    target_probs fp32 [num_seqs, max_draft + 1, vocab]; draft_probs fp32 [num_seqs,
    max_draft, vocab] or None (certain drafts); their rows may be padded (a slice of a
    wider vocabulary).  Returns (out_tokens, num_accepted, new_lens or None): new_lens
    is made when context_lens is given.
    """
    if stream is None and _fast is not None:
        st = _fast.verify_drafts(target_probs, draft_probs, draft_tokens, accept_u, sample_u, draft_lens,
                                  context_lens, out_tokens, num_accepted, new_lens)
        if st == PA_OK:
            return out_tokens, num_accepted, new_lens
        if st is not None:
            raise PagedAttnError("pa_verify_drafts", st)
    dev = _device_of(target_probs)
    if draft_tokens.dim() != 2:
        raise ValueError("draft_tokens must be [num_seqs, max_draft]")
    n, k = draft_tokens.shape
    i32, per_seq = torch.int32, (n,)
    p_ptr, p_st = _prob_rows(target_probs, "target_probs", n, k + 1, dev)
    vocab = target_probs.shape[2]
    q_ptr, q_st = None, 0
    if draft_probs is not None:
        q_ptr, q_st = _prob_rows(draft_probs, "draft_probs", n, k, dev)
        if draft_probs.shape[2] != vocab:
            raise ValueError("draft_probs must have target_probs' vocabulary")
    _shape(accept_u, "accept_u", (n, k))
    _shape(sample_u, "sample_u", per_seq)
    dl = cl = nl = None
    if draft_lens is not None:
        _shape(draft_lens, "draft_lens", per_seq)
        dl = _ptr(draft_lens, "draft_lens", i32, dev)
    if context_lens is not None:
        _shape(context_lens, "context_lens", per_seq)
        cl = _ptr(context_lens, "context_lens", i32, dev)
        if new_lens is None:
            new_lens = _made(per_seq, torch.int32, context_lens.device, stream)
    if new_lens is not None:
        if context_lens is None:
            raise ValueError("new_lens needs context_lens")
        _shape(new_lens, "new_lens", per_seq)
        nl = _ptr(new_lens, "new_lens", i32, dev)
    if out_tokens is None:
        out_tokens = _made((n, k + 1), i32, target_probs.device, stream)
    _shape(out_tokens, "out_tokens", (n, k + 1))
    if num_accepted is None:
        num_accepted = _made(per_seq, i32, target_probs.device, stream)
    _shape(num_accepted, "num_accepted", per_seq)
    st = (_lib or load()).pa_verify_drafts(
        _ptr(out_tokens, "out_tokens", i32, dev), _ptr(num_accepted, "num_accepted", i32, dev), nl, cl,
        p_ptr, q_ptr, _ptr(draft_tokens, "draft_tokens", i32, dev), dl,
        _ptr(accept_u, "accept_u", torch.float32, dev), _ptr(sample_u, "sample_u", torch.float32, dev),
        n, k, vocab, p_st, q_st, _stream_on(stream, dev))
    if st != PA_OK:
        raise PagedAttnError("pa_verify_drafts", st)
    return out_tokens, num_accepted, new_lens
