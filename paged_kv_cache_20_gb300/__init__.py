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
  kv_scales         fp32 [num_blocks, num_kv_heads, 2]  (K, V; a block-scaled FP8 cache)
  ref_counts        int32 [num_blocks]

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
PA_FP32 = 2   # the logits of pa_adjust_logits alone
_DTYPE = {torch.float16: PA_FP16, torch.bfloat16: PA_BF16}
_LOGIT_DTYPE = {**_DTYPE, torch.float32: PA_FP32}

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
    "pa_append_kv_block_scaled": (_c_int, [_c_vp] * 7 + [_c_int] * 8 + [_c_i64, _c_i64, _c_vp]),
    "pa_decode_block_scaled": (_c_int, [_c_vp] * 7 + [_c_int] * 5 + [_c_float] + [_c_int] * 5 +
                               [_c_vp, _c_size, _c_vp]),
    "pa_pages_workspace_size": (_c_size, [_c_int] * 2),
    "pa_free_blocks": (_c_int, [_c_vp] * 3 + [_c_int] * 4 + [_c_vp]),
    "pa_reserve_blocks": (_c_int, [_c_vp] * 4 + [_c_int] * 4 + [_c_vp, _c_size, _c_vp]),
    "pa_fork_blocks": (_c_int, [_c_vp] * 8 + [_c_int] * 5 + [_c_vp, _c_size, _c_vp]),
    "pa_compact_blocks": (_c_int, [_c_vp] * 7 + [_c_int] * 3 + [_c_vp, _c_size, _c_vp]),
    "pa_copy_pages": (_c_int, [_c_vp] * 6 + [_c_int] * 6 + [_c_vp]),
    "pa_adjust_logits": (_c_int, [_c_vp] * 13 + [_c_int] * 7 + [_c_i64] * 4 + [_c_vp]),
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


# ------------------------------------------------------ block-scaled FP8 cache
def _scaled_caches(k_cache, v_cache, kv_scales, dev: int):
    """Pointers of a block-scaled pool's codes and scales, and its shape."""
    cache = _cache_shape(k_cache)
    dt = k_cache.dtype
    if dt not in _FP8_CACHE:
        raise TypeError(f"k_cache must hold e4m3 codes (uint8 or float8_e4m3fn), got {dt}")
    _shape(v_cache, "v_cache", cache)
    _shape(kv_scales, "kv_scales", (cache[0], cache[1], 2))
    return (_ptr(k_cache, "k_cache", dt, dev), _ptr(v_cache, "v_cache", dt, dev),
            _ptr(kv_scales, "kv_scales", torch.float32, dev), cache)


def _tables(block_tables, dev: int) -> tuple:
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq]")
    return (_ptr(block_tables, "block_tables", torch.int32, dev), *block_tables.shape)


def pa_append_kv_block_scaled(k_cache: torch.Tensor, v_cache: torch.Tensor, kv_scales: torch.Tensor,
                              k_new: torch.Tensor, v_new: torch.Tensor, block_tables: torch.Tensor,
                              context_lens: torch.Tensor, q_len: int = 1, stream=None) -> None:
    """Quantise the last q_len positions of every sequence into a block-scaled FP8 cache,
    each block's scale grown where its rows need it.

    k_new, v_new [num_seqs * q_len, num_kv_heads, head_dim], 16-bit; tokens may be strided.
    """
    if stream is None and _fast is not None:
        st = _fast.append_kv_block_scaled(k_cache, v_cache, kv_scales, k_new, v_new, block_tables,
                                          context_lens, q_len)
        if st == PA_OK:
            return
        if st is not None:
            raise PagedAttnError("pa_append_kv_block_scaled", st)
    dev = _device_of(k_new)
    kc, vc, sp, (num_blocks, h_kv, block_size, head_dim) = _scaled_caches(k_cache, v_cache, kv_scales, dev)
    bt, num_seqs, maxb = _tables(block_tables, dev)
    _shape(context_lens, "context_lens", (num_seqs,))
    dt = _elt(k_new, "k_new")
    shape = (num_seqs * q_len, h_kv, head_dim)
    k_ptr, k_st = _tokens3(k_new, "k_new", k_new.dtype, dev, shape)
    v_ptr, v_st = _tokens3(v_new, "v_new", k_new.dtype, dev, shape)
    cl = _ptr(context_lens, "context_lens", torch.int32, dev)
    if num_seqs == 0:
        return
    st = (_lib or load()).pa_append_kv_block_scaled(
        kc, vc, sp, k_ptr, v_ptr, bt, cl, num_seqs, h_kv, head_dim, block_size, maxb, num_blocks, q_len,
        dt, k_st, v_st, _stream_on(stream, dev))
    if st != PA_OK:
        raise PagedAttnError("pa_append_kv_block_scaled", st)


def pa_decode_block_scaled(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           kv_scales: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                           scale: float, q_len: int = 1, num_splits: int = 1,
                           workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Paged attention over a block-scaled FP8 cache; writes and returns ``out`` (shape of
    q).  num_splits > 1 uses the split-KV pair."""
    if stream is None and _fast is not None:
        st = _fast.decode_block_scaled(out, q, k_cache, v_cache, kv_scales, block_tables, context_lens, scale,
                                       q_len, num_splits, workspace)
        if st == PA_OK:
            return out
        if st is not None:
            raise PagedAttnError("pa_decode_block_scaled", st)
    dev = _device_of(q)
    kc, vc, sp, (num_blocks, h_kv, block_size, head_dim) = _scaled_caches(k_cache, v_cache, kv_scales, dev)
    bt, num_seqs, maxb = _tables(block_tables, dev)
    dt, elt, q_shape = _elt(q, "q"), q.dtype, q.shape
    if len(q_shape) < 3:
        raise ValueError("q must be [num_seqs, q_len, num_q_heads, head_dim]")
    h_q = q_shape[-2]
    if q_shape != (num_seqs, q_len, h_q, head_dim) and (q_len != 1 or q_shape != (num_seqs, h_q, head_dim)):
        raise ValueError("q must be [num_seqs, q_len, num_q_heads, head_dim]")
    _shape(out, "out", q_shape)
    _shape(context_lens, "context_lens", (num_seqs,))
    ws, ws_bytes = None, 0
    if num_splits > 1:
        if workspace is None:
            nbytes = pa_decode_workspace_size(num_seqs, h_q, q_len, head_dim, num_splits)
            workspace = _made((nbytes,), torch.uint8, q.device, stream)
        ws, ws_bytes = _ptr(workspace, "workspace", workspace.dtype, dev), workspace.nbytes
    st = (_lib or load()).pa_decode_block_scaled(
        _ptr(out, "out", elt, dev), _ptr(q, "q", elt, dev), kc, vc, sp, bt,
        _ptr(context_lens, "context_lens", torch.int32, dev), num_seqs, h_q, h_kv, head_dim, block_size,
        scale, maxb, num_blocks, q_len, dt, num_splits, ws, ws_bytes, _stream_on(stream, dev))
    if st != PA_OK:
        raise PagedAttnError("pa_decode_block_scaled", st)
    return out


# ------------------------------------------------------------ the pool's blocks
def pa_pages_workspace_size(num_blocks: int, num_forks: int = 0) -> int:
    """Bytes of the bookkeeping calls' workspace (0 for invalid sizes)."""
    return int(load().pa_pages_workspace_size(num_blocks, num_forks))


def _pool(block_tables, ref_counts) -> tuple:
    """(device, table pointer, num_seqs, width, counts pointer, num_blocks)"""
    dev = _device_of(block_tables)
    if ref_counts.dim() != 1:
        raise ValueError("ref_counts must be [num_blocks]")
    return (dev, *_tables(block_tables, dev), _ptr(ref_counts, "ref_counts", torch.int32, dev),
            ref_counts.shape[0])


def _i32(t, name: str, shape: tuple, dev: int) -> int:
    _shape(t, name, shape)
    return _ptr(t, name, torch.int32, dev)


def _pages_room(workspace, num_blocks: int, num_forks: int, device, stream, dev: int) -> tuple:
    if workspace is None:
        workspace = _made((pa_pages_workspace_size(num_blocks, num_forks),), torch.uint8, device, stream)
    return workspace, _ptr(workspace, "workspace", workspace.dtype, dev), workspace.nbytes


def pa_free_blocks(block_tables: torch.Tensor, ref_counts: torch.Tensor, keep_lens: torch.Tensor,
                   block_size: int, stream=None) -> None:
    """Give up every sequence's blocks past its first keep_lens[i] tokens: their counts
    fall by one, their entries become -1."""
    if stream is None and _fast is not None:
        st = _fast.free_blocks(block_tables, ref_counts, keep_lens, block_size)
        if st == PA_OK:
            return
        if st is not None:
            raise PagedAttnError("pa_free_blocks", st)
    dev, bt, n, width, rc, num_blocks = _pool(block_tables, ref_counts)
    kl = _i32(keep_lens, "keep_lens", (n,), dev)
    st = (_lib or load()).pa_free_blocks(bt, rc, kl, n, width, num_blocks, block_size, _stream_on(stream, dev))
    if st != PA_OK:
        raise PagedAttnError("pa_free_blocks", st)


def pa_reserve_blocks(block_tables: torch.Tensor, ref_counts: torch.Tensor, lens: torch.Tensor, block_size: int,
                      missing: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """Blocks for every sequence's first lens[i] tokens where it has none: the lowest free
    ones, in the order of sequences.  Returns ``missing`` (int32 [1]): entries that found
    no free block."""
    if stream is None and _fast is not None:
        st = _fast.reserve_blocks(block_tables, ref_counts, lens, block_size, missing, workspace)
        if st == PA_OK:
            return missing
        if st is not None:
            raise PagedAttnError("pa_reserve_blocks", st)
    dev, bt, n, width, rc, num_blocks = _pool(block_tables, ref_counts)
    ln = _i32(lens, "lens", (n,), dev)
    if missing is None:
        missing = _made((1,), torch.int32, lens.device, stream)
    mp = _i32(missing, "missing", (1,), dev)
    workspace, ws, ws_bytes = _pages_room(workspace, num_blocks, 0, lens.device, stream, dev)
    st = (_lib or load()).pa_reserve_blocks(bt, rc, ln, mp, n, width, num_blocks, block_size, ws, ws_bytes,
                                            _stream_on(stream, dev))
    if st != PA_OK:
        raise PagedAttnError("pa_reserve_blocks", st)
    return missing


def pa_fork_blocks(block_tables: torch.Tensor, context_lens: torch.Tensor, ref_counts: torch.Tensor,
                   src_seqs: torch.Tensor, dst_seqs: torch.Tensor, block_size: int,
                   src_blocks: torch.Tensor | None = None, dst_blocks: torch.Tensor | None = None,
                   counts: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Sequences dst_seqs[f] become copies of src_seqs[f]: full blocks shared, partial last
    blocks to be copied.  Returns (src_blocks, dst_blocks, counts): the copies to make with
    pa_copy_pages, counts[0] of them; counts[1] forks found no free block."""
    if stream is None and _fast is not None:
        st = _fast.fork_blocks(block_tables, context_lens, ref_counts, src_seqs, dst_seqs, block_size, src_blocks,
                               dst_blocks, counts, workspace)
        if st == PA_OK:
            return src_blocks, dst_blocks, counts
        if st is not None:
            raise PagedAttnError("pa_fork_blocks", st)
    dev, bt, n, width, rc, num_blocks = _pool(block_tables, ref_counts)
    cl = _i32(context_lens, "context_lens", (n,), dev)
    if src_seqs.dim() != 1:
        raise ValueError("src_seqs must be [num_forks]")
    f = src_seqs.shape[0]
    ss, ds = _i32(src_seqs, "src_seqs", (f,), dev), _i32(dst_seqs, "dst_seqs", (f,), dev)
    device = block_tables.device
    if src_blocks is None:
        src_blocks = _made((f,), torch.int32, device, stream)
    if dst_blocks is None:
        dst_blocks = _made((f,), torch.int32, device, stream)
    if counts is None:
        counts = _made((2,), torch.int32, device, stream)
    sb, db = _i32(src_blocks, "src_blocks", (f,), dev), _i32(dst_blocks, "dst_blocks", (f,), dev)
    cp = _i32(counts, "counts", (2,), dev)
    workspace, ws, ws_bytes = _pages_room(workspace, num_blocks, f, device, stream, dev)
    st = (_lib or load()).pa_fork_blocks(bt, cl, rc, ss, ds, sb, db, cp, f, n, width, num_blocks, block_size, ws,
                                         ws_bytes, _stream_on(stream, dev))
    if st != PA_OK:
        raise PagedAttnError("pa_fork_blocks", st)
    return src_blocks, dst_blocks, counts


def pa_compact_blocks(block_tables: torch.Tensor, ref_counts: torch.Tensor,
                      block_tables_out: torch.Tensor | None = None, ref_counts_out: torch.Tensor | None = None,
                      src_blocks: torch.Tensor | None = None, dst_blocks: torch.Tensor | None = None,
                      counts: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Give the blocks in use the pool's lowest ids, in tables and counts (in place unless
    both outputs are given).  Returns (src_blocks, dst_blocks, counts): the copies to make
    with pa_copy_pages, counts[0] of them; counts[1] blocks are in use."""
    if stream is None and _fast is not None:
        st = _fast.compact_blocks(block_tables, ref_counts, block_tables_out, ref_counts_out, src_blocks,
                                  dst_blocks, counts, workspace)
        if st == PA_OK:
            return src_blocks, dst_blocks, counts
        if st is not None:
            raise PagedAttnError("pa_compact_blocks", st)
    dev, bt, n, width, rc, num_blocks = _pool(block_tables, ref_counts)
    if (block_tables_out is None) != (ref_counts_out is None):
        raise ValueError("give both block_tables_out and ref_counts_out, or neither")
    to, ro = bt, rc
    if block_tables_out is not None:
        to = _i32(block_tables_out, "block_tables_out", (n, width), dev)
        ro = _i32(ref_counts_out, "ref_counts_out", (num_blocks,), dev)
    device, most = block_tables.device, num_blocks // 2
    if src_blocks is None:
        src_blocks = _made((most,), torch.int32, device, stream)
    if dst_blocks is None:
        dst_blocks = _made((most,), torch.int32, device, stream)
    if counts is None:
        counts = _made((2,), torch.int32, device, stream)
    sb, db = _i32(src_blocks, "src_blocks", (most,), dev), _i32(dst_blocks, "dst_blocks", (most,), dev)
    cp = _i32(counts, "counts", (2,), dev)
    workspace, ws, ws_bytes = _pages_room(workspace, num_blocks, 0, device, stream, dev)
    st = (_lib or load()).pa_compact_blocks(to, ro, bt, rc, sb, db, cp, n, width, num_blocks, ws, ws_bytes,
                                            _stream_on(stream, dev))
    if st != PA_OK:
        raise PagedAttnError("pa_compact_blocks", st)
    return src_blocks, dst_blocks, counts


def pa_copy_pages(k_cache: torch.Tensor, v_cache: torch.Tensor, src_blocks: torch.Tensor, dst_blocks: torch.Tensor,
                  counts: torch.Tensor, kv_scales: torch.Tensor | None = None, stream=None) -> None:
    """Copy the first counts[0] listed blocks src_blocks[p] -> dst_blocks[p] of both caches
    (16-bit or FP8), with their scales where kv_scales is given."""
    if stream is None and _fast is not None:
        st = _fast.copy_pages(k_cache, v_cache, src_blocks, dst_blocks, counts, kv_scales)
        if st == PA_OK:
            return
        if st is not None:
            raise PagedAttnError("pa_copy_pages", st)
    dev = _device_of(k_cache)
    cache = num_blocks, h_kv, block_size, head_dim = _cache_shape(k_cache)
    elt = k_cache.dtype
    if elt not in _DTYPE and elt not in _FP8_CACHE:
        raise TypeError(f"k_cache must be 16-bit or hold e4m3 codes, got {elt}")
    _shape(v_cache, "v_cache", cache)
    sp = None
    if kv_scales is not None:
        _shape(kv_scales, "kv_scales", (num_blocks, h_kv, 2))
        sp = _ptr(kv_scales, "kv_scales", torch.float32, dev)
    if src_blocks.dim() != 1:
        raise ValueError("src_blocks must be [max_pairs]")
    most = src_blocks.shape[0]
    sb, db = _i32(src_blocks, "src_blocks", (most,), dev), _i32(dst_blocks, "dst_blocks", (most,), dev)
    _shape(counts, "counts", (2,))
    kc, vc = _ptr(k_cache, "k_cache", elt, dev), _ptr(v_cache, "v_cache", elt, dev)
    cp = _ptr(counts, "counts", torch.int32, dev)
    if most == 0:
        return
    st = (_lib or load()).pa_copy_pages(kc, vc, sp, sb, db, cp, most, h_kv, head_dim, block_size, num_blocks,
                                        2 if elt in _DTYPE else 1, _stream_on(stream, dev))
    if st != PA_OK:
        raise PagedAttnError("pa_copy_pages", st)


# ---------------------------------------------------------------------- logits
def _logit_rows(t, name: str, dtype, dev: int) -> tuple[int, int]:
    """Pointer and row stride of [n, r, vocab], rows dense and evenly spaced (a slice of a
    padded vocabulary is fine)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev:
        raise TypeError(f"{name} must be a {dtype} tensor on cuda:{dev}")
    n, r, vocab = t.shape
    if t.is_contiguous():
        return t.data_ptr(), vocab
    s0, s1, s2 = t.stride()
    row = s1 if r > 1 else s0 if n > 1 else vocab
    if (vocab > 1 and s2 != 1) or (n > 1 and s0 != r * row):
        raise ValueError(f"{name}: rows must be dense and evenly spaced")
    return t.data_ptr(), row


def pa_adjust_logits(out: torch.Tensor | None, logits: torch.Tensor, history: torch.Tensor | None = None,
                     history_lens: torch.Tensor | None = None, prompt_lens: torch.Tensor | None = None,
                     drafts: torch.Tensor | None = None, repetition: torch.Tensor | None = None,
                     presence: torch.Tensor | None = None, frequency: torch.Tensor | None = None,
                     bias_ids: torch.Tensor | None = None, bias_values: torch.Tensor | None = None,
                     mask: torch.Tensor | None = None, temperature: torch.Tensor | None = None,
                     probs: bool = False, stream=None) -> torch.Tensor:
    """Penalties for repeated tokens, biases and a grammar's mask on logits [num_seqs, rows,
    vocab] (fp16, bf16 or fp32), row j behind drafts[:, :j]; with ``probs`` the fp32
    probabilities at ``temperature`` that pa_verify_drafts takes.

    history int32 [num_seqs, max_history] with history_lens (and prompt_lens: where the
    prompt ends); drafts int32 [num_seqs, rows - 1]; the penalties and the temperature fp32
    [num_seqs]; bias_ids, bias_values [num_seqs, num_bias]; mask int32 [num_seqs, rows,
    ceil(vocab / 32)], which may be expanded over rows or sequences.  ``out`` (logits itself
    is fine) is made when None.
    """
    if stream is None and _fast is not None and out is not None:
        st = _fast.adjust_logits(out, logits, history, history_lens, prompt_lens, drafts, repetition, presence,
                                 frequency, bias_ids, bias_values, mask, temperature, probs)
        if st == PA_OK:
            return out
        if st is not None:
            raise PagedAttnError("pa_adjust_logits", st)
    dev = _device_of(logits)
    if logits.dtype not in _LOGIT_DTYPE:
        raise TypeError(f"logits must be float16, bfloat16 or float32, got {logits.dtype}")
    if logits.dim() != 3:
        raise ValueError("logits must be [num_seqs, rows, vocab]")
    n, r, vocab = logits.shape
    out_type = torch.float32 if probs else logits.dtype
    if out is None:
        out = _made((n, r, vocab), out_type, logits.device, stream)
    _shape(out, "out", (n, r, vocab))
    i_ptr, i_st = _logit_rows(logits, "logits", logits.dtype, dev)
    o_ptr, o_st = _logit_rows(out, "out", out_type, dev)
    if (history is None) != (history_lens is None):
        raise ValueError("give both history and history_lens, or neither")
    if prompt_lens is not None and history is None:
        raise ValueError("prompt_lens needs history")
    hp = hl = pl = None
    longest = 0
    if history is not None:
        if history.dim() != 2 or history.shape[0] != n:
            raise ValueError(f"history must be [{n}, max_history]")
        longest = history.shape[1]
        hp = _ptr(history, "history", torch.int32, dev)
        hl = _i32(history_lens, "history_lens", (n,), dev)
        if prompt_lens is not None:
            pl = _i32(prompt_lens, "prompt_lens", (n,), dev)
        if longest == 0:
            hp = hl = pl = None
    dp = _i32(drafts, "drafts", (n, r - 1), dev) if drafts is not None else None
    per = []
    for name, t in (("repetition", repetition), ("presence", presence), ("frequency", frequency),
                    ("temperature", temperature)):
        if t is not None:
            _shape(t, name, (n,))
        per.append(None if t is None else _ptr(t, name, torch.float32, dev))
    if (bias_ids is None) != (bias_values is None):
        raise ValueError("give both bias_ids and bias_values, or neither")
    bi = bv = None
    num_bias = 0
    if bias_ids is not None:
        if bias_ids.dim() != 2 or bias_ids.shape[0] != n:
            raise ValueError(f"bias_ids must be [{n}, num_bias]")
        num_bias = bias_ids.shape[1]
        bi = _ptr(bias_ids, "bias_ids", torch.int32, dev)
        _shape(bias_values, "bias_values", (n, num_bias))
        bv = _ptr(bias_values, "bias_values", torch.float32, dev)
        if num_bias == 0:
            bi = bv = None
    mp, m_seq, m_row = None, 0, 0
    if mask is not None:
        words = (vocab + 31) // 32
        _shape(mask, "mask", (n, r, words))
        if mask.dtype is not torch.int32 or mask.get_device() != dev:
            raise TypeError(f"mask must be an int32 tensor on cuda:{dev}")
        m_seq, m_row, one = mask.stride()
        if one != 1 and words > 1:
            raise ValueError("mask: the words of a row must be dense")
        mp, m_seq, m_row = mask.data_ptr(), m_seq if n > 1 else 0, m_row if r > 1 else 0
    if n == 0 or r == 0:
        return out
    st = (_lib or load()).pa_adjust_logits(
        o_ptr, i_ptr, hp, hl, pl, dp, per[0], per[1], per[2], bi, bv, mp, per[3], n, r, vocab, longest, num_bias,
        _LOGIT_DTYPE[logits.dtype], 1 if probs else 0, o_st, i_st, m_seq, m_row, _stream_on(stream, dev))
    if st != PA_OK:
        raise PagedAttnError("pa_adjust_logits", st)
    return out
