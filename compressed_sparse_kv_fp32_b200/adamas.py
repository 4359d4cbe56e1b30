"""Python binding of libadamas.so (C ABI in include/adamas.h).

Argument marshalling only: every step of the method runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors; calls are enqueued on the current torch
stream, or on `stream`, to which the tensors that such a call makes then belong
(another stream waits for it before it reads them, and is recorded on them before
they are given up).  The library must have been built
(compressed_sparse_kv_fp32_b200.build); there is no fallback of any kind.

Method: ADAMAS long-context sparse attention article (lnwmold.com/news/826806),
§2.1 Hadamard rotation, §2.2 dynamic 2-bit bucketing, §3.1 packed code cache,
§2.3 Manhattan-distance scoring, §5.2 token budget.  The cache operators at the end
(rope_append, chunk_attend, accumulate_kept, accumulate_chunk, evict) are what a
serving loop runs around the decode step on the same cache.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import Optional, Tuple

import torch

from .build import LIBRARY

HEAD_DIM = 128
DEVERR_SEQLEN = 0x1
DEVERR_TIMEOUT = 0x2

_lock = threading.Lock()
_lib = None

SYMBOLS = (
    "adamas_status_string", "adamas_version", "adamas_last_error_string", "adamas_workspace_bytes", "adamas_workspace_init",
    "adamas_encode_keys", "adamas_decode_step", "adamas_score", "adamas_get_device_error",
    "adamas_decode_step_static", "adamas_decode_step_append", "adamas_decode_step_ex",
    "adamas_static_device_error", "adamas_debug_withhold_stage",
    "adamas_shard_workspace_bytes", "adamas_shard_score", "adamas_shard_attend", "adamas_merge_partials",
    "adamas_rope_append", "adamas_chunk_workspace_bytes", "adamas_chunk_attend", "adamas_accumulate_chunk",
    "adamas_accumulate_kept", "adamas_evict",
)

SELECT_PER_HEAD = 0
SELECT_GROUP_SHARED = 1
DEVERR_INTERNAL = 0x4
DEVERR_TABLE = 0x8
DEVERR_OFFSETS = 0x10


class DecodeArgs(ctypes.Structure):
    """Mirror of adamas_decode_args (include/adamas.h), field for field."""

    _fields_ = [
        ("q", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("K", ctypes.c_void_p), ("V", ctypes.c_void_p),
        ("seq_lens", ctypes.c_void_p),
        ("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("Nmax", ctypes.c_int64),
        ("d", ctypes.c_int), ("budget", ctypes.c_int),
        ("out", ctypes.c_void_p), ("idx", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("append_pos", ctypes.c_void_p), ("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int),
        ("max_pages", ctypes.c_int), ("n_sink", ctypes.c_int), ("n_recent", ctypes.c_int), ("policy", ctypes.c_int),
    ]


_P, _I, _I64, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
_PAGED = [("block_table", _P), ("n_pages", _I64), ("page_size", _I), ("max_pages", _I)]
_WORKSPACE = [("workspace", _P), ("workspace_bytes", _SZ)]


class RopeArgs(ctypes.Structure):
    """Mirror of adamas_rope_args (include/adamas.h), field for field."""

    _fields_ = [("q", _P), ("k", _P), ("v", _P), ("q_stride", _I64), ("k_stride", _I64), ("v_stride", _I64),
                ("cu_new", _P), ("cache_lens", _P), ("positions", _P), ("freqs", _P), ("rot_dim", _I),
                ("interleaved", _I), ("mscale", ctypes.c_double), ("T", _I), ("B", _I), ("Hq", _I), ("Hkv", _I),
                ("Nmax", _I64), ("d", _I), ("q_out", _P), ("K", _P), ("V", _P), ("codes", _P),
                *_PAGED, *_WORKSPACE]


class ChunkArgs(ctypes.Structure):
    """Mirror of adamas_chunk_args (include/adamas.h), field for field."""

    _fields_ = [("q", _P), ("K", _P), ("V", _P), ("cu_q", _P), ("seq_lens", _P), ("T", _I), ("B", _I), ("Hq", _I),
                ("Hkv", _I), ("Nmax", _I64), ("d", _I), ("out", _P), ("lse", _P), ("mass", _P),
                *_PAGED, *_WORKSPACE]


class KeptArgs(ctypes.Structure):
    """Mirror of adamas_kept_args (include/adamas.h), field for field."""

    _fields_ = [("q", _P), ("K", _P), ("idx", _P), ("seq_lens", _P), ("B", _I), ("Hq", _I), ("Hkv", _I),
                ("Nmax", _I64), ("d", _I), ("budget", _I), ("policy", _I), ("mass", _P), *_PAGED, *_WORKSPACE]


class EvictArgs(ctypes.Structure):
    """Mirror of adamas_evict_args (include/adamas.h), field for field."""

    _fields_ = [("K", _P), ("V", _P), ("codes", _P), ("mass", _P), ("seq_lens", _P), ("B", _I), ("Hkv", _I),
                ("Nmax", _I64), ("d", _I), ("keep", _I), ("n_sink", _I), ("n_recent", _I), ("kept", _P),
                ("new_lens", _P), *_PAGED, ("K_out", _P), ("V_out", _P), ("codes_out", _P), ("mass_out", _P),
                ("Nmax_out", _I64), ("block_table_out", _P), ("n_pages_out", _I64), ("page_size_out", _I),
                ("max_pages_out", _I), *_WORKSPACE]


class AdamasError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = f": {load().adamas_last_error_string().decode()}" if status == -4 else ""
        super().__init__(f"{where}: {status_string(status)} ({status}){detail}")


def load(path: str = LIBRARY) -> ctypes.CDLL:
    """Load libadamas.so and declare its signatures (raises if it was not built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it with `python -m compressed_sparse_kv_fp32_b200.build`")
        l = ctypes.CDLL(path)
        P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        l.adamas_status_string.argtypes = [I]
        l.adamas_status_string.restype = ctypes.c_char_p
        l.adamas_version.argtypes = []
        l.adamas_version.restype = I
        l.adamas_last_error_string.argtypes = []
        l.adamas_last_error_string.restype = ctypes.c_char_p
        l.adamas_workspace_bytes.argtypes = [I, I, I, I64, I, I]
        l.adamas_workspace_bytes.restype = SZ
        l.adamas_workspace_init.argtypes = [P, SZ, P]
        l.adamas_workspace_init.restype = I
        l.adamas_encode_keys.argtypes = [P, P, P, I, I, I, I64, I, P]
        l.adamas_encode_keys.restype = I
        l.adamas_decode_step.argtypes = [P, P, P, P, P, I, I, I, I64, I, I, P, P, P, SZ, P]
        l.adamas_decode_step.restype = I
        l.adamas_score.argtypes = [P, P, P, I, I, I, I64, I, P, P]
        l.adamas_score.restype = I
        l.adamas_get_device_error.argtypes = [P, SZ, ctypes.POINTER(ctypes.c_uint32), P]
        l.adamas_get_device_error.restype = I
        l.adamas_decode_step_static.argtypes = [P, P, P, P, P, I, I, I, I64, I, I, P, P, P]
        l.adamas_decode_step_static.restype = I
        l.adamas_decode_step_append.argtypes = [P, P, P, P, P, P, I, I, I, I64, I, I, P, P, P, SZ, P]
        l.adamas_decode_step_append.restype = I
        l.adamas_decode_step_ex.argtypes = [ctypes.POINTER(DecodeArgs), P]
        l.adamas_decode_step_ex.restype = I
        l.adamas_static_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32), P]
        l.adamas_static_device_error.restype = I
        l.adamas_shard_workspace_bytes.argtypes = [I, I, I, I64, I, I]
        l.adamas_shard_workspace_bytes.restype = SZ
        l.adamas_shard_score.argtypes = [P, P, P, I, I, I, I64, I, I, P, P, SZ, P]
        l.adamas_shard_score.restype = I
        l.adamas_shard_attend.argtypes = [P, P, P, P, I, I, I, I64, I, I, P, I, I, P, P, P, SZ, P]
        l.adamas_shard_attend.restype = I
        l.adamas_merge_partials.argtypes = [P, I, I, I, P, P]
        l.adamas_merge_partials.restype = I
        for name, args in (("rope_append", RopeArgs), ("chunk_attend", ChunkArgs), ("accumulate_chunk", ChunkArgs),
                           ("accumulate_kept", KeptArgs), ("evict", EvictArgs)):
            fn = getattr(l, "adamas_" + name)
            fn.argtypes = [ctypes.POINTER(args), P]
            fn.restype = I
        l.adamas_chunk_workspace_bytes.argtypes = [I, I, I, I, I]
        l.adamas_chunk_workspace_bytes.restype = SZ
        l.adamas_debug_withhold_stage.argtypes = [I]
        l.adamas_debug_withhold_stage.restype = None
        _lib = l
        return l


def status_string(status: int) -> str:
    return load().adamas_status_string(int(status)).decode()


def _check(rc: int, where: str):
    if rc != 0:
        raise AdamasError(rc, where)


def _stream(stream: Optional[torch.cuda.Stream]) -> int:
    if stream is not None:
        return stream.cuda_stream
    # the current stream's handle alone: making a Stream object for it takes 3 us
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _make(fill, shape: tuple, dtype: torch.dtype, device, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """A tensor that a call makes for its results, by torch.empty or torch.zeros, as of the
    stream that the call goes to: on the current one its fill could land behind the
    call's kernels, and so could work that still writes to memory given back there."""
    if stream is None:
        return fill(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return fill(shape, dtype=dtype, device=device)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape: Optional[tuple] = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def workspace_bytes(B: int, Hq: int, Hkv: int, Nmax: int, budget: int, d: int = HEAD_DIM) -> int:
    n = load().adamas_workspace_bytes(B, Hq, Hkv, Nmax, d, budget)
    if n == 0:
        raise AdamasError(-2, "adamas_workspace_bytes")
    return int(n)


def shard_workspace_bytes(B: int, Hq: int, Hkv: int, Nmax: int, budget: int, d: int = HEAD_DIM) -> int:
    n = load().adamas_shard_workspace_bytes(B, Hq, Hkv, Nmax, d, budget)
    if n == 0:
        raise AdamasError(-2, "adamas_shard_workspace_bytes")
    return int(n)


class Workspace:
    """Device workspace of adamas_decode_step (or, with sharded=True, of the
    sequence-sharded step's two halves), zero-filled on creation."""

    def __init__(self, B: int, Hq: int, Hkv: int, Nmax: int, budget: int, device=None,
                 stream: Optional[torch.cuda.Stream] = None, sharded: bool = False):
        self.nbytes = (shard_workspace_bytes if sharded else workspace_bytes)(B, Hq, Hkv, Nmax, budget)
        self.buffer = _make(torch.empty, (self.nbytes,), torch.uint8, device if device is not None else "cuda", stream)
        self.reset(stream)

    def reset(self, stream: Optional[torch.cuda.Stream] = None):
        _check(load().adamas_workspace_init(self.buffer.data_ptr(), self.nbytes, _stream(stream)),
               "adamas_workspace_init")

    def device_error(self, stream: Optional[torch.cuda.Stream] = None) -> int:
        """Synchronise the stream and return the device error word (DEVERR_* bits)."""
        word = ctypes.c_uint32(0)
        rc = load().adamas_get_device_error(self.buffer.data_ptr(), self.nbytes, ctypes.byref(word),
                                            _stream(stream))
        if rc not in (0, -5):
            raise AdamasError(rc, "adamas_get_device_error")
        return int(word.value)


def encode_keys(K: torch.Tensor, codes: torch.Tensor, pos_begin: Optional[torch.Tensor] = None,
                count: Optional[int] = None, stream: Optional[torch.cuda.Stream] = None):
    """Encode K [B,Hkv,Nmax,128] bf16 into codes [B,Hkv,Nmax,32] uint8 at positions
    [pos_begin[b], pos_begin[b] + count) (all positions by default)."""
    _need(K, "K", torch.bfloat16)
    if K.dim() != 4 or K.shape[-1] != HEAD_DIM:
        raise ValueError("K must be [B, Hkv, Nmax, 128]")
    B, Hkv, Nmax, d = K.shape
    _need(codes, "codes", torch.uint8, (B, Hkv, Nmax, d // 4))
    if pos_begin is not None:
        _need(pos_begin, "pos_begin", torch.int32, (B,))
    n = Nmax if count is None else int(count)
    _check(load().adamas_encode_keys(K.data_ptr(), codes.data_ptr(), _ptr(pos_begin), n, B, Hkv, Nmax, d,
                                     _stream(stream)), "adamas_encode_keys")
    return codes


def _decode_args(q, codes, K, V, seq_lens, budget, out, idx, stream):
    _need(q, "q", torch.bfloat16)
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, 128]")
    B, Hq, d = q.shape
    _need(K, "K", torch.bfloat16)
    if K.dim() != 4:
        raise ValueError("K must be [B, Hkv, Nmax, 128]")
    _, Hkv, Nmax, _ = K.shape
    _need(K, "K", torch.bfloat16, (B, Hkv, Nmax, d))
    _need(V, "V", torch.bfloat16, (B, Hkv, Nmax, d))
    _need(codes, "codes", torch.uint8, (B, Hkv, Nmax, d // 4))
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    if out is None:
        out = _make(torch.empty, (B, Hq, d), torch.float32, q.device, stream)
    if idx is None:
        idx = _make(torch.empty, (B, Hq, budget), torch.int32, q.device, stream)
    _need(out, "out", torch.float32, (B, Hq, d))
    _need(idx, "idx", torch.int32, (B, Hq, budget))
    return B, Hq, Hkv, Nmax, d, out, idx


def decode_step(q: torch.Tensor, codes: torch.Tensor, K: torch.Tensor, V: torch.Tensor,
                seq_lens: torch.Tensor, budget: int, workspace: Workspace,
                out: Optional[torch.Tensor] = None, idx: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """One decode step: returns (out [B,Hq,128] fp32, idx [B,Hq,budget] int32)."""
    B, Hq, Hkv, Nmax, d, out, idx = _decode_args(q, codes, K, V, seq_lens, budget, out, idx, stream)
    rc = load().adamas_decode_step(q.data_ptr(), codes.data_ptr(), K.data_ptr(), V.data_ptr(),
                                   seq_lens.data_ptr(), B, Hq, Hkv, Nmax, d, budget, out.data_ptr(),
                                   idx.data_ptr() if budget > 0 else None,
                                   workspace.buffer.data_ptr(), workspace.nbytes, _stream(stream))
    _check(rc, "adamas_decode_step")
    return out, idx


def decode_step_append(q: torch.Tensor, codes: torch.Tensor, K: torch.Tensor, V: torch.Tensor,
                       seq_lens: torch.Tensor, append_pos: torch.Tensor, budget: int, workspace: Workspace,
                       out: Optional[torch.Tensor] = None, idx: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """encode_keys of the key at append_pos[b] (int32 [B]; out of [0, Nmax): none)
    followed by decode_step, in one launch; codes is updated in place."""
    B, Hq, Hkv, Nmax, d, out, idx = _decode_args(q, codes, K, V, seq_lens, budget, out, idx, stream)
    _need(append_pos, "append_pos", torch.int32, (B,))
    rc = load().adamas_decode_step_append(q.data_ptr(), codes.data_ptr(), K.data_ptr(), V.data_ptr(),
                                          seq_lens.data_ptr(), append_pos.data_ptr(), B, Hq, Hkv, Nmax, d,
                                          budget, out.data_ptr(), idx.data_ptr() if budget > 0 else None,
                                          workspace.buffer.data_ptr(), workspace.nbytes, _stream(stream))
    _check(rc, "adamas_decode_step_append")
    return out, idx


def score(q: torch.Tensor, codes: torch.Tensor, seq_lens: torch.Tensor, Hkv: Optional[int] = None,
          stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """L1 code distances [B,Hq,Nmax] (uint16 values in an int16 tensor; 0xFFFF past each length)."""
    _need(q, "q", torch.bfloat16)
    B, Hq, d = q.shape
    _need(codes, "codes", torch.uint8)
    _, Hkv, Nmax, _ = codes.shape
    _need(codes, "codes", torch.uint8, (B, Hkv, Nmax, d // 4))
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    dist = _make(torch.empty, (B, Hq, Nmax), torch.int16, q.device, stream)
    _check(load().adamas_score(q.data_ptr(), codes.data_ptr(), seq_lens.data_ptr(), B, Hq, Hkv, Nmax, d,
                               dist.data_ptr(), _stream(stream)), "adamas_score")
    return dist


def decode(q: torch.Tensor, codes: torch.Tensor, K: torch.Tensor, V: torch.Tensor, seq_lens: torch.Tensor,
           budget: int, workspace: Workspace, *, append_pos: Optional[torch.Tensor] = None,
           k_new: Optional[torch.Tensor] = None, v_new: Optional[torch.Tensor] = None,
           block_table: Optional[torch.Tensor] = None, n_sink: int = 0, n_recent: int = 0,
           policy: int = SELECT_PER_HEAD, out: Optional[torch.Tensor] = None, idx: Optional[torch.Tensor] = None,
           stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """adamas_decode_step_ex: the decode step with every option.

    Contiguous cache: codes [B,Hkv,Nmax,32], K/V [B,Hkv,Nmax,128].  Paged cache
    (block_table int32 [B, max_pages]): codes [n_pages,Hkv,P,32], K/V
    [n_pages,Hkv,P,128] with P the page size.  append_pos int32 [B] encodes the key
    at that position first; k_new/v_new bf16 [B,Hkv,128] are also written into the
    cache there by the launch.  n_sink/n_recent force the first/last tokens of each
    sequence into the kept set.  policy SELECT_GROUP_SHARED keeps one budget per kv
    head (idx [B,Hkv,budget]).  Returns (out [B,Hq,128] fp32, idx)."""
    _need(q, "q", torch.bfloat16)
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, 128]")
    B, Hq, d = q.shape
    _need(K, "K", torch.bfloat16)
    if K.dim() != 4:
        raise ValueError("K must be 4-dimensional")
    paged = block_table is not None
    if paged:
        n_pages, Hkv, page_size, _ = K.shape
        _need(block_table, "block_table", torch.int32)
        if block_table.dim() != 2 or block_table.shape[0] != B:
            raise ValueError("block_table must be [B, max_pages]")
        max_pages = block_table.shape[1]
        Nmax = max_pages * page_size
        _need(K, "K", torch.bfloat16, (n_pages, Hkv, page_size, d))
        _need(V, "V", torch.bfloat16, (n_pages, Hkv, page_size, d))
        _need(codes, "codes", torch.uint8, (n_pages, Hkv, page_size, d // 4))
    else:
        _, Hkv, Nmax, _ = K.shape
        n_pages = page_size = max_pages = 0
        _need(K, "K", torch.bfloat16, (B, Hkv, Nmax, d))
        _need(V, "V", torch.bfloat16, (B, Hkv, Nmax, d))
        _need(codes, "codes", torch.uint8, (B, Hkv, Nmax, d // 4))
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    rows = Hkv if policy == SELECT_GROUP_SHARED else Hq
    if out is None:
        out = _make(torch.empty, (B, Hq, d), torch.float32, q.device, stream)
    if idx is None:
        idx = _make(torch.empty, (B, rows, budget), torch.int32, q.device, stream)
    _need(out, "out", torch.float32, (B, Hq, d))
    _need(idx, "idx", torch.int32, (B, rows, budget))
    if append_pos is not None:
        _need(append_pos, "append_pos", torch.int32, (B,))
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new go together")
    if k_new is not None:
        _need(k_new, "k_new", torch.bfloat16, (B, Hkv, d))
        _need(v_new, "v_new", torch.bfloat16, (B, Hkv, d))
    a = DecodeArgs(q.data_ptr(), codes.data_ptr(), K.data_ptr(), V.data_ptr(), seq_lens.data_ptr(),
                   B, Hq, Hkv, Nmax, d, budget, out.data_ptr(), idx.data_ptr() if budget > 0 else None,
                   workspace.buffer.data_ptr(), workspace.nbytes, _ptr(append_pos), _ptr(k_new), _ptr(v_new),
                   _ptr(block_table), n_pages, page_size, max_pages, n_sink, n_recent, policy)
    _check(load().adamas_decode_step_ex(ctypes.byref(a), _stream(stream)), "adamas_decode_step_ex")
    return out, idx


# ---------------------------------------------------------------- sequence-sharded step
HIST_STRIDE = 388      # ADAMAS_HIST_STRIDE: uint32 bins per (b, query head) of an exchanged histogram
PARTIAL_FLOATS = 132   # ADAMAS_PARTIAL_FLOATS: fp32 per (b, query head) of a softmax state


def _shard_shapes(q, codes_or_K, seq_lens):
    _need(q, "q", torch.bfloat16)
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, 128]")
    B, Hq, d = q.shape
    if codes_or_K.dim() != 4:
        raise ValueError("the cache must be [B, Hkv, Nmax, ...]")
    _, Hkv, Nmax, _ = codes_or_K.shape
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    return B, Hq, Hkv, Nmax, d


def shard_score(q: torch.Tensor, codes: torch.Tensor, seq_lens: torch.Tensor, budget: int, workspace: Workspace,
                hist: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """First half of the sharded step on this GPU's slice: returns its histograms
    [B, Hq, HIST_STRIDE] int32 (uint32 counts), to be all-gathered in rank order."""
    B, Hq, Hkv, Nmax, d = _shard_shapes(q, codes, seq_lens)
    _need(codes, "codes", torch.uint8, (B, Hkv, Nmax, d // 4))
    if hist is None:
        hist = _make(torch.empty, (B, Hq, HIST_STRIDE), torch.int32, q.device, stream)
    _need(hist, "hist", torch.int32, (B, Hq, HIST_STRIDE))
    _check(load().adamas_shard_score(q.data_ptr(), codes.data_ptr(), seq_lens.data_ptr(), B, Hq, Hkv, Nmax, d,
                                     budget, hist.data_ptr(), workspace.buffer.data_ptr(), workspace.nbytes,
                                     _stream(stream)), "adamas_shard_score")
    return hist


def shard_attend(q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, seq_lens: torch.Tensor, budget: int,
                 hist_all: torch.Tensor, rank: int, workspace: Workspace, partial: Optional[torch.Tensor] = None,
                 idx: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Second half on this GPU's slice, with hist_all [world, B, Hq, HIST_STRIDE] of
    every slice: returns (partial [B, Hq, PARTIAL_FLOATS] fp32, idx [B, Hq, budget]
    int32 holding the global indices of this slice's kept tokens, -1 elsewhere)."""
    B, Hq, Hkv, Nmax, d = _shard_shapes(q, K, seq_lens)
    _need(K, "K", torch.bfloat16, (B, Hkv, Nmax, d))
    _need(V, "V", torch.bfloat16, (B, Hkv, Nmax, d))
    if hist_all.dim() != 4:
        raise ValueError("hist_all must be [world, B, Hq, HIST_STRIDE]")
    world = hist_all.shape[0]
    _need(hist_all, "hist_all", torch.int32, (world, B, Hq, HIST_STRIDE))
    if partial is None:
        partial = _make(torch.empty, (B, Hq, PARTIAL_FLOATS), torch.float32, q.device, stream)
    if idx is None:
        idx = _make(torch.empty, (B, Hq, budget), torch.int32, q.device, stream)
    _need(partial, "partial", torch.float32, (B, Hq, PARTIAL_FLOATS))
    _need(idx, "idx", torch.int32, (B, Hq, budget))
    _check(load().adamas_shard_attend(q.data_ptr(), K.data_ptr(), V.data_ptr(), seq_lens.data_ptr(), B, Hq, Hkv,
                                      Nmax, d, budget, hist_all.data_ptr(), world, int(rank), partial.data_ptr(),
                                      idx.data_ptr() if budget > 0 else None, workspace.buffer.data_ptr(),
                                      workspace.nbytes, _stream(stream)), "adamas_shard_attend")
    return partial, idx


def merge_partials(partials: torch.Tensor, out: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention output [B, Hq, 128] fp32 from the states [n, B, Hq, PARTIAL_FLOATS] of n slices."""
    if partials.dim() != 4:
        raise ValueError("partials must be [n, B, Hq, PARTIAL_FLOATS]")
    n, B, Hq, _ = partials.shape
    _need(partials, "partials", torch.float32, (n, B, Hq, PARTIAL_FLOATS))
    if out is None:
        out = _make(torch.empty, (B, Hq, HEAD_DIM), torch.float32, partials.device, stream)
    _need(out, "out", torch.float32, (B, Hq, HEAD_DIM))
    _check(load().adamas_merge_partials(partials.data_ptr(), n, B, Hq, out.data_ptr(), _stream(stream)),
           "adamas_merge_partials")
    return out


# ---------------------------------------------------------------- cache operators
def chunk_workspace_bytes(T: int, B: int, Hq: int, Hkv: int, d: int = HEAD_DIM) -> int:
    n = load().adamas_chunk_workspace_bytes(T, B, Hq, Hkv, d)
    if n == 0:
        raise AdamasError(-2, "adamas_chunk_workspace_bytes")
    return int(n)


class ChunkWorkspace(Workspace):
    """Device workspace of chunk_attend for up to T packed rows (the other cache
    operators take it, or any other Workspace, as well), zero-filled on creation."""

    def __init__(self, T: int, B: int, Hq: int, Hkv: int, device=None, stream: Optional[torch.cuda.Stream] = None):
        self.nbytes = chunk_workspace_bytes(T, B, Hq, Hkv)
        self.buffer = _make(torch.empty, (self.nbytes,), torch.uint8, device if device is not None else "cuda", stream)
        self.reset(stream)


def rope_frequencies(rot_dim: int = HEAD_DIM, base: float = 10000.0, *, scaling: Optional[str] = None,
                     factor: float = 1.0, original_len: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
                     device=None) -> Tuple[torch.Tensor, float]:
    """The frequency table of rope_append and its factor on cos and sin: (freqs int64
    [rot_dim / 2], mscale).  Pair j turns by base^(-2j / rot_dim) per position.

    scaling, for contexts `factor` times the trained length original_len:
      None      as trained
      "linear"  every frequency divided by factor (positions interpolated)
      "ntk"     base * factor^(rot_dim / (rot_dim - 2)): the slowest pair is slowed by
                factor, the fastest hardly
      "yarn"    pairs that turn more than beta_fast times within original_len as
                trained, those below beta_slow turns divided by factor, a linear ramp
                over the pairs between; mscale = 0.1 ln(factor) + 1
    Evaluated in 64 bits; the table holds each frequency as a fraction of a turn times
    2^64, so that far positions lose nothing."""
    if rot_dim % 2 or not 0 <= rot_dim <= HEAD_DIM:
        raise ValueError("rot_dim must be even and at most 128")
    if base <= 1.0 or factor < 1.0:
        raise ValueError("base must be above 1 and factor at least 1")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    half, mscale = rot_dim // 2, 1.0
    if scaling == "ntk":
        if rot_dim <= 2:
            raise ValueError("ntk scaling needs rot_dim above 2")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freq = [base ** (-2.0 * j / rot_dim) for j in range(half)]
    if scaling == "linear":
        freq = [f / factor for f in freq]
    if scaling == "yarn":
        def pair_of(turns):  # the pair that turns this often within original_len
            return rot_dim * math.log(original_len / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        lo = max(0, math.floor(pair_of(beta_fast)))
        hi = min(rot_dim - 1, math.ceil(pair_of(beta_slow)))  # may lie behind the last pair: none is that slow
        ramp = [min(1.0, max(0.0, (j - lo) / max(hi - lo, 1e-3))) for j in range(half)]
        freq = [f * (1.0 - r) + f / factor * r for f, r in zip(freq, ramp)]
        mscale = 0.1 * math.log(factor) + 1.0
    turns = [round(f / (2.0 * math.pi) * 2.0 ** 64) for f in freq]
    return torch.tensor(turns, dtype=torch.int64, device=device if device is not None else "cuda"), mscale


def _on(dev: int, t: Optional[torch.Tensor], name: str, dtype: torch.dtype, shape: tuple):
    """An argument of a cache operator: on CUDA device `dev`, dense, of this type and
    shape; its address (None for None).  (A call checks about ten of them.)"""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _device_of(t: torch.Tensor, name: str) -> int:
    """The device of a call: that of its first tensor, which must be the current one
    (the launch goes to the current device's stream)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _scratch(dev: int, workspace: Workspace) -> Tuple[int, int]:
    """Address and size of a call's workspace, which must be on the call's device."""
    if workspace.buffer.get_device() != dev:
        raise ValueError(f"workspace must be on cuda:{dev}, got {workspace.buffer.device}")
    return workspace.buffer.data_ptr(), workspace.nbytes


def _run(name: str, args: ctypes.Structure, stream: Optional[torch.cuda.Stream]):
    rc = getattr(_lib if _lib is not None else load(), name)(ctypes.byref(args), _stream(stream))
    if rc != 0:
        raise AdamasError(rc, name)


def _cache_of(dev, K, V, codes, B, block_table, suffix=""):
    """Geometry of a cache: (Hkv, Nmax, (K, V, codes) addresses, (table, n_pages, page_size, max_pages))."""
    if not isinstance(K, torch.Tensor) or K.dim() != 4 or K.shape[3] != HEAD_DIM:
        raise ValueError(f"K{suffix} must be [B, Hkv, Nmax, 128] or [n_pages, Hkv, page_size, 128]")
    lead, Hkv, rows, d = K.shape
    if block_table is None:
        if lead != B:
            raise ValueError(f"K{suffix} must hold {B} sequences, got {lead}")
        Nmax, paged = rows, (None, 0, 0, 0)
    else:
        if block_table.dim() != 2:
            raise ValueError(f"block_table{suffix} must be [B, max_pages]")
        pages = block_table.shape[1]
        paged = (_on(dev, block_table, "block_table" + suffix, torch.int32, (B, pages)), lead, rows, pages)
        Nmax = pages * rows
    ptrs = (_on(dev, K, "K" + suffix, torch.bfloat16, K.shape), _on(dev, V, "V" + suffix, torch.bfloat16, K.shape),
            _on(dev, codes, "codes" + suffix, torch.uint8, (lead, Hkv, rows, d // 4)))
    return Hkv, Nmax, ptrs, paged


def _packed_rows(dev, x: Optional[torch.Tensor], name: str):
    """A packed batch [T, heads, 128] whose rows may be spaced: (T, heads, stride, address)."""
    if x is None:
        return None, 0, 0, None
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {x.dtype}")
    if x.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {x.device}")
    if x.dim() != 3 or x.shape[2] != HEAD_DIM:
        raise ValueError(f"{name} must be [T, heads, 128]")
    T, H, d = x.shape
    row, head, one = x.stride()
    if T and (one != 1 or (H > 1 and head != d)):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return T, H, row if T > 1 else H * d, x.data_ptr()  # one row has no spacing


def rope_append(q: Optional[torch.Tensor], k: Optional[torch.Tensor], v: Optional[torch.Tensor],
                cu_new: torch.Tensor, cache_lens: torch.Tensor, K: torch.Tensor, V: torch.Tensor,
                freqs: torch.Tensor, workspace: Workspace, *, positions: Optional[torch.Tensor] = None,
                interleaved: bool = False, mscale: float = 1.0, codes: Optional[torch.Tensor] = None,
                block_table: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> Optional[torch.Tensor]:
    """Rotary positions of new rows, and their append to the cache (adamas_rope_append).

    q [T, Hq, 128], k and v [T, Hkv, 128] bf16, packed by cu_new int32 [B + 1]; rows
    may be spaced (parts of one projection's output).  Token i of sequence b is
    rotated by positions[row] (int32 [T]; default: its slot) and goes to slot
    cache_lens[b] + i (int32 [B]).  freqs, mscale: rope_frequencies.  The first
    2 * len(freqs) dimensions are rotated.  codes (uint8, optional) receives the rotated keys' codes.
    K, V, codes are written in place; returns the rotated queries [T, Hq, 128] (out;
    may be q itself), rows of no sequence left as they were (in a new tensor: 0)."""
    dev = _device_of(K, "K")
    if (k is None) != (v is None):
        raise ValueError("k and v go together")
    if q is None and k is None:
        raise ValueError("neither q nor k, v given")
    if not isinstance(cache_lens, torch.Tensor) or cache_lens.dim() != 1:
        raise ValueError("cache_lens must be [B]")
    B = cache_lens.shape[0]
    Hkv, Nmax, ptrs, paged = _cache_of(dev, K, V, codes, B, block_table)
    Tq, Hq, sq, pq = _packed_rows(dev, q, "q")
    Tk, Hk, sk, pk = _packed_rows(dev, k, "k")
    Tv, Hv, sv, pv = _packed_rows(dev, v, "v")
    T = Tk if q is None else Tq
    if k is not None and (Tk != T or Tv != T or Hk != Hkv or Hv != Hkv):
        raise ValueError(f"k and v must be [{T}, {Hkv}, 128]")
    if freqs.dim() != 1:
        raise ValueError("freqs must be [rot_dim / 2]")
    if q is None:
        if out is not None:
            raise ValueError("out without q")
    elif out is None:
        out = _make(torch.zeros, (T, Hq, HEAD_DIM), torch.bfloat16, q.device, stream)
    a = RopeArgs(pq, pk, pv, sq, sk, sv, _on(dev, cu_new, "cu_new", torch.int32, (B + 1,)),
                 _on(dev, cache_lens, "cache_lens", torch.int32, (B,)),
                 _on(dev, positions, "positions", torch.int32, (T,)),
                 _on(dev, freqs, "freqs", torch.int64, freqs.shape), 2 * freqs.shape[0], int(interleaved), mscale,
                 T, B, Hq or Hkv, Hkv, Nmax, HEAD_DIM, _on(dev, out, "out", torch.bfloat16, (T, Hq, HEAD_DIM)),
                 *ptrs, *paged, *_scratch(dev, workspace))
    _run("adamas_rope_append", a, stream)
    return out


def _chunk_args(dev, q, K, V, cu_q, seq_lens, block_table):
    if q.dim() != 3:
        raise ValueError("q must be [T, Hq, 128]")
    if not isinstance(seq_lens, torch.Tensor) or seq_lens.dim() != 1:
        raise ValueError("seq_lens must be [B]")
    T, Hq, _ = q.shape
    B = seq_lens.shape[0]
    Hkv, Nmax, (pk, pv, _), paged = _cache_of(dev, K, V, None, B, block_table)
    head = (_on(dev, q, "q", torch.bfloat16, (T, Hq, HEAD_DIM)), pk, pv,
            _on(dev, cu_q, "cu_q", torch.int32, (B + 1,)), _on(dev, seq_lens, "seq_lens", torch.int32, (B,)),
            T, B, Hq, Hkv, Nmax, HEAD_DIM)
    return head, paged


def chunk_attend(q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, cu_q: torch.Tensor, seq_lens: torch.Tensor,
                 workspace: Workspace, *, block_table: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Causal attention of a chunk of new tokens over the cache (adamas_chunk_attend).

    q [T, Hq, 128] bf16 packed by cu_q int32 [B + 1]; sequence b's rows are the last
    ones of its seq_lens[b] cached tokens (K, V already appended).  Returns (out [T,
    Hq, 128] bf16, lse [T, Hq] fp32, natural logarithm); rows of no sequence are left
    as they were (in new tensors: 0).  workspace: ChunkWorkspace of at least T rows."""
    dev = _device_of(q, "q")
    head, paged = _chunk_args(dev, q, K, V, cu_q, seq_lens, block_table)
    T, Hq = head[5], head[7]
    if out is None:
        out = _make(torch.zeros, (T, Hq, HEAD_DIM), torch.bfloat16, q.device, stream)
    if lse is None:
        lse = _make(torch.zeros, (T, Hq), torch.float32, q.device, stream)
    a = ChunkArgs(*head, _on(dev, out, "out", torch.bfloat16, (T, Hq, HEAD_DIM)),
                  _on(dev, lse, "lse", torch.float32, (T, Hq)), None, *paged, *_scratch(dev, workspace))
    _run("adamas_chunk_attend", a, stream)
    return out, lse


def accumulate_chunk(q: torch.Tensor, K: torch.Tensor, lse: torch.Tensor, cu_q: torch.Tensor, seq_lens: torch.Tensor,
                     mass: torch.Tensor, workspace: Workspace, *, block_table: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Adds to mass [B, Hkv, Nmax] fp32 the attention weight each cached token received
    from the chunk's rows (adamas_accumulate_chunk); q, cu_q, seq_lens and lse as of
    chunk_attend (or its last rows alone).  Returns mass."""
    dev = _device_of(q, "q")
    head, paged = _chunk_args(dev, q, K, None, cu_q, seq_lens, block_table)
    T, B, Hq, Hkv, Nmax = head[5:10]
    a = ChunkArgs(*head, None, _on(dev, lse, "lse", torch.float32, (T, Hq)),
                  _on(dev, mass, "mass", torch.float32, (B, Hkv, Nmax)), *paged, *_scratch(dev, workspace))
    _run("adamas_accumulate_chunk", a, stream)
    return mass


def accumulate_kept(q: torch.Tensor, K: torch.Tensor, idx: torch.Tensor, seq_lens: torch.Tensor, mass: torch.Tensor,
                    workspace: Workspace, *, policy: int = SELECT_PER_HEAD,
                    block_table: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Adds to mass [B, Hkv, Nmax] fp32 the attention weights of a decode step's kept
    tokens (adamas_accumulate_kept): q [B, Hq, 128] and idx as of decode_step / decode,
    [B, Hq, budget] or, group-shared, [B, Hkv, budget].  Returns mass."""
    dev = _device_of(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, 128]")
    B, Hq, _ = q.shape
    Hkv, Nmax, (pk, _, _), paged = _cache_of(dev, K, None, None, B, block_table)
    if idx.dim() != 3:
        raise ValueError("idx must be [B, Hq, budget] or, group-shared, [B, Hkv, budget]")
    budget = idx.shape[2]
    rows = Hkv if policy == SELECT_GROUP_SHARED else Hq
    a = KeptArgs(_on(dev, q, "q", torch.bfloat16, (B, Hq, HEAD_DIM)), pk,
                 _on(dev, idx, "idx", torch.int32, (B, rows, budget)),
                 _on(dev, seq_lens, "seq_lens", torch.int32, (B,)), B, Hq, Hkv, Nmax, HEAD_DIM, budget, policy,
                 _on(dev, mass, "mass", torch.float32, (B, Hkv, Nmax)), *paged, *_scratch(dev, workspace))
    _run("adamas_accumulate_kept", a, stream)
    return mass


def evict(K: torch.Tensor, V: torch.Tensor, mass: torch.Tensor, seq_lens: torch.Tensor, keep: int,
          workspace: Workspace, *, codes: Optional[torch.Tensor] = None, n_sink: int = 0, n_recent: int = 0,
          block_table: Optional[torch.Tensor] = None, K_out: Optional[torch.Tensor] = None,
          V_out: Optional[torch.Tensor] = None, codes_out: Optional[torch.Tensor] = None,
          mass_out: Optional[torch.Tensor] = None, table_out: Optional[torch.Tensor] = None,
          kept: Optional[torch.Tensor] = None, new_lens: Optional[torch.Tensor] = None,
          stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Keeps the `keep` tokens of largest mass per (b, kv head), sinks and recent tokens
    first, and moves their K, V, codes and mass to the front in their old order
    (adamas_evict): in place, or into K_out, V_out, codes_out, mass_out (table_out:
    their block table).  Returns (kept int32 [B, Hkv, keep]: the old slots, -1 past the
    sequence's count; new_lens int32 [B])."""
    dev = _device_of(K, "K")
    if not isinstance(seq_lens, torch.Tensor) or seq_lens.dim() != 1:
        raise ValueError("seq_lens must be [B]")
    B = seq_lens.shape[0]
    Hkv, Nmax, ptrs, paged = _cache_of(dev, K, V, codes, B, block_table)
    in_place = K_out is None
    if in_place:
        if V_out is not None or codes_out is not None or mass_out is not None or table_out is not None:
            raise ValueError("V_out, codes_out, mass_out and table_out go with K_out")
        ptrs_out, Nmax_out, paged_out = (None, None, None), 0, (None, 0, 0, 0)
    else:
        if V_out is None or mass_out is None or (codes is None) != (codes_out is None):
            raise ValueError("K_out goes with V_out, mass_out and, when codes is given, codes_out")
        Hkv_out, Nmax_out, ptrs_out, paged_out = _cache_of(dev, K_out, V_out, codes_out, B, table_out, "_out")
        if Hkv_out != Hkv:
            raise ValueError(f"K_out must have {Hkv} kv heads, got {Hkv_out}")
    if kept is None:
        kept = _make(torch.empty, (B, Hkv, max(keep, 0)), torch.int32, K.device, stream)
    if new_lens is None:
        new_lens = _make(torch.empty, (B,), torch.int32, K.device, stream)
    a = EvictArgs(*ptrs, _on(dev, mass, "mass", torch.float32, (B, Hkv, Nmax)),
                  _on(dev, seq_lens, "seq_lens", torch.int32, (B,)), B, Hkv, Nmax, HEAD_DIM, keep, n_sink, n_recent,
                  _on(dev, kept, "kept", torch.int32, (B, Hkv, max(keep, 0))),
                  _on(dev, new_lens, "new_lens", torch.int32, (B,)), *paged, *ptrs_out,
                  _on(dev, mass_out, "mass_out", torch.float32, (B, Hkv, Nmax_out)), Nmax_out, *paged_out,
                  *_scratch(dev, workspace))
    _run("adamas_evict", a, stream)
    return kept, new_lens
