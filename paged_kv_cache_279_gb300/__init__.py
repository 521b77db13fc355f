"""Paged KV cache for GB300: Python binding of libpkv (include/pkv.h).

Argument marshalling only: every step of the hot path runs in the library's
CUDA kernels or its C++ allocator.  PyTorch supplies device memory and the
current CUDA stream.  If the library has not been built the calls raise; there
is no CPU or PyTorch fallback.

    kv_cache_write(k_new, v_new, k_cache, v_cache, slot_mapping)
    paged_attention_decode(out, q, k_cache, v_cache, block_tables, seq_lens,
                           scale, max_seq_len, partition_size=0, workspace=None)
    paged_attention_decode_append(...)    # store the step's new tokens, then attend
    paged_attention_decode_grouped(...)   # beams sharing prefix blocks: each read once
    paged_attention_multi_token(...)      # several causal query tokens per sequence
    kv_cache_write_fp8(...), paged_attention_decode_fp8(...),
    paged_attention_decode_append_fp8(...)  # E4M3 cache, per-tensor scales
    kv_cache_write_fp8_rows(...), kv_cache_read_fp8_rows(...)  # E4M3 cache, a scale per row
    paged_attention_decode_scored(...), paged_attention_decode_scored_fp8_rows(...),
    paged_attention_multi_token_scored(...)  # capped or biased scores, windows, documents, prefixes
    rotary_frequencies(...), rotary_embed(...), kv_cache_write_rotary(...)  # positions by rotation
    latent_cache_write(...), paged_latent_attention_decode(...),
    paged_latent_attention_multi_token(...)  # one latent row a token, shared by all heads
    block_copy(k_caches, v_caches, block_pairs)
    BlockAllocator(num_blocks, block_size)   # host allocator: CoW, prefix cache, truncation
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence

import numpy as np
import torch

from . import _lib

(PKV_OK, PKV_ERR_INVALID, PKV_ERR_OOM, PKV_ERR_CUDA, PKV_ERR_UNSUPPORTED, PKV_ERR_TIMEOUT,
 PKV_ERR_TOO_LARGE) = range(7)
NOALLOC_SCRATCH_BYTES = 16 << 20
PKV_F32, PKV_BF16 = 0, 1
LATENT_ROPE_DIM = 64
DEVERR_BLOCK_ID, DEVERR_SEQ_LEN, DEVERR_SLOT, DEVERR_COPY_PAIR, DEVERR_TIMEOUT, DEVERR_PREFIX = (
    1, 2, 4, 8, 16, 32)

__all__ = [
    "PkvError", "kv_cache_write", "kv_cache_write_fp8", "paged_attention_decode",
    "paged_attention_decode_fp8", "paged_attention_decode_append_fp8", "paged_attention_workspace_size",
    "paged_attention_multi_token", "paged_attention_multi_token_workspace_size",
    "paged_attention_decode_append", "paged_attention_decode_grouped",
    "kv_cache_write_fp8_rows", "kv_cache_read_fp8_rows", "paged_attention_decode_scored",
    "paged_attention_decode_scored_fp8_rows", "paged_attention_decode_scored_workspace_size",
    "paged_attention_multi_token_scored", "paged_attention_multi_token_scored_workspace_size",
    "rotary_frequencies", "rotary_embed", "kv_cache_write_rotary", "latent_cache_write",
    "paged_latent_attention_decode", "paged_latent_attention_multi_token", "paged_latent_attention_workspace_size",
    "paged_attention_grouped_workspace_size", "block_copy", "read_device_errors", "BlockAllocator",
    "library_path",
]


class PkvError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = int(status)
        msg = _lib.load().pkv_status_string(int(status)).decode()
        super().__init__(f"{what}: {msg} (status {status})")


def _check(status: int, what: str) -> None:
    if status != PKV_OK:
        raise PkvError(status, what)


def library_path() -> str:
    return _lib.library_path()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return PKV_F32
    if t.dtype == torch.bfloat16:
        return PKV_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _dev(t: torch.Tensor, name: str, dtype=None, ndim=None) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def kv_cache_write(k_new, v_new, k_cache, v_cache, slot_mapping, stream=None) -> None:
    """Scatter new K/V rows [T, Hkv, D] into the caches [NB, Hkv, B, D] at
    slot_mapping[t] (int64; negative = skip)."""
    lib = _lib.load()
    NB, Hkv, B, D = k_cache.shape
    T = k_new.shape[0]
    if tuple(k_new.shape) != (T, Hkv, D) or k_new.shape != v_new.shape or k_cache.shape != v_cache.shape:
        raise ValueError("shape mismatch between new tokens and caches")
    if slot_mapping.shape[0] != T:
        raise ValueError("slot_mapping needs one entry per token")
    dt = _dtype_code(k_cache)
    for t, n in ((k_new, "k_new"), (v_new, "v_new"), (v_cache, "v_cache")):
        if t.dtype != k_cache.dtype:
            raise TypeError(f"{n} dtype differs from k_cache")
    st = lib.kv_cache_write(_dev(k_new, "k_new"), _dev(v_new, "v_new"), _dev(k_cache, "k_cache"),
                            _dev(v_cache, "v_cache"), _dev(slot_mapping, "slot_mapping", torch.int64, 1),
                            T, Hkv, D, B, NB, dt, _stream(stream))
    _check(st, "kv_cache_write")


def paged_attention_workspace_size(num_seqs: int, num_heads: int, head_dim: int,
                                   max_seq_len: int, partition_size: int = 0) -> int:
    return int(_lib.load().paged_attention_workspace_size(num_seqs, num_heads, head_dim,
                                                          max_seq_len, partition_size))


def paged_attention_decode(out, q, k_cache, v_cache, block_tables, seq_lens, scale: float,
                           max_seq_len: int, partition_size: int = 0,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[s, h] = softmax(scale * q[s, h] . K_s^T) V_s over the paged cache.

    q/out [S, Hq, D]; caches [NB, Hkv, B, D]; block_tables int32 [S, maxB];
    seq_lens int32 [S].  ``workspace`` (uint8 CUDA tensor) is allocated from
    PyTorch's caching allocator when not given."""
    lib = _lib.load()
    S, Hq, D = q.shape
    NB, Hkv, B, Dk = k_cache.shape
    if Dk != D or tuple(out.shape) != (S, Hq, D) or v_cache.shape != k_cache.shape:
        raise ValueError("shape mismatch")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or seq_lens.shape[0] != S:
        raise ValueError("block_tables must be [S, maxB] and seq_lens [S]")
    dt = _dtype_code(q)
    for t, n in ((out, "out"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.dtype != q.dtype:
            raise TypeError(f"{n} dtype differs from q")
    need = paged_attention_workspace_size(S, Hq, D, max_seq_len, partition_size)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _dev(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.paged_attention_decode(
        _dev(out, "out"), _dev(q, "q"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
        _dev(block_tables, "block_tables", torch.int32, 2), _dev(seq_lens, "seq_lens", torch.int32, 1),
        S, Hq, Hkv, D, B, block_tables.shape[1], NB, int(max_seq_len), float(scale),
        int(partition_size), ws_ptr, ws_bytes, dt, _stream(stream))
    _check(st, "paged_attention_decode")
    return out


def paged_attention_multi_token_workspace_size(num_q_tokens: int, num_heads: int, head_dim: int,
                                               max_seq_len: int) -> int:
    return int(_lib.load().paged_attention_multi_token_workspace_size(num_q_tokens, num_heads, head_dim,
                                                                      max_seq_len))


def paged_attention_multi_token(out, q, k_cache, v_cache, block_tables, seq_lens, q_starts, scale: float,
                                max_q_len: int, max_seq_len: int, workspace: Optional[torch.Tensor] = None,
                                stream=None) -> torch.Tensor:
    """Causal attention of each sequence's last Q_s positions (chunked prefill,
    verification of drafted tokens): q/out bf16 [T, Hq, D] with sequence s
    owning rows q_starts[s] .. q_starts[s+1]-1 (int32 [S+1]); caches
    [NB, Hkv, B, D]; block_tables int32 [S, maxB]; seq_lens int32 [S] (the
    contexts including the query tokens)."""
    lib = _lib.load()
    T, Hq, D = q.shape
    NB, Hkv, B, Dk = k_cache.shape
    S = seq_lens.shape[0]
    if Dk != D or tuple(out.shape) != (T, Hq, D) or v_cache.shape != k_cache.shape:
        raise ValueError("shape mismatch")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or q_starts.shape[0] != S + 1:
        raise ValueError("block_tables must be [S, maxB] and q_starts [S + 1]")
    need = paged_attention_multi_token_workspace_size(T, Hq, D, max_seq_len)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _dev(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.paged_attention_multi_token(
        _dev(out, "out", torch.bfloat16), _dev(q, "q", torch.bfloat16), _dev(k_cache, "k_cache", torch.bfloat16),
        _dev(v_cache, "v_cache", torch.bfloat16), _dev(block_tables, "block_tables", torch.int32, 2),
        _dev(seq_lens, "seq_lens", torch.int32, 1), _dev(q_starts, "q_starts", torch.int32, 1), S, T, Hq, Hkv,
        D, B, block_tables.shape[1], NB, int(max_q_len), int(max_seq_len), float(scale), ws_ptr, ws_bytes,
        _stream(stream))
    _check(st, "paged_attention_multi_token")
    return out


def kv_cache_write_fp8(k_new, v_new, k_cache, v_cache, slot_mapping, k_scale: float, v_scale: float,
                       stream=None) -> None:
    """Quantise bf16 K/V rows [T, Hkv, D] to E4M3 codes and store them: K in
    k_cache uint8 [NB, Hkv, B, D], V transposed in v_cache uint8 [NB, Hkv, D, B]
    (code = e4m3(x / scale), nearest even, saturating)."""
    lib = _lib.load()
    NB, Hkv, B, D = k_cache.shape
    T = k_new.shape[0]
    if tuple(k_new.shape) != (T, Hkv, D) or k_new.shape != v_new.shape or \
            tuple(v_cache.shape) != (NB, Hkv, D, B):
        raise ValueError("shape mismatch between new tokens and FP8 caches")
    if slot_mapping.shape[0] != T:
        raise ValueError("slot_mapping needs one entry per token")
    st = lib.kv_cache_write_fp8(
        _dev(k_new, "k_new", torch.bfloat16), _dev(v_new, "v_new", torch.bfloat16),
        _dev(k_cache, "k_cache", torch.uint8), _dev(v_cache, "v_cache", torch.uint8),
        _dev(slot_mapping, "slot_mapping", torch.int64, 1), T, Hkv, D, B, NB,
        float(k_scale), float(v_scale), _stream(stream))
    _check(st, "kv_cache_write_fp8")


def paged_attention_decode_fp8(out, q, k_cache, v_cache, block_tables, seq_lens, scale: float,
                               k_scale: float, v_scale: float, max_seq_len: int,
                               workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Decode attention over an FP8 (E4M3) cache: K codes [NB, Hkv, B, D], V
    codes transposed [NB, Hkv, D, B], values code * k_scale / code * v_scale.
    q/out bf16 [S, Hq, D]; block_tables int32 [S, maxB]; seq_lens int32 [S]."""
    lib = _lib.load()
    S, Hq, D = q.shape
    NB, Hkv, B, Dk = k_cache.shape
    if Dk != D or tuple(out.shape) != (S, Hq, D) or tuple(v_cache.shape) != (NB, Hkv, D, B):
        raise ValueError("shape mismatch")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or seq_lens.shape[0] != S:
        raise ValueError("block_tables must be [S, maxB] and seq_lens [S]")
    need = paged_attention_workspace_size(S, Hq, D, max_seq_len, 0)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _dev(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.paged_attention_decode_fp8(
        _dev(out, "out", torch.bfloat16), _dev(q, "q", torch.bfloat16), _dev(k_cache, "k_cache", torch.uint8),
        _dev(v_cache, "v_cache", torch.uint8), _dev(block_tables, "block_tables", torch.int32, 2),
        _dev(seq_lens, "seq_lens", torch.int32, 1), S, Hq, Hkv, D, B, block_tables.shape[1], NB,
        int(max_seq_len), float(scale), float(k_scale), float(v_scale), ws_ptr, ws_bytes, _stream(stream))
    _check(st, "paged_attention_decode_fp8")
    return out


def paged_attention_decode_append_fp8(out, q, k_new, v_new, k_cache, v_cache, block_tables, seq_lens,
                                      scale: float, k_scale: float, v_scale: float, max_seq_len: int,
                                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One FP8 decode step: quantise and store each sequence's new token (bf16
    k_new/v_new [S, Hkv, D]) at position seq_lens[s] - 1, then attend; the
    store happens inside the attention kernel."""
    lib = _lib.load()
    S, Hq, D = q.shape
    NB, Hkv, B, Dk = k_cache.shape
    if Dk != D or tuple(out.shape) != (S, Hq, D) or tuple(v_cache.shape) != (NB, Hkv, D, B):
        raise ValueError("shape mismatch")
    if tuple(k_new.shape) != (S, Hkv, D) or k_new.shape != v_new.shape:
        raise ValueError("k_new / v_new must be [S, Hkv, D]")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or seq_lens.shape[0] != S:
        raise ValueError("block_tables must be [S, maxB] and seq_lens [S]")
    need = paged_attention_workspace_size(S, Hq, D, max_seq_len, 0)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _dev(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.paged_attention_decode_append_fp8(
        _dev(out, "out", torch.bfloat16), _dev(q, "q", torch.bfloat16), _dev(k_new, "k_new", torch.bfloat16),
        _dev(v_new, "v_new", torch.bfloat16), _dev(k_cache, "k_cache", torch.uint8),
        _dev(v_cache, "v_cache", torch.uint8), _dev(block_tables, "block_tables", torch.int32, 2),
        _dev(seq_lens, "seq_lens", torch.int32, 1), S, Hq, Hkv, D, B, block_tables.shape[1], NB,
        int(max_seq_len), float(scale), float(k_scale), float(v_scale), ws_ptr, ws_bytes, _stream(stream))
    _check(st, "paged_attention_decode_append_fp8")
    return out


def paged_attention_decode_append(out, q, k_new, v_new, k_cache, v_cache, block_tables, seq_lens,
                                  scale: float, max_seq_len: int, partition_size: int = 0,
                                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One decode step: store k_new[s] / v_new[s] ([S, Hkv, D]) at position
    seq_lens[s] - 1 of each sequence, then attend as paged_attention_decode."""
    lib = _lib.load()
    S, Hq, D = q.shape
    NB, Hkv, B, Dk = k_cache.shape
    if Dk != D or tuple(out.shape) != (S, Hq, D) or v_cache.shape != k_cache.shape:
        raise ValueError("shape mismatch")
    if tuple(k_new.shape) != (S, Hkv, D) or v_new.shape != k_new.shape:
        raise ValueError("k_new/v_new must be [S, Hkv, D]")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or seq_lens.shape[0] != S:
        raise ValueError("block_tables must be [S, maxB] and seq_lens [S]")
    dt = _dtype_code(q)
    for t, n in ((out, "out"), (k_cache, "k_cache"), (v_cache, "v_cache"), (k_new, "k_new"), (v_new, "v_new")):
        if t.dtype != q.dtype:
            raise TypeError(f"{n} dtype differs from q")
    need = paged_attention_workspace_size(S, Hq, D, max_seq_len, partition_size)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _dev(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.paged_attention_decode_append(
        _dev(out, "out"), _dev(q, "q"), _dev(k_new, "k_new"), _dev(v_new, "v_new"),
        _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
        _dev(block_tables, "block_tables", torch.int32, 2), _dev(seq_lens, "seq_lens", torch.int32, 1),
        S, Hq, Hkv, D, B, block_tables.shape[1], NB, int(max_seq_len), float(scale),
        int(partition_size), ws_ptr, ws_bytes, dt, _stream(stream))
    _check(st, "paged_attention_decode_append")
    return out


def paged_attention_grouped_workspace_size(num_seqs: int, num_heads: int, head_dim: int,
                                           max_seq_len: int) -> int:
    return int(_lib.load().paged_attention_grouped_workspace_size(num_seqs, num_heads, head_dim,
                                                                  max_seq_len))


def paged_attention_decode_grouped(out, q, k_cache, v_cache, block_tables, seq_lens, group_offsets,
                                   prefix_lens, scale: float, max_seq_len: int, k_new=None, v_new=None,
                                   workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Decode where the sequences of group g (group_offsets[g] .. [g+1]-1,
    int32 on the device) share the blocks of their first prefix_lens[g]
    tokens; each shared block is read once for the whole group.  With k_new /
    v_new the new tokens are stored first, as in paged_attention_decode_append."""
    lib = _lib.load()
    S, Hq, D = q.shape
    NB, Hkv, B, Dk = k_cache.shape
    if Dk != D or tuple(out.shape) != (S, Hq, D) or v_cache.shape != k_cache.shape:
        raise ValueError("shape mismatch")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or seq_lens.shape[0] != S:
        raise ValueError("block_tables must be [S, maxB] and seq_lens [S]")
    G = prefix_lens.shape[0]
    if group_offsets.shape[0] != G + 1:
        raise ValueError("group_offsets needs num_groups + 1 entries")
    if (k_new is None) != (v_new is None):
        raise ValueError("give both k_new and v_new, or neither")
    if k_new is not None and (tuple(k_new.shape) != (S, Hkv, D) or v_new.shape != k_new.shape):
        raise ValueError("k_new/v_new must be [S, Hkv, D]")
    need = paged_attention_grouped_workspace_size(S, Hq, D, max_seq_len)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _dev(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.paged_attention_decode_grouped(
        _dev(out, "out"), _dev(q, "q"),
        _dev(k_new, "k_new") if k_new is not None else None,
        _dev(v_new, "v_new") if v_new is not None else None,
        _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
        _dev(block_tables, "block_tables", torch.int32, 2), _dev(seq_lens, "seq_lens", torch.int32, 1),
        _dev(group_offsets, "group_offsets", torch.int32, 1), _dev(prefix_lens, "prefix_lens", torch.int32, 1),
        G, S, Hq, Hkv, D, B, block_tables.shape[1], NB, int(max_seq_len), float(scale), ws_ptr, ws_bytes,
        _dtype_code(q), _stream(stream))
    _check(st, "paged_attention_decode_grouped")
    return out


_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _device_of(t, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _ptr(t, name: str, dtype, dev: int) -> int:
    """Address of a contiguous tensor of that type on device `dev`."""
    try:
        if t.get_device() == dev and t.dtype is dtype and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        if not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        raise ValueError(f"{name} is on {t.device}, other tensors of the call on cuda:{dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be contiguous")


def _opt_ptr(t, name: str, dtype, dev: int):
    return None if t is None else _ptr(t, name, dtype, dev)


def _stream_on(stream, dev: int) -> int:
    """The stream a call runs on: the given one, else the current stream of its tensors' device."""
    if stream is None:
        return _current_raw_stream(dev) if _current_raw_stream else int(torch.cuda.current_stream(dev).cuda_stream)
    return _stream(stream)


@functools.lru_cache(maxsize=None)
def _cuda_device(dev: int) -> torch.device:
    return torch.device("cuda", dev)


def _scratch(workspace, need: int, stream, dev: int):
    """(address, bytes) of the caller's workspace, or of one taken here."""
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=_cuda_device(dev))
        if stream is not None:  # its memory must outlive the work on that stream, not on the current one
            workspace.record_stream(stream if hasattr(stream, "cuda_stream") else
                                    torch.cuda.ExternalStream(int(stream), device=dev))
        return workspace.data_ptr(), need
    if workspace.get_device() != dev:
        raise ValueError("workspace must be a tensor on the device of the call's tensors")
    return _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()


def _run_on(dev: int, what: str, fn, args) -> None:
    """Call the library with the tensors' device current."""
    if dev == _current_device():
        st = fn(*args)
    else:
        with torch.cuda.device(dev):
            st = fn(*args)
    if st != PKV_OK:
        raise PkvError(st, what)


_raw_alloc = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)
_raw_free = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None)


def _run_with_scratch(dev: int, what: str, fn, size_fn, sizes, head, workspace, tail, stream) -> None:
    """_run_on with a workspace, the caller's or, for this call, one of size_fn(*sizes) bytes: head, its address, its bytes,
    tail (whose last entry is the stream)."""
    if workspace is None and _raw_alloc is not None and _raw_free is not None and dev == _current_device():
        # the allocator's block of the call's stream, without a tensor around it (5 us less)
        need = size_fn(*sizes)
        ws = _raw_alloc(need, tail[-1]) if need else None
        try:
            st = fn(*head, ws, need, *tail)
        finally:
            if ws is not None:
                _raw_free(ws)  # work on that stream may reuse it, after this call's
        if st != PKV_OK:
            raise PkvError(st, what)
        return
    ws, n = _scratch(workspace, 0 if workspace is not None else size_fn(*sizes), stream, dev)
    _run_on(dev, what, fn, (*head, ws, n, *tail))


def _fp8_rows_call(what: str, k, v, k_cache, v_cache, k_scales, v_scales, slot_mapping, stream) -> None:
    NB, Hkv, B, D = k_cache.shape
    T = k.shape[0]
    if k.shape != (T, Hkv, D) or v.shape != k.shape or v_cache.shape != k_cache.shape:
        raise ValueError("shape mismatch between token rows and FP8 caches")
    if k_scales.shape != (NB, Hkv, B) or v_scales.shape != (NB, Hkv, B):
        raise ValueError("scales must be [NB, Hkv, B]")
    if slot_mapping.shape != (T,):
        raise ValueError("slot_mapping needs one entry per token")
    dev, dt, u8 = _device_of(k, "K rows"), k.dtype, torch.uint8
    _run_on(dev, what, getattr(_lib.load(), what), (
        _ptr(k, "K rows", dt, dev), _ptr(v, "V rows", dt, dev), _ptr(k_cache, "k_cache", u8, dev),
        _ptr(v_cache, "v_cache", u8, dev), _ptr(k_scales, "k_scales", u8, dev), _ptr(v_scales, "v_scales", u8, dev),
        _ptr(slot_mapping, "slot_mapping", torch.int64, dev), T, Hkv, D, B, NB, _dtype_code(k), _stream_on(stream, dev)))


def kv_cache_write_fp8_rows(k_new, v_new, k_cache, v_cache, k_scales, v_scales, slot_mapping, stream=None) -> None:
    """Quantise K/V rows [T, Hkv, D] (bf16 or float32) to E4M3 codes with one
    power-of-two scale per row, chosen here, and store both: codes in k_cache /
    v_cache uint8 [NB, Hkv, B, D], scales in k_scales / v_scales uint8
    [NB, Hkv, B] (exponent + 127), at slot_mapping[t] (int64; negative = skip)."""
    _fp8_rows_call("kv_cache_write_fp8_rows", k_new, v_new, k_cache, v_cache, k_scales, v_scales, slot_mapping, stream)


def kv_cache_read_fp8_rows(k_out, v_out, k_cache, v_cache, k_scales, v_scales, slot_mapping, stream=None):
    """The values of the cache rows at slot_mapping[t], into k_out / v_out
    [T, Hkv, D] (bf16, exact, or float32).  Rows of negative slots are left as
    they were.  Returns (k_out, v_out)."""
    _fp8_rows_call("kv_cache_read_fp8_rows", k_out, v_out, k_cache, v_cache, k_scales, v_scales, slot_mapping, stream)
    return k_out, v_out


def paged_attention_decode_scored_workspace_size(num_seqs: int, num_heads: int, head_dim: int, max_seq_len: int,
                                                 dtype: Optional[torch.dtype] = None) -> int:
    """Bytes of workspace that paged_attention_decode_scored (q of that dtype) or, for bfloat16,
    paged_attention_decode_scored_fp8_rows needs; without a dtype as much as any of them needs."""
    lib, size = _lib.load(), (int(num_seqs), int(num_heads), int(head_dim), _int32(max_seq_len))
    if dtype is None:
        return int(lib.paged_attention_decode_scored_workspace_size(*size))
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    return int(lib.paged_attention_decode_scored_workspace_size_for(*size, PKV_F32 if dtype == torch.float32 else PKV_BF16))


def paged_attention_multi_token_scored_workspace_size(num_q_tokens: int, num_heads: int, head_dim: int,
                                                      max_seq_len: int) -> int:
    return int(_lib.load().paged_attention_multi_token_scored_workspace_size(num_q_tokens, num_heads, head_dim,
                                                                             max_seq_len))


def _int32(x) -> int:
    """A limit as the library's int: beyond its range the largest value, or -1 (refused)."""
    x = int(x)
    return x if -1 <= x < 2 ** 31 else 2 ** 31 - 1 if x > 0 else -1


def _scored_shapes(out, q, k_cache, v_cache, block_tables, seq_lens, alibi_slopes, prefix_lens, key_starts):
    """(T, Hq, D, NB, Hkv, B, S, maxB) of a scored attention call."""
    T, Hq, D = q.shape
    NB, Hkv, B, Dk = k_cache.shape
    S = seq_lens.shape[0]
    if Dk != D or out.shape != q.shape or v_cache.shape != k_cache.shape:
        raise ValueError("shape mismatch")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or seq_lens.dim() != 1:
        raise ValueError("block_tables must be [S, maxB] and seq_lens [S]")
    if alibi_slopes is not None and alibi_slopes.shape != (Hq,):
        raise ValueError("alibi_slopes must be [Hq]")
    if prefix_lens is not None and prefix_lens.shape != (S,):
        raise ValueError("prefix_lens must be [S]")
    if key_starts is not None and key_starts.shape != (T,):
        raise ValueError("key_starts needs one entry per query")
    return T, Hq, D, NB, Hkv, B, S, block_tables.shape[1]


def paged_attention_decode_scored(out, q, k_cache, v_cache, block_tables, seq_lens, scale: float, max_seq_len: int,
                                  softcap: float = 0.0, alibi_slopes=None, window: int = 0, prefix_lens=None,
                                  key_starts=None, k_new=None, v_new=None, workspace: Optional[torch.Tensor] = None,
                                  stream=None) -> torch.Tensor:
    """paged_attention_decode with capped or biased scores and masked keys: with
    p = seq_lens[s] - 1, x = scale * q.k, then softcap * tanh(x / softcap) if
    softcap > 0, then - alibi_slopes[h] * (p - t) (float32 [Hq]); key t is seen
    if t >= key_starts[s] and (t < prefix_lens[s] or window == 0 or
    p - t < window) (int32 [S] each).  With k_new / v_new [S, Hkv, D] the new
    tokens are stored first.  A query that sees nothing gets zeros."""
    S, Hq, D, NB, Hkv, B, n, maxb = _scored_shapes(out, q, k_cache, v_cache, block_tables, seq_lens, alibi_slopes,
                                                   prefix_lens, key_starts)
    if n != S:
        raise ValueError("one query per sequence")
    if (k_new is None) != (v_new is None):
        raise ValueError("give both k_new and v_new, or neither")
    if k_new is not None and (k_new.shape != (S, Hkv, D) or v_new.shape != k_new.shape):
        raise ValueError("k_new/v_new must be [S, Hkv, D]")
    lib, code, dt, i32 = _lib.load(), _dtype_code(q), q.dtype, torch.int32
    dev, max_len = _device_of(q, "q"), _int32(max_seq_len)
    _run_with_scratch(dev, "paged_attention_decode_scored", lib.paged_attention_decode_scored,
                      lib.paged_attention_decode_scored_workspace_size_for, (S, Hq, D, max_len, code), (
        _ptr(out, "out", dt, dev), _ptr(q, "q", dt, dev), _opt_ptr(k_new, "k_new", dt, dev),
        _opt_ptr(v_new, "v_new", dt, dev), _ptr(k_cache, "k_cache", dt, dev), _ptr(v_cache, "v_cache", dt, dev),
        _ptr(block_tables, "block_tables", i32, dev), _ptr(seq_lens, "seq_lens", i32, dev), S, Hq, Hkv, D, B, maxb, NB,
        max_len, float(scale), float(softcap), _opt_ptr(alibi_slopes, "alibi_slopes", torch.float32, dev),
        _int32(window),
        _opt_ptr(prefix_lens, "prefix_lens", i32, dev), _opt_ptr(key_starts, "key_starts", i32, dev)), workspace,
        (code, _stream_on(stream, dev)), stream)
    return out


def paged_attention_decode_scored_fp8_rows(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, seq_lens,
                                           scale: float, max_seq_len: int, softcap: float = 0.0, alibi_slopes=None,
                                           window: int = 0, prefix_lens=None, key_starts=None,
                                           workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """paged_attention_decode_scored over a row-scaled FP8 cache (codes uint8
    [NB, Hkv, B, D], scales uint8 [NB, Hkv, B]); q / out bf16 [S, Hq, D]."""
    S, Hq, D, NB, Hkv, B, n, maxb = _scored_shapes(out, q, k_cache, v_cache, block_tables, seq_lens, alibi_slopes,
                                                   prefix_lens, key_starts)
    if n != S:
        raise ValueError("one query per sequence")
    if k_scales.shape != (NB, Hkv, B) or v_scales.shape != (NB, Hkv, B):
        raise ValueError("scales must be [NB, Hkv, B]")
    lib, bf, u8, i32 = _lib.load(), torch.bfloat16, torch.uint8, torch.int32
    dev, max_len = _device_of(q, "q"), _int32(max_seq_len)
    _run_with_scratch(dev, "paged_attention_decode_scored_fp8_rows", lib.paged_attention_decode_scored_fp8_rows,
                      lib.paged_attention_decode_scored_workspace_size_for, (S, Hq, D, max_len, PKV_BF16), (
        _ptr(out, "out", bf, dev), _ptr(q, "q", bf, dev), _ptr(k_cache, "k_cache", u8, dev),
        _ptr(v_cache, "v_cache", u8, dev), _ptr(k_scales, "k_scales", u8, dev), _ptr(v_scales, "v_scales", u8, dev),
        _ptr(block_tables, "block_tables", i32, dev), _ptr(seq_lens, "seq_lens", i32, dev), S, Hq, Hkv, D, B, maxb, NB,
        max_len, float(scale), float(softcap), _opt_ptr(alibi_slopes, "alibi_slopes", torch.float32, dev),
        _int32(window),
        _opt_ptr(prefix_lens, "prefix_lens", i32, dev), _opt_ptr(key_starts, "key_starts", i32, dev)), workspace,
        (_stream_on(stream, dev),), stream)
    return out


def paged_attention_multi_token_scored(out, q, k_cache, v_cache, block_tables, seq_lens, q_starts, scale: float,
                                       max_q_len: int, max_seq_len: int, softcap: float = 0.0, alibi_slopes=None,
                                       window: int = 0, prefix_lens=None, key_starts=None,
                                       workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """paged_attention_multi_token with capped or biased scores and masked keys
    (see paged_attention_decode_scored): a query at position p sees key t if
    t >= key_starts[row] (int32 [T], not decreasing over a sequence's queries)
    and (t < prefix_lens[s], or t <= p and (window == 0 or p - t < window)); the
    bias is - alibi_slopes[h] * |p - t|."""
    T, Hq, D, NB, Hkv, B, S, maxb = _scored_shapes(out, q, k_cache, v_cache, block_tables, seq_lens, alibi_slopes,
                                                   prefix_lens, key_starts)
    if q_starts.shape != (S + 1,):
        raise ValueError("q_starts must be [S + 1]")
    lib, bf, i32 = _lib.load(), torch.bfloat16, torch.int32
    dev, max_len = _device_of(q, "q"), _int32(max_seq_len)
    _run_with_scratch(dev, "paged_attention_multi_token_scored", lib.paged_attention_multi_token_scored,
                      lib.paged_attention_multi_token_scored_workspace_size, (T, Hq, D, max_len), (
        _ptr(out, "out", bf, dev), _ptr(q, "q", bf, dev), _ptr(k_cache, "k_cache", bf, dev),
        _ptr(v_cache, "v_cache", bf, dev), _ptr(block_tables, "block_tables", i32, dev),
        _ptr(seq_lens, "seq_lens", i32, dev), _ptr(q_starts, "q_starts", i32, dev), S, T, Hq, Hkv, D, B, maxb, NB,
        _int32(max_q_len), max_len, float(scale), float(softcap),
        _opt_ptr(alibi_slopes, "alibi_slopes", torch.float32, dev), _int32(window),
        _opt_ptr(prefix_lens, "prefix_lens", i32, dev), _opt_ptr(key_starts, "key_starts", i32, dev)), workspace,
        (_stream_on(stream, dev),), stream)
    return out


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, factor: float = 1.0, original_len: float = 0.0,
                       low_turns: float = 1.0, high_turns: float = 32.0, device=None) -> torch.Tensor:
    """Radians per position of the rotary_dim / 2 pairs, float64: base ** (-2 i / rotary_dim), for longer contexts
    divided by `factor`; with original_len, by parts: a pair that turns high_turns times or more in that length
    keeps its frequency, one that turns low_turns times or less has it divided, between them a ramp."""
    if int(rotary_dim) < 2 or int(rotary_dim) % 2:
        raise ValueError("rotary_dim must be even and positive")
    out = torch.empty(int(rotary_dim) // 2, dtype=torch.float64)
    _check(_lib.load().rotary_frequencies(out.data_ptr(), int(rotary_dim), float(base), float(factor), float(original_len),
                                          float(low_turns), float(high_turns)), "rotary_frequencies")
    return out if device is None else out.to(device)


# The calls below check the shapes and strides of a call once for each combination they meet: the functions
# under lru_cache see sizes alone, never a tensor, and give what the library's call takes of them.  Types, devices and
# addresses are looked at in every call.
_plans = functools.lru_cache(maxsize=4096)
_codes = {torch.float32: PKV_F32, torch.bfloat16: PKV_BF16}


def _code(t) -> int:
    code = _codes.get(t.dtype)
    return _dtype_code(t) if code is None else code


def _rows(name: str, shape, stride):
    """Token and head stride of rows [T, H, D] whose entries are contiguous."""
    if len(shape) != 3:
        raise ValueError(f"{name} must have 3 dimensions")
    if stride[2] != 1 and shape[2] > 1:
        raise ValueError(f"the entries of a row of {name} must be contiguous")
    # strides of dimensions of one entry say nothing, and are not held against the call
    return stride[0] if shape[0] > 1 else 0, stride[1] if shape[1] > 1 else 0


def _vector(name: str, shape, T: int) -> None:
    if shape != (T,):
        raise ValueError(f"{name} needs one entry per token")


def _pairs(shape, rotary_dim: Optional[int] = None) -> int:
    if len(shape) != 1:
        raise ValueError("frequencies must be a vector, one entry per rotated pair")
    if rotary_dim is not None and 2 * shape[0] != rotary_dim:
        raise ValueError(f"frequencies needs {rotary_dim // 2} entries")
    return 2 * shape[0]


def _row_ptr(t, name: str, dtype, dev: int) -> int:
    """Address of a tensor of that type on device `dev`, whatever its strides."""
    try:
        if t.get_device() == dev and t.dtype is dtype:
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} is on {t.device}, other tensors of the call on cuda:{dev}")


@_plans
def _embed_plan(x, x_stride, out, out_stride, positions, frequencies):
    if len(x) != 3 or out != x:
        raise ValueError("x and out must have the same shape [T, H, D]")
    _vector("positions", positions, x[0])
    return (*x, _pairs(frequencies)), (ctypes.c_int64 * 4)(*_rows("out", out, out_stride), *_rows("x", x, x_stride))


def rotary_embed(out, x, positions, frequencies, amplitude: float = 1.0, interleaved: bool = False, offset: int = 0,
                 stream=None) -> torch.Tensor:
    """Rotate rows x [T, H, D] (bf16 or float32) by their positions (int32 [T]) into out, which may be x itself: the
    entries from `offset` on, in pairs (i, i + R / 2) or, interleaved, (2 i, 2 i + 1), R = 2 * len(frequencies)
    (float64, radians per position); pair i turns by position * frequencies[i], scaled by `amplitude`.  Tokens
    and heads may be strided, in steps of 16 bytes; rows of out must not overlap."""
    size, strides = _embed_plan(x.shape, x.stride(), out.shape, out.stride(), positions.shape, frequencies.shape)
    dev, dt = _device_of(x, "x"), x.dtype
    _run_on(dev, "rotary_embed", _lib.load().rotary_embed, (
        _row_ptr(out, "out", dt, dev), x.data_ptr(), _ptr(positions, "positions", torch.int32, dev),
        _ptr(frequencies, "frequencies", torch.float64, dev), *size, offset, strides, amplitude, bool(interleaved),
        _code(x), _stream_on(stream, dev)))
    return out


@_plans
def _write_plan(k, k_stride, v, v_stride, k_cache, v_cache, slots, positions, frequencies, q, q_stride, out, out_stride):
    if len(k_cache) != 4 or v_cache != k_cache:
        raise ValueError("caches must be [NB, Hkv, B, D], and alike")
    NB, Hkv, B, D = k_cache
    if len(k) != 3 or k[1:] != (Hkv, D) or v != k:
        raise ValueError("shape mismatch between new tokens and caches")
    T, Hq, qs = k[0], 0, (0, 0, 0, 0)
    _vector("slot_mapping", slots, T)
    _vector("positions", positions, T)
    if (q is None) != (out is None):
        raise ValueError("give both q and q_out, or neither")
    if q is not None:
        if len(q) != 3 or q[0] != T or q[2] != D or out != q:
            raise ValueError("q and q_out must be [T, Hq, D]")
        Hq, qs = q[1], _rows("q_out", out, out_stride) + _rows("q", q, q_stride)
    return (T, Hq, Hkv, D, _pairs(frequencies)), (B, NB), (ctypes.c_int64 * 8)(*qs, *_rows("k_new", k, k_stride), *_rows("v_new", v, v_stride))


def kv_cache_write_rotary(k_new, v_new, k_cache, v_cache, slot_mapping, positions, frequencies, q=None, q_out=None,
                          amplitude: float = 1.0, interleaved: bool = False, offset: int = 0, stream=None):
    """kv_cache_write with the keys rotated by their positions on the way (see rotary_embed), and with q [T, Hq, D]
    the queries too, into q_out (which may be q), in one launch.  k_new, v_new, q and q_out may be strided.
    Queries are rotated whatever the token's slot.  Returns q_out."""
    some, out = q is not None, q_out is not None
    size, blocks, strides = _write_plan(
        k_new.shape, k_new.stride(), v_new.shape, v_new.stride(), k_cache.shape, v_cache.shape, slot_mapping.shape, positions.shape,
        frequencies.shape, q.shape if some else None, q.stride() if some else None, q_out.shape if out else None,
        q_out.stride() if out else None)
    some = some and size[1] > 0
    dev, dt = _device_of(k_cache, "k_cache"), k_cache.dtype
    _run_on(dev, "kv_cache_write_rotary", _lib.load().kv_cache_write_rotary, (
        _row_ptr(q_out, "q_out", dt, dev) if some else None, _row_ptr(q, "q", dt, dev) if some else None,
        _row_ptr(k_new, "k_new", dt, dev), _row_ptr(v_new, "v_new", dt, dev), _ptr(k_cache, "k_cache", dt, dev),
        _ptr(v_cache, "v_cache", dt, dev), _ptr(slot_mapping, "slot_mapping", torch.int64, dev),
        _ptr(positions, "positions", torch.int32, dev), _ptr(frequencies, "frequencies", torch.float64, dev), *size, offset, *blocks,
        strides, amplitude, bool(interleaved), _code(k_cache), _stream_on(stream, dev)))
    return q_out


@_plans
def _latent_write_plan(latent, latent_stride, key, key_stride, cache, slots, positions, frequencies, q, q_stride, out, out_stride):
    if len(cache) != 3 or len(latent) != 2:
        raise ValueError("cache must be [NB, B, V + %d], latent [T, V]" % LATENT_ROPE_DIM)
    (NB, B, W), (T, V) = cache, latent
    if W != V + LATENT_ROPE_DIM or key != (T, LATENT_ROPE_DIM):
        raise ValueError("cache rows must be [latent | %d], k_rope [T, %d]" % (LATENT_ROPE_DIM, LATENT_ROPE_DIM))
    _vector("slot_mapping", slots, T)
    _vector("positions", positions, T)
    _pairs(frequencies, LATENT_ROPE_DIM)
    H, qs = 0, (0, 0, 0, 0)
    if (q is None) != (out is None):
        raise ValueError("give both q_rope and q_out, or neither")
    if q is not None:
        if len(q) != 3 or q[0] != T or q[2] != LATENT_ROPE_DIM or out != q:
            raise ValueError("q_rope and q_out must be [T, H, %d]" % LATENT_ROPE_DIM)
        H, qs = q[1], _rows("q_out", out, out_stride) + _rows("q_rope", q, q_stride)
    rows = [_rows(n, (x[0], 1, x[1]), (st[0], 0, st[1]))[0] for n, x, st in (("latent", latent, latent_stride), ("k_rope", key, key_stride))]
    return (T, H, V, B, NB), (ctypes.c_int64 * 6)(*qs, *rows)


def latent_cache_write(latent, k_rope, cache, slot_mapping, positions, frequencies, q_rope=None, q_out=None,
                       amplitude: float = 1.0, interleaved: bool = False, stream=None):
    """Store one row a token, [latent | k_rope rotated], in cache [NB, B, V + 64] at slot_mapping[t] (int64; negative =
    skip): latent [T, V], k_rope [T, 64].  With q_rope [T, H, 64] the queries' rotary part is rotated too, into q_out
    [T, H, 64], say q[..., V:] of the attention's queries.  Rows may be strided, in steps of 16 bytes.  Returns
    q_out."""
    some, out = q_rope is not None, q_out is not None
    size, strides = _latent_write_plan(
        latent.shape, latent.stride(), k_rope.shape, k_rope.stride(), cache.shape, slot_mapping.shape, positions.shape,
        frequencies.shape, q_rope.shape if some else None, q_rope.stride() if some else None, q_out.shape if out else None,
        q_out.stride() if out else None)
    some = some and size[1] > 0
    dev, dt = _device_of(cache, "cache"), cache.dtype
    _run_on(dev, "latent_cache_write", _lib.load().latent_cache_write, (
        _row_ptr(q_out, "q_out", dt, dev) if some else None, _row_ptr(q_rope, "q_rope", dt, dev) if some else None,
        _row_ptr(latent, "latent", dt, dev), _row_ptr(k_rope, "k_rope", dt, dev), _ptr(cache, "cache", dt, dev),
        _ptr(slot_mapping, "slot_mapping", torch.int64, dev), _ptr(positions, "positions", torch.int32, dev),
        _ptr(frequencies, "frequencies", torch.float64, dev), *size, strides, amplitude, bool(interleaved), _code(cache),
        _stream_on(stream, dev)))
    return q_out


def paged_latent_attention_workspace_size(num_q_tokens: int, num_heads: int, latent_dim: int, max_seq_len: int,
                                          dtype: torch.dtype = torch.bfloat16) -> int:
    """Bytes of workspace of either latent attention call (num_q_tokens: the sequences of a decode)."""
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    return int(_lib.load().paged_latent_attention_workspace_size(num_q_tokens, num_heads, latent_dim, _int32(max_seq_len),
                                                                 PKV_F32 if dtype == torch.float32 else PKV_BF16))


@_plans
def _latent_plan(out, q, cache, tables, lens, starts):
    """(S, T, H, V, B, maxB, NB); starts None: a decode."""
    if len(q) != 3 or len(cache) != 3 or cache[2] != q[2] or q[2] <= LATENT_ROPE_DIM or out != (*q[:2], q[2] - LATENT_ROPE_DIM):
        raise ValueError("q must be [T, H, V + %d], cache [NB, B, V + %d], out [T, H, V]" % (LATENT_ROPE_DIM, LATENT_ROPE_DIM))
    if len(lens) != 1 or len(tables) != 2 or tables[0] != lens[0]:
        raise ValueError("block_tables must be [S, maxB] and seq_lens [S]")
    if starts is None and lens[0] != q[0]:
        raise ValueError("one query per sequence")
    if starts is not None and starts != (lens[0] + 1,):
        raise ValueError("q_starts must be [S + 1]")
    return lens[0], q[0], q[1], q[2] - LATENT_ROPE_DIM, cache[1], tables[1], cache[0]


@_plans
def _latent_workspace(dev: int, T: int, H: int, V: int, max_len: int, code: int) -> int:
    with torch.cuda.device(dev):
        return _lib.load().paged_latent_attention_workspace_size(T, H, V, max_len, code)


def paged_latent_attention_decode(out, q, cache, block_tables, seq_lens, scale: float, max_seq_len: int,
                                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[s, h] = sum_t softmax_t(scale * q[s, h] . c_t) c_t[:V] over the rows c_t = [latent | key part] of
    sequence s's tokens: q [S, H, V + 64], out [S, H, V] (bf16 or float32), cache [NB, B, V + 64],
    block_tables int32 [S, maxB], seq_lens int32 [S]."""
    S, _, H, V, B, maxb, NB = _latent_plan(out.shape, q.shape, cache.shape, block_tables.shape, seq_lens.shape, None)
    lib, code, dt, i32 = _lib.load(), _code(q), q.dtype, torch.int32
    dev, max_len = _device_of(q, "q"), _int32(max_seq_len)
    _run_with_scratch(dev, "paged_latent_attention_decode", lib.paged_latent_attention_decode,
                      _latent_workspace, (dev, S, H, V, max_len, code), (
        _ptr(out, "out", dt, dev), _ptr(q, "q", dt, dev), _ptr(cache, "cache", dt, dev),
        _ptr(block_tables, "block_tables", i32, dev), _ptr(seq_lens, "seq_lens", i32, dev), S, H, V, B, maxb, NB, max_len,
        scale), workspace, (code, _stream_on(stream, dev)), stream)
    return out


def paged_latent_attention_multi_token(out, q, cache, block_tables, seq_lens, q_starts, scale: float, max_q_len: int,
                                       max_seq_len: int, workspace: Optional[torch.Tensor] = None,
                                       stream=None) -> torch.Tensor:
    """paged_latent_attention_decode for each sequence's last Q_s positions, causal: sequence s owns the rows
    q_starts[s] .. q_starts[s + 1] - 1 of q [T, H, V + 64] and out [T, H, V] (int32 [S + 1])."""
    S, T, H, V, B, maxb, NB = _latent_plan(out.shape, q.shape, cache.shape, block_tables.shape, seq_lens.shape, q_starts.shape)
    lib, code, dt, i32 = _lib.load(), _code(q), q.dtype, torch.int32
    dev, max_len = _device_of(q, "q"), _int32(max_seq_len)
    _run_with_scratch(dev, "paged_latent_attention_multi_token", lib.paged_latent_attention_multi_token,
                      _latent_workspace, (dev, T, H, V, max_len, code), (
        _ptr(out, "out", dt, dev), _ptr(q, "q", dt, dev), _ptr(cache, "cache", dt, dev),
        _ptr(block_tables, "block_tables", i32, dev), _ptr(seq_lens, "seq_lens", i32, dev),
        _ptr(q_starts, "q_starts", i32, dev), S, T, H, V, B, maxb, NB, _int32(max_q_len), max_len, scale), workspace,
        (code, _stream_on(stream, dev)), stream)
    return out


def block_copy(k_caches: Sequence[torch.Tensor], v_caches: Sequence[torch.Tensor],
               block_pairs: torch.Tensor, stream=None) -> None:
    """For every layer, K and V: block dst := block src for each (src, dst)
    row of block_pairs (int64 [N, 2] on the device)."""
    lib = _lib.load()
    L = len(k_caches)
    if len(v_caches) != L:
        raise ValueError("one V cache per K cache")
    if L == 0:
        return
    NB = k_caches[0].shape[0]
    block_bytes = k_caches[0][0].numel() * k_caches[0].element_size()
    for t in list(k_caches) + list(v_caches):
        if t.shape != k_caches[0].shape or t.dtype != k_caches[0].dtype:
            raise ValueError("all caches must share shape and dtype")
    if block_pairs.dim() != 2 or block_pairs.shape[1] != 2:
        raise ValueError("block_pairs must be [N, 2]")
    kp = (ctypes.c_void_p * L)(*[_dev(t, "k_cache") for t in k_caches])
    vp = (ctypes.c_void_p * L)(*[_dev(t, "v_cache") for t in v_caches])
    st = lib.block_copy(kp, vp, L, _dev(block_pairs, "block_pairs", torch.int64, 2),
                        block_pairs.shape[0], NB, block_bytes, _stream(stream))
    _check(st, "block_copy")


def read_device_errors(clear: bool = True, stream=None) -> int:
    """PKV_DEVERR_* bits raised by kernels since the last clear (waits for the stream)."""
    flags = ctypes.c_uint32(0)
    _check(_lib.load().pkv_read_device_errors(ctypes.byref(flags), int(clear), _stream(stream)),
           "pkv_read_device_errors")
    return int(flags.value)


def bounded_wait_check(flags: Optional[torch.Tensor], tag: int, arrive: bool, polls: int,
                       stream=None) -> None:
    """Runs the attention kernels' two bounded waits once with `polls` as the
    limit: the flag wait on the int64 words of `flags` (None: skipped) for
    `tag`, then an mbarrier wait that completes only with `arrive`.  A wait
    that runs out sets DEVERR_TIMEOUT (read_device_errors)."""
    ptr, n = 0, 0
    if flags is not None:
        ptr, n = _dev(flags, "flags", torch.int64, 1), flags.numel()
    _check(_lib.load().pkv_bounded_wait_check(ptr, n, int(tag), int(bool(arrive)), int(polls), _stream(stream)),
           "pkv_bounded_wait_check")


class BlockAllocator:
    """Host block allocator (C++): free stack, block tables, refcounts, CoW."""

    def __init__(self, num_blocks: int, block_size: int):
        self._lib = _lib.load()
        self._h = self._lib.block_allocator_create(int(num_blocks), int(block_size))
        if not self._h:
            raise PkvError(PKV_ERR_INVALID, "block_allocator_create")
        self.num_blocks = int(num_blocks)
        self.block_size = int(block_size)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            self._lib.block_allocator_destroy(h)
            self._h = None

    def add_seq(self, seq: int, num_tokens: int) -> int:
        return self._lib.block_allocator_add_seq(self._h, int(seq), int(num_tokens))

    def add_seq_cached(self, seq: int, tokens):
        """A prompt whose leading full blocks may already be in the pool
        (prefix caching).  Returns (status, cached_tokens): the caller writes
        K/V for positions cached_tokens .. len(tokens) - 1 only."""
        ids = np.ascontiguousarray(np.asarray(tokens, dtype=np.int32))
        cached = ctypes.c_int64(0)
        st = self._lib.block_allocator_add_seq_cached(self._h, int(seq), ids.ctypes.data if ids.size else None,
                                                      int(ids.size), ctypes.byref(cached))
        return st, int(cached.value)

    def cache_stats(self) -> dict:
        """Prefix cache counters: hits, misses, cached_blocks, evictable_blocks."""
        h, m = ctypes.c_int64(0), ctypes.c_int64(0)
        c, e = ctypes.c_int(0), ctypes.c_int(0)
        _check(self._lib.block_allocator_cache_stats(self._h, ctypes.byref(h), ctypes.byref(m), ctypes.byref(c),
                                                     ctypes.byref(e)), "cache_stats")
        return {"hits": h.value, "misses": m.value, "cached_blocks": c.value, "evictable_blocks": e.value}

    def cache_clear(self) -> int:
        return self._lib.block_allocator_cache_clear(self._h)

    def append_slot(self, seq: int):
        """(status, slot, cow_src, cow_dst)."""
        slot, src, dst = ctypes.c_int64(-1), ctypes.c_int32(-1), ctypes.c_int32(-1)
        st = self._lib.block_allocator_append_slot(self._h, int(seq), ctypes.byref(slot),
                                                   ctypes.byref(src), ctypes.byref(dst))
        return st, slot.value, src.value, dst.value

    def append_slots(self, seqs):
        """One token for each of the distinct sequences ``seqs``.  Returns
        (status, slots int64 [n], cow_pairs int64 [k, 2])."""
        ids = np.ascontiguousarray(np.asarray(seqs, dtype=np.int64))
        slots = np.full(len(ids), -1, dtype=np.int64)
        pairs = np.empty((max(1, len(ids)), 2), dtype=np.int64)
        ncow = ctypes.c_int(0)
        st = self._lib.block_allocator_append_slots(self._h, ids.ctypes.data, len(ids),
                                                    slots.ctypes.data, pairs.ctypes.data,
                                                    ctypes.byref(ncow))
        return st, slots, pairs[:ncow.value]

    def append_step(self, seqs, tables: np.ndarray, lens: np.ndarray):
        """append_slots that also updates the dense tables (int32 [n, cap],
        row i for seqs[i]) and lens (int32 [n]) in place, writing only the
        entry of each new token's block.  Both arrays must be C-contiguous
        (pinned host views are fine).  Returns (status, slots, cow_pairs)."""
        ids = np.ascontiguousarray(np.asarray(seqs, dtype=np.int64))
        if (tables.dtype != np.int32 or lens.dtype != np.int32 or tables.ndim != 2 or
                not tables.flags.c_contiguous or not lens.flags.c_contiguous or
                tables.shape[0] != len(ids) or lens.shape[0] != len(ids)):
            raise ValueError("tables must be int32 [n, cap] and lens int32 [n], C-contiguous")
        slots = np.full(len(ids), -1, dtype=np.int64)
        pairs = np.empty((max(1, len(ids)), 2), dtype=np.int64)
        ncow = ctypes.c_int(0)
        st = self._lib.block_allocator_append_step(self._h, ids.ctypes.data, len(ids), tables.ctypes.data,
                                                   tables.shape[1], lens.ctypes.data, slots.ctypes.data,
                                                   pairs.ctypes.data, ctypes.byref(ncow))
        return st, slots, pairs[:ncow.value]

    def extend(self, seq: int, count: int):
        """Slots for ``count`` more tokens of seq (all or nothing).  Returns
        (status, slots int64 [count], cow_src, cow_dst)."""
        slots = np.zeros(max(int(count), 1), dtype=np.int64)
        src, dst = ctypes.c_int32(-1), ctypes.c_int32(-1)
        st = int(self._lib.block_allocator_extend(self._h, int(seq), int(count),
                                                  slots.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
                                                  ctypes.byref(src), ctypes.byref(dst)))
        if st != PKV_OK:
            return st, slots[:0], -1, -1
        return st, slots[:int(count)], int(src.value), int(dst.value)

    def truncate(self, seq: int, num_tokens: int) -> int:
        """Keep the first num_tokens tokens of seq (roll back rejected drafts)."""
        return int(self._lib.block_allocator_truncate(self._h, int(seq), int(num_tokens)))

    def fork(self, parent: int, child: int) -> int:
        return self._lib.block_allocator_fork(self._h, int(parent), int(child))

    def free_seq(self, seq: int) -> int:
        return self._lib.block_allocator_free_seq(self._h, int(seq))

    def num_tokens(self, seq: int) -> int:
        return int(self._lib.block_allocator_num_tokens(self._h, int(seq)))

    def block_table(self, seq: int):
        n = self.num_tokens(seq)
        if n < 0:
            raise PkvError(PKV_ERR_INVALID, "block_table")
        cap = max(1, -(-n // self.block_size) + 1)
        buf = np.empty(cap, dtype=np.int32)
        cnt = ctypes.c_int(0)
        _check(self._lib.block_allocator_block_table(self._h, int(seq), buf.ctypes.data, cap,
                                                     ctypes.byref(cnt)), "block_table")
        return buf[:cnt.value].tolist()

    def block_tables(self, seqs, cap: int, pad: int = -1):
        """(tables int32 [n, cap], seq_lens int32 [n]) as numpy arrays."""
        ids = np.ascontiguousarray(np.asarray(seqs, dtype=np.int64))
        tables = np.empty((len(ids), max(1, cap)), dtype=np.int32)
        lens = np.empty(len(ids), dtype=np.int32)
        _check(self._lib.block_allocator_block_tables(self._h, ids.ctypes.data, len(ids),
                                                      tables.ctypes.data, tables.shape[1],
                                                      int(pad), lens.ctypes.data), "block_tables")
        return tables, lens

    def prefix_groups(self, seqs):
        """(group_offsets int32 [G + 1], prefix_lens int32 [G]) for the
        sequences in the given order (runs that start with the same blocks)."""
        ids = np.ascontiguousarray(np.asarray(seqs, dtype=np.int64))
        offs = np.zeros(len(ids) + 1, dtype=np.int32)
        pre = np.zeros(max(1, len(ids)), dtype=np.int32)
        ng = ctypes.c_int(0)
        _check(self._lib.block_allocator_prefix_groups(self._h, ids.ctypes.data, len(ids), offs.ctypes.data,
                                                       pre.ctypes.data, ctypes.byref(ng)), "prefix_groups")
        return offs[:ng.value + 1].copy(), pre[:ng.value].copy()

    def slots(self, seq: int, start: int, count: int) -> np.ndarray:
        out = np.empty(max(0, count), dtype=np.int64)
        _check(self._lib.block_allocator_slots(self._h, int(seq), int(start), int(count),
                                               out.ctypes.data), "slots")
        return out

    def num_free(self) -> int:
        return int(self._lib.block_allocator_num_free(self._h))

    def refcount(self, block: int) -> int:
        return int(self._lib.block_allocator_refcount(self._h, int(block)))

    def waste(self):
        used, alloc = ctypes.c_int64(0), ctypes.c_int64(0)
        _check(self._lib.block_allocator_waste(self._h, ctypes.byref(used), ctypes.byref(alloc)),
               "waste")
        return used.value, alloc.value
