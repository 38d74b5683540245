"""Binding of the query/key norm with rotation, the 8-bit KV cache and the
block-sparse decode (include/gqa_attn.h).

As in the package's other functions: torch CUDA tensors are checked and their
pointers passed to the C entry point of the same name on the tensors' own
device, on ``stream`` (default: that device's current stream).  The checks are
native (csrc/marshal.cpp).  Codes are ``torch.float8_e4m3fn`` tensors.
"""

from __future__ import annotations

import contextlib
import ctypes
import importlib.util
import threading

import torch

from . import AttnError, _DEBUG_WORKSPACES, _build, _raise, attn_debug_build, load_library

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_native = None
_address: dict = {}
_loading = threading.Lock()


def _load():
    """The native checks and the addresses of the C entry points (built in-tree first if needed)."""
    global _native
    with _loading:
        if _native is None:
            lib = load_library()
            spec = importlib.util.spec_from_file_location("_gqa_marshal", _build.build_marshal())
            native = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(native)
            for name in ("attn_qk_norm_rope", "attn_qk_norm_rope_append", "attn_kv8_append",
                         "attn_decode_step_kv8", "attn_decode_step_kv8_blocks",
                         "attn_decode_step_kv8_sparse", "attn_block_scores", "attn_block_select"):
                _address[name] = ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
            _native = native  # last: other threads go on from here
    return _native


def _stream(stream, t) -> int:
    """The stream handle for a call on t's device (0 where t is no CUDA tensor: the call's checks
    refuse it before the handle is used)."""
    if stream is None:
        device = t.get_device() if isinstance(t, torch.Tensor) else -1
        return torch._C._cuda_getCurrentRawStream(device) if device >= 0 else 0
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _made_on(stream, device):
    """Where a call makes its output or workspace itself: memory of the stream the call runs on,
    so that it is filled and handed back in that stream's order."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def _empty(shape, dtype, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _made_on(stream, device):
        return torch.empty(shape, dtype=dtype, device=device)


def _on(t, name, dtype=_BF16):
    """t's device, for the outputs a call makes itself."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _dims(t, name, *ndims):
    if t.dim() not in ndims:
        raise ValueError(f"{name} must have {ndims} dims, got shape {tuple(t.shape)}")
    return t.shape


def attn_qk_norm_rope(q, k, q_weight, k_weight, eps: float, positions, cos_table=None,
                      sin_table=None, q_out=None, k_out=None, stream=None):
    """RMS norm of every head of q [N,Hq,D] and k [N,Hkv,D] (weights [D] or
    None), then the rotation at positions [N] by rows of cos_table/sin_table
    [L,D] float32 (or none).  q and k may be views with a token stride.
    Returns (q_out, k_out), dense bf16."""
    m = _native or _load()
    if q_out is None:
        q_out = _empty(q.shape, _BF16, _on(q, "q"), stream)
    if k_out is None:
        k_out = _empty(k.shape, _BF16, _on(k, "k"), stream)
    code = m.qk_norm_rope(_address["attn_qk_norm_rope"], _stream(stream, q), q, k, q_weight,
                          k_weight, eps, positions, cos_table, sin_table, q_out, k_out)
    if code:
        _raise(code, "attn_qk_norm_rope")
    return q_out, k_out


def attn_qk_norm_rope_append(q, k_new, v_new, q_weight, k_weight, eps: float, positions, k_cache,
                             v_cache, cos_table=None, sin_table=None, q_out=None,
                             stream=None) -> torch.Tensor:
    """attn_qk_norm_rope for q [B,S,Hq,D], k_new and v_new [B,S,Hkv,D] (or
    without S, for one token), the keys and values written to rows
    positions[b] + t of the bf16 caches [B,Hkv,L,D].  Returns q_out."""
    m = _native or _load()
    if q_out is None:
        q_out = _empty(q.shape, _BF16, _on(q, "q"), stream)
    code = m.qk_norm_rope_append(_address["attn_qk_norm_rope_append"], _stream(stream, q), q,
                                 k_new, v_new, q_weight, k_weight, eps, positions, k_cache,
                                 v_cache, cos_table, sin_table, q_out)
    if code:
        _raise(code, "attn_qk_norm_rope_append")
    return q_out


def attn_kv8_append(k_new, v_new, positions, k_cache, v_cache, k_scale, v_scale, block: int,
                    k_bounds=None, stream=None) -> None:
    """Rows k_new/v_new [B,S,Hkv,D] (or [B,Hkv,D]; views with a token stride
    will do) into rows positions[b] + t of the 8-bit caches [B,Hkv,L,D], in
    place, with the blocks' scales [B,Hkv,NB] and, if given, the keys' bounds
    [B,Hkv,NB,2,D]."""
    m = _native or _load()
    code = m.kv8_append(_address["attn_kv8_append"], _stream(stream, k_cache), k_new, v_new,
                        positions, k_cache, v_cache, k_scale, v_scale, block, k_bounds)
    if code:
        _raise(code, "attn_kv8_append")


def attn_kv8_workspace_size(B: int, Hq: int, Hkv: int, L: int, D: int) -> int:
    return int(load_library().attn_kv8_workspace_size(B, Hq, Hkv, L, D))


def attn_kv8_sparse_workspace_size(B: int, Hq: int, Hkv: int, L: int, D: int, block: int,
                                   count: int) -> int:
    return int(load_library().attn_kv8_sparse_workspace_size(B, Hq, Hkv, L, D, block, count))


def _zeros(n, where, device):
    if n == 0:
        raise AttnError(2, where)
    ws = torch.zeros(n, dtype=torch.uint8, device=device or "cuda")
    if attn_debug_build():
        _DEBUG_WORKSPACES.append(ws)
    return ws


def kv8_workspace(B: int, Hq: int, Hkv: int, L: int, D: int, device=None) -> torch.Tensor:
    """A zero-filled workspace of the size the 8-bit decode calls need."""
    return _zeros(attn_kv8_workspace_size(B, Hq, Hkv, L, D), "attn_kv8_workspace_size", device)


def kv8_sparse_workspace(B: int, Hq: int, Hkv: int, L: int, D: int, block: int, count: int,
                         device=None) -> torch.Tensor:
    """A zero-filled workspace of the size attn_decode_step_kv8_sparse needs."""
    return _zeros(attn_kv8_sparse_workspace_size(B, Hq, Hkv, L, D, block, count),
                  "attn_kv8_sparse_workspace_size", device)


def attn_decode_step_kv8(q, positions, k_cache, v_cache, k_scale, v_scale, block: int,
                         scale: float, out=None, workspace=None, stream=None) -> torch.Tensor:
    """attn_decode_step over the 8-bit cache (q [B,Hq,D]; codes [B,Hkv,L,D];
    scales [B,Hkv,ceil(L/block)])."""
    m = _native or _load()
    if out is None:
        out = _empty(q.shape, _BF16, _on(q, "q"), stream)
    if workspace is None:
        B, Hq, D = _dims(q, "q", 3)
        _, Hkv, L, _ = _dims(k_cache, "k_cache", 4)
        with _made_on(stream, q.device):
            workspace = kv8_workspace(B, Hq, Hkv, L, D, q.device)
    code = m.decode_kv8(_address["attn_decode_step_kv8"], _stream(stream, q), q, positions,
                        k_cache, v_cache, k_scale, v_scale, block, scale, out, workspace)
    if code:
        _raise(code, "attn_decode_step_kv8")
    return out


def attn_block_scores(q, positions, k_bounds, L: int, block: int, out=None,
                      stream=None) -> torch.Tensor:
    """scores [B,Hkv,NB]: what the g query heads of a KV head can score at
    most with each block's keys as they were appended (before their rounding to
    8 bits), summed over the heads; -inf past the position's block.
    L is the cache's length, k_bounds [B,Hkv,NB,2,D]."""
    m = _native or _load()
    if out is None:
        device = _on(q, "q")
        out = _empty(_dims(k_bounds, "k_bounds", 5)[:3], _F32, device, stream)
    code = m.block_scores(_address["attn_block_scores"], _stream(stream, q), q, positions,
                          k_bounds, L, block, out)
    if code:
        _raise(code, "attn_block_scores")
    return out


def attn_block_select(scores, positions, L: int, block: int, count: int, first: int = 1,
                      recent: int = 1, out=None, stream=None) -> torch.Tensor:
    """Indices [B,Hkv,count] int32 of the blocks to attend: the first `first`,
    the last `recent` and the best-scored others up to each position,
    ascending, -1 behind the last."""
    m = _native or _load()
    if out is None:
        device = _on(scores, "scores", _F32)
        if count < 1:
            raise AttnError(1, "attn_block_select")
        out = _empty((*_dims(scores, "scores", 3)[:2], count), _I32, device, stream)
    code = m.block_select(_address["attn_block_select"], _stream(stream, scores), scores,
                          positions, L, block, count, first, recent, out)
    if code:
        _raise(code, "attn_block_select")
    return out


def attn_decode_step_kv8_blocks(q, positions, k_cache, v_cache, k_scale, v_scale, block: int,
                                block_index, scale: float, out=None, workspace=None,
                                stream=None) -> torch.Tensor:
    """attn_decode_step_kv8 over the rows of the blocks listed in block_index
    [B,Hkv,count] int32 (-1: none), up to each position."""
    m = _native or _load()
    if out is None:
        out = _empty(q.shape, _BF16, _on(q, "q"), stream)
    if workspace is None:
        B, Hq, D = _dims(q, "q", 3)
        _, Hkv, L, _ = _dims(k_cache, "k_cache", 4)
        with _made_on(stream, q.device):
            workspace = kv8_workspace(B, Hq, Hkv, L, D, q.device)
    code = m.decode_kv8_blocks(_address["attn_decode_step_kv8_blocks"], _stream(stream, q), q,
                               positions, k_cache, v_cache, k_scale, v_scale, block, block_index,
                               scale, out, workspace)
    if code:
        _raise(code, "attn_decode_step_kv8_blocks")
    return out


def attn_decode_step_kv8_sparse(q, positions, k_cache, v_cache, k_scale, v_scale, k_bounds,
                                block: int, count: int, scale: float, first: int = 1,
                                recent: int = 1, out=None, workspace=None,
                                stream=None) -> torch.Tensor:
    """attn_block_scores, attn_block_select and attn_decode_step_kv8_blocks in
    one call: a decode step that attends `count` blocks per KV head."""
    m = _native or _load()
    if out is None:
        out = _empty(q.shape, _BF16, _on(q, "q"), stream)
    if workspace is None:
        B, Hq, D = _dims(q, "q", 3)
        _, Hkv, L, _ = _dims(k_cache, "k_cache", 4)
        with _made_on(stream, q.device):
            workspace = kv8_sparse_workspace(B, Hq, Hkv, L, D, block, count, q.device)
    code = m.decode_kv8_sparse(_address["attn_decode_step_kv8_sparse"], _stream(stream, q), q,
                               positions, k_cache, v_cache, k_scale, v_scale, block, k_bounds,
                               count, first, recent, scale, out, workspace)
    if code:
        _raise(code, "attn_decode_step_kv8_sparse")
    return out
