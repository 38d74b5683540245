"""Binding of the query/key norm with rotation, the 8-bit KV cache and the
block-sparse decode (include/gqa_attn.h).

As in the package's other functions: torch CUDA tensors are checked and their
pointers passed to the C entry point of the same name on the tensors' own
device, on ``stream`` (default: that device's current stream).  Codes are
``torch.float8_e4m3fn`` tensors.
"""

from __future__ import annotations

import torch

from . import AttnError, _DEBUG_WORKSPACES, _raise, attn_debug_build, load_library

_BF16, _F32, _I32, _E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


def _want(where, t, name, dtype, shape, device):
    """t is a dense CUDA tensor of this dtype, shape and device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.shape != shape:
        raise ValueError(f"{where}: {name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{where}: {name} is on {t.device}, not on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _lead(t, name, dtype, ndims):
    """The tensor whose shape and device the others follow."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() not in ndims:
        raise ValueError(f"{name} must have {ndims} dims, got shape {tuple(t.shape)}")
    return t.device


def _call(where, fn, device, stream, *args):
    """One C call on `device` and its status."""
    if stream is None:
        stream = torch.cuda.current_stream(device).cuda_stream
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    else:
        stream = int(stream)
    if torch.cuda.current_device() == device.index:
        code = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            code = fn(*args, stream)
    if code:
        _raise(code, where)


def _blocks(L, block):
    if block not in (16, 32, 64, 128):
        raise AttnError(2, "block")
    return (L + block - 1) // block


def _rows(where, t, name, shape, device):
    """(pointer, token stride) of [tokens.., heads, D] rows: heads of a token dense, tokens
    evenly spaced (a view of a fused projection buffer will do)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not _BF16:
        raise TypeError(f"{name} must be {_BF16}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.shape != shape:
        raise ValueError(f"{where}: {name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{where}: {name} is on {t.device}, not on {device}")
    H, D = shape[-2:]
    if t.is_contiguous():
        return t.data_ptr(), H * D
    st = t.stride()
    ok = (D == 1 or st[-1] == 1) and (H == 1 or st[-2] == D)
    if len(shape) == 3:
        token = st[0] if shape[0] > 1 else H * D
    else:
        B, S = shape[:2]
        token = st[1] if S > 1 else st[0] if B > 1 else H * D
        ok = ok and (B == 1 or S == 1 or st[0] == S * st[1])
    if not ok:
        raise ValueError(f"{where}: the heads of a token of {name} must be dense and its tokens "
                         f"evenly spaced, got strides {tuple(st)}")
    return t.data_ptr(), token


def _norm_args(where, q, k, kname, q_weight, k_weight, cos_table, sin_table, L, device):
    Hkv, D = k.shape[-2], q.shape[-1]
    qp, qs = _rows(where, q, "q", q.shape, device)
    kp, ks = _rows(where, k, kname, q.shape[:-2] + (Hkv, D), device)
    wq = None if q_weight is None else _want(where, q_weight, "q_weight", _BF16, (D,), device)
    wk = None if k_weight is None else _want(where, k_weight, "k_weight", _BF16, (D,), device)
    if (cos_table is None) != (sin_table is None):
        raise ValueError(f"{where}: give both cos_table and sin_table, or neither")
    cos = sin = None
    if cos_table is not None:
        cos = _want(where, cos_table, "cos_table", _F32, (L, D), device)
        sin = _want(where, sin_table, "sin_table", _F32, (L, D), device)
    return qp, qs, kp, ks, wq, wk, cos, sin


def attn_qk_norm_rope(q, k, q_weight, k_weight, eps: float, positions, cos_table=None,
                      sin_table=None, q_out=None, k_out=None, stream=None):
    """RMS norm of every head of q [N,Hq,D] and k [N,Hkv,D] (weights [D] or
    None), then the rotation at positions [N] by rows of cos_table/sin_table
    [L,D] float32 (or none).  q and k may be views with a token stride.
    Returns (q_out, k_out), dense bf16."""
    where = "attn_qk_norm_rope"
    device = _lead(q, "q", _BF16, (3,))
    _lead(k, "k", _BF16, (3,))
    N, Hq, D = q.shape
    Hkv = k.shape[1]
    # without tables any position will do
    L = cos_table.shape[0] if cos_table is not None else 0x7fffffff
    qp, qs, kp, ks, wq, wk, cos, sin = _norm_args(where, q, k, "k", q_weight, k_weight, cos_table,
                                                  sin_table, L, device)
    pos = _want(where, positions, "positions", _I32, (N,), device)
    if q_out is None:
        q_out = torch.empty((N, Hq, D), dtype=_BF16, device=device)
    if k_out is None:
        k_out = torch.empty((N, Hkv, D), dtype=_BF16, device=device)
    _call(where, load_library().attn_qk_norm_rope, device, stream, qp, kp, qs, ks, wq, wk,
          float(eps), pos, cos, sin, N, Hq, Hkv, D, L,
          _want(where, q_out, "q_out", _BF16, (N, Hq, D), device),
          _want(where, k_out, "k_out", _BF16, (N, Hkv, D), device))
    return q_out, k_out


def attn_qk_norm_rope_append(q, k_new, v_new, q_weight, k_weight, eps: float, positions, k_cache,
                             v_cache, cos_table=None, sin_table=None, q_out=None,
                             stream=None) -> torch.Tensor:
    """attn_qk_norm_rope for q [B,S,Hq,D], k_new and v_new [B,S,Hkv,D] (or
    without S, for one token), the keys and values written to rows
    positions[b] + t of the bf16 caches [B,Hkv,L,D].  Returns q_out."""
    where = "attn_qk_norm_rope_append"
    device = _lead(q, "q", _BF16, (3, 4))
    _lead(k_new, "k_new", _BF16, (q.dim(),))
    _lead(k_cache, "k_cache", _BF16, (4,))
    B, Hq, D = q.shape[0], q.shape[-2], q.shape[-1]
    S = q.shape[1] if q.dim() == 4 else 1
    Hkv, L = k_new.shape[-2], k_cache.shape[2]
    qp, qs, kp, ks, wq, wk, cos, sin = _norm_args(where, q, k_new, "k_new", q_weight, k_weight,
                                                  cos_table, sin_table, L, device)
    vp, vs = _rows(where, v_new, "v_new", k_new.shape, device)
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=_BF16, device=device)
    cache = (B, Hkv, L, D)
    _call(where, load_library().attn_qk_norm_rope_append, device, stream, qp, kp, vp, qs, ks, vs,
          wq, wk, float(eps), _want(where, positions, "positions", _I32, (B,), device), cos, sin,
          _want(where, k_cache, "k_cache", _BF16, cache, device),
          _want(where, v_cache, "v_cache", _BF16, cache, device), B, S, Hq, Hkv, D, L,
          _want(where, q_out, "q_out", _BF16, q.shape, device))
    return q_out


def attn_kv8_append(k_new, v_new, positions, k_cache, v_cache, k_scale, v_scale, block: int,
                    k_bounds=None, stream=None) -> None:
    """Rows k_new/v_new [B,S,Hkv,D] (or [B,Hkv,D]) into rows positions[b] + t
    of the 8-bit caches [B,Hkv,L,D], in place, with the blocks' scales
    [B,Hkv,NB] and, if given, the keys' bounds [B,Hkv,NB,2,D]."""
    where = "attn_kv8_append"
    device = _lead(k_cache, "k_cache", _E4M3, (4,))
    _lead(k_new, "k_new", _BF16, (3, 4))
    B, Hkv, L, D = k_cache.shape
    S = k_new.shape[1] if k_new.dim() == 4 else 1
    nb = _blocks(L, block)
    new = (B, S, Hkv, D) if k_new.dim() == 4 else (B, Hkv, D)
    cache, scales = (B, Hkv, L, D), (B, Hkv, nb)
    _call(where, load_library().attn_kv8_append, device, stream,
          _want(where, k_new, "k_new", _BF16, new, device),
          _want(where, v_new, "v_new", _BF16, new, device),
          _want(where, positions, "positions", _I32, (B,), device),
          _want(where, k_cache, "k_cache", _E4M3, cache, device),
          _want(where, v_cache, "v_cache", _E4M3, cache, device),
          _want(where, k_scale, "k_scale", _F32, scales, device),
          _want(where, v_scale, "v_scale", _F32, scales, device),
          None if k_bounds is None else
          _want(where, k_bounds, "k_bounds", _BF16, (B, Hkv, nb, 2, D), device),
          B, S, Hkv, L, D, block)


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


def _decode_args(where, q, positions, k_cache, v_cache, k_scale, v_scale, block, out):
    device = _lead(q, "q", _BF16, (3,))
    _lead(k_cache, "k_cache", _E4M3, (4,))
    B, Hq, D = q.shape
    Hkv, L = k_cache.shape[1], k_cache.shape[2]
    nb = _blocks(L, block)
    cache, scales = (B, Hkv, L, D), (B, Hkv, nb)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=_BF16, device=device)
    ptrs = (_want(where, q, "q", _BF16, (B, Hq, D), device),
            _want(where, positions, "positions", _I32, (B,), device),
            _want(where, k_cache, "k_cache", _E4M3, cache, device),
            _want(where, v_cache, "v_cache", _E4M3, cache, device),
            _want(where, k_scale, "k_scale", _F32, scales, device),
            _want(where, v_scale, "v_scale", _F32, scales, device))
    return (device, B, Hq, Hkv, L, D, nb, out, ptrs,
            _want(where, out, "out", _BF16, (B, Hq, D), device))


def _workspace(where, ws, device):
    if not isinstance(ws, torch.Tensor) or not ws.is_contiguous() or ws.device != device:
        raise ValueError(f"{where}: workspace must be a contiguous tensor on {device}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def attn_decode_step_kv8(q, positions, k_cache, v_cache, k_scale, v_scale, block: int,
                         scale: float, out=None, workspace=None, stream=None) -> torch.Tensor:
    """attn_decode_step over the 8-bit cache (q [B,Hq,D]; codes [B,Hkv,L,D];
    scales [B,Hkv,ceil(L/block)])."""
    where = "attn_decode_step_kv8"
    device, B, Hq, Hkv, L, D, _, out, ptrs, op = _decode_args(
        where, q, positions, k_cache, v_cache, k_scale, v_scale, block, out)
    if workspace is None:
        workspace = kv8_workspace(B, Hq, Hkv, L, D, device)
    _call(where, load_library().attn_decode_step_kv8, device, stream, *ptrs, B, Hq, Hkv, L, D,
          block, float(scale), op, *_workspace(where, workspace, device))
    return out


def attn_block_scores(q, positions, k_bounds, L: int, block: int, out=None,
                      stream=None) -> torch.Tensor:
    """scores [B,Hkv,NB]: what the g query heads of a KV head can score in
    each block at most, summed over the heads; -inf past the position's block.
    L is the cache's length, k_bounds [B,Hkv,NB,2,D]."""
    where = "attn_block_scores"
    device = _lead(q, "q", _BF16, (3,))
    _lead(k_bounds, "k_bounds", _BF16, (5,))
    B, Hq, D = q.shape
    Hkv, nb = k_bounds.shape[1], _blocks(L, block)
    if out is None:
        out = torch.empty((B, Hkv, nb), dtype=_F32, device=device)
    _call(where, load_library().attn_block_scores, device, stream,
          _want(where, q, "q", _BF16, (B, Hq, D), device),
          _want(where, positions, "positions", _I32, (B,), device),
          _want(where, k_bounds, "k_bounds", _BF16, (B, Hkv, nb, 2, D), device),
          B, Hq, Hkv, L, D, block, _want(where, out, "out", _F32, (B, Hkv, nb), device))
    return out


def attn_block_select(scores, positions, L: int, block: int, count: int, first: int = 1,
                      recent: int = 1, out=None, stream=None) -> torch.Tensor:
    """Indices [B,Hkv,count] int32 of the blocks to attend: the first `first`,
    the last `recent` and the best-scored others up to each position,
    ascending, -1 behind the last."""
    where = "attn_block_select"
    device = _lead(scores, "scores", _F32, (3,))
    B, Hkv = scores.shape[:2]
    nb = _blocks(L, block)
    if out is None:
        out = torch.empty((B, Hkv, count), dtype=_I32, device=device)
    _call(where, load_library().attn_block_select, device, stream,
          _want(where, scores, "scores", _F32, (B, Hkv, nb), device),
          _want(where, positions, "positions", _I32, (B,), device), B, Hkv, L, block, count,
          first, recent, _want(where, out, "out", _I32, (B, Hkv, count), device))
    return out


def attn_decode_step_kv8_blocks(q, positions, k_cache, v_cache, k_scale, v_scale, block: int,
                                block_index, scale: float, out=None, workspace=None,
                                stream=None) -> torch.Tensor:
    """attn_decode_step_kv8 over the rows of the blocks listed in block_index
    [B,Hkv,count] int32 (-1: none), up to each position."""
    where = "attn_decode_step_kv8_blocks"
    device, B, Hq, Hkv, L, D, _, out, ptrs, op = _decode_args(
        where, q, positions, k_cache, v_cache, k_scale, v_scale, block, out)
    _lead(block_index, "block_index", _I32, (3,))
    count = block_index.shape[2]
    ip = _want(where, block_index, "block_index", _I32, (B, Hkv, count), device)
    if workspace is None:
        workspace = kv8_workspace(B, Hq, Hkv, L, D, device)
    _call(where, load_library().attn_decode_step_kv8_blocks, device, stream, *ptrs, ip, count, B,
          Hq, Hkv, L, D, block, float(scale), op, *_workspace(where, workspace, device))
    return out


def attn_decode_step_kv8_sparse(q, positions, k_cache, v_cache, k_scale, v_scale, k_bounds,
                                block: int, count: int, scale: float, first: int = 1,
                                recent: int = 1, out=None, workspace=None,
                                stream=None) -> torch.Tensor:
    """attn_block_scores, attn_block_select and attn_decode_step_kv8_blocks in
    one call: a decode step that attends `count` blocks per KV head."""
    where = "attn_decode_step_kv8_sparse"
    device, B, Hq, Hkv, L, D, nb, out, ptrs, op = _decode_args(
        where, q, positions, k_cache, v_cache, k_scale, v_scale, block, out)
    bp = _want(where, k_bounds, "k_bounds", _BF16, (B, Hkv, nb, 2, D), device)
    if workspace is None:
        workspace = kv8_sparse_workspace(B, Hq, Hkv, L, D, block, count, device)
    _call(where, load_library().attn_decode_step_kv8_sparse, device, stream, *ptrs, bp, count,
          first, recent, B, Hq, Hkv, L, D, block, float(scale), op,
          *_workspace(where, workspace, device))
    return out
