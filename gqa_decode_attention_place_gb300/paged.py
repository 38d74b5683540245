"""Binding of the paged bf16 cache: append, decode step, and the pages' calls
(include/gqa_attn.h).

As in kv8.py: torch CUDA tensors, checked natively, on the tensors' own device
and on ``stream`` (default: that device's current stream).  k_pages and v_pages
are [P,Hkv,page,D] bf16 with dense rows and any other strides, alike for both:
views of a token-major pool or of one buffer for both will do.
"""

from __future__ import annotations

import ctypes

import torch

from . import AttnError, _raise, kv8, load_library
from .kv8 import _BF16, _I32, _dims, _empty, _made_on, _on, _stream, _zeros

_native = None
_address: dict = {}


def _load():
    """The native checks (kv8.py's) and the addresses of the C entry points."""
    global _native
    m = kv8._native or kv8._load()
    lib = load_library()
    for name in ("attn_paged_append", "attn_decode_step_paged", "attn_pages_reserve",
                 "attn_pages_fork", "attn_pages_compact"):
        _address[name] = ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
    _native = m  # last: other threads go on from here
    return m


def attn_paged_append(k_new, v_new, positions, page_table, k_pages, v_pages, lengths=None,
                      stream=None) -> None:
    """Rows k_new/v_new [B,S,Hkv,D] (or [B,Hkv,D]; views with a token stride
    will do) into rows positions[b] + t, t < lengths[b] (default S), of the
    pages that page_table [B,M] names, in place."""
    m = _native or _load()
    code = m.paged_append(_address["attn_paged_append"], _stream(stream, k_new), k_new, v_new,
                          positions, lengths, page_table, k_pages, v_pages)
    if code:
        _raise(code, "attn_paged_append")


def attn_paged_workspace_size(B: int, S: int, Hq: int, Hkv: int, D: int) -> int:
    return int(load_library().attn_paged_workspace_size(B, S, Hq, Hkv, D))


def attn_pages_workspace_size(B: int, S: int, P: int, page: int) -> int:
    return int(load_library().attn_pages_workspace_size(B, S, P, page))


def paged_workspace(B: int, S: int, Hq: int, Hkv: int, D: int, device=None) -> torch.Tensor:
    """A zero-filled workspace of the size attn_decode_step_paged needs."""
    return _zeros(attn_paged_workspace_size(B, S, Hq, Hkv, D), "attn_paged_workspace_size", device)


def pages_workspace(B: int, S: int, P: int, page: int, device=None) -> torch.Tensor:
    """A zero-filled workspace for attn_pages_reserve (of up to S new tokens),
    attn_pages_fork and attn_pages_compact."""
    return _zeros(attn_pages_workspace_size(B, S, P, page), "attn_pages_workspace_size", device)


def attn_decode_step_paged(q, positions, page_table, k_pages, v_pages, scale: float, lengths=None,
                           out=None, workspace=None, stream=None) -> torch.Tensor:
    """Attention of q [B,S,Hq,D] (or [B,Hq,D], one token) over the pages: token
    t of sequence b sees rows 0 .. positions[b] + t; tokens past lengths[b]
    (default S) get zeros."""
    m = _native or _load()
    if out is None:
        out = _empty(q.shape, _BF16, _on(q, "q"), stream)
    if workspace is None:
        shape = _dims(q, "q", 3, 4)
        S = shape[1] if len(shape) == 4 else 1
        Hkv = _dims(k_pages, "k_pages", 4)[1]
        with _made_on(stream, q.device):
            workspace = paged_workspace(shape[0], S, shape[-2], Hkv, shape[-1], q.device)
    code = m.decode_paged(_address["attn_decode_step_paged"], _stream(stream, q), q, positions,
                          lengths, page_table, k_pages, v_pages, scale, out, workspace)
    if code:
        _raise(code, "attn_decode_step_paged")
    return out


def attn_pages_reserve(page_table, page_refs, positions, k_pages, v_pages, tokens: int,
                       lengths=None, taken=None, workspace=None, stream=None) -> torch.Tensor:
    """Pages of their own for the rows positions[b] .. of each sequence's new
    tokens (lengths [B], or `tokens` each): free ones where there are none, and
    copies of those that sequences share.  page_table [B,M] and page_refs [P]
    int32 are changed in place.  Returns taken [B]: the pages each sequence
    took, -1 where the pool is too small (nothing of it is changed)."""
    m = _native or _load()
    device = _on(page_table, "page_table", _I32)
    if taken is None:
        taken = _empty(_dims(page_table, "page_table", 2)[:1], _I32, device, stream)
    if workspace is None:
        P, _, page, _ = _dims(k_pages, "k_pages", 4)
        if tokens < 1:
            raise AttnError(1, "attn_pages_reserve")
        with _made_on(stream, device):
            workspace = pages_workspace(_dims(page_table, "page_table", 2)[0], tokens, P, page,
                                        device)
    code = m.pages_reserve(_address["attn_pages_reserve"], _stream(stream, page_table), page_table,
                           page_refs, positions, lengths, k_pages, v_pages, tokens, taken,
                           workspace)
    if code:
        _raise(code, "attn_pages_reserve")
    return taken


def attn_pages_fork(page_table, page_refs, page: int, parents=None, lengths=None, workspace=None,
                    stream=None) -> None:
    """Every sequence becomes a copy of what sequence parents[b] was (-1: it
    ends; None: all stay), cut to the pages of its first lengths[b] rows (None:
    none is cut).  Pages are shared, not copied; page_table [B,M] and page_refs
    [P] are changed in place."""
    m = _native or _load()
    if workspace is None:
        device = _on(page_table, "page_table", _I32)
        with _made_on(stream, device):
            workspace = torch.zeros(256, dtype=torch.uint8, device=device)
    code = m.pages_fork(_address["attn_pages_fork"], _stream(stream, page_table), page_table,
                        page_refs, page, parents, lengths, workspace)
    if code:
        _raise(code, "attn_pages_fork")


def attn_pages_compact(page_table, page_refs, k_pages, v_pages, page_map=None, workspace=None,
                       stream=None) -> torch.Tensor:
    """Moves the n pages in use to pages 0 .. n - 1, with their rows, counts and
    table entries.  Returns page_map [P]: where each page went, -1 for a free
    one."""
    m = _native or _load()
    device = _on(page_refs, "page_refs", _I32)
    if page_map is None:
        page_map = _empty(page_refs.shape, _I32, device, stream)
    if workspace is None:
        P, _, page, _ = _dims(k_pages, "k_pages", 4)
        with _made_on(stream, device):
            workspace = pages_workspace(1, 1, P, page, device)
    code = m.pages_compact(_address["attn_pages_compact"], _stream(stream, page_refs), page_table,
                           page_refs, k_pages, v_pages, page_map, workspace)
    if code:
        _raise(code, "attn_pages_compact")
    return page_map
