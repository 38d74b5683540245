"""Refusals of the paged cache's calls: on the host, before any launch (no GPU
needed)."""

import os
import re

import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from gqa_decode_attention_place_gb300 import _build

P = 0x1000  # fake but 16-byte aligned "device" pointer: never dereferenced
Q = 0x2000
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
POOL = dict(kp=P, vp=Q, ps=8 * 16 * 128, hs=16 * 128, rs=128, Hkv=8, D=128, pages=9, page=16, M=4)
BAD_POOL = [(dict(kp=None), INVALID), (dict(vp=None), INVALID), (dict(kp=P + 8), INVALID),
            (dict(vp=Q + 2), INVALID), (dict(Hkv=0), INVALID), (dict(D=0), INVALID),
            (dict(pages=0), INVALID), (dict(page=0), INVALID), (dict(page=-16), INVALID),
            (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=256), UNSUPPORTED),
            (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED), (dict(M=1 << 27), UNSUPPORTED),
            (dict(pages=(1 << 26) + 1), UNSUPPORTED),
            (dict(rs=120), INVALID), (dict(rs=132), INVALID), (dict(rs=0), INVALID),
            (dict(rs=-128), INVALID), (dict(hs=128), INVALID), (dict(hs=16 * 128 - 8), INVALID),
            (dict(ps=16 * 128), INVALID), (dict(ps=0), INVALID), (dict(ps=1 << 38), INVALID),
            (dict(hs=4), INVALID)]


@pytest.fixture(scope="module")
def lib():
    return ga.load_library()


def _append(lib, kn=P, vn=P, kst=1024, vst=1024, pos=P, lens=P, table=P, B=2, S=3, **kw):
    c = dict(POOL, **kw)
    return lib.attn_paged_append(kn, vn, kst, vst, pos, lens, table, c["kp"], c["vp"], c["ps"],
                                 c["hs"], c["rs"], B, S, c["Hkv"], c["D"], c["pages"], c["page"],
                                 c["M"], None)


def test_append(lib):
    for bad in (dict(kn=None), dict(vn=None), dict(pos=None), dict(table=None), dict(kn=P + 8),
                dict(vn=P + 4), dict(pos=P + 1), dict(lens=P + 2), dict(table=P + 3), dict(B=0),
                dict(S=-1), dict(M=0), dict(kst=1016), dict(vst=1028), dict(vst=0), dict(kp=Q)):
        assert _append(lib, **bad) == INVALID, bad
    for bad, code in BAD_POOL:
        assert _append(lib, **bad) == code, bad
    assert _append(lib, S=0, kn=None, vn=None) == 0
    # a stride that nothing steps by counts for nothing, any order of the others will do
    assert _append(lib, S=0, Hkv=1, hs=0, ps=2048) == 0
    assert _append(lib, S=0, pages=1, ps=-8) == 0
    assert _append(lib, S=0, rs=1024, hs=128, ps=16384) == 0
    assert _append(lib, S=0, rs=2048 + 128, hs=256, ps=128) == INVALID


def test_decode(lib):
    need = ga.attn_paged_workspace_size(2, 2, 16, 8, 128)
    assert need > 0 and need % 256 == 0

    def call(q=P, pos=P, lens=None, table=P, B=2, S=2, Hq=16, out=P, ws=P, n=need, **kw):
        c = dict(POOL, **kw)
        return lib.attn_decode_step_paged(q, pos, lens, table, c["kp"], c["vp"], c["ps"], c["hs"],
                                          c["rs"], B, S, Hq, c["Hkv"], c["D"], c["pages"],
                                          c["page"], c["M"], 1.0, out, ws, n, None)
    for bad in (dict(q=None), dict(pos=None), dict(table=None), dict(out=None), dict(q=P + 8),
                dict(out=P + 2), dict(pos=P + 1), dict(lens=P + 2), dict(table=P + 1), dict(B=0),
                dict(S=0), dict(S=-1), dict(Hq=0), dict(Hq=12), dict(M=0)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(S=17), dict(S=1, Hq=33 * 8), dict(B=4097), dict(S=1 << 30)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad, code in BAD_POOL:
        assert call(**bad) == code, bad
    for bad in (dict(ws=None), dict(ws=P + 4), dict(n=need - 1), dict(n=0)):
        assert call(**bad) == WORKSPACE, bad


def test_workspace_sizes():
    size = ga.attn_paged_workspace_size
    for bad in ((0, 1, 8, 8, 128), (1, 0, 8, 8, 128), (1, 1, 12, 8, 128), (1, 1, 8, 8, 96),
                (1, 33, 8, 8, 128), (4097, 1, 8, 8, 128), (1, 1, 8, 0, 64)):
        assert size(*bad) == 0, bad
        with pytest.raises(ga.AttnError):
            ga.paged_workspace(*bad)
    assert size(4096, 32, 8, 8, 64) > 0
    size = ga.attn_pages_workspace_size
    for bad in ((0, 1, 1, 16), (1, 0, 1, 16), (1, 1, 0, 16), (1, 1, 1, 24), (65537, 1, 1, 16),
                (65536, 1 << 30, 1, 16)):
        assert size(*bad) == 0, bad
        with pytest.raises(ga.AttnError):
            ga.pages_workspace(*bad)
    assert size(1, 1, 100, 16) >= 256


def test_reserve(lib):
    need = ga.attn_pages_workspace_size(2, 3, 9, 16)

    def call(table=P, refs=P, pos=P, lens=None, B=2, S=3, taken=P, ws=P, n=need, **kw):
        c = dict(POOL, **kw)
        return lib.attn_pages_reserve(table, refs, pos, lens, c["kp"], c["vp"], c["ps"], c["hs"],
                                      c["rs"], B, S, c["Hkv"], c["D"], c["pages"], c["page"],
                                      c["M"], taken, ws, n, None)
    for bad in (dict(table=None), dict(refs=None), dict(pos=None), dict(taken=None),
                dict(table=P + 1), dict(refs=P + 2), dict(pos=P + 3), dict(lens=P + 1),
                dict(taken=P + 2), dict(B=0), dict(S=0), dict(M=0), dict(kp=Q)):
        assert call(**bad) == INVALID, bad
    for bad, code in BAD_POOL:
        assert call(**bad) == code, bad
    assert call(B=65537) == UNSUPPORTED
    for bad in (dict(ws=None), dict(ws=P + 4), dict(n=256)):
        assert call(**bad) == WORKSPACE, bad


def test_fork(lib):
    def call(table=P, refs=P, parents=P, lens=P, B=2, M=4, pages=9, page=16, ws=P, n=256):
        return lib.attn_pages_fork(table, refs, parents, lens, B, M, pages, page, ws, n, None)
    for bad in (dict(table=None), dict(refs=None), dict(table=P + 1), dict(refs=P + 2),
                dict(parents=P + 2), dict(lens=P + 1), dict(B=0), dict(M=0), dict(pages=0),
                dict(page=0)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(page=8), dict(B=4097), dict(B=65537, parents=None), dict(M=1 << 27),
                dict(pages=(1 << 26) + 1)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(ws=None), dict(ws=P + 8), dict(n=255)):
        assert call(**bad) == WORKSPACE, bad
    assert call(parents=None, lens=None) == 0  # nothing changes


def test_compact(lib):
    need = ga.attn_pages_workspace_size(1, 1, 9, 16)

    def call(table=P, refs=P, B=2, page_map=P, ws=P, n=need, **kw):
        c = dict(POOL, **kw)
        return lib.attn_pages_compact(table, refs, c["kp"], c["vp"], c["ps"], c["hs"], c["rs"], B,
                                      c["M"], c["Hkv"], c["D"], c["pages"], c["page"], page_map,
                                      ws, n, None)
    for bad in (dict(table=None), dict(refs=None), dict(page_map=None), dict(table=P + 1),
                dict(refs=P + 2), dict(page_map=P + 1), dict(B=-1), dict(M=-1), dict(kp=Q)):
        assert call(**bad) == INVALID, bad
    for bad, code in BAD_POOL:
        assert call(**bad) == code, bad
    for bad in (dict(ws=None), dict(ws=P + 8), dict(n=511)):
        assert call(**bad) == WORKSPACE, bad


def test_the_binding_wants_cuda_tensors():
    t = torch.zeros((2, 3), dtype=torch.int32)
    kv = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    for call in (lambda: ga.attn_decode_step_paged(q, t[0], t, kv, kv, 1.0),
                 lambda: ga.attn_pages_reserve(t, t[0], t[0], kv, kv, 1),
                 lambda: ga.attn_pages_fork(t, t[0], 16),
                 lambda: ga.attn_pages_compact(t, t[0], kv, kv),
                 lambda: ga.attn_paged_append(q, q, t[0], t, kv, kv)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        ga.attn_paged_append(None, None, None, None, kv, kv)
    with pytest.raises(TypeError):
        ga.attn_pages_fork(q, t[0], 16)


@pytest.mark.parametrize("name", ["paged.cu", "paged_decode.cuh", "paged_cluster.cuh", "pages.cu"])
def test_no_sm_count_is_written_in(name):
    with open(os.path.join(_build.CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"\b152(?:ll|u|\b)", code)


CHECK = re.compile(r"\b(?:range_ok|range_ok_count|slot_ok)\(")
PLACES = [  # file, the function's first words, range checks in its body at least
    ("paged.cu", "paged_append_kernel(\n", 1),
    ("paged_decode.cuh", "void store4(", 1),
    ("paged_decode.cuh", "void merge_parts(", 1),
    ("paged_decode.cuh", "void put_piece(", 1),              # a part's slot
    ("paged_decode.cuh", "void short_segments(", 1),         # a table entry
    ("paged_decode.cuh", "paged_decode_kernel(const", 1),    # likewise
    ("paged_cluster.cuh", "paged_cluster_kernel(const", 1),  # landing places
    ("pages.cu", "void copy_rows(", 1),
    ("pages.cu", "void give(", 1),
    ("pages.cu", "pages_reserve_solo_kernel(const", 1),
    ("pages.cu", "pages_reserve_kernel(const", 2),
    ("pages.cu", "pages_compact_solo_kernel(const", 2),
    ("pages.cu", "pages_plan_kernel(const", 2),
]


@pytest.mark.parametrize("name,words,least", PLACES)
def test_computed_addresses_are_checked(name, words, least):
    with open(os.path.join(_build.CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = text.index("{", text.index(")", text.index(words)))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            break
    assert len(CHECK.findall(text[at:i])) >= least
