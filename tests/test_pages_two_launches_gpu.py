"""attn_pages_reserve and attn_pages_compact above the sizes that take one launch,
with pages of several 16-row units, several heads and both head dims: tables,
counts and rows exactly, every other byte untouched."""

import random

import numpy as np
import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from _paged import i32, i64, pools
from oracle import paged
from test_pages_gpu import same_counts, state

pytestmark = pytest.mark.gpu


def bits(x):
    return x.contiguous().view(torch.int16)


@pytest.mark.parametrize("B,S,M,P,page,Hkv,D,layout", [
    (600, 1, 4, 17000, 128, 1, 64, "pair"), (1100, 3, 4, 2600, 64, 2, 128, "rows"),
    (700, 40, 6, 4000, 32, 3, 64, "heads"), (300, 200, 12, 2500, 64, 2, 128, "woven"),
    (1500, 1, 5, 3000, 128, 2, 128, "heads")])
def test_reserve(B, S, M, P, page, Hkv, D, layout):
    for seed in range(2):
        r = random.Random(seed + 50)
        table, refs, rows = state(B, M, P, page, seed)
        lengths = [r.choice([1, S, r.randint(0, S)]) for _ in range(B)] if seed else None
        gen = torch.Generator(device="cuda").manual_seed(seed)
        k, v = pools(P, Hkv, page, D, gen, layout, poison=False)
        want_k, want_v = k.clone(), v.clone()
        t, c = i32(table.tolist()), i32(refs.tolist())
        taken = ga.attn_pages_reserve(t, c, i32(rows), k, v, S, lengths=i32(lengths))
        want_taken, copies = paged.reserve(table, refs, rows, lengths, S, page)
        # whole 16-row units, units cut short and pages that end inside one are among them
        assert len(copies) > 20 and any(n % 16 for *_, n in copies) and max(
            n for *_, n in copies) > page - 16
        for src, dst, n in copies:
            want_k[dst, :, :n], want_v[dst, :, :n] = want_k[src, :, :n], want_v[src, :, :n]
        assert (i64(taken) == want_taken).all()
        assert (i64(t) == table).all() and (i64(c) == refs).all()
        assert torch.equal(bits(k), bits(want_k)) and torch.equal(bits(v), bits(want_v))
        same_counts(table, refs)


@pytest.mark.parametrize("P,page,Hkv,D,layout", [
    (3000, 128, 3, 128, "rows"), (9000, 32, 2, 64, "pair"), (1000, 64, 16, 128, "woven"),
    (12000, 16, 3, 128, "heads"), (8300, 128, 1, 64, "heads")])
@pytest.mark.parametrize("share", [0.02, 0.6, 0.97])
def test_compact(P, page, Hkv, D, layout, share):
    assert P > 8192 or P * Hkv * page > 786432
    gen = torch.Generator(device="cuda").manual_seed(P)
    r = np.random.default_rng(P)
    used = np.flatnonzero(r.random(P) < share)
    table = np.full(2 * len(used) + 6, -1, dtype=np.int64)
    table[r.permutation(len(table))[:len(used)]] = used
    extra = r.permutation(np.flatnonzero(table < 0))[:5]
    table[extra] = r.choice(used, len(extra))
    refs = np.bincount(table[table >= 0], minlength=P)
    table = table.reshape(2, -1)
    k, v = pools(P, Hkv, page, D, gen, layout, poison=False)
    want_k, want_v = k.clone(), v.clone()
    t, c = i32(table.tolist()), i32(refs.tolist())
    page_map = ga.attn_pages_compact(t, c, k, v)
    want_map, moves = paged.compact(table, refs)
    assert moves
    src, dst = (torch.tensor(x, device="cuda") for x in zip(*moves))
    want_k[dst], want_v[dst] = want_k[src], want_v[src]
    assert (i64(page_map) == want_map).all()
    assert (i64(t) == table).all() and (i64(c) == refs).all()
    assert torch.equal(bits(k), bits(want_k)) and torch.equal(bits(v), bits(want_v))


def test_both_operands_behind_32_bits():
    """Pages of two units whose elements lie behind 2^31 of the base: copied and moved."""
    P, Hkv, page, D = 140000, 8, 32, 64  # 2.3e9 elements, 4.6 GB an operand
    gen = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.empty((P, Hkv, page, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    for x in (k, v):
        x[-8:] = torch.randn((8, Hkv, page, D), generator=gen, device="cuda").bfloat16()
    refs = torch.ones(P, dtype=torch.int32, device="cuda")
    refs[P - 1], refs[P - 3] = 0, 2
    table = i32([[P - 3], [P - 3]])
    before = k[P - 1].clone(), v[P - 1].clone()
    taken = ga.attn_pages_reserve(table, refs, i32([21, 32]), k, v, 1, lengths=i32([1, 0]))
    assert taken.tolist() == [1, 0] and table.tolist() == [[P - 1], [P - 3]]
    for x, old in zip((k, v), before):
        assert torch.equal(bits(x[P - 1, :, :21]), bits(x[P - 3, :, :21]))
        assert torch.equal(bits(x[P - 1, :, 21:]), bits(old[:, 21:]))
    refs.zero_()
    refs[P - 1] = refs[P - 3] = 1
    want = [x[[P - 3, P - 1]].clone() for x in (k, v)]
    page_map = ga.attn_pages_compact(table, refs, k, v)
    assert table.tolist() == [[1], [0]] and page_map[P - 1] == 1 and page_map[P - 3] == 0
    for x, y in zip((k, v), want):
        assert torch.equal(bits(x[:2]), bits(y))
