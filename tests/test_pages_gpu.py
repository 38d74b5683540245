"""attn_pages_reserve, attn_pages_fork and attn_pages_compact against the oracle:
tables, counts and rows exactly."""

import random

import numpy as np
import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from _paged import f64, i32, i64, pools
from oracle import paged

pytestmark = pytest.mark.gpu


def state(B, M, P, page, seed, shared=0.5, fullness=0.6):
    """A consistent random state: (table, refs, rows held by each sequence)."""
    r = random.Random(seed)
    free = list(range(P))
    r.shuffle(free)
    table = np.full((B, M), -1, dtype=np.int64)
    rows = []
    for b in range(B):
        n = r.randint(0, int(M * fullness))
        src = r.randrange(b) if b and r.random() < shared else None
        keep = 0 if src is None else min(n, -(-rows[src] // page))
        for j in range(n):
            if j < keep:
                table[b, j] = table[src, j]
            elif free:
                table[b, j] = free.pop()
            else:
                n = j
                break
        rows.append(max(0, n * page - r.randint(0, page - 1)) if n else 0)
    refs = np.bincount(table[table >= 0], minlength=P)
    return table, refs, rows


def same_counts(table, refs):
    assert (np.bincount(table[(table >= 0) & (table < len(refs))], minlength=len(refs))
            == refs).all()


@pytest.mark.parametrize("B,S,M,P,page,Hkv,D,layout", [
    (1, 1, 1, 1, 16, 1, 64, "heads"), (9, 1, 6, 40, 16, 2, 128, "rows"),
    (40, 3, 9, 300, 32, 1, 64, "pair"), (6, 100, 20, 110, 16, 2, 64, "heads"),
    (300, 1, 5, 900, 16, 1, 64, "woven"), (3, 700, 60, 5000, 16, 1, 64, "heads"),
    (70, 5, 4, 120, 128, 1, 64, "heads"), (1100, 1, 3, 2500, 16, 1, 64, "heads"),
    (300, 700, 60, 13000, 16, 1, 64, "heads"), (2, 1, 3, 20000, 16, 1, 64, "pair")])
def test_reserve(B, S, M, P, page, Hkv, D, layout):
    for seed in range(3):
        r = random.Random(seed + 100)
        table, refs, rows = state(B, M, P, page, seed)
        lengths = [r.choice([0, 1, S, r.randint(0, S)]) for _ in range(B)] if seed else None
        positions = list(rows)
        if seed == 2 and B > 5:  # a few that do not fit, and a rolled-back one
            positions[1], positions[3] = -1, M * page
            lengths[4] = S + 1
            positions[5] = max(0, rows[5] - page - 3)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        k, v = pools(P, Hkv, page, D, gen, layout, poison=False)
        want_k, want_v = f64(k), f64(v)
        t, c = i32(table.tolist()), i32(refs.tolist())
        ws = ga.pages_workspace(B, S, P, page)
        taken = ga.attn_pages_reserve(t, c, i32(positions), k, v, S, lengths=i32(lengths),
                                      workspace=ws)
        want_taken, copies = paged.reserve(table, refs, positions, lengths, S, page)
        for src, dst, n in copies:
            want_k[dst, :, :n], want_v[dst, :, :n] = want_k[src, :, :n], want_v[src, :, :n]
        assert (i64(taken) == want_taken).all()
        assert (i64(t) == table).all() and (i64(c) == refs).all()
        assert (f64(k) == want_k).all() and (f64(v) == want_v).all()
        same_counts(table, refs)
        bad = any(n and not (0 < n <= S and paged.rows_fit(p, n, M * page))
                  for p, n in zip(positions, lengths or [S] * B))
        assert ga.attn_read_device_status(ws) == (ga.ATTN_DEV_BAD_POSITION if bad else 0)


def test_reserve_beams_leave_their_page():
    """All sequences that share a page get copies of it, and it is free again."""
    table, refs = np.array([[3, 1], [3, 1], [3, 1]]), np.array([0, 3, 0, 3, 0, 0])
    gen = torch.Generator(device="cuda").manual_seed(1)
    k, v = pools(6, 2, 16, 64, gen, poison=False)
    before = f64(k)
    t, c = i32(table.tolist()), i32(refs.tolist())
    taken = ga.attn_pages_reserve(t, c, i32([21, 21, 21]), k, v, 1)
    assert i64(taken).tolist() == [1, 1, 1]
    assert i64(t).tolist() == [[3, 0], [3, 2], [3, 4]] and i64(c).tolist() == [1, 0, 1, 3, 1, 0]
    for p in (0, 2, 4):
        assert (f64(k)[p, :, :5] == before[1, :, :5]).all()
        assert (f64(k)[p, :, 5:] == before[p, :, 5:]).all()


@pytest.mark.parametrize("B,M,P,page", [(1, 1, 1, 16), (5, 33, 100, 32), (64, 70, 3000, 16),
                                        (1024, 5, 900, 128), (1025, 11, 4000, 16),
                                        (4096, 9, 9000, 64)])
def test_fork(B, M, P, page):
    for seed in range(4):
        r = random.Random(seed)
        table, refs, rows = state(B, M, P, page, seed)
        parents = [r.choice([b, r.randrange(B), -1]) for b in range(B)]
        lengths = [r.choice([0, 10 ** 9, r.randint(-3, M * page)]) for _ in range(B)]
        status = 0
        if seed == 0:
            parents = None
        if seed == 1:
            lengths = None
        if seed == 3:
            parents[0], parents[-1] = B, -2
            table[0, 0], status = P + 7, ga.ATTN_DEV_BAD_PARENT
            refs = np.bincount(table[(table >= 0) & (table < P)], minlength=P)
        t, c = i32(table.tolist()), i32(refs.tolist())
        ws = ga.pages_workspace(B, 1, P, page)
        ga.attn_pages_fork(t, c, page, parents=i32(parents), lengths=i32(lengths), workspace=ws)
        paged.fork(table, refs, parents, lengths, page)
        assert (i64(t) == table).all() and (i64(c) == refs).all()
        same_counts(table, refs)
        assert ga.attn_read_device_status(ws) == status


@pytest.mark.parametrize("P,share", [(1, 0.0), (1, 1.0), (33, 0.5), (257, 0.9), (300, 0.0),
                                     (300, 1.0), (5000, 0.3), (70001, 0.6)])
def test_compact(P, share):
    gen = torch.Generator(device="cuda").manual_seed(P)
    r = np.random.default_rng(P)
    D, page, Hkv, layout = (64, 16, 1, "pair") if P > 300 else (128, 32, 3, "rows")
    used = np.flatnonzero(r.random(P) < share)
    table = np.full(max(4, 2 * len(used)), -1, dtype=np.int64)
    table[r.permutation(len(table))[:len(used)]] = used
    if len(used):
        extra = r.permutation(np.flatnonzero(table < 0))[:5]
        table[extra] = r.choice(used, len(extra))
    table[np.flatnonzero(table < 0)[:1]] = P + 3  # an entry that names no page stays
    refs = np.bincount(table[(table >= 0) & (table < P)], minlength=P)
    table = table.reshape(2, -1)
    k, v = pools(P, Hkv, page, D, gen, layout, poison=False)
    want_k, want_v = k.clone(), v.clone()
    t, c = i32(table.tolist()), i32(refs.tolist())
    page_map = ga.attn_pages_compact(t, c, k, v)
    want_map, moves = paged.compact(table, refs)
    if moves:
        src, dst = (torch.tensor(x, device="cuda") for x in zip(*moves))
        want_k[dst], want_v[dst] = want_k[src], want_v[src]
    assert (i64(page_map) == want_map).all()
    assert (i64(t) == table).all() and (i64(c) == refs).all()
    assert torch.equal(k, want_k) and torch.equal(v, want_v)
    n = int((refs > 0).sum())
    assert (refs[:n] > 0).all() and (refs[n:] == 0).all()
