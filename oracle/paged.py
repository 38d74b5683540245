"""fp64 oracle of the paged cache (include/gqa_attn.h): append, decode step, and
the calls that give out, pass on, free and move pages.  Plain Python loops over
numpy arrays; test infrastructure only."""

import numpy as np


def rows_fit(pos, n, cap):
    return n >= 1 and pos >= 0 and pos + n <= cap


def append(k_pages, v_pages, k_new, v_new, positions, lengths, table):
    """In place: k_new, v_new [B, S, Hkv, D] into pages [P, Hkv, page, D]."""
    P, _, page, _ = k_pages.shape
    B, M = table.shape
    S = k_new.shape[1]
    for b in range(B):
        n = S if lengths is None else int(lengths[b])
        if n > S or not rows_fit(int(positions[b]), n, M * page):
            continue
        for t in range(n):
            row = int(positions[b]) + t
            pg = int(table[b, row // page])
            if 0 <= pg < P:
                k_pages[pg, :, row % page] = k_new[b, t]
                v_pages[pg, :, row % page] = v_new[b, t]


def decode(q, k_pages, v_pages, positions, lengths, table, scale):
    """out [B, S, Hq, D]; also, for error bounds, per output row the sum of
    w |v| (spread), the load sum_d |q_d k_d| scale of its worst row, and the
    number of rows."""
    P, Hkv, page, D = k_pages.shape
    B, S, Hq, _ = q.shape
    g = Hq // Hkv
    M = table.shape[1]
    out = np.zeros(q.shape)
    spread, load, count = np.zeros(q.shape), np.zeros((B, S, Hq)), np.zeros((B, S), dtype=int)
    for b in range(B):
        n = S if lengths is None else int(lengths[b])
        if n == 0:
            continue
        if n > S or not rows_fit(int(positions[b]), n, M * page):
            out[b] = np.nan
            continue
        for t in range(n):
            rows = np.arange(int(positions[b]) + t + 1)
            pg = table[b, rows // page].astype(int)
            ok = (pg >= 0) & (pg < P)
            rows, pg = rows[ok], pg[ok]
            count[b, t] = len(rows)
            if not len(rows):
                continue
            for h in range(Hkv):
                K, V = k_pages[pg, h, rows % page], v_pages[pg, h, rows % page]
                sl = slice(h * g, (h + 1) * g)
                x = scale * (q[b, t, sl] @ K.T)
                w = np.exp(x - x.max(axis=1, keepdims=True))
                w /= w.sum(axis=1, keepdims=True)
                out[b, t, sl] = w @ V
                spread[b, t, sl] = w @ np.abs(V)
                load[b, t, sl] = abs(scale) * (np.abs(q[b, t, sl]) @ np.abs(K).T).max(axis=1)
    return out, spread, load, count


def reserve(table, refs, positions, lengths, S, page):
    """In place on table and refs; returns (taken, copies), copies of
    (from, to, rows) in any order."""
    B, M = table.shape
    P = len(refs)
    was = refs.copy()
    free = [p for p in range(P) if was[p] <= 0]
    at, taken, copies = 0, np.zeros(B, dtype=np.int64), []
    for b in range(B):
        n = S if lengths is None else int(lengths[b])
        pos = int(positions[b])
        if n == 0:
            continue
        if n < 0 or n > S or not rows_fit(pos, n, M * page):
            taken[b] = -1
            continue
        need = []
        for j in range(pos // page, (pos + n - 1) // page + 1):
            e = int(table[b, j])
            if not 0 <= e < P:
                need.append((j, -1))
            elif was[e] > 1:
                need.append((j, e))
        first, at = at, at + len(need)
        if need and at > len(free):
            taken[b] = -1
            continue
        taken[b] = len(need)
        for k, (j, e) in enumerate(need):
            new = free[first + k]
            table[b, j] = new
            refs[new] = 1
            if e >= 0:
                refs[e] -= 1
                if j == pos // page and pos % page:
                    copies.append((e, new, pos % page))
    return taken, copies


def fork(table, refs, parents, lengths, page):
    """In place on table and refs."""
    B, M = table.shape
    old = table.copy()
    for b in range(B):
        src = b if parents is None else int(parents[b])
        if src < -1 or src >= B:
            src = b
        for j in range(M):
            new = -1 if src < 0 else old[src, j]
            if lengths is not None and j * page >= lengths[b]:
                new = -1
            if new == old[b, j]:
                continue
            table[b, j] = new
            if 0 <= new < len(refs):
                refs[new] += 1
            if 0 <= old[b, j] < len(refs):
                refs[old[b, j]] -= 1


def compact(table, refs):
    """In place on table and refs; returns (page_map, moves), moves of (from, to)."""
    P = len(refs)
    n = int((refs > 0).sum())
    high = [p for p in range(n, P) if refs[p] > 0]
    low = [p for p in range(n) if refs[p] <= 0]
    page_map = np.where(refs > 0, np.arange(P), -1)
    for src, dst in zip(high, low):
        page_map[src] = dst
        refs[dst], refs[src] = refs[src], 0
    for i, e in np.ndenumerate(table):
        if 0 <= e < P:
            table[i] = page_map[e]
    return page_map, list(zip(high, low))
