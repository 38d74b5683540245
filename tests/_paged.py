"""Shared pieces of the paged cache's tests: pools in every layout, tables of
pages in random order, the elementwise error bounds, and a comparison against
oracle/paged.py."""

import numpy as np
import torch

from oracle import paged

BF16_HALF = 2.0 ** -8   # half a bf16 step, relative
F32_HALF = 2.0 ** -24


def f64(t):
    return t.detach().cpu().double().numpy()


def i64(t):
    return None if t is None else t.detach().cpu().numpy().astype(np.int64)


def i32(x, device="cuda"):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device=device)


def pools(P, Hkv, page, D, gen, layout="heads", poison=True):
    """k_pages, v_pages [P, Hkv, page, D]: NaN throughout (poison) or random."""
    shape = {"heads": (2, P, Hkv, page, D), "rows": (2, P, page, Hkv, D),
             "pair": (P, 2, Hkv, page, D), "woven": (P, Hkv, page, 2, D)}[layout]
    if poison:
        both = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    else:
        both = torch.randn(shape, generator=gen, device="cuda").bfloat16()
    if layout == "pair":
        return both[:, 0], both[:, 1]
    if layout == "woven":
        return both[..., 0, :], both[..., 1, :]
    if layout == "rows":
        return both[0].transpose(1, 2), both[1].transpose(1, 2)
    return both[0], both[1]


def random_table(rows, page, M, gen, spare=2):
    """Pages in random order for `rows[b]` rows of each sequence; (table, P)."""
    n = [-(-r // page) for r in rows]
    P = sum(n) + spare
    order = torch.randperm(P, generator=gen, device="cuda").tolist()
    table, at = [], 0
    for k in n:
        table.append(order[at:at + k] + [-1] * (M - k))
        at += k
    return i32(table), P


def fill(k_pages, v_pages, table, rows, gen, gain=1.0):
    """Random rows 0 .. rows[b] - 1 of every sequence; the rest stays as it is."""
    P, Hkv, page, D = k_pages.shape
    for b, r in enumerate(rows):
        if r == 0:
            continue
        j = torch.arange(r, device="cuda")
        pg = table[b].long()[j // page]
        for x in (k_pages, v_pages):
            x[pg, :, j % page] = (torch.randn((r, Hkv, D), generator=gen, device="cuda")
                                  * gain).bfloat16()


def out_bound(want, spread, load, n, parts):
    """Elementwise bound on a decode output.  Rounding to bf16: half a step of
    the result.  A probability comes from a score whose D <= 128 products and
    sums in fp32 are off by 130 half-steps of the row's load (and as many again
    for the exponent's own roundings) and from ex2 (2^-22), for numerator and
    sum; it is rounded to bf16 once, or in two parts to 2^-16; the product sums n
    rows in fp32."""
    rounding = BF16_HALF if parts == 1 else 2.0 ** -16
    rel = rounding + 2 * (2 * 130 * F32_HALF * load[..., None] + 2.0 ** -20) + \
        n[..., None, None] * F32_HALF / 8
    return BF16_HALF * np.abs(want) + (1 + BF16_HALF) * rel * spread + 1e-30


def check_decode(out, q, k_pages, v_pages, positions, lengths, table, scale, what=""):
    """Every output row against the oracle."""
    q4, o4 = (x if x.dim() == 4 else x[:, None] for x in (q, out))
    S, g = q4.shape[1], q4.shape[2] // k_pages.shape[1]
    k, v = f64(k_pages), f64(v_pages)
    want, spread, load, n = paged.decode(f64(q4), k, v, positions, lengths, i64(table), scale)
    got = f64(o4)
    assert (np.isnan(got) == np.isnan(want)).all(), f"{what}: NaN where there is none, or missing"
    err = np.abs(got - want)
    bound = out_bound(want, spread, load, n, 1 if S * g > 16 and q.shape[-1] == 64 else 2)
    bad = ~(err <= bound) & ~np.isnan(want)
    worst = np.unravel_index(np.argmax(np.where(bad, err - bound, -1)), err.shape)
    assert not bad.any(), (f"{what} at {worst}: off {err[worst]:.3e}, bound {bound[worst]:.3e}, "
                           f"want {want[worst]:.3e}, {bad.sum()} of {bad.size}")
