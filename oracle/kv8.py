"""Plain fp64 definitions of the query/key norm with rotation, the 8-bit cache
and the block-sparse decode (test infrastructure, see the package docstring).

Codes are numpy uint8 arrays of e4m3 bit patterns: sign, 4 exponent bits with
bias 7, 3 mantissa bits; exponent 0 subnormal; 0x7f and 0xff NaN; no infinity;
largest value 448.
"""

from __future__ import annotations

import math

import numpy as np


def _code_value(code: int) -> float:
    sign = -1.0 if code & 0x80 else 1.0
    e, m = (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return math.nan
    return sign * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))


E4M3 = np.array([_code_value(c) for c in range(256)])
E_MIN, E_MAX = -60, 60


def e4m3_decode(codes) -> np.ndarray:
    return E4M3[np.asarray(codes, dtype=np.uint8)]


def e4m3_encode(x) -> np.ndarray:
    """Nearest code, ties to the even mantissa, beyond 448 the largest, NaN 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    fine = np.where(np.isnan(a), 0.0, a)
    with np.errstate(divide="ignore"):
        e = np.where(fine > 0, np.floor(np.log2(np.where(fine > 0, fine, 1.0))), -6.0)
    # log2 next to a power of two may land on the wrong side
    e = np.where(np.exp2(e) > fine, e - 1, e)
    e = np.where(np.exp2(e + 1) <= fine, e + 1, e)
    step = np.exp2(np.maximum(e, -6.0) - 3)
    v = np.minimum(np.rint(fine / step) * step, 448.0)  # rint: ties to even
    code = np.searchsorted(E4M3[:127], v).astype(np.uint8)
    code = np.where(np.signbit(x), code | 0x80, code).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), code)


def block_exponent(amax: float) -> int:
    """Least e with amax <= 448 * 2^e, kept in [E_MIN, E_MAX]."""
    if amax == 0:
        return E_MIN
    m, x = math.frexp(amax)  # amax = m * 2^x, m in [0.5, 1); 448 = 0.875 * 2^9
    e = x - 9 if m <= 0.875 else x - 8
    return max(E_MIN, min(E_MAX, e))


def kv8_append(codes, scale, new, positions, block, bounds=None):
    """One operand: codes [B,H,L,D] uint8, scale [B,H,NB], new [B,S,H,D],
    bounds [B,H,NB,2,D] or None.  Returns new (codes, scale, bounds)."""
    codes, scale = codes.copy(), scale.astype(np.float64).copy()
    bounds = None if bounds is None else bounds.copy()
    B, H, L, _ = codes.shape
    S = new.shape[1]
    for b in range(B):
        p = int(positions[b])
        if p < 0 or p + S > L:
            continue
        for h in range(H):
            for j in range(p // block, (p + S - 1) // block + 1):
                lo, hi = max(p, j * block), min(p + S, (j + 1) * block)
                x = new[b, lo - p:hi - p, h].astype(np.float64)
                finite = np.abs(x[np.isfinite(x)])
                s = 2.0 ** block_exponent(float(finite.max()) if finite.size else 0.0)
                had = j * block < p
                if had:
                    old = scale[b, h, j]
                    s = max(s, old)
                    if s > old:
                        r = slice(j * block, p)
                        codes[b, h, r] = e4m3_encode(e4m3_decode(codes[b, h, r]) * (old / s))
                scale[b, h, j] = s
                codes[b, h, lo:hi] = e4m3_encode(x / s)
                if bounds is not None:
                    top = np.fmax.reduce(x, axis=0, initial=-np.inf)
                    low = np.fmin.reduce(x, axis=0, initial=np.inf)
                    if had:
                        top = np.fmax(top, bounds[b, h, j, 0])
                        low = np.fmin(low, bounds[b, h, j, 1])
                    bounds[b, h, j, 0], bounds[b, h, j, 1] = top, low
    return codes, scale, bounds


def kv8_rows(codes, scale, rows, block):
    """Values of the listed rows of one (sequence, KV head)."""
    return e4m3_decode(codes[rows]) * np.asarray(scale, dtype=np.float64)[rows // block, None]


def decode_rows_of(position, L, block, blocks=None):
    """Rows a step attends: 0..position, or those of the listed blocks up to it."""
    if blocks is None:
        return np.arange(position + 1)
    nb = -(-L // block)
    parts = [np.arange(j * block, min((j + 1) * block, position + 1))
             for j in blocks if 0 <= j < nb and j * block <= position]
    return np.concatenate(parts) if parts else np.zeros(0, dtype=np.int64)


def attend(q, K, V, scale):
    """q [g, D] over rows K, V [n, D]: (out [g, D], spread [g, D], load [g]).
    spread is sum_j p_j |v_j| and load the largest sum_d |scale q_d k_jd| of
    a row: what an error bound of the product and of a score hangs on."""
    if not len(K):
        z = np.zeros(q.shape)
        return z, z, np.zeros(len(q))
    s = scale * (q @ K.T)
    w = np.exp(s - s.max(axis=1, keepdims=True))
    w /= w.sum(axis=1, keepdims=True)
    load = (abs(scale) * (np.abs(q) @ np.abs(K).T)).max(axis=1)
    return w @ V, w @ np.abs(V), load


def block_scores(q, bounds, position, block, g):
    """One sequence: q [Hq, D], bounds [Hkv, NB, 2, D] -> (scores, magnitude) [Hkv, NB]."""
    Hkv, NB = bounds.shape[:2]
    out, mag = np.full((Hkv, NB), -np.inf), np.zeros((Hkv, NB))
    n = position // block + 1
    for h in range(Hkv):
        for i in range(g):
            x = q[h * g + i]
            t = np.maximum(x * bounds[h, :n, 0], x * bounds[h, :n, 1])
            out[h, :n] = t.sum(-1) if i == 0 else out[h, :n] + t.sum(-1)
            mag[h, :n] += np.maximum(np.abs(x * bounds[h, :n, 0]),
                                     np.abs(x * bounds[h, :n, 1])).sum(-1)
    return out, mag


def block_select(scores, position, L, block, count, first, recent):
    """Indices chosen from one row of scores, ascending, padded with -1."""
    n = position // block + 1 if 0 <= position < L else 0
    if n <= count:
        chosen = list(range(n))
    else:
        forced = set(range(first)) | set(range(n - recent, n))
        rest = [j for j in range(n) if j not in forced]
        key = lambda j: -math.inf if math.isnan(scores[j]) else float(scores[j])  # noqa: E731
        rest.sort(key=lambda j: (-key(j), j))
        chosen = sorted(forced | set(rest[:count - first - recent]))
    return np.array(chosen + [-1] * (count - len(chosen)), dtype=np.int32)


def norm_rope(x, w, eps, cos, sin):
    """x [..., D], w [D] or None, cos and sin broadcastable to x, or None."""
    y = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    if w is not None:
        y = y * w
    if cos is None:
        return y
    half = x.shape[-1] // 2
    return y * cos + np.concatenate([-y[..., half:], y[..., :half]], axis=-1) * sin
