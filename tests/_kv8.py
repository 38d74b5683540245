"""Shared pieces of the 8-bit cache's tests: caches of random codes, the
elementwise error bounds, and a comparison against oracle/kv8.py."""

import numpy as np
import torch

from oracle import kv8

D = 128
BF16_HALF = 2.0 ** -8   # half a bf16 step, relative
F16_HALF = 2.0 ** -11   # half an fp16 step, relative
F32_HALF = 2.0 ** -24


def u8(t):
    return t.detach().view(torch.uint8).cpu().numpy()


def f64(t):
    return t.detach().cpu().double().numpy()


def codes_cache(B, Hkv, L, gen, nan_tail=None):
    """Random codes (normal values x 100); rows past nan_tail[b] hold NaN codes."""
    x = torch.randn((B, Hkv, L, D), generator=gen, device="cuda") * 100
    c = x.clamp(-448, 448).to(torch.float8_e4m3fn)
    if nan_tail is not None:
        raw = c.view(torch.uint8)
        for b, p in enumerate(nan_tail):
            raw[b, :, max(0, p + 1):] = 0x7F
    return c


def scales(B, Hkv, L, block, gen, lo=-9, hi=-5):
    nb = -(-L // block)
    e = torch.randint(lo, hi, (B, Hkv, nb), generator=gen, device="cuda")
    return torch.ldexp(torch.ones((), device="cuda"), e).float().contiguous()


def out_bound(want, spread, load, n, vmax):
    """Elementwise bound on a decode output.  Rounding to bf16: half a step of
    the result.  Each probability is rounded to fp16 once (half a step), comes
    from an exponent whose error is a score's (128 products and sums in fp32:
    130 half-steps of the row's load, and as many again for the exponent's own
    rounding) and from ex2 (2^-22): all of it twice, for numerator and sum;
    the product sums n rows in fp32.  Probabilities below 2^-20 of the largest
    are fp16 subnormals: 2^-31 absolute each."""
    rel = F16_HALF + 2 * (2 * 130 * F32_HALF * load[:, None] + 2.0 ** -20) + n * F32_HALF / 8
    sum_part = BF16_HALF * np.abs(want) + (1 + BF16_HALF) * rel * spread
    return sum_part + n * 2.0 ** -31 * vmax + 1e-30


def check_decode(out, q, positions, kc, vc, ks, vs, L, block, scale, index=None, seqs=None,
                 what=""):
    """Every head of the listed sequences against the oracle."""
    B, Hq, _ = q.shape
    Hkv = kc.shape[1]
    g = Hq // Hkv
    got, qf = f64(out), f64(q)
    ksf, vsf = f64(ks), f64(vs)
    for b in seqs if seqs is not None else range(B):
        kb, vb = u8(kc[b]), u8(vc[b])
        for h in range(Hkv):
            rows = kv8.decode_rows_of(positions[b], L, block,
                                      None if index is None else index[b][h])
            K = kv8.kv8_rows(kb[h], ksf[b, h], rows, block)
            V = kv8.kv8_rows(vb[h], vsf[b, h], rows, block)
            sl = slice(h * g, (h + 1) * g)
            want, spread, load = kv8.attend(qf[b, sl], K, V, scale)
            err = np.abs(got[b, sl] - want)
            bound = out_bound(want, spread, load, len(rows), np.abs(V).max() if len(V) else 0.0)
            worst = np.unravel_index(np.argmax(err - bound), err.shape)
            assert (err <= bound).all(), (
                f"{what} b={b} kvh={h} n={len(rows)}: off {err[worst]:.3e}, bound "
                f"{bound[worst]:.3e}, want {want[worst]:.3e}")
