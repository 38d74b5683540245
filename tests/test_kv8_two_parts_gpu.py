"""The 8-bit decode at up to 8 heads to a KV head holds probabilities in two
fp16 parts: outputs of few rows lie where the exact ones round to."""

import numpy as np
import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from oracle import kv8
from _kv8 import BF16_HALF, D, F32_HALF, codes_cache, f64, scales, u8

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5


def _bound(want, spread, load, n, vmax):
    """_kv8.out_bound with the probability's rounding to 22 bits in place of 11, and what fp16
    cannot hold of it (2^-25 of its own scale, 2^-31 of the largest) as there."""
    rel = 2.0 ** -22 + 2 * (2 * 130 * F32_HALF * load[:, None] + 2.0 ** -20) + n * F32_HALF / 8
    return BF16_HALF * np.abs(want) + (1 + BF16_HALF) * rel * spread + n * 2.0 ** -31 * vmax


@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("schedule", [0, 8])
@pytest.mark.parametrize("g", [1, 3, 8])
def test_few_rows(g, schedule, listed):
    pos, Hkv, L, block = [1, 3, 7, 15, 40], 4, 48, 16
    gen = torch.Generator(device="cuda").manual_seed(300 + g)
    kc, vc = (codes_cache(len(pos), Hkv, L, gen) for _ in "kv")
    ks, vs = (scales(len(pos), Hkv, L, block, gen) for _ in "kv")
    q = (torch.randn((len(pos), Hkv * g, D), generator=gen, device="cuda") * 0.05).bfloat16()
    at = torch.tensor(pos, dtype=torch.int32, device="cuda")
    index = torch.arange(3, dtype=torch.int32, device="cuda").repeat(len(pos), Hkv, 1).contiguous()
    ga.attn_test_force_schedule(schedule)
    try:
        if listed:
            out = ga.attn_decode_step_kv8_blocks(q, at, kc, vc, ks, vs, block, index, SCALE)
        else:
            out = ga.attn_decode_step_kv8(q, at, kc, vc, ks, vs, block, SCALE)
        torch.cuda.synchronize()
    finally:
        ga.attn_test_force_schedule(-1)
    got, qf = f64(out), f64(q)
    for b, p in enumerate(pos):
        for h in range(Hkv):
            rows = np.arange(p + 1)
            K, V = (kv8.kv8_rows(u8(c[b, h]), f64(s[b, h]), rows, block)
                    for c, s in ((kc, ks), (vc, vs)))
            sl = slice(h * g, (h + 1) * g)
            want, spread, load = kv8.attend(qf[b, sl], K, V, SCALE)
            err, bound = np.abs(got[b, sl] - want), _bound(want, spread, load, p + 1,
                                                           np.abs(V).max())
            assert (err <= bound).all(), (b, h, float((err - bound).max()))
