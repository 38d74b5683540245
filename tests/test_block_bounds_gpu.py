"""What a block's score is a bound of: the keys as they were appended, and their
codes but for the codes' rounding."""

import numpy as np
import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from oracle import kv8
from _kv8 import D, F32_HALF, f64, u8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("g", [1, 4])
@pytest.mark.parametrize("block", [16, 128])
def test_no_appended_key_scores_above_its_block(g, block):
    B, Hkv, S, L = 2, 3, 500, 512
    gen = torch.Generator(device="cuda").manual_seed(400 + g)
    k, v = (torch.randn((B, S, Hkv, D), generator=gen, device="cuda").bfloat16() for _ in "kv")
    q = torch.randn((B, Hkv * g, D), generator=gen, device="cuda").bfloat16()
    # one query along its block's largest values, where the bound is met
    q[0, 0] = torch.sign(k[0, 3, 0])
    nb = -(-L // block)
    kc, vc = (torch.zeros((B, Hkv, L, D), dtype=torch.uint8, device="cuda")
              .view(torch.float8_e4m3fn) for _ in "kv")
    ks, vs = (torch.ones((B, Hkv, nb), device="cuda") for _ in "kv")
    bounds = torch.zeros((B, Hkv, nb, 2, D), dtype=torch.bfloat16, device="cuda")
    ga.attn_kv8_append(k, v, torch.zeros(B, dtype=torch.int32, device="cuda"), kc, vc, ks, vs,
                       block, k_bounds=bounds)
    at = torch.full((B,), S - 1, dtype=torch.int32, device="cuda")
    scores = f64(ga.attn_block_scores(q, at, bounds, L, block))
    kf, qf, ksf = f64(k), f64(q), f64(ks)
    rows = np.arange(S)
    for b in range(B):
        _, mag = kv8.block_scores(qf[b], f64(bounds[b]), S - 1, block, g)
        for h in range(Hkv):
            qh = qf[b, h * g:(h + 1) * g].sum(0), np.abs(qf[b, h * g:(h + 1) * g]).sum(0)
            top = scores[b, h][rows // block]
            slack = (256 + g) * F32_HALF * mag[h][rows // block]
            keys = kf[b, :, h]
            assert (keys @ qh[0] <= top + slack).all()
            codes = kv8.kv8_rows(u8(kc[b, h]), ksf[b, h], rows, block)
            # half a step: 2^-4 of the value, and 2^-10 of the scale below the normal codes
            off = np.abs(keys) * 2.0 ** -4 + 2.0 ** -10 * ksf[b, h][rows // block, None]
            assert (codes @ qh[0] <= top + slack + off @ qh[1]).all()
