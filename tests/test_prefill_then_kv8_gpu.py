"""A prompt through the causal prefill, the bf16 cache and the 8-bit cache: the
last token's row of the prefill, the bf16 decode of its query and the 8-bit
decode, each against fp64."""

import numpy as np
import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from oracle import kv8
from _kv8 import BF16_HALF, D, F32_HALF, check_decode, f64, u8

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5


@pytest.mark.parametrize("S", [1, 129, 500])
@pytest.mark.parametrize("Hq,Hkv,block", [(8, 2, 64), (16, 16, 16)])
def test_last_token(S, Hq, Hkv, block):
    L, g = 512, Hq // Hkv
    gen = torch.Generator(device="cuda").manual_seed(600 + S)
    q, k, v = (torch.randn((S, h, D), generator=gen, device="cuda").bfloat16()
               for h in (Hq, Hkv, Hkv))
    nb = -(-L // block)
    k16, v16 = (torch.zeros((1, Hkv, L, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    k16[0, :, :S], v16[0, :, :S] = k.transpose(0, 1), v.transpose(0, 1)
    k8, v8 = (torch.zeros((1, Hkv, L, D), dtype=torch.uint8, device="cuda")
              .view(torch.float8_e4m3fn) for _ in "kv")
    ks, vs = (torch.ones((1, Hkv, nb), device="cuda") for _ in "kv")
    ga.attn_kv8_append(k[None], v[None], torch.zeros(1, dtype=torch.int32, device="cuda"), k8, v8,
                       ks, vs, block)
    at = torch.full((1,), S - 1, dtype=torch.int32, device="cuda")
    last = q[None, S - 1].contiguous()
    rows = {"prefill": ga.attn_prefill_causal(q, k, v, 0, SCALE)[S - 1],
            "bf16 decode": ga.attn_decode_step(last, at, k16, v16, SCALE)[0]}
    out8 = ga.attn_decode_step_kv8(last, at, k8, v8, ks, vs, block, SCALE)
    torch.cuda.synchronize()
    for h in range(Hkv):
        sl = slice(h * g, (h + 1) * g)
        want, spread, load = kv8.attend(f64(q[S - 1, sl]), f64(k[:, h]), f64(v[:, h]), SCALE)
        # a probability rounded to bf16, in the product and perhaps in the sum, the scores' sums
        # in fp32 as in _kv8.out_bound, and the output's rounding
        rel = 2 * (BF16_HALF + 2 * 130 * F32_HALF * load[:, None] + 2.0 ** -20) + S * F32_HALF
        bound = BF16_HALF * np.abs(want) + (1 + BF16_HALF) * rel * spread
        for what, got in rows.items():
            assert (np.abs(f64(got[sl]) - want) <= bound).all(), (what, h)
    # the 8-bit cache holds each value to half an e4m3 step, and its decode attends those
    for c, s, x in ((k8, ks, k), (v8, vs, v)):
        for h in range(Hkv):
            held = kv8.kv8_rows(u8(c[0, h]), f64(s[0, h]), np.arange(S), block)
            unit = f64(s[0, h])[np.arange(S) // block, None]
            exact = f64(x[:, h])
            assert (np.abs(held - exact) <= np.maximum(np.abs(exact) * 2.0 ** -4,
                                                       unit * 2.0 ** -10)).all()
    check_decode(out8, last, [S - 1], k8, v8, ks, vs, L, block, SCALE)
