"""Appends into blocks whose rows came with a scale that is no power of two: it
stays, the new codes are of x times its fp32 reciprocal, or the block moves to
the new rows' power of two; and the decode reads both."""

import numpy as np
import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from oracle import kv8
from _kv8 import D, check_decode, codes_cache, f64, scales, u8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S", [1, 9])
@pytest.mark.parametrize("gain", [0.01, 1e4])
def test_append(S, gain):
    B, Hkv, L, block, pos = 2, 3, 64, 32, [40, 5]
    gen = torch.Generator(device="cuda").manual_seed(500 + S)
    kc, vc = (codes_cache(B, Hkv, L, gen) for _ in "kv")
    ks, vs = (scales(B, Hkv, L, block, gen) * 0.7 for _ in "kv")
    new = [(torch.randn((B, S, Hkv, D), generator=gen, device="cuda") * gain).bfloat16()
           for _ in "kv"]
    before = [(u8(c), s.cpu().numpy()) for c, s in ((kc, ks), (vc, vs))]
    at = torch.tensor(pos, dtype=torch.int32, device="cuda")
    ga.attn_kv8_append(new[0], new[1], at, kc, vc, ks, vs, block)
    torch.cuda.synchronize()
    one = np.float32(1.0)
    for (codes, scale), x, c, s in zip(before, new, (kc, vc), (ks, vs)):
        x, got, got_s = f64(x).astype(np.float32), u8(c), s.cpu().numpy()
        for b, p in enumerate(pos):
            j, rows = p // block, slice(p // block * block, p)
            for h in range(Hkv):
                s_new = np.float32(2.0 ** kv8.block_exponent(float(np.abs(x[b, :, h]).max())))
                want_s = max(scale[b, h, j], s_new)
                assert got_s[b, h, j] == want_s
                inv = one / want_s
                assert np.array_equal(got[b, h, p:p + S], kv8.e4m3_encode(x[b, :, h] * inv))
                old = codes[b, h, rows]
                if want_s > scale[b, h, j]:
                    ratio = np.float32(scale[b, h, j] * inv)
                    old = kv8.e4m3_encode(kv8.e4m3_decode(old).astype(np.float32) * ratio)
                assert np.array_equal(got[b, h, rows], old)
    q = torch.randn((B, Hkv * 2, D), generator=gen, device="cuda").bfloat16()
    last = [p + S - 1 for p in pos]
    out = ga.attn_decode_step_kv8(q, torch.tensor(last, dtype=torch.int32, device="cuda"), kc, vc,
                                  ks, vs, block, 1e-3 * D ** -0.5)
    check_decode(out, q, last, kc, vc, ks, vs, L, block, 1e-3 * D ** -0.5)
