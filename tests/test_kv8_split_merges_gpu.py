"""The flat-list 8-bit decode where a CTA has the split part of one segment and
then its last piece: every run gives the oracle's result, and the same bits."""

import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from _kv8 import D, check_decode, codes_cache, scales

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5


@pytest.mark.parametrize("g", [2, 16])
@pytest.mark.parametrize("B,Hkv,tiles", [(50, 2, 20), (70, 2, 9), (10, 3, 60), (76, 2, 13)])
def test_a_split_piece_before_the_last(B, Hkv, tiles, g):
    L, block = tiles * 128, 64
    gen = torch.Generator(device="cuda").manual_seed(100 + B)
    pos = [L - 1 - (b % 3) * 50 for b in range(B)]
    kc, vc = (codes_cache(B, Hkv, L, gen) for _ in "kv")
    ks, vs = (scales(B, Hkv, L, block, gen) for _ in "kv")
    q = torch.randn((B, Hkv * g, D), generator=gen, device="cuda").bfloat16()
    at = torch.tensor(pos, dtype=torch.int32, device="cuda")
    ws = ga.kv8_workspace(B, Hkv * g, Hkv, L, D)
    ga.attn_test_force_schedule(0)
    try:
        first = ga.attn_decode_step_kv8(q, at, kc, vc, ks, vs, block, SCALE, workspace=ws)
        wrong = torch.zeros((), dtype=torch.int64, device="cuda")
        for _ in range(300):
            again = ga.attn_decode_step_kv8(q, at, kc, vc, ks, vs, block, SCALE, workspace=ws)
            wrong += (again.view(torch.int16) != first.view(torch.int16)).sum()
        torch.cuda.synchronize()
    finally:
        ga.attn_test_force_schedule(-1)
    assert int(wrong) == 0 and ga.attn_read_device_status(ws) == 0
    check_decode(first, q, pos, kc, vc, ks, vs, L, block, SCALE, seqs=range(0, B, 9))
