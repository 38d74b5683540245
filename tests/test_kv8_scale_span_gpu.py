"""The 8-bit decode where value scales lie as far apart as they may: rows that
weigh in the softmax's sum and, their values being tiny, not in its product."""

import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from _kv8 import D, check_decode

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5
BLOCK = 16
KS = 2.0 ** -6
# a key of this code in every dim, with a query of ones: this many bits of score
CODE_OF_BITS = {7: 28.0, 13: 52.0}  # 128 * 28 * 2^-6 / sqrt(128) * log2(e) = 7.1; 52: 13.3


def _run(L, g, big, small, big_blocks, bits, sign, schedule, listed):
    """Blocks `big_blocks` at scale 2^big with their first row at score 0, every other row `bits`
    lower (sign -1) or higher (sign 1), every other block at scale 2^small."""
    gen = torch.Generator(device="cuda").manual_seed(200 + g)
    nb = -(-L // BLOCK)
    k = torch.full((1, 1, L, D), sign * CODE_OF_BITS[bits], device="cuda")
    v = torch.randn((1, 1, L, D), generator=gen, device="cuda").abs() * 100
    ks = torch.full((1, 1, nb), KS, device="cuda")
    vs = torch.full((1, 1, nb), 2.0 ** small, device="cuda")
    for j in big_blocks:
        k[0, 0, j * BLOCK] = 0.0
        vs[0, 0, j] = 2.0 ** big
    kc, vc = (x.clamp(-448, 448).to(torch.float8_e4m3fn) for x in (k, v))
    q = torch.ones((1, g, D), device="cuda").bfloat16()
    at = torch.tensor([L - 1], dtype=torch.int32, device="cuda")
    index = torch.arange(nb, dtype=torch.int32, device="cuda")[None, None].contiguous()
    ga.attn_test_force_schedule(schedule)
    try:
        if listed:
            out = ga.attn_decode_step_kv8_blocks(q, at, kc, vc, ks, vs, BLOCK, index, SCALE)
        else:
            out = ga.attn_decode_step_kv8(q, at, kc, vc, ks, vs, BLOCK, SCALE)
        torch.cuda.synchronize()
    finally:
        ga.attn_test_force_schedule(-1)
    check_decode(out, q, [L - 1], kc, vc, ks, vs, L, BLOCK, SCALE,
                 index=index.tolist() if listed else None)


@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("schedule", [0, 1, 8])
@pytest.mark.parametrize("g", [2, 16])
@pytest.mark.parametrize("big_blocks", [[0], [1255], [600, 700]])
@pytest.mark.parametrize("bits,sign", [(7, -1), (13, -1), (7, 1)])
def test_the_ends_of_the_range(big_blocks, bits, sign, g, schedule, listed):
    _run(20096, g, 60, -60, big_blocks, bits, sign, schedule, listed)


@pytest.mark.parametrize("big,small", [(55, -55), (60, -8), (-8, -60), (52, -50)])
@pytest.mark.parametrize("schedule", [0, 8])
def test_inside_the_range(big, small, schedule):
    _run(20096, 4, big, small, [0, 900], 13, -1, schedule, False)


@pytest.mark.parametrize("schedule", [0, 8])
def test_one_tile_holds_all(schedule):
    _run(100, 4, 60, -60, [3], 13, -1, schedule, False)
    _run(300, 4, 60, -60, [0], 13, -1, schedule, False)
