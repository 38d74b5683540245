"""attn_block_scores and attn_block_select against oracle/kv8.py."""

import math

import numpy as np
import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from oracle import kv8
from _kv8 import D, F32_HALF, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("B,Hkv,g,L,positions", [
    (1, 1, 1, 1, [0]),
    (1, 8, 2, 9000, [8999]),
    (4, 3, 5, 1000, [0, 15, 16, 999]),
    (2, 2, 16, 5001, [5000, 2047]),
    (3, 2, 8, 300, [-1, 300, 128]),
])
def test_scores(B, Hkv, g, L, positions, block):
    gen = torch.Generator(device="cuda").manual_seed(60)
    nb = -(-L // block)
    q = torch.randn((B, Hkv * g, D), generator=gen, device="cuda").bfloat16()
    mid = torch.randn((B, Hkv, nb, D), generator=gen, device="cuda")
    rad = torch.randn((B, Hkv, nb, D), generator=gen, device="cuda").abs()
    bounds = torch.stack([mid + rad, mid - rad], dim=3).bfloat16()
    for b, p in enumerate(positions):  # bounds past the position are not read
        bounds[b, :, (p // block + 1 if 0 <= p < L else 0):] = float("nan")
    pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
    got = f64(ga.attn_block_scores(q, pos, bounds, L, block))
    for b, p in enumerate(positions):
        if not 0 <= p < L:
            assert np.isneginf(got[b]).all()
            continue
        want, mag = kv8.block_scores(f64(q[b]), f64(bounds[b]), p, block, g)
        n = p // block + 1
        assert np.isneginf(got[b, :, n:]).all()
        # g sums and 256 fused products and sums, half a step each, of the terms' size
        tol = (256 + g) * F32_HALF * mag[:, :n] + 1e-30
        assert (np.abs(got[b, :, :n] - want[:, :n]) <= tol).all()


def _select(scores, positions, L, block, count, first, recent):
    pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
    B, Hkv = scores.shape[:2]
    whole = torch.full((B * Hkv * count + 4096,), -77, dtype=torch.int32, device="cuda")
    out = whole[2048:2048 + B * Hkv * count].view(B, Hkv, count)
    got = ga.attn_block_select(scores, pos, L, block, count, first, recent, out=out).cpu().numpy()
    assert (whole[:2048] == -77).all() and (whole[-2048:] == -77).all()  # nothing written outside
    s = scores.cpu().numpy()
    for b, p in enumerate(positions):
        for h in range(s.shape[1]):
            want = kv8.block_select(s[b, h], p, L, block, count, first, recent)
            assert np.array_equal(got[b, h], want), (b, h, got[b, h], want)


@pytest.mark.parametrize("L,block,count,first,recent", [
    (1, 16, 1, 0, 0), (100, 16, 3, 1, 1), (100, 16, 7, 1, 1), (100, 16, 20, 2, 3),
    (16384, 16, 64, 1, 2), (16400, 16, 1, 0, 0), (16400, 16, 1, 1, 0), (16400, 16, 1, 0, 1),
    (40000, 16, 64, 0, 64), (40000, 16, 65, 64, 1), (70000, 16, 512, 4, 16),
    (140000, 16, 100, 1, 2), (262144, 16, 16000, 1, 1), (300000, 16, 37, 1, 1),
])
def test_select(L, block, count, first, recent):
    """From one block to more than the kernel holds in registers."""
    nb = -(-L // block)
    gen = torch.Generator(device="cuda").manual_seed(61)
    scores = torch.randn((3, 2, nb), generator=gen, device="cuda")
    _select(scores, [L - 1, L // 2, L // 3], L, block, count, first, recent)


@pytest.mark.parametrize("nb", [4, 2045, 2046, 2047, 2048, 2049, 8188, 8189, 8190, 8191, 8192, 8193,
                                16384])
def test_select_row_lengths_at_the_kernels_limits(nb):
    """Rows that just fill, and just pass, what a block's threads hold, on and off 16 bytes; full
    rows and the lengths next to them."""
    gen = torch.Generator(device="cuda").manual_seed(63)
    scores = torch.randn((4, 3, nb), generator=gen, device="cuda")
    pos = [nb * 16 - 1, (nb - 1) * 16 - 1, (nb - 2) * 16 - 1, (nb - 3) * 16 - 1]
    for count in (1, min(nb - 1, 65), min(nb - 1, 2000)):
        _select(scores, pos, nb * 16, 16, count, 0, 0)
        _select(scores, pos, nb * 16, 16, count, 1, count - 1)
        if count > 2:
            _select(scores, pos, nb * 16, 16, count, 1, 1)
    # the same rows from a base that is not on 16 bytes
    shifted = torch.empty(scores.numel() + 1, device="cuda")[1:].view_as(scores).copy_(scores)
    _select(shifted, pos, nb * 16, 16, min(nb - 1, 65), 0, 1)


def test_select_ties_signs_and_non_finite():
    nb = 3000
    gen = torch.Generator(device="cuda").manual_seed(62)
    s = torch.randint(-2, 3, (6, 2, nb), generator=gen, device="cuda").float() * 0.5
    s[1] = 0.0
    s[1, 0, ::2] = -0.0
    s[2, :, 100:2000] = math.inf
    s[3, :, 5:] = -math.inf
    s[4, :, ::3] = math.nan
    s[5] = torch.finfo(torch.float32).min
    for count, first, recent in ((1, 0, 0), (50, 1, 1), (1500, 0, 3), (2999, 1, 0)):
        _select(s, [nb * 16 - 1] * 6, nb * 16, 16, count, first, recent)


def test_select_bad_positions():
    s = torch.zeros((4, 2, 10), device="cuda")
    _select(s, [-1, 160, 2 ** 31 - 1, 5], 160, 16, 3, 1, 1)


def test_scores_past_the_position_are_ignored():
    s = torch.zeros((1, 1, 400), device="cuda")
    s[..., 200:] = math.inf
    _select(s, [200 * 16 - 1], 6400, 16, 10, 1, 1)


@pytest.mark.parametrize("nb", [300, 2048, 8189, 8192])
@pytest.mark.parametrize("shape", ["close", "outlier", "tiny", "huge", "two", "wide", "coarse",
                                   "stairs", "one_low"])
def test_select_distributions(shape, nb):
    """Scores that spread evenly over their range, and ones of which most lie in a small part."""
    gen = torch.Generator(device="cuda").manual_seed(64)
    r = torch.randn((3, 2, nb), generator=gen, device="cuda")
    s = {
        "close": 1000 + r,
        "outlier": torch.where(r == r.amax(-1, keepdim=True), torch.full_like(r, 1e20), r),
        "tiny": r * 1e-33,
        "huge": r * 1e37,
        "two": torch.where(r > 0, r * 1e-3 + 5, r * 1e-3 - 5),
        "wide": torch.exp(r * 12),
        "coarse": (r * 20).bfloat16().float(),
        "stairs": torch.floor(r * 3),
        "one_low": torch.where(r == r.amin(-1, keepdim=True), torch.full_like(r, -math.inf), r),
    }[shape]
    pos = [nb * 16 - 1, nb * 16 - 17, nb * 8]
    for count, first, recent in ((1, 0, 0), (40, 1, 2), (nb // 2, 0, 1), (nb - 3, 1, 1)):
        _select(s, pos, nb * 16, 16, count, first, recent)
