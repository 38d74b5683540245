"""Pins of oracle/kv8.py against things other than itself: PyTorch's e4m3
type, hand-worked scales, the attention oracle, and closed forms."""

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import kv8


def test_e4m3_table_and_rounding_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(kv8.e4m3_decode(codes.numpy()), want, equal_nan=True)
    g = torch.Generator().manual_seed(0)
    x = torch.randn(20000, generator=g) * torch.exp2(torch.randint(-12, 9, (20000,), generator=g))
    mid = torch.tensor(kv8.E4M3[:126] + kv8.E4M3[1:127]) / 2  # the ties
    x = torch.cat([x, mid.float(), -mid.float(), torch.tensor([0.0, 448.0, 2.0 ** -10, math.nan])])
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = kv8.e4m3_encode(x.numpy())
    assert np.array_equal(got[~np.isnan(x.numpy())], want[~np.isnan(x.numpy())])
    assert got[-1] == 0x7F
    assert kv8.e4m3_encode(np.array([1e9]))[0] == 0x7E


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.1, 1), (449.0, 1), (224.0, -1), (1.0, -8),
                                    (0.0, -60), (1e-30, -60), (1e30, 60), (1.75, -8),
                                    (1.7578125, -7)])
def test_block_exponent(amax, e):
    assert kv8.block_exponent(amax) == e
    if -60 < e < 60:
        assert amax <= 448 * 2.0 ** e and (amax > 448 * 2.0 ** (e - 1))


def test_append_small_by_hand():
    """Block of 16: three rows in, then one a hundred times larger: the scale grows, the old
    codes move, the bounds widen, and a block reached at its first row starts anew."""
    rng = np.random.default_rng(0)
    codes = np.full((1, 1, 40, 4), 0x7F, dtype=np.uint8)
    scale = np.full((1, 1, 3), 2.0 ** 50)
    bounds = np.full((1, 1, 3, 2, 4), 99.0)
    a = rng.standard_normal((1, 3, 1, 4))
    codes, scale, bounds = kv8.kv8_append(codes, scale, a, [16], 16, bounds)
    e = kv8.block_exponent(np.abs(a).max())
    assert scale[0, 0].tolist() == [2.0 ** 50, 2.0 ** e, 2.0 ** 50]
    assert np.array_equal(bounds[0, 0, 1, 0], a[0, :, 0].max(0))
    assert (codes[0, 0, :16] == 0x7F).all() and (codes[0, 0, 19:] == 0x7F).all()
    big = a[:, :1] * 100
    codes2, scale2, bounds2 = kv8.kv8_append(codes, scale, big, [19], 16, bounds)
    s2 = scale2[0, 0, 1]
    assert s2 == 2.0 ** kv8.block_exponent(np.abs(big).max()) and s2 > 2.0 ** e
    assert np.array_equal(bounds2[0, 0, 1, 1], np.minimum(a[0, :, 0].min(0), big[0, 0, 0]))
    back = kv8.e4m3_decode(codes2[0, 0, 16:19]) * s2
    once = kv8.e4m3_decode(codes[0, 0, 16:19]) * 2.0 ** e
    assert np.all(np.abs(back - once) <= np.maximum(np.abs(once) * 2.0 ** -4, s2 * 2.0 ** -10))


def test_decode_matches_the_bf16_oracle():
    """With scale 1 and values that e4m3 holds, the 8-bit decode is the plain decode."""
    rng = np.random.default_rng(1)
    L, D, g = 50, 128, 4
    codes = rng.integers(0, 0x7F, (2, L, D)).astype(np.uint8)
    codes |= (rng.integers(0, 2, codes.shape) * 0x80).astype(np.uint8)
    K, V = (kv8.kv8_rows(c, np.full(4, 0.01), np.arange(L), 16) for c in codes)
    q = rng.standard_normal((1, g, D))
    out, spread, _ = kv8.attend(q[0], K[:31], V[:31], D ** -0.5)
    want = oracle.decode(q, K[None, None], V[None, None], [30], D ** -0.5)[0]
    assert np.allclose(out, want, rtol=1e-12, atol=1e-14)
    assert np.all(spread >= np.abs(out) - 1e-12)


def test_rows_of_lists():
    assert kv8.decode_rows_of(40, 64, 16).tolist() == list(range(41))
    got = kv8.decode_rows_of(40, 64, 16, [2, -1, 0, 3, 7, -5]).tolist()
    assert got == list(range(32, 41)) + list(range(16))
    assert kv8.decode_rows_of(40, 64, 16, [-1, 3]).size == 0


def test_scores_bound_every_key():
    rng = np.random.default_rng(2)
    K = rng.standard_normal((1, 64, 128))
    q = rng.standard_normal((2, 128))
    bounds = np.stack([K.reshape(1, 4, 16, 128).max(2), K.reshape(1, 4, 16, 128).min(2)], axis=2)
    s, _ = kv8.block_scores(q, bounds, 50, 16, 2)
    top = (q @ K[0].T).reshape(2, 4, 16).max(-1).sum(0)
    assert np.all(s[0] >= top) and np.isfinite(s).all()
    s, _ = kv8.block_scores(q, bounds, 31, 16, 2)
    assert np.isneginf(s[0, 2:]).all() and np.isfinite(s[0, :2]).all()


def test_select_rules():
    s = np.array([5.0, 1.0, 7.0, 7.0, np.nan, 2.0, -np.inf, 0.0])
    pick = lambda pos, count, first, recent: kv8.block_select(s, pos, 128, 16, count, first,  # noqa: E731
                                                              recent).tolist()
    assert pick(127, 3, 0, 0) == [0, 2, 3]
    assert pick(127, 1, 0, 0) == [2]                # the tie's lower index
    assert pick(127, 4, 1, 1) == [0, 2, 3, 7]
    assert pick(30, 4, 1, 1) == [0, 1, -1, -1]
    assert pick(-1, 2, 0, 0) == [-1, -1] and pick(128, 2, 0, 0) == [-1, -1]
    assert pick(127, 7, 0, 0) == [0, 1, 2, 3, 4, 5, 7]  # NaN and -inf alike: the lower index


def test_norm_rope_closed_forms():
    x = np.array([3.0, 4.0, 0.0, 0.0])
    y = kv8.norm_rope(x, None, 0.0, None, None)
    assert np.allclose(y, x / 2.5) and np.isclose((y * y).mean(), 1.0)
    c, s = math.cos(0.3), math.sin(0.3)
    r = kv8.norm_rope(x, np.array([1.0, 2.0, 1.0, 1.0]), 0.0, np.full(4, c), np.full(4, s))
    assert np.allclose(r, [1.2 * c, 3.2 * c, 1.2 * s, 3.2 * s])
    ora = oracle.rope_f32(y.astype(np.float32)[None], np.full((1, 4), c, np.float32),
                          np.full((1, 4), s, np.float32))
    assert np.allclose(kv8.norm_rope(x, None, 0.0, np.full(4, c), np.full(4, s)), ora[0], atol=1e-6)
