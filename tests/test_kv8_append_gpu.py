"""attn_kv8_append against oracle/kv8.py: codes, scales and bounds equal bit
for bit, and no other byte changes."""

import numpy as np
import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from oracle import kv8
from _kv8 import D, codes_cache, f64, scales, u8

pytestmark = pytest.mark.gpu


def _state(B, S, Hkv, L, block, seed, gain=1.0, lo=-9, hi=-5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nb = -(-L // block)
    st = dict(kc=codes_cache(B, Hkv, L, g), vc=codes_cache(B, Hkv, L, g),
              ks=scales(B, Hkv, L, block, g, lo, hi), vs=scales(B, Hkv, L, block, g, lo, hi),
              bounds=torch.randn((B, Hkv, nb, 2, D), generator=g, device="cuda").bfloat16(),
              kn=(torch.randn((B, S, Hkv, D), generator=g, device="cuda") * gain).bfloat16(),
              vn=(torch.randn((B, S, Hkv, D), generator=g, device="cuda") * gain).bfloat16())
    return st


def _check(st, positions, block, bounds=True):
    pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
    wk = kv8.kv8_append(u8(st["kc"]), f64(st["ks"]), f64(st["kn"]), positions, block,
                        f64(st["bounds"]))
    wv = kv8.kv8_append(u8(st["vc"]), f64(st["vs"]), f64(st["vn"]), positions, block)
    kept = st["bounds"].clone()
    ga.attn_kv8_append(st["kn"], st["vn"], pos, st["kc"], st["vc"], st["ks"], st["vs"], block,
                       k_bounds=st["bounds"] if bounds else None)
    torch.cuda.synchronize()
    assert np.array_equal(f64(st["ks"]), wk[1]) and np.array_equal(f64(st["vs"]), wv[1])
    assert np.array_equal(u8(st["kc"]), wk[0])
    assert np.array_equal(u8(st["vc"]), wv[0])
    if bounds:
        assert np.array_equal(f64(st["bounds"]), wk[2])
    else:
        assert torch.equal(kept.view(torch.int16), st["bounds"].view(torch.int16))


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("B,S,Hkv,L,positions", [
    (1, 1, 8, 1, [0]),
    (4, 1, 2, 200, [0, 15, 16, 199]),
    (3, 1, 3, 129, [127, 128, 31]),
    (2, 7, 1, 77, [0, 70]),
    (2, 130, 2, 300, [0, 170]),
    (1, 257, 5, 400, [63]),
])
def test_append(B, S, Hkv, L, positions, block):
    _check(_state(B, S, Hkv, L, block, seed=1), positions, block)


@pytest.mark.parametrize("gain,lo,hi", [(1e4, -9, -5), (1e-6, -9, -5), (1.0, -60, -50),
                                        (1.0, 20, 61), (3e19, 0, 40), (1e-25, -60, -59)])
def test_scales_that_grow_stay_and_clamp(gain, lo, hi):
    """New rows far above and far below the block's scale; the ends of the scale's range."""
    for S in (1, 20):
        _check(_state(2, S, 2, 96, 32, seed=2, gain=gain, lo=lo, hi=hi), [33, 60], 32)


def test_token_by_token_fills_blocks():
    """41 single appends into blocks of 16, each checked, with rows of growing size."""
    st = _state(1, 41, 2, 48, 16, seed=3)
    rows_k, rows_v = st["kn"].clone(), st["vn"].clone()
    for t in range(41):
        st["kn"] = (rows_k[:, t:t + 1] * 1.3 ** t).bfloat16()
        st["vn"] = (rows_v[:, t:t + 1] * 0.8 ** t).bfloat16()
        _check(st, [t], 16)


def test_without_bounds_and_3d_rows():
    _check(_state(2, 5, 2, 64, 32, seed=4), [3, 40], 32, bounds=False)
    st = _state(2, 1, 2, 64, 32, seed=5)
    four = {k: v.clone() for k, v in st.items()}
    pos = torch.tensor([3, 40], dtype=torch.int32, device="cuda")
    for s, cut in ((st, lambda x: x[:, 0].contiguous()), (four, lambda x: x)):
        ga.attn_kv8_append(cut(s["kn"]), cut(s["vn"]), pos, s["kc"], s["vc"], s["ks"], s["vs"], 32)
    torch.cuda.synchronize()
    assert torch.equal(st["kc"].view(torch.uint8), four["kc"].view(torch.uint8))


@pytest.mark.parametrize("S", [1, 45])
def test_rows_as_views_of_a_fused_buffer(S):
    """Keys and values at a token stride of their projections' buffer; the same with and without
    the token axis for one token."""
    B, Hq, Hkv, L, block = 3, 4, 2, 90, 32
    st = _state(B, S, Hkv, L, block, seed=10)
    qkv = torch.randn((B, S, Hq + 2 * Hkv, D), device="cuda").bfloat16()
    st["kn"], st["vn"] = qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    if S == 1:
        alone = {k: v.clone() for k, v in st.items() if k not in ("kn", "vn")}
        pos = torch.tensor([0, 31, 45], dtype=torch.int32, device="cuda")
        ga.attn_kv8_append(st["kn"][:, 0], st["vn"][:, 0], pos, alone["kc"], alone["vc"],
                           alone["ks"], alone["vs"], block, k_bounds=alone["bounds"])
    _check(st, [0, 31, 45], block)
    if S == 1:
        for k in alone:
            assert torch.equal(alone[k].view(torch.uint8), st[k].view(torch.uint8))


def test_non_finite_values():
    """NaN is kept as a NaN code, infinities saturate, and neither sets the scale; a block of
    nothing finite takes the smallest scale; NaN leaves the bounds alone."""
    st = _state(1, 4, 1, 64, 32, seed=6)
    st["kn"][0, 0, 0, 3] = float("nan")
    st["kn"][0, 1, 0, 4] = float("inf")
    st["kn"][0, 2, 0, 5] = float("-inf")
    st["vn"][:] = float("nan")
    st["vn"][0, 1, 0, ::2] = 0.0
    pos = torch.tensor([32], dtype=torch.int32, device="cuda")
    wk = kv8.kv8_append(u8(st["kc"]), f64(st["ks"]), f64(st["kn"]), [32], 32, f64(st["bounds"]))
    wv = kv8.kv8_append(u8(st["vc"]), f64(st["vs"]), f64(st["vn"]), [32], 32)
    ga.attn_kv8_append(st["kn"], st["vn"], pos, st["kc"], st["vc"], st["ks"], st["vs"], 32,
                       k_bounds=st["bounds"])
    torch.cuda.synchronize()
    for got, (codes, scale, *_), sc in ((st["kc"], wk, st["ks"]), (st["vc"], wv, st["vs"])):
        assert np.array_equal(f64(sc), scale)
        assert np.array_equal(kv8.e4m3_decode(u8(got)), kv8.e4m3_decode(codes), equal_nan=True)
    assert np.array_equal(f64(st["bounds"]), wk[2])


@pytest.mark.parametrize("pos", [32, 40])
def test_non_finite_single_tokens(pos):
    """One token with NaN and infinities, at a block's first row and inside it: a channel that has
    only been NaN keeps the empty bounds."""
    st = _state(1, 1, 2, 64, 32, seed=9)
    st["kn"][0, 0, 0, :3] = torch.tensor([float("nan"), float("inf"), float("-inf")])
    st["vn"][0, 0, 1] = float("nan")
    wk = kv8.kv8_append(u8(st["kc"]), f64(st["ks"]), f64(st["kn"]), [pos], 32, f64(st["bounds"]))
    wv = kv8.kv8_append(u8(st["vc"]), f64(st["vs"]), f64(st["vn"]), [pos], 32)
    at = torch.tensor([pos], dtype=torch.int32, device="cuda")
    ga.attn_kv8_append(st["kn"], st["vn"], at, st["kc"], st["vc"], st["ks"], st["vs"], 32,
                       k_bounds=st["bounds"])
    torch.cuda.synchronize()
    for got, (codes, scale, *_), sc in ((st["kc"], wk, st["ks"]), (st["vc"], wv, st["vs"])):
        assert np.array_equal(f64(sc), scale)
        assert np.array_equal(kv8.e4m3_decode(u8(got)), kv8.e4m3_decode(codes), equal_nan=True)
    assert np.array_equal(f64(st["bounds"]), wk[2])


def test_rows_outside_the_cache_are_skipped():
    st = _state(5, 3, 2, 50, 16, seed=7)
    before = {k: v.clone() for k, v in st.items()}
    pos = [48, -1, 2 ** 31 - 1, -2 ** 31, 47]
    _check(st, pos, 16)
    for k in ("kc", "vc"):
        assert torch.equal(before[k].view(torch.uint8)[:4], st[k].view(torch.uint8)[:4])
    for k in ("ks", "vs", "bounds"):
        assert torch.equal(before[k][:4], st[k][:4])


def test_nothing_to_append_changes_nothing():
    st = _state(2, 1, 2, 50, 16, seed=8)
    before = st["kc"].clone()
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    ga.attn_kv8_append(st["kn"][:, :0], st["vn"][:, :0], pos, st["kc"], st["vc"], st["ks"],
                       st["vs"], 16)
    torch.cuda.synchronize()
    assert torch.equal(before.view(torch.uint8), st["kc"].view(torch.uint8))
