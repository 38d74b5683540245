"""attn_qk_norm_rope and attn_qk_norm_rope_append against oracle/kv8.py."""

import numpy as np
import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from oracle import kv8
from _kv8 import BF16_HALF, F32_HALF, f64

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _tables(L, D, gen):
    a = torch.rand((L, D), generator=gen, device="cuda") * 6.3  # halves need not be alike
    return torch.cos(a), torch.sin(a)


def _close(got, x, w, cos, sin, what=""):
    """Half a bf16 step of the result, and fp32 work: D products and sums under the root (half
    of it, for the root), the root, two scalings, and two products and a sum."""
    want = kv8.norm_rope(x, w, EPS, cos, sin)
    y = kv8.norm_rope(x, w, EPS, None, None)
    D = x.shape[-1]
    size = np.abs(y) + np.abs(np.roll(y, D // 2, axis=-1))
    tol = BF16_HALF * np.abs(want) + (1 + BF16_HALF) * (D / 2 + 12) * F32_HALF * size + 1e-38
    assert got.shape == want.shape
    assert (np.abs(got - want) <= tol).all(), what


@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 128, 192, 256])
@pytest.mark.parametrize("N,Hq,Hkv", [(1, 1, 1), (3, 16, 8), (130, 6, 2)])
def test_prompt_rows(N, Hq, Hkv, D):
    gen = torch.Generator(device="cuda").manual_seed(70)
    qkv = (torch.randn((N, Hq + 2 * Hkv, D), generator=gen, device="cuda") * 3).bfloat16()
    w = (torch.randn((2, D), generator=gen, device="cuda") * 0.2 + 1).bfloat16()
    L = 300
    cos, sin = _tables(L, D, gen)
    pos = torch.randint(0, L, (N,), generator=gen, device="cuda", dtype=torch.int32)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]  # views of one buffer
    p = pos.long().cpu().numpy()
    c, s = f64(cos)[p][:, None], f64(sin)[p][:, None]
    for qi, ki in ((q, k), (q.contiguous(), k.contiguous())):
        qo, ko = ga.attn_qk_norm_rope(qi, ki, w[0], w[1], EPS, pos, cos, sin)
        _close(f64(qo), f64(q), f64(w[0]), c, s, "q")
        _close(f64(ko), f64(k), f64(w[1]), c, s, "k")
    qo, ko = ga.attn_qk_norm_rope(q, k, None, None, EPS, pos)
    _close(f64(qo), f64(q), None, None, None)
    qc, kc = (t.clone(memory_format=torch.contiguous_format) for t in (q, k))
    ga.attn_qk_norm_rope(qc, kc, None, w[1], EPS, pos, cos, sin, q_out=qc, k_out=kc)  # in place
    _close(f64(qc), f64(q), None, c, s)
    _close(f64(kc), f64(k), f64(w[1]), c, s)


@pytest.mark.parametrize("B,S,positions", [(1, 1, [0]), (1, 1, [99]), (3, 1, [0, 98, 40]),
                                           (2, 37, [0, 63]), (1, 100, [0])])
@pytest.mark.parametrize("D", [64, 80, 128])
def test_append(B, S, positions, D):
    gen = torch.Generator(device="cuda").manual_seed(71)
    Hq, Hkv, L = 6, 3, 100
    qkv = (torch.randn((B, S, Hq + 2 * Hkv, D), generator=gen, device="cuda") * 2).bfloat16()
    w = (torch.randn((2, D), generator=gen, device="cuda") * 0.2 + 1).bfloat16()
    cos, sin = _tables(L, D, gen)
    kc = torch.randn((B, Hkv, L, D), generator=gen, device="cuda").bfloat16()
    vc = torch.randn((B, Hkv, L, D), generator=gen, device="cuda").bfloat16()
    k0, v0 = kc.clone(), vc.clone()
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
    qo = ga.attn_qk_norm_rope_append(q, k, v, w[0], w[1], EPS, pos, kc, vc, cos, sin)
    torch.cuda.synchronize()
    for b, p in enumerate(positions):
        rows = np.arange(p, p + S)
        c, s = f64(cos)[rows][:, None], f64(sin)[rows][:, None]
        _close(f64(qo[b]), f64(q[b]), f64(w[0]), c, s, "q")
        _close(f64(kc[b, :, p:p + S]).transpose(1, 0, 2), f64(k[b]), f64(w[1]), c, s, "k")
        assert torch.equal(vc[b, :, p:p + S], v[b].transpose(0, 1))
        kc[b, :, p:p + S] = k0[b, :, p:p + S]
        vc[b, :, p:p + S] = v0[b, :, p:p + S]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)  # no other row changed


def test_one_token_without_the_token_axis():
    gen = torch.Generator(device="cuda").manual_seed(72)
    x = torch.randn((2, 6, 64), generator=gen, device="cuda").bfloat16()
    pos = torch.tensor([3, 5], dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros((2, 2, 9, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    a = ga.attn_qk_norm_rope_append(x[:, :2], x[:, 2:4], x[:, 4:], None, None, EPS, pos, kc, vc)
    k2, v2 = torch.zeros_like(kc), torch.zeros_like(vc)
    b = ga.attn_qk_norm_rope_append(x[:, None, :2], x[:, None, 2:4], x[:, None, 4:], None, None,
                                    EPS, pos, k2, v2)
    assert torch.equal(a, b[:, 0]) and torch.equal(kc, k2) and torch.equal(vc, v2)


def test_bad_positions():
    gen = torch.Generator(device="cuda").manual_seed(73)
    D, L = 64, 20
    q = torch.randn((4, 2, D), generator=gen, device="cuda").bfloat16()
    cos, sin = _tables(L, D, gen)
    pos = torch.tensor([-1, 19, 20, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    qo, ko = ga.attn_qk_norm_rope(q, q.clone(), None, None, EPS, pos, cos, sin)
    for t in (qo, ko):
        assert torch.isnan(t[[0, 2, 3]]).all() and torch.isfinite(t[1]).all()
    kc, vc = (torch.zeros((4, 2, L, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    q2 = q[:, None].expand(4, 2, 2, D).contiguous()
    pos = torch.tensor([-1, 18, 19, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    qo = ga.attn_qk_norm_rope_append(q2, q2, q2, None, None, EPS, pos, kc, vc, cos, sin)
    assert torch.isnan(qo[[0, 2, 3]]).all() and torch.isfinite(qo[1]).all()
    assert (kc[[0, 2, 3]] == 0).all() and (vc[[0, 2, 3]] == 0).all() and (vc[1, :, 18:] != 0).any()


def test_zero_rows_and_zero_tokens():
    z = torch.zeros((2, 3, 128), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    qo, ko = ga.attn_qk_norm_rope(z, z, None, None, EPS, pos)
    assert (qo == 0).all() and (ko == 0).all()
    qo, _ = ga.attn_qk_norm_rope(z[:0], z[:0], None, None, EPS, pos[:0])
    assert qo.shape == (0, 3, 128)
