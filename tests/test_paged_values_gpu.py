"""attn_decode_step_paged where values or the score scale are not finite: the
output is what the formula gives, in the cluster, flat-list and warp-a-segment
forms and for every group of query rows."""

import numpy as np
import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from _paged import f64, fill, i32, i64, out_bound, pools, random_table
from oracle import paged

pytestmark = pytest.mark.gpu

SHAPES = [(1, 2, 128), (1, 4, 64), (1, 16, 128), (1, 12, 64), (1, 32, 128), (1, 24, 64),
          (3, 2, 128), (4, 4, 128), (4, 4, 64), (4, 8, 128), (4, 8, 64), (8, 1, 64)]
INF = float("inf")


def cache(B, S, Hq, Hkv, D, page, positions, seed, lengths=None):
    """Random attended rows and NaN everywhere else."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows = [p + n for p, n in zip(positions, lengths or [S] * B)]
    table, P = random_table(rows, page, -(-max(rows) // page), gen)
    k, v = pools(P, Hkv, page, D, gen)
    fill(k, v, table, rows, gen)
    return torch.randn((B, S, Hq, D), generator=gen, device="cuda").bfloat16(), table, k, v


def put(v, table, b, row, dims, x):
    page = v.shape[2]
    v[int(table[b, row // page]), :, row % page, dims] = x


def run(schedule, *args, **kw):
    ga.attn_test_force_schedule(schedule)
    try:
        return f64(ga.attn_decode_step_paged(*args, **kw))
    finally:
        ga.attn_test_force_schedule(-1)


def check(out, q, k, v, positions, lengths, table, scale):
    """Infinities and NaN where the formula has them, the bound of _paged.py elsewhere."""
    S, g = q.shape[1], q.shape[2] // k.shape[1]
    with np.errstate(invalid="ignore"):
        want, spread, load, n = paged.decode(f64(q), f64(k), f64(v), positions, lengths, i64(table),
                                             scale)
    for what, there in (("NaN", np.isnan), ("+inf", np.isposinf), ("-inf", np.isneginf)):
        off = there(out) != there(want)
        assert not off.any(), (f"{what}: {off.sum()} of {off.size} differ, the first at "
                               f"{np.argwhere(off)[0]}: {out[off][0]}, want {want[off][0]}")
    fine = np.isfinite(want)
    bound = out_bound(want, spread, load, n, 1 if S * g > 16 and q.shape[-1] == 64 else 2)
    assert (np.abs(out[fine] - want[fine]) <= bound[fine]).all()


def infinities(v, table, positions, S):
    """+inf, -inf and both in dims of their own: in an old row, in the last row that
    all tokens see, and in a drafted token's."""
    for b, p in enumerate(positions):
        put(v, table, b, p // 2, slice(0, None, 7), INF)
        put(v, table, b, p // 3, slice(1, None, 7), -INF)
        put(v, table, b, p, slice(2, None, 7), INF)
        put(v, table, b, 0, slice(3, None, 7), INF)
        put(v, table, b, p, slice(3, None, 7), -INF)
        if S > 1:
            put(v, table, b, p + 1, slice(4, None, 7), INF)
            put(v, table, b, p + S - 1, slice(5, None, 7), -INF)


@pytest.mark.parametrize("schedule", [0, 2])
@pytest.mark.parametrize("S,g,D", SHAPES)
def test_infinite_values(S, g, D, schedule):
    positions, Hkv = [1, 14, 126, 129, 500, 901], 2
    q, table, k, v = cache(6, S, Hkv * g, Hkv, D, 16, positions, 1)
    infinities(v, table, positions, S)
    out = run(schedule, q, i32(positions), table, k, v, 0.09)
    check(out, q, k, v, positions, None, table, 0.09)


@pytest.mark.parametrize("S,g,D", SHAPES)
def test_infinite_values_of_many_short_sequences(S, g, D):
    positions = (np.random.default_rng(2).integers(1, 100, 400)).tolist()
    q, table, k, v = cache(400, S, g, 1, D, 32, positions, 2)
    infinities(v, table, positions, S)
    out = run(0, q, i32(positions), table, k, v, 0.09)
    check(out, q, k, v, positions, None, table, 0.09)


@pytest.mark.parametrize("schedule", [0, 2])
@pytest.mark.parametrize("S,g,D", [(1, 4, 128), (1, 16, 128), (1, 32, 128), (1, 32, 64),
                                   (4, 8, 128)])
def test_infinite_values_of_little_weight(S, g, D, schedule):
    """Weights from 2^-90 up: the infinite row comes before the largest score and behind it."""
    q, table, k, v = cache(2, S, g, 1, D, 16, [600, 600], 3)
    k.copy_(torch.where(k.isnan(), k, torch.zeros_like(k)))
    q[..., 0] = 1.0
    q[..., 1:] = 0.0
    for b, (low, high) in enumerate(((100, 400), (400, 100))):
        put(k, table, b, low, slice(0, 1), -30.0)   # 60 below the largest score: 2^-86
        put(k, table, b, high, slice(0, 1), 30.0)
        put(v, table, b, low, slice(0, None, 3), INF)
    out = run(schedule, q, i32([600, 600]), table, k, v, 1.0)
    check(out, q, k, v, [600, 600], None, table, 1.0)


@pytest.mark.parametrize("schedule", [0, 2])
@pytest.mark.parametrize("S,g,D", [(1, 2, 128), (1, 16, 128), (1, 32, 64), (4, 8, 128)])
def test_scores_that_are_all_minus_infinity(S, g, D, schedule):
    """Zeros for a token that sees no other row; one finite row is all that another sees."""
    positions = [0, 40, 300]
    q, table, k, v = cache(3, S, g, 1, D, 16, positions, 5)
    q[..., 0] = 1.0
    k[..., 0] = torch.where(k[..., 0].isnan(), k[..., 0], -INF)
    last = positions[2] + S - 1  # seen by the last token alone
    k[int(table[2, last // 16]), 0, last % 16] = 0.5
    out = run(schedule, q, i32(positions), table, k, v, 0.1)
    assert (out[:2] == 0).all() and (out[2, :S - 1] == 0).all()
    assert (out[2, S - 1] == f64(v[int(table[2, last // 16]), 0, last % 16])).all()


@pytest.mark.parametrize("schedule", [0, 2])
@pytest.mark.parametrize("S,g", [(1, 2), (1, 16), (4, 8)])
def test_a_scale_that_is_nan(S, g, schedule):
    """NaN in every row of a token that is there, zeros in the others, as ever."""
    lengths = [S, 0, 1]
    q, table, k, v = cache(3, S, g, 1, 128, 16, [100, 0, 300], 4, lengths)
    out = run(schedule, q, i32([100, 0, 300]), table, k, v, float("nan"), lengths=i32(lengths))
    for b, n in enumerate(lengths):
        assert np.isnan(out[b, :n]).all() and (out[b, n:] == 0).all()
