"""attn_decode_step_paged and attn_paged_append against the fp64 oracle."""

import numpy as np
import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from _paged import check_decode, f64, fill, i32, i64, pools, random_table
from oracle import paged

pytestmark = pytest.mark.gpu


def make(B, S, Hq, Hkv, D, page, positions, gen, lengths=None, layout="heads", M=None, gain=1.0):
    """A cache whose attended rows are random and everything else NaN."""
    n = lengths or [S] * B
    rows = [p + k if k else 0 for p, k in zip(positions, n)]
    M = M or max(1, -(-max(rows) // page))
    table, P = random_table(rows, page, M, gen)
    k, v = pools(P, Hkv, page, D, gen, layout)
    fill(k, v, table, rows, gen, gain)
    q = torch.randn((B, S, Hq, D), generator=gen, device="cuda").bfloat16()
    return q, table, k, v


def run(B, S, Hq, Hkv, D, page, positions, lengths=None, layout="heads", M=None, seed=0, gain=1.0,
        scale=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q, table, k, v = make(B, S, Hq, Hkv, D, page, positions, gen, lengths, layout, M, gain)
    scale = scale or D ** -0.5
    out = ga.attn_decode_step_paged(q, i32(positions), table, k, v, scale, lengths=i32(lengths))
    torch.cuda.synchronize()
    check_decode(out, q, k, v, positions, lengths, table, scale)
    return out


@pytest.mark.parametrize("schedule", [-1, 0, 1, 3])
@pytest.mark.parametrize("D,page", [(128, 16), (64, 16), (128, 128), (64, 64), (128, 32)])
def test_sizes_and_splits(D, page, schedule):
    """Positions around pages and tiles, by every split."""
    ga.attn_test_force_schedule(schedule)
    try:
        run(7, 1, 8, 2, D, page, [0, 15, 16, 127, 128, 300, 1000])
    finally:
        ga.attn_test_force_schedule(-1)


@pytest.mark.parametrize("schedule", [0, 2])
@pytest.mark.parametrize("S,g,D", [(1, 1, 128), (1, 3, 64), (2, 4, 128), (1, 9, 128), (3, 5, 64),
                                   (1, 16, 128), (2, 16, 128), (4, 8, 64), (32, 1, 128),
                                   (5, 6, 128), (8, 1, 128), (17, 1, 64)])
def test_rows(S, g, D, schedule):
    """Heads and tokens of every row group, the new block across tiles and pages."""
    ga.attn_test_force_schedule(schedule)
    try:
        run(4, S, 3 * g, 3, D, 32, [0, 126, 500, 255], seed=1)
    finally:
        ga.attn_test_force_schedule(-1)


@pytest.mark.parametrize("layout", ["heads", "rows", "pair", "woven"])
def test_layouts(layout):
    run(3, 2, 8, 4, 128, 16, [5, 77, 260], layout=layout, seed=2)
    run(2, 1, 4, 1, 64, 128, [5, 400], layout=layout, seed=3)


@pytest.mark.parametrize("schedule", [-1, 0, 2])
def test_padded_batch(schedule):
    """Tokens past a sequence's own give zeros; a sequence without any is not looked at."""
    ga.attn_test_force_schedule(schedule)
    try:
        lengths = [4, 0, 1, 3, 0]
        out = run(5, 4, 8, 2, 128, 16, [60, 0, 0, 130, 10 ** 9], lengths=lengths, seed=4)
        for b, n in enumerate(lengths):
            assert (out[b, n:] == 0).all()
    finally:
        ga.attn_test_force_schedule(-1)


@pytest.mark.parametrize("schedule", [-1, 0, 2])
def test_bad_positions_lengths_and_pages(schedule):
    gen = torch.Generator(device="cuda").manual_seed(5)
    pos, lengths = [-1, 200, 250, 10, 300, 2 ** 31 - 1], [1, 2, 2, 3, -1, 2]
    good = [0, 200, 250, 10, 0, 0]
    q, table, k, v = make(6, 2, 4, 2, 128, 16, good, gen, [1, 2, 2, 2, 1, 1], M=16)
    table[2, 3], table[2, 5] = -1, 10 ** 6
    fill(k, v, torch.where(table < 0, 0, table.clamp(max=k.shape[0] - 1)), [0] * 6, gen)
    ws = ga.paged_workspace(6, 2, 4, 2, 128)
    ga.attn_test_force_schedule(schedule)
    try:
        out = ga.attn_decode_step_paged(q, i32(pos), table, k, v, 0.1, lengths=i32(lengths),
                                        workspace=ws)
    finally:
        ga.attn_test_force_schedule(-1)
    assert ga.attn_read_device_status(ws) == ga.ATTN_DEV_BAD_POSITION | ga.ATTN_DEV_BAD_PAGE
    check_decode(out, q, k, v, pos, lengths, table, 0.1)
    assert out[0].isnan().all() and out[3].isnan().all() and not out[2].isnan().any()
    # no page at all: zeros
    out = ga.attn_decode_step_paged(q, i32(good), torch.full_like(table, -1), k, v, 0.1)
    assert (out == 0).all()


@pytest.mark.parametrize("schedule", [0, 2])
@pytest.mark.parametrize("S,g", [(4, 2), (4, 4), (4, 8)])
def test_odd_values_of_a_later_token_stay_there(S, g, schedule):
    """A drafted token's NaN and infinities reach the tokens that see it, and no others."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    pos = [126, 40, 500]
    q, table, k, v = make(3, S, 2 * g, 2, 128, 16, pos, gen)
    want, _, _, _ = paged.decode(f64(q), f64(k), f64(v), pos, None, i64(table), 0.09)
    for b, p in enumerate(pos):
        for t, x in ((2, float("nan")), (3, float("inf"))):
            row = p + t
            v[int(table[b, row // 16]), :, row % 16, ::3] = x
    ga.attn_test_force_schedule(schedule)
    try:
        out = f64(ga.attn_decode_step_paged(q, i32(pos), table, k, v, 0.09))
    finally:
        ga.attn_test_force_schedule(-1)
    assert np.abs(out[:, :2] - want[:, :2]).max() < 0.05
    assert np.isnan(out[:, 2:, :, ::3]).all()
    clean = np.delete(np.arange(128), np.arange(0, 128, 3))
    assert np.abs(out[:, 2:][..., clean] - want[:, 2:][..., clean]).max() < 0.05


@pytest.mark.parametrize("schedule", [0, 2])
def test_scores_that_grow_and_fall(schedule):
    """Scores that rise by more than 2^64 from tile to tile, and fall again: the
    reference moves before the weights, after them, or not at all."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    q, table, k, v = make(2, 1, 4, 2, 128, 32, [1400, 900], gen)
    for b, p in enumerate([1400, 900]):
        for tile in range((p + 1) // 128):
            gain = [0.05, 20.0, 21.0, 0.1, 60.0, 59.0, 1.0, 300.0, 2.0, 310.0][tile % 10]
            j = torch.arange(tile * 128, tile * 128 + 128, device="cuda")
            pg = table[b].long()[j // 32]
            k[pg, :, j % 32] = (k[pg, :, j % 32].float() * gain).bfloat16()
    ga.attn_test_force_schedule(schedule)
    try:
        out = ga.attn_decode_step_paged(q, i32([1400, 900]), table, k, v, 128 ** -0.5)
    finally:
        ga.attn_test_force_schedule(-1)
    check_decode(out, q, k, v, [1400, 900], None, table, 128 ** -0.5)


def test_long_and_ragged():
    """Many segments cut anywhere, and one long one over all CTAs."""
    g = torch.Generator(device="cuda").manual_seed(8)
    pos = torch.randint(0, 3000, (37,), generator=g, device="cuda").tolist()
    run(37, 1, 8, 2, 128, 16, pos, seed=9)
    run(1, 1, 4, 1, 128, 64, [60000], seed=10)
    ga.attn_test_force_schedule(0)
    try:
        run(1, 2, 8, 1, 64, 16, [50001], seed=11)
    finally:
        ga.attn_test_force_schedule(-1)


def test_pages_shared_by_sequences():
    gen = torch.Generator(device="cuda").manual_seed(12)
    q, table, k, v = make(4, 1, 8, 2, 128, 16, [100] * 4, gen)
    table[1:, :5] = table[0, :5]
    out = ga.attn_decode_step_paged(q[:, 0].contiguous(), i32([100] * 4), table, k, v, 0.09)
    check_decode(out, q[:, 0], k, v, [100] * 4, None, table, 0.09)


@pytest.mark.parametrize("layout", ["heads", "rows", "pair", "woven"])
@pytest.mark.parametrize("D,page,Hkv", [(128, 16, 8), (64, 128, 3), (128, 64, 1)])
def test_append(D, page, Hkv, layout):
    gen = torch.Generator(device="cuda").manual_seed(13)
    B, S = 5, 150
    pos, lengths = [0, 15, 333, 7, 600], [150, 1, 149, 0, 40]
    M = -(-640 // page)
    table, P = random_table([p + n for p, n in zip(pos, lengths)], page, M, gen)
    table[4, 610 // page] = -1
    k, v = pools(P, Hkv, page, D, gen, layout, poison=False)
    fused = torch.randn((B, S, 2 * Hkv + 1, D), generator=gen, device="cuda").bfloat16()
    kn, vn = fused[:, :, :Hkv], fused[:, :, Hkv + 1:]
    want_k, want_v = f64(k), f64(v)
    paged.append(want_k, want_v, f64(kn), f64(vn), pos, lengths, i64(table))
    ga.attn_paged_append(kn, vn, i32(pos), table, k, v, lengths=i32(lengths))
    assert (f64(k) == want_k).all() and (f64(v) == want_v).all()


def test_append_skips_what_does_not_fit():
    gen = torch.Generator(device="cuda").manual_seed(14)
    pos, lengths = [-1, 63, 60, 0, 2 ** 31 - 1], [1, 2, 4, 9, 3]
    table, P = random_table([64] * 5, 16, 4, gen)
    k, v = pools(P, 2, 16, 64, gen, poison=False)
    kn, vn = (torch.randn((5, 4, 2, 64), generator=gen, device="cuda").bfloat16() for _ in "kv")
    want_k, want_v = f64(k), f64(v)
    paged.append(want_k, want_v, f64(kn), f64(vn), pos, lengths, i64(table))
    ga.attn_paged_append(kn, vn, i32(pos), table, k, v, lengths=i32(lengths))
    assert (f64(k) == want_k).all() and (f64(v) == want_v).all()
    ga.attn_paged_append(kn[:, 0], vn[:, 0], i32([16 * i for i in range(5)]), table, k, v)
    paged.append(want_k, want_v, f64(kn[:, :1]), f64(vn[:, :1]), [16 * i for i in range(5)], None,
                 i64(table))
    assert (f64(k) == want_k).all() and (f64(v) == want_v).all()


@pytest.mark.parametrize("S,g", [(1, 2), (1, 16), (2, 16)])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
def test_score_scales(S, g, scale):
    """A negative scale, zero (the mean of the rows), and one that leaves a single row."""
    gen = torch.Generator(device="cuda").manual_seed(15)
    pos = [0, 129, 400]
    q, table, k, v = make(3, S, 2 * g, 2, 128, 16, pos, gen)
    out = ga.attn_decode_step_paged(q, i32(pos), table, k, v, scale)
    check_decode(out, q, k, v, pos, None, table, scale)


@pytest.mark.parametrize("schedule", [0, 2])
@pytest.mark.parametrize("S,g,D", [(3, 2, 128), (3, 5, 128), (3, 8, 64), (3, 8, 128)])
def test_odd_keys_reach_who_sees_them(S, g, D, schedule):
    """NaN, +inf and -inf scores: in a drafted token's row, and in one that all see."""
    gen = torch.Generator(device="cuda").manual_seed(16)
    pos = [126, 40, 500, 300]
    q, table, k, v = make(4, S, g, 1, D, 16, pos, gen)
    want, _, _, _ = paged.decode(f64(q), f64(k), f64(v), pos, None, i64(table), 0.09)
    k[int(table[0, 127 // 16]), :, 127 % 16] = float("nan")       # the second token's own row
    k[int(table[1, 3 // 16]), :, 3] = float("nan")                # an old row
    k[int(table[2, 502 // 16]), :, 502 % 16] = q[2, 0, 0, 0].sign() * float("inf")  # the third's
    row = k[int(table[3, 7 // 16]), :, 7]
    row.zero_()
    row[..., 5] = float("inf")  # a score of +inf or -inf, by the sign of a query's dim 5
    ga.attn_test_force_schedule(schedule)
    try:
        out = f64(ga.attn_decode_step_paged(q, i32(pos), table, k, v, 0.09))
    finally:
        ga.attn_test_force_schedule(-1)
    assert np.abs(out[0, 0] - want[0, 0]).max() < 0.05 and np.isnan(out[0, 1:]).all()
    assert np.isnan(out[1]).all()
    assert np.abs(out[2, :2] - want[2, :2]).max() < 0.05 and np.isnan(out[2, 2]).all()
    # +inf: no weight is finite; -inf: the row has none
    up = f64(q)[3, :, :, 5] > 0
    assert np.isnan(out[3][up]).all()
    without = table.clone()
    kz, vz = f64(k), f64(v)
    kz[int(without[3, 0]), :, 7] = 0.0
    rest = np.delete(np.arange(303), 7)
    pg = i64(table)[3, rest // 16]
    for t in range(S):
        seen = rest <= 300 + t
        K, V = kz[pg[seen], 0, rest[seen] % 16], vz[pg[seen], 0, rest[seen] % 16]
        x = 0.09 * (f64(q)[3, t] @ K.T)
        w = np.exp(x - x.max(axis=1, keepdims=True))
        exact = (w @ V) / w.sum(axis=1, keepdims=True)
        down = f64(q)[3, t, :, 5] < 0
        assert np.abs(out[3, t][down] - exact[down]).max(initial=0) < 0.05


@pytest.mark.parametrize("S,g,D,page,layout", [
    (1, 1, 128, 16, "heads"), (1, 4, 128, 128, "rows"), (1, 4, 64, 32, "pair"),
    (1, 16, 128, 32, "woven"), (3, 4, 64, 16, "heads"), (2, 16, 128, 64, "rows"),
    (4, 8, 64, 128, "heads"), (5, 1, 128, 64, "pair"), (17, 1, 128, 16, "rows")])
@pytest.mark.parametrize("longest", [1, 17, 128, 250])
def test_many_short_sequences(S, g, D, page, layout, longest):
    """More segments than CTAs, none longer than two tiles: padded, idle and bad ones among them."""
    B, Hkv = 400, 3
    r = np.random.default_rng(17)
    lengths = r.integers(0, S + 1, B).tolist()
    pos = [int(r.integers(0, max(1, longest + 1 - n))) for n in lengths]
    gen = torch.Generator(device="cuda").manual_seed(17)
    q, table, k, v = make(B, S, Hkv * g, Hkv, D, page, pos, gen, lengths, layout)
    b = lengths.index(S)
    pos[b] = 10 ** 6
    ws = ga.paged_workspace(B, S, Hkv * g, Hkv, D)
    ga.attn_test_force_schedule(0)
    try:
        out = ga.attn_decode_step_paged(q, i32(pos), table, k, v, 0.1, lengths=i32(lengths),
                                        workspace=ws)
        first = ga.attn_decode_step_paged(q[:, :1].contiguous(), i32(pos), table, k, v, 0.1,
                                          lengths=i32([min(n, 1) for n in lengths]))
    finally:
        ga.attn_test_force_schedule(-1)
    assert ga.attn_read_device_status(ws) == ga.ATTN_DEV_BAD_POSITION
    check_decode(out, q, k, v, pos, lengths, table, 0.1)
    check_decode(first, q[:, :1], k, v, pos, [min(n, 1) for n in lengths], table, 0.1)


@pytest.mark.parametrize("S,g,D", [(1, 4, 128), (1, 16, 128), (1, 32, 128), (3, 2, 128),
                                   (8, 4, 128), (1, 4, 64), (5, 6, 64)])
def test_most_sequences_of_a_launch_short(S, g, D):
    """4096 sequences leave the rows in flight less room than fewer do."""
    B, page = 4096, 16
    r = np.random.default_rng(19)
    pos = r.integers(0, 130 - S, B).tolist()
    gen = torch.Generator(device="cuda").manual_seed(19)
    q, table, k, v = make(B, S, g, 1, D, page, pos, gen)
    out = ga.attn_decode_step_paged(q, i32(pos), table, k, v, 0.1)
    check_decode(out, q, k, v, pos, None, table, 0.1)


def test_many_short_sequences_with_bad_pages_and_odd_values():
    B, S, g, D, page = 500, 3, 4, 128, 16
    r = np.random.default_rng(18)
    pos = r.integers(0, 126, B).tolist()
    gen = torch.Generator(device="cuda").manual_seed(18)
    q, table, k, v = make(B, S, g, 1, D, page, pos, gen)
    for b in range(0, B, 7):
        table[b, int(r.integers(0, (pos[b] + S - 1) // page + 1))] = int(r.choice([-1, 10 ** 6]))
    ws = ga.paged_workspace(B, S, g, 1, D)
    for schedule in (0, 1):
        ga.attn_test_force_schedule(schedule)
        try:
            out = ga.attn_decode_step_paged(q, i32(pos), table, k, v, 0.1, workspace=ws)
        finally:
            ga.attn_test_force_schedule(-1)
        assert ga.attn_read_device_status(ws) == ga.ATTN_DEV_BAD_PAGE
        check_decode(out, q, k, v, pos, None, table, 0.1)
    # a last token's values that are not finite stay with it
    good = (table[:, :15] >= -1).all(1).tolist()
    for b in range(1, B, 7):
        row = pos[b] + S - 1
        v[int(table[b, row // page]), :, row % page, ::2] = float("nan")
    ga.attn_test_force_schedule(0)
    try:
        out = f64(ga.attn_decode_step_paged(q, i32(pos), table, k, v, 0.1))
    finally:
        ga.attn_test_force_schedule(-1)
    for b in range(1, B, 7):
        assert good[b] and not np.isnan(out[b, :S - 1]).any()
        assert np.isnan(out[b, S - 1, :, ::2]).all() and not np.isnan(out[b, S - 1, :, 1::2]).any()
