"""attn_decode_step_kv8 and attn_decode_step_kv8_blocks against the fp64
oracle, with the elementwise bounds of _kv8.out_bound."""

import numpy as np
import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from _kv8 import D, check_decode, codes_cache, scales

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5


def _case(B, Hkv, g, L, block, positions, seed, lo=-9, hi=-5, qgain=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    tail = [p if 0 <= p < L else L for p in positions]
    st = dict(kc=codes_cache(B, Hkv, L, gen, tail), vc=codes_cache(B, Hkv, L, gen, tail),
              ks=scales(B, Hkv, L, block, gen, lo, hi), vs=scales(B, Hkv, L, block, gen, lo, hi),
              q=(torch.randn((B, Hkv * g, D), generator=gen, device="cuda") * qgain).bfloat16(),
              pos=torch.tensor(positions, dtype=torch.int32, device="cuda"))
    for b, p in enumerate(tail):  # scales of blocks past the position may hold anything
        st["ks"][b, :, p // block + 1:] = float("nan")
        st["vs"][b, :, p // block + 1:] = float("nan")
    return st


def _run(st, block, **kw):
    return ga.attn_decode_step_kv8(st["q"], st["pos"], st["kc"], st["vc"], st["ks"], st["vs"],
                                   block, SCALE, **kw)


def _run_blocks(st, block, index, **kw):
    return ga.attn_decode_step_kv8_blocks(st["q"], st["pos"], st["kc"], st["vc"], st["ks"],
                                          st["vs"], block, index, SCALE, **kw)


def _check(out, st, L, block, positions, index=None, seqs=None, what=""):
    torch.cuda.synchronize()
    check_decode(out, st["q"], positions, st["kc"], st["vc"], st["ks"], st["vs"], L, block, SCALE,
                 index=index, seqs=seqs, what=what)


@pytest.mark.parametrize("g", [1, 2, 3, 4, 7, 8, 9, 16])
def test_group_sizes(g):
    pos = [0, 1, 15, 16, 127, 128, 300]
    st = _case(7, 2, g, 301, 32, pos, seed=10 + g)
    _check(_run(st, 32), st, 301, 32, pos)


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("B,Hkv,g,L,positions", [
    (1, 1, 1, 1, [0]),
    (1, 8, 2, 5000, [4999]),          # split over the grid
    (1, 1, 16, 40000, [39990]),       # one segment over every CTA
    (40, 8, 4, 700, "ragged"),
    (3, 5, 5, 777, [776, 0, 400]),
])
def test_sizes(B, Hkv, g, L, positions, block):
    if positions == "ragged":
        positions = [(b * 37 + 5) % L for b in range(B)]
    st = _case(B, Hkv, g, L, block, positions, seed=30)
    _check(_run(st, block), st, L, block, positions, seqs=range(min(B, 8)))


def test_large_batch_of_short_sequences():
    """More sequences than the first scan chunk, and fewer pipeline stages beside them."""
    B = 700
    pos = [(b * 11) % 130 for b in range(B)]
    st = _case(B, 2, 2, 130, 16, pos, seed=31)
    _check(_run(st, 16), st, 130, 16, pos, seqs=range(0, B, 13))


def test_largest_batch():
    """8192 sequences at 16 heads to a KV head: the fewest pipeline stages beside their scan."""
    B = 8192
    pos = [(b * 7) % 40 for b in range(B)]
    st = _case(B, 2, 16, 40, 16, pos, seed=53)
    _check(_run(st, 16), st, 40, 16, pos, seqs=range(0, B, 331))
    index = torch.tensor([2, 0], dtype=torch.int32, device="cuda").expand(B, 2, 2).contiguous()
    _check(_run_blocks(st, 16, index), st, 40, 16, pos, index=index.tolist(),
           seqs=range(0, B, 331))


@pytest.mark.parametrize("lo,hi", [(-60, -20), (-60, 61), (40, 61)])
def test_block_scales_far_apart(lo, hi):
    """V scales over the whole range: a probability must keep its weight whatever its block's
    scale.  K scales stay ordinary (scores of 2^60 would leave one row)."""
    st = _case(2, 2, 4, 600, 16, [599, 300], seed=32)
    g = torch.Generator(device="cuda").manual_seed(33)
    vs = scales(2, 2, 600, 16, g, lo, hi)
    st["vs"] = torch.where(st["vs"].isnan(), st["vs"], vs)
    _check(_run(st, 16), st, 600, 16, [599, 300])


def test_scales_that_are_no_powers_of_two():
    st = _case(2, 2, 4, 300, 32, [299, 77], seed=34)
    for k in ("ks", "vs"):
        st[k] *= 0.7
    _check(_run(st, 32), st, 300, 32, [299, 77])


@pytest.mark.parametrize("qgain", [1e-30, 1e-3, 30.0, 1e3])
def test_query_sizes(qgain):
    """Tiny queries (a flat softmax) and large ones (one row takes all)."""
    st = _case(2, 2, 4, 500, 64, [499, 200], seed=35, qgain=qgain)
    _check(_run(st, 64), st, 500, 64, [499, 200])


def test_query_with_elements_far_apart():
    st = _case(1, 1, 4, 300, 64, [299], seed=36)
    st["q"][:, :, ::2] *= 1e-6
    _check(_run(st, 64), st, 300, 64, [299])


def test_long_flat_softmax():
    """130000 rows of near-equal weight, with values of one sign: lost small weights would show."""
    L = 130001
    st = _case(1, 1, 2, L, 128, [L - 1], seed=37, qgain=0.01)
    st["vc"].view(torch.uint8).bitwise_and_(0x7F)
    _check(_run(st, 128), st, L, 128, [L - 1])


def test_one_row_over_many_small_ones():
    """Two rows 2^12 and 2^20 above all others in weight: the many keep their share of 1.4%."""
    L = 20000
    st = _case(1, 1, 2, L, 128, [L - 1], seed=38, qgain=0.01)
    st["q"][:] = 1.0
    st["kc"].view(torch.uint8).zero_()
    st["ks"].fill_(2.0 ** -6)
    for row, v in ((17, 48.0), (9000, 80.0)):  # scores 128 * v * 2^-6 / sqrt(128)
        st["kc"][0, 0, row] = torch.full((D,), v, device="cuda").to(torch.float8_e4m3fn)
    st["vc"].view(torch.uint8).bitwise_and_(0x7F)
    _check(_run(st, 128), st, L, 128, [L - 1])


def test_offsets_past_32_bits():
    """Caches of 4.5 GB: the last sequences lie past byte 2^32."""
    B, Hkv, L = 35, 4, 262144
    g = torch.Generator(device="cuda").manual_seed(39)
    kc = torch.empty((B, Hkv, L, D), dtype=torch.float8_e4m3fn, device="cuda")
    vc = torch.empty_like(kc)
    kc.view(torch.uint8).zero_()
    vc.view(torch.uint8).zero_()
    pos = [5] * (B - 2) + [L - 1, 1000]
    for c in (kc, vc):
        for b, n in ((0, 6), (B - 2, L), (B - 1, 1001)):
            c[b, :, :n] = codes_cache(1, Hkv, n, g)[0]
    st = dict(kc=kc, vc=vc, ks=scales(B, Hkv, L, 64, g), vs=scales(B, Hkv, L, 64, g),
              q=torch.randn((B, Hkv * 2, D), generator=g, device="cuda").bfloat16(),
              pos=torch.tensor(pos, dtype=torch.int32, device="cuda"))
    assert kc.numel() > 2 ** 32
    _check(_run(st, 64), st, L, 64, pos, seqs=[0, B - 2, B - 1])
    index = torch.tensor([0, 15, L // 64 - 1, -1], dtype=torch.int32, device="cuda").repeat(
        B, Hkv, 1).contiguous()
    _check(_run_blocks(st, 64, index), st, L, 64, pos, index=index.cpu().tolist(),
           seqs=[0, B - 2, B - 1])


def test_bad_positions_give_nan_and_status():
    pos = [10, -1, 64, 63]
    st = _case(4, 2, 4, 64, 16, pos, seed=40)
    ws = ga.kv8_workspace(4, 8, 2, 64, D)
    out = _run(st, 16, workspace=ws)
    assert ga.attn_read_device_status(ws) == ga.ATTN_DEV_BAD_POSITION
    assert torch.isnan(out[1:3]).all()
    _check(out, st, 64, 16, pos, seqs=[0, 3])
    index = torch.zeros((4, 2, 3), dtype=torch.int32, device="cuda")
    out = _run_blocks(st, 16, index, workspace=ws)
    assert ga.attn_read_device_status(ws) == ga.ATTN_DEV_BAD_POSITION
    assert torch.isnan(out[1:3]).all() and torch.isfinite(out[0]).all()


@pytest.mark.parametrize("g", [2, 16])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_listed_blocks(block, g):
    """Any order, repeats, none (-1) in between, blocks past the position, a last block cut by
    the position, and lists without a row (zeros)."""
    L = 1000
    nb = -(-L // block)
    pos = [999, 500, 0, block - 1, block]
    st = _case(5, 2, g, L, block, pos, seed=41)
    gen = torch.Generator().manual_seed(42)
    index = torch.randint(-1, nb, (5, 2, 11), generator=gen).int()
    index[0, 0] = torch.tensor([0, 0, nb - 1, 3, -1, 3, 1, 2, -1, nb - 1, 0])
    index[1, 0] = -1
    index[2, 1] = nb - 1                     # all past the position
    index[4, 0, 0] = 1
    out = _run_blocks(st, block, index.cuda())
    _check(out, st, L, block, pos, index=index.tolist())
    assert (out[1, :g] == 0).all() and (out[2, g:] == 0).all()


@pytest.mark.parametrize("count", [1, 2, 5, 64, 300])
def test_list_lengths(count):
    L, block = 5000, 16
    pos = [4999, 2500]
    st = _case(2, 3, 4, L, block, pos, seed=43)
    gen = torch.Generator().manual_seed(44)
    index = torch.stack([torch.randperm(156, generator=gen)[:count] if count <= 156 else
                         torch.cat([torch.arange(156), torch.full((count - 156,), -1)])
                         for _ in range(6)]).view(2, 3, count).int()
    _check(_run_blocks(st, block, index.cuda()), st, L, block, pos, index=index.tolist())


def test_all_blocks_listed_is_the_full_decode():
    pos = [4000, 4999]
    st = _case(2, 2, 4, 5000, 64, pos, seed=45)
    index = torch.arange(79, dtype=torch.int32, device="cuda").repeat(2, 2, 1).contiguous()
    a, b = _run(st, 64), _run_blocks(st, 64, index)
    assert torch.equal(a, b) or (a.float() - b.float()).abs().max() < 2e-2
    _check(b, st, 5000, 64, pos)


def test_bad_block_indices_are_skipped_and_reported():
    st = _case(1, 1, 2, 100, 32, [99], seed=46)
    ws = ga.kv8_workspace(1, 2, 1, 100, D)
    index = torch.tensor([[[1, -2, 4, 2 ** 31 - 1, -2 ** 31, 3]]], dtype=torch.int32,
                         device="cuda")
    out = _run_blocks(st, 32, index, workspace=ws)
    assert ga.attn_read_device_status(ws) == ga.ATTN_DEV_BAD_BLOCK
    _check(out, st, 100, 32, [99], index=[[[1, 3]]])


def test_same_bits_every_time_and_workspace_reuse():
    pos = [3000, 17, 4095]
    st = _case(3, 4, 4, 4096, 64, pos, seed=47)
    ws = ga.kv8_workspace(3, 16, 4, 4096, D)
    first = _run(st, 64, workspace=ws).clone()
    for _ in range(20):
        assert torch.equal(first, _run(st, 64, workspace=ws))
    assert ga.attn_read_device_status(ws) == 0


def test_nan_in_attended_rows_reaches_the_output():
    st = _case(1, 2, 2, 64, 16, [40], seed=48)
    st["vc"].view(torch.uint8)[0, 0, 7, 9] = 0x7F
    st["q"][0, 3, 0] = float("nan")
    out = _run(st, 16).float()
    torch.cuda.synchronize()
    assert torch.isnan(out[0, :2, 9]).all() and torch.isfinite(out[0, :2, :9]).all()
    assert torch.isfinite(out[0, 2]).all() and torch.isnan(out[0, 3]).all()


@pytest.mark.parametrize("cluster", [0, 1, 3, 8, 16])
@pytest.mark.parametrize("g", [2, 5, 16])
def test_every_way_of_splitting(cluster, g):
    """The flat list (0) and clusters of each size, with more and with fewer CTAs than a segment
    has tiles, and a sequence at a bad position among them."""
    L, block = 3100, 32
    pos = [3099, 0, -1, 700, 129]
    st = _case(5, 2, g, L, block, pos, seed=49)
    gen = torch.Generator().manual_seed(50)
    index = torch.randint(-1, 97, (5, 2, 21), generator=gen).int()
    ws = ga.kv8_workspace(5, 2 * g, 2, L, D)
    ga.attn_test_force_schedule(cluster)
    try:
        for _ in range(3):
            dense = _run(st, block, workspace=ws)
            listed = _run_blocks(st, block, index.cuda(), workspace=ws)
        torch.cuda.synchronize()
    finally:
        ga.attn_test_force_schedule(-1)
    assert ga.attn_read_device_status(ws) == ga.ATTN_DEV_BAD_POSITION
    assert torch.isnan(dense[2]).all() and torch.isnan(listed[2]).all()
    good = [0, 1, 3, 4]
    _check(dense, st, L, block, pos, seqs=good, what=f"cluster {cluster}")
    _check(listed, st, L, block, pos, index=index.tolist(), seqs=good, what=f"cluster {cluster}")


@pytest.mark.parametrize("seed", range(12))
def test_ragged_batches_split_anywhere(seed):
    """Batches of all kinds of lengths through the flat list, so that its cuts fall at, next to
    and inside segments, with bad positions in between; the same bits on a second run."""
    rng = np.random.default_rng(1000 + seed)
    B, Hkv, g = int(rng.integers(1, 90)), int(rng.integers(1, 6)), int(rng.integers(1, 5))
    L = int(rng.integers(100, 3000)) if B < 40 else int(rng.integers(100, 1000))
    pos = [int(p) for p in rng.integers(0, L, B)]
    if B > 4:
        for b in rng.integers(0, B, 2):
            pos[b] = L + 5
    st = _case(B, Hkv, g, L, 64, pos, seed=52)
    good = [b for b in range(B) if pos[b] < L]
    ga.attn_test_force_schedule(0)
    try:
        out, again = _run(st, 64), _run(st, 64)
        torch.cuda.synchronize()
    finally:
        ga.attn_test_force_schedule(-1)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    _check(out, st, L, 64, pos, seqs=good)


@pytest.mark.parametrize("g", [2, 16])
@pytest.mark.parametrize("longest", [130, 700, 5000])
def test_short_segments_beside_long_ones(longest, g):
    """Hundreds of segments of one to five tiles, which are kept whole, with a long one here and
    there that is split; the same for lists of which whole tiles hold no row."""
    B, Hkv, block = 150, 3, 16
    rng = np.random.default_rng(longest + g)
    pos = [int(p) for p in rng.integers(0, min(longest, 640), B)]
    for b in (0, 70, 149):
        pos[b] = longest - 1
    pos[5] = -3
    st = _case(B, Hkv, g, longest, block, pos, seed=53)
    index = torch.from_numpy(rng.integers(0, -(-longest // block), (B, Hkv, 37))).int()
    index[::2, :, 8:24] = -1  # two whole tiles
    index[::3, :, 30:] = -1
    index[9] = -1
    ga.attn_test_force_schedule(0)
    try:
        dense, listed = _run(st, block), _run_blocks(st, block, index.cuda())
        torch.cuda.synchronize()
    finally:
        ga.attn_test_force_schedule(-1)
    assert torch.isnan(dense[5]).all() and torch.isnan(listed[5]).all()
    assert (listed[9] == 0).all()
    seqs = [0, 1, 2, 3, 9, 70, 71, 100, 148, 149]
    _check(dense, st, longest, block, pos, seqs=seqs, what="dense")
    _check(listed, st, longest, block, pos, index=index.tolist(), seqs=seqs, what="listed")


@pytest.mark.parametrize("cluster", [0, 8])
@pytest.mark.parametrize("listed", [False, True])
def test_a_wait_that_runs_out_is_reported(cluster, listed):
    """A tile that never comes (its copy is not issued): the waits give up, the status says so,
    and the context and a zeroed workspace go on working."""
    pos = [2000]
    st = _case(1, 1, 4, 2001, 64, pos, seed=51)
    index = torch.arange(32, dtype=torch.int32, device="cuda")[None, None].contiguous()
    run = (lambda **kw: _run_blocks(st, 64, index, **kw)) if listed else \
        (lambda **kw: _run(st, 64, **kw))
    ws = ga.kv8_workspace(1, 4, 1, 2001, D)
    ga.attn_test_force_schedule(cluster)
    ga.attn_test_skip_tile(3)
    try:
        run(workspace=ws)
        bits = ga.attn_read_device_status(ws)
    finally:
        ga.attn_test_skip_tile(-1)
        ga.attn_test_force_schedule(-1)
    assert bits & ga.ATTN_DEV_TIMEOUT
    ws.zero_()
    _check(run(workspace=ws), st, 2001, 64, pos,
           index=index.cpu().tolist() if listed else None)
    assert ga.attn_read_device_status(ws) == 0
