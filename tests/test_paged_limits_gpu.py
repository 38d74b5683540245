"""The paged cache at its limits: offsets past 32 bits, the largest batch, a
wait that runs out, workspaces of other sizes."""

import numpy as np
import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from _paged import check_decode, f64, fill, i32, i64, pools, random_table
from oracle import paged

pytestmark = pytest.mark.gpu


def test_offsets_past_32_bits():
    """Pages whose elements lie behind 2^31 of the pool's base, in every call."""
    P, Hkv, page, D = 270000, 8, 16, 64  # 2.2e9 elements, 4.4 GB an operand
    k, v = (torch.empty((P, Hkv, page, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    gen = torch.Generator(device="cuda").manual_seed(1)
    top = list(range(P - 12, P))
    table = i32([[top[0], 3, top[5], -1], [top[8], top[2], top[9], top[11]]])
    low = dict(zip([3] + top, range(13)))
    fill(k, v, table, [48, 64], gen)
    kn, vn = (torch.randn((2, 1, Hkv, D), generator=gen, device="cuda").bfloat16() for _ in "kv")
    q = torch.randn((2, 1, 16, D), generator=gen, device="cuda").bfloat16()
    pos = i32([40, 63])
    ga.attn_paged_append(kn, vn, pos, table, k, v)
    at = [3] + top
    small_k, small_v = k[at], v[at]  # the same pages, close together
    small = i32([[low.get(e, -1) for e in row] for row in table.tolist()])
    assert torch.equal(small_k[low[top[5]], :, 8], kn[0, 0])
    assert torch.equal(small_v[low[top[11]], :, 15], vn[1, 0])
    out = ga.attn_decode_step_paged(q, pos, table, k, v, 0.1)
    check_decode(out, q, small_k, small_v, [40, 63], None, small, 0.1)
    # a shared page at the end of the pool, copied to the last free one, and back to the front
    refs = torch.ones(P, dtype=torch.int32, device="cuda")
    refs[P - 1], refs[P - 3] = 0, 2
    both = i32([[P - 3], [P - 3]])
    taken = ga.attn_pages_reserve(both, refs, i32([7, 16]), k, v, 1, lengths=i32([1, 0]))
    assert taken.tolist() == [1, 0] and both.tolist() == [[P - 1], [P - 3]]
    assert torch.equal(k[P - 1, :, :7], k[P - 3, :, :7])
    assert torch.equal(v[P - 1, :, :7], v[P - 3, :, :7])
    refs.zero_()
    refs[P - 1] = refs[P - 3] = 1
    want = k[[P - 3, P - 1]].clone()
    page_map = ga.attn_pages_compact(both, refs, k, v)
    assert both.tolist() == [[1], [0]] and page_map[P - 1] == 1 and page_map[P - 3] == 0
    assert torch.equal(k[:2], want)


def test_largest_batch():
    g = torch.Generator(device="cuda").manual_seed(2)
    B, page = 4096, 16
    r = torch.randint(0, 40, (B,), generator=g, device="cuda").tolist()
    lengths = [b % 3 for b in range(B)]
    table, P = random_table([p + n for p, n in zip(r, lengths)], page, 3, g)
    k, v = pools(P, 1, page, 64, g, poison=False)
    q = torch.randn((B, 2, 2, 64), generator=g, device="cuda").bfloat16()
    for schedule in (-1, 0):
        ga.attn_test_force_schedule(schedule)
        try:
            out = ga.attn_decode_step_paged(q, i32(r), table, k, v, 0.2, lengths=i32(lengths))
        finally:
            ga.attn_test_force_schedule(-1)
        check_decode(out, q, k, v, r, lengths, table, 0.2)


@pytest.mark.parametrize("schedule", [0, 2])
@pytest.mark.parametrize("S,g,D", [(1, 4, 128), (2, 8, 64), (4, 8, 128)])
def test_wait_runs_out_and_the_context_stays_usable(S, g, D, schedule):
    """A tile that is never copied: the call ends by itself, with the status."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    pos = [700, 300, 20]
    table, P = random_table([p + S for p in pos], 32, 24, gen)
    k, v = pools(P, 2, 32, D, gen, poison=False)
    q = torch.randn((3, S, 2 * g, D), generator=gen, device="cuda").bfloat16()
    args = (q, i32(pos), table, k, v, 0.1)
    ws = ga.paged_workspace(3, S, 2 * g, 2, D)
    ga.attn_test_force_schedule(schedule)
    ga.attn_test_skip_tile(1)
    try:
        ga.attn_decode_step_paged(*args, workspace=ws)
        bits = ga.attn_read_device_status(ws)  # synchronises
        ga.attn_test_skip_tile(-1)
        assert bits == ga.ATTN_DEV_TIMEOUT
        ws.zero_()
        out = ga.attn_decode_step_paged(*args, workspace=ws)
        assert ga.attn_read_device_status(ws) == 0
    finally:
        ga.attn_test_skip_tile(-1)
        ga.attn_test_force_schedule(-1)
    check_decode(out, q, k, v, pos, None, table, 0.1)


def test_one_workspace_for_pages_calls_of_many_sizes():
    """The scratch of one call does not reach into the next, whatever its sizes."""
    g = torch.Generator(device="cuda").manual_seed(4)
    ws = ga.pages_workspace(1200, 400, 20000, 16)
    for B, S, P in ((1200, 1, 20000), (3, 400, 200), (1, 1, 1), (600, 3, 9000), (1200, 1, 20000)):
        M = -(-(S + 40) // 16)
        k, v = pools(P, 1, 16, 64, g, poison=False)
        pos = torch.randint(0, 30, (B,), generator=g, device="cuda")
        t, c = np.full((B, M), -1), np.zeros(P, dtype=np.int64)
        table, refs = i32(t.tolist()), i32(c.tolist())
        for _ in range(2):
            taken = ga.attn_pages_reserve(table, refs, pos.to(torch.int32), k, v, S, workspace=ws)
            want, copies = paged.reserve(t, c, i64(pos), None, S, 16)
            assert (i64(taken) == want).all() and not copies
            ga.attn_pages_fork(table, refs, 16, parents=i32(list(range(B))[::-1]), workspace=ws)
            paged.fork(t, c, list(range(B))[::-1], None, 16)
            ga.attn_pages_compact(table, refs, k, v, workspace=ws)
            paged.compact(t, c)
            assert (i64(table) == t).all() and (i64(refs) == c).all()
    assert ga.attn_read_device_status(ws) == 0


def test_values_behind_the_last_row_and_unused_pages_stay():
    """Nothing but the new rows is written: by the append, and by none of the decode's calls."""
    g = torch.Generator(device="cuda").manual_seed(5)
    table, P = random_table([100, 37], 16, 9, g, spare=4)
    k, v = pools(P, 2, 16, 128, g, poison=False)
    before = f64(k), f64(v), i64(table)
    kn, vn = (torch.randn((2, 3, 2, 128), generator=g, device="cuda").bfloat16() for _ in "kv")
    ga.attn_paged_append(kn, vn, i32([90, 30]), table, k, v, lengths=i32([3, 2]))
    q = torch.randn((2, 3, 4, 128), generator=g, device="cuda").bfloat16()
    ga.attn_decode_step_paged(q, i32([90, 30]), table, k, v, 0.1, lengths=i32([3, 2]))
    want_k, want_v, t = before
    paged.append(want_k, want_v, f64(kn), f64(vn), [90, 30], [3, 2], t)
    assert (f64(k) == want_k).all() and (f64(v) == want_v).all() and (i64(table) == t).all()
