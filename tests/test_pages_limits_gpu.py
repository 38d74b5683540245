"""attn_pages_reserve with the most new tokens that a call may allow for."""

import numpy as np
import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from _paged import f64, i32, i64, pools
from oracle import paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S", [2 ** 31 - 128, 2 ** 31 - 1])
def test_reserve_for_up_to_all_tokens(S):
    """Some rows behind the first sequence's, which leave the page that it shares; then all S of
    them, which do not fit."""
    page, P, M = 128, 9, 6
    table, refs = np.full((1, M), -1), np.zeros(P, dtype=np.int64)
    table[0, :2], refs[4], refs[7] = (4, 7), 1, 2
    gen = torch.Generator(device="cuda").manual_seed(1)
    k, v = pools(P, 2, page, 64, gen, poison=False)
    want_k, want_v = f64(k), f64(v)
    t, c = i32(table.tolist()), i32(refs.tolist())
    ws = ga.pages_workspace(1, S, P, page)
    for positions, lengths in (([200], [300]), ([0], None)):
        taken = ga.attn_pages_reserve(t, c, i32(positions), k, v, S, lengths=i32(lengths),
                                      workspace=ws)
        if lengths:
            want, copies = paged.reserve(table, refs, positions, lengths, S, page)
            for src, dst, n in copies:
                want_k[dst, :, :n], want_v[dst, :, :n] = want_k[src, :, :n], want_v[src, :, :n]
            assert want.tolist() == [3] and len(copies) == 1
            assert ga.attn_read_device_status(ws) == 0
        else:
            want = np.array([-1])
            assert ga.attn_read_device_status(ws) == ga.ATTN_DEV_BAD_POSITION
        assert (i64(taken) == want).all()
        assert (i64(t) == table).all() and (i64(c) == refs).all()
        assert (f64(k) == want_k).all() and (f64(v) == want_v).all()
