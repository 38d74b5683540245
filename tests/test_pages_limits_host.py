"""Sizes at the limits of the pages' calls: on the host, before any launch (no
GPU needed)."""

import pytest

import gqa_decode_attention_place_gb300 as ga

MOST = 2 ** 31 - 1
ITEMS = 1 << 28  # B * ceil((S - 1) / page + 1) may reach this


def needs(B, S, page):
    """Bytes that a reserve needs: 24 a sequence, 8 for each page its rows can touch."""
    up = lambda x: -(-x // 256) * 256
    return up(up(256 + 24 * B) + 8 * B * (-(-(S - 1) // page) + 1))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("S", [1, 2, 129, 2 ** 30, MOST - 128, MOST - 127, MOST - 16, MOST - 1, MOST])
def test_workspace_of_a_reserve_of_up_to_all_tokens(S, page):
    for B in (1, 2, 3):
        fits = B * (-(-(S - 1) // page) + 1) <= ITEMS
        assert ga.attn_pages_workspace_size(B, S, 1, page) == (needs(B, S, page) if fits else 0), B


@pytest.mark.parametrize("S", [MOST - 127, MOST])
def test_a_reserve_of_the_most_tokens_wants_that_workspace(S):
    """A byte less is refused; the last size that is not is refused for the next argument."""
    lib, P, Q = ga.load_library(), 0x1000, 0x2000  # never dereferenced

    def call(n, B=1, refs=P):
        return lib.attn_pages_reserve(P, refs, P, None, P, Q, 1024, 1024, 64, B, S, 1, 64, 1, 16, 1,
                                      P, P, n, None)
    assert call(needs(1, S, 16) - 1) == 3   # workspace
    assert call(needs(1, S, 16), B=3) == 2  # more items than there can be
    assert call(needs(1, S, 16), refs=None) == 1
