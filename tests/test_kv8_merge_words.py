"""The shared-memory words that the two merge warps of the flat-list 8-bit
decode pass to each other: no word is written between two of their barriers in
which the other warp may still read it.  The order of barriers, writes and reads
is taken from the kernel's text, as the window is too short for a run to show."""

import itertools
import os
import re

import pytest

from gqa_decode_attention_place_gb300 import _build

EVENT = re.compile(r"(msync\(lane\))|(misc\[(\d+)\](?:\+\+)? = )|misc\[(\d+)\]")


def _events(text):
    """Barriers, writes and reads of misc words, in order; comments left out."""
    out = []
    for m in EVENT.finditer(re.sub(r"//[^\n]*", "", text)):
        if m.group(1):
            out.append(("barrier", None))
        elif m.group(2):
            out.append(("write", int(m.group(3))))
        else:
            out.append(("read", int(m.group(4))))
    return out


def races(pieces):
    """(words) written by thread 0 in a stretch without a barrier in which the other warp reads."""
    found, wrote, read = set(), set(), set()
    for kind, word in itertools.chain(*pieces, [("barrier", None)]):
        if kind == "barrier":
            found |= wrote & read
            wrote, read = set(), set()
        else:
            (wrote if kind == "write" else read).add(word)
    return found


def _merge_branch():
    with open(os.path.join(_build.CSRC, "kv8_decode.cu")) as f:
        text = f.read()
    start = text.index("ConsumerSync msync")
    branch = text[start:text.index("mbar_arrive(smem_u32(merged))", start)]
    cut = branch.index("if (w.u >= w.end) {  // the last piece")
    end = branch.index("break;", cut)
    split = branch[branch.index("if (!whole) {", end):]
    return _events(branch[cut:end]), _events(split)


def test_the_checker_sees_a_word_written_while_it_may_be_read():
    piece = [("barrier", None), ("write", 2), ("barrier", None), ("read", 2)]
    assert races([piece, piece]) == set()
    assert races([piece, piece[1:]]) == {2}


@pytest.mark.parametrize("before", [0, 1, 2])
def test_no_word_is_written_while_the_other_warp_may_read_it(before):
    """Up to two split pieces, then the CTA's last."""
    last, split = _merge_branch()
    assert ("barrier", None) in last and any(k == "write" for k, _ in last)
    assert ("barrier", None) in split and any(k == "write" for k, _ in split)
    assert races([split] * before + [last]) == set()
