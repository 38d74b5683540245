"""Launch rules ask the device for its SMs: the launchers of the norm, 8-bit
cache and block selection hold no count of one machine."""

import os
import re

import pytest

from gqa_decode_attention_place_gb300 import _build


@pytest.mark.parametrize("name", ["qk_norm_rope.cu", "kv8_append.cu", "kv8_decode.cu",
                                  "kv8_cluster.cuh", "block_select.cu"])
def test_no_sm_count_is_written_in(name):
    with open(os.path.join(_build.CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"\b152(?:ll|u|\b)", code)
