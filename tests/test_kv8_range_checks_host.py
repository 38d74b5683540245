"""What the range-checked build checks in the norm, 8-bit cache and block
selection kernels: every function that writes to memory at an address of its own
making tests it there, by the kernels' text."""

import ctypes
import os
import re

import pytest

import gqa_decode_attention_place_gb300 as ga
from gqa_decode_attention_place_gb300 import _build

CHECK = re.compile(r"\b(?:range_ok|range_ok_count|slot_ok)\(")

# file, the function's first words, checks in its body at least
PLACES = [
    ("kv8_decode.cu", "void store_column(", 1),         # an output's columns
    ("kv8_decode.cu", "bool slot_ok(", 1),              # a part's slot
    ("kv8_decode.cu", "void store_part(", 1),
    ("kv8_decode.cu", "void merge_few(", 1),
    ("kv8_decode.cu", "void merge_many(", 2),
    ("kv8_decode.cu", "kv8_decode_kernel(const", 5),    # tiles, scales, parts and what is left over
    ("kv8_cluster.cuh", "kv8_cluster_kernel(const", 4),  # tiles, scales, landing places
    ("kv8_append.cu", "kv8_append_kernel(\n", 3),       # block, older and new rows
    ("kv8_append.cu", "kv8_append_token_kernel(\n", 1),
    ("block_select.cu", "block_scores_kernel(\n", 1),
    ("block_select.cu", "block_select_kernel(\n", 4),   # row, both lists, the chosen
    ("qk_norm_rope.cu", "qk_norm_rope_kernel(const", 2),
]


def _body(name, words):
    with open(os.path.join(_build.CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = text.index("{", text.index(")", text.index(words)))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i]
    raise AssertionError(f"{name}: {words} has no end")


@pytest.mark.parametrize("name,words,least", PLACES, ids=[f"{p[0]}:{p[1].split('(')[0]}"
                                                         for p in PLACES])
def test_computed_addresses_are_checked(name, words, least):
    assert len(CHECK.findall(_body(name, words))) >= least


def test_calls_without_a_workspace_have_a_count():
    """Their kernels count into the word that attn_read_range_skips reads."""
    lib = ga.load_library()
    assert isinstance(lib.attn_read_range_skips, ctypes._CFuncPtr)
    assert "attn_read_range_skips" in ga.__all__
