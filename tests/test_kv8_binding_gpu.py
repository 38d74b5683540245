"""The 8-bit cache's binding: memory that a call makes itself, and tensors too large to name."""

import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from _kv8 import D, check_decode, codes_cache, scales

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5


def test_a_call_on_a_given_stream_makes_its_memory_there():
    """Workspace and output made by the call belong to the stream it runs on: not to the current
    one, which is busy, and whose freed memory holds ones."""
    L, block, pos = 3000, 64, [2999, 17, 700]
    gen = torch.Generator(device="cuda").manual_seed(7)
    kc, vc = (codes_cache(3, 2, L, gen, pos) for _ in "kv")
    ks, vs = (scales(3, 2, L, block, gen) for _ in "kv")
    q = torch.randn((3, 8, D), generator=gen, device="cuda").bfloat16()
    at = torch.tensor(pos, dtype=torch.int32, device="cuda")
    index = torch.arange(20, dtype=torch.int32, device="cuda").expand(3, 2, 20).contiguous()
    s = torch.cuda.Stream()

    def both(stream):
        ga.attn_test_force_schedule(0)
        try:
            return (ga.attn_decode_step_kv8(q, at, kc, vc, ks, vs, block, SCALE, stream=stream),
                    ga.attn_decode_step_kv8_blocks(q, at, kc, vc, ks, vs, block, index, SCALE,
                                                   stream=stream))
        finally:
            ga.attn_test_force_schedule(-1)

    both(s)  # kernels loaded and the stream's first memory made: both may wait for the device
    for handle in (s, s.cuda_stream):
        junk = torch.full((ga.attn_kv8_workspace_size(3, 8, 2, L, D),), 255, dtype=torch.uint8,
                          device="cuda")
        torch.cuda.synchronize()
        del junk
        torch.cuda._sleep(50_000_000)
        busy = torch.cuda.Event()
        busy.record()
        dense, listed = both(handle)
        s.synchronize()
        assert not busy.query()  # nothing above waited for the current stream
        check_decode(dense, q, pos, kc, vc, ks, vs, L, block, SCALE)
        check_decode(listed, q, pos, kc, vc, ks, vs, L, block, SCALE, index=index.tolist())


def test_sizes_past_32_bits_are_refused():
    """A dense tensor without elements may have any length."""
    L = 2 ** 31 + 1
    q = torch.empty((1, 0, D), dtype=torch.bfloat16, device="cuda")
    cache = torch.empty((1, 0, L, D), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty((1, 0, -(-L // 16)), device="cuda")
    at = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(1024, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        with pytest.raises(ValueError, match="out of range"):
            ga.attn_decode_step_kv8(q, at, cache, cache, scale, scale, 16, SCALE, workspace=ws)
