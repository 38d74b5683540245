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


def test_calls_from_several_threads():
    """Four threads, each with its own stream, workspace and output; the same bits as alone."""
    import threading

    L, block, B = 2000, 32, 5
    gen = torch.Generator(device="cuda").manual_seed(8)
    kc, vc = (codes_cache(B, 2, L, gen) for _ in "kv")
    ks, vs = (scales(B, 2, L, block, gen) for _ in "kv")
    bounds = torch.randn((B, 2, -(-L // block), 2, D), generator=gen, device="cuda")
    bounds = bounds.sort(dim=3, descending=True).values.bfloat16()
    q = [torch.randn((B, 16, D), generator=gen, device="cuda").bfloat16() for _ in range(4)]
    at = torch.tensor([0, 1999, 300, 1024, 77], dtype=torch.int32, device="cuda")

    def step(x, **kw):
        return (ga.attn_decode_step_kv8(x, at, kc, vc, ks, vs, block, SCALE, **kw),
                ga.attn_decode_step_kv8_sparse(x, at, kc, vc, ks, vs, bounds, block, 9, SCALE,
                                               **kw))

    want = [step(x) for x in q]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(4)

    def many(i):
        s = torch.cuda.Stream()
        start.wait()
        for _ in range(50):
            got = step(q[i], stream=s)
            s.synchronize()
            if not all(torch.equal(a.view(torch.int16), b.view(torch.int16))
                       for a, b in zip(got, want[i])):
                wrong.append(i)
                return

    threads = [threading.Thread(target=many, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


CAPTURE_FIRST = """
import torch, gqa_decode_attention_place_gb300 as ga
B, Hkv, L, block = 3, 2, 700, 16
g = torch.Generator(device="cuda").manual_seed(9)
codes = lambda: (torch.randn((B, Hkv, L, 128), generator=g, device="cuda") * 50).to(torch.float8_e4m3fn)
kc, vc = codes(), codes()
nb = -(-L // block)
ks, vs = (torch.full((B, Hkv, nb), 2.0 ** -7, device="cuda") for _ in "kv")
bounds = torch.zeros((B, Hkv, nb, 2, 128), dtype=torch.bfloat16, device="cuda")
q = torch.randn((B, 8, 128), generator=g, device="cuda").bfloat16()
k = torch.randn((B, Hkv, 128), generator=g, device="cuda").bfloat16()
at = torch.tensor([5, 699, 350], dtype=torch.int32, device="cuda")
ws = ga.kv8_sparse_workspace(B, 8, Hkv, L, 128, block, 6)
out, qn, kn = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k)
def step():
    ga.attn_qk_norm_rope(q, k, None, None, 1e-6, at, q_out=qn, k_out=kn)
    ga.attn_kv8_append(kn, kn, at, kc, vc, ks, vs, block, k_bounds=bounds)
    ga.attn_decode_step_kv8_sparse(qn, at, kc, vc, ks, vs, bounds, block, 6, 0.1, out=out, workspace=ws)
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
first = out.clone()
out.zero_()
step()
torch.cuda.synchronize()
assert torch.equal(first.view(torch.int16), out.view(torch.int16)) and torch.isfinite(first).all()
print("same")
"""


def test_a_process_whose_first_calls_are_captured():
    """Nothing has to run before a capture: what the calls find out about the device at their first
    use needs no stream."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CAPTURE_FIRST], capture_output=True, text=True,
                       cwd=root, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr
