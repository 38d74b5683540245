"""The paged cache as a serving program uses it: prompts, decode steps with
beams that change places and share pages, drafted tokens that are dropped, a
pool that is compacted; eagerly, on another stream, captured and replayed, from
several threads."""

import threading

import numpy as np
import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from _paged import check_decode, f64, i32, i64, pools
from oracle import paged

pytestmark = pytest.mark.gpu


class Server:
    """B sequences over one pool, with the oracle's copy of everything beside it."""

    def __init__(self, B, Hq, Hkv, D, page, P, M, S, seed, layout="heads"):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.Hq, self.Hkv, self.D, self.page, self.S = B, Hq, Hkv, D, page, S
        self.k, self.v = pools(P, Hkv, page, D, self.g, layout)
        self.table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(P, dtype=torch.int32, device="cuda")
        self.pos = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.pages_ws = ga.pages_workspace(B, S, P, page)
        self.ws = ga.paged_workspace(B, S, Hq, Hkv, D)
        # rows held by each sequence, as a program without pages would keep them
        self.rows = [[np.zeros((Hkv, 0, D)) for _ in "kv"] for _ in range(B)]

    def step(self, n, stream=None):
        """n[b] new tokens of each sequence: pages, rows, attention; checked."""
        B, S, lengths = self.B, self.S, i32(n)
        new = torch.randn((B, S, self.Hq + 2 * self.Hkv, self.D), generator=self.g,
                          device="cuda").bfloat16()
        q = new[:, :, :self.Hq].contiguous()
        kn, vn = new[:, :, self.Hq:self.Hq + self.Hkv], new[:, :, self.Hq + self.Hkv:]
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        taken = ga.attn_pages_reserve(self.table, self.refs, self.pos, self.k, self.v, S,
                                      lengths=lengths, workspace=self.pages_ws, stream=stream)
        ga.attn_paged_append(kn, vn, self.pos, self.table, self.k, self.v, lengths=lengths,
                             stream=stream)
        out = ga.attn_decode_step_paged(q, self.pos, self.table, self.k, self.v, self.D ** -0.5,
                                        lengths=lengths, workspace=self.ws, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        assert (taken >= 0).all()
        check_decode(out, q, self.k, self.v, i64(self.pos), n, self.table, self.D ** -0.5)
        for b in range(B):
            for x, y in zip((0, 1), (kn, vn)):
                self.rows[b][x] = np.concatenate(
                    [self.rows[b][x], f64(y[b, :n[b]]).transpose(1, 0, 2)], axis=1)
        self.pos += lengths
        self.check()

    def fork(self, parents, kept):
        """Sequence b goes on from parents[b] with its first kept[b] rows."""
        ga.attn_pages_fork(self.table, self.refs, self.page, parents=i32(parents),
                           lengths=i32(kept), workspace=self.pages_ws)
        old = self.rows
        self.rows = [[x[:, :kept[b]] for x in old[p]] if p >= 0 else
                     [np.zeros((self.Hkv, 0, self.D)) for _ in "kv"] for b, p in enumerate(parents)]
        self.pos.copy_(i32([r[0].shape[1] for r in self.rows]))
        self.check()

    def check(self):
        """Every sequence's rows where its table says, the counts those of the table."""
        table, refs, k, v = i64(self.table), i64(self.refs), f64(self.k), f64(self.v)
        assert (np.bincount(table[table >= 0], minlength=len(refs)) == refs).all()
        for b, rows in enumerate(self.rows):
            j = np.arange(rows[0].shape[1])
            assert len(j) == int(self.pos[b])
            assert (table[b, -(-len(j) // self.page):] == -1).all()
            pg = table[b, j // self.page]
            for x, y in zip((k, v), rows):
                assert (x[pg, :, j % self.page].transpose(1, 0, 2) == y).all(), b
        assert ga.attn_read_device_status(self.pages_ws) == 0
        assert ga.attn_read_device_status(self.ws) == 0


@pytest.mark.parametrize("D,page,layout", [(128, 16, "heads"), (64, 32, "pair"),
                                           (128, 128, "rows")])
def test_serving(D, page, layout):
    s = Server(6, 8, 2, D, page, 400 if page == 16 else 90, -(-600 // page), 8, 1, layout)
    s.step([8, 3, 8, 1, 0, 8])
    for k in range(6):
        s.step([8, 7, 0, 8, 5 * (k % 2), 8])
    s.step([1] * 6, stream=torch.cuda.Stream())
    # beams: sequences 0 .. 3 go on from 0 and 1, 4 ends, 5 drops its last rows
    s.fork([0, 0, 1, 0, -1, 5], [2 ** 30, 2 ** 30, 50, 2 ** 30, 0, int(s.pos[5]) - 9])
    for _ in range(3):
        s.step([1, 1, 1, 1, 1, 8])
    before = int((s.refs > 0).sum())
    page_map = i64(ga.attn_pages_compact(s.table, s.refs, s.k, s.v, workspace=s.pages_ws))
    assert sorted(page_map[page_map >= 0].tolist()) == list(range(before))
    s.check()
    s.fork([3, 2, 1, 0, 5, 5], [2 ** 30] * 6)
    s.step([2, 0, 8, 1, 4, 1])
    s.fork([0, 1, 2, 3, 4, 5], [int(p) // 2 for p in s.pos])
    s.step([8] * 6)
    s.fork([-1] * 6, [0] * 6)
    assert (s.refs == 0).all()


def test_norm_with_rotation_feeds_the_pages():
    """attn_qk_norm_rope in front of the append and the decode."""
    B, Hq, Hkv, D, page = 3, 8, 2, 128, 16
    g = torch.Generator(device="cuda").manual_seed(2)
    pos = [5, 40, 63]
    k, v = pools(12, Hkv, page, D, g, poison=False)
    table = i32([[0, 1, 2, 3], [4, 5, 6, -1], [8, 9, 10, 11]])
    qkv = torch.randn((B, Hq + 2 * Hkv, D), generator=g, device="cuda").bfloat16()
    a = torch.arange(64, device="cuda")[:, None] * \
        10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D)
    cos, sin = torch.cos(torch.cat([a, a], 1)), torch.sin(torch.cat([a, a], 1))
    q, kn = ga.attn_qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], None, None, 1e-6, i32(pos), cos,
                                 sin)
    ga.attn_paged_append(kn, qkv[:, Hq + Hkv:], i32(pos), table, k, v)
    out = ga.attn_decode_step_paged(q, i32(pos), table, k, v, D ** -0.5)
    for b, p in enumerate(pos):
        assert torch.equal(k[int(table[b, p // page]), :, p % page], kn[b])
    check_decode(out, q, k, v, pos, None, table, D ** -0.5)


def test_matches_the_contiguous_cache():
    """The same rows in a static cache: the same step to rounding."""
    B, Hq, Hkv, L, D = 5, 16, 4, 512, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    pos = i32([0, 100, 511, 300, 17])
    kc, vc = (torch.randn((B, Hkv, L, D), generator=g, device="cuda").bfloat16() for _ in "kv")
    q = torch.randn((B, Hq, D), generator=g, device="cuda").bfloat16()
    order = torch.randperm(B * L // 32, generator=g, device="cuda")
    k, v = (torch.empty((B * L // 32, Hkv, 32, D), dtype=torch.bfloat16, device="cuda")
            for _ in "kv")
    for x, c in ((k, kc), (v, vc)):
        x[order] = c.view(B, Hkv, L // 32, 32, D).transpose(1, 2).reshape(-1, Hkv, 32, D)
    table = order.view(B, -1).to(torch.int32)
    a = ga.attn_decode_step(q, pos, kc, vc, D ** -0.5).float()
    b = ga.attn_decode_step_paged(q, pos, table, k, v, D ** -0.5).float()
    # both are within their bounds of the exact output; outputs are below 8, a bf16 step 2^-5
    assert (a - b).abs().max() <= 2.0 ** -5


def _state(seed, B=40, S=1, page=16, D=128):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = torch.randint(0, 1500, (B,), generator=g, device="cuda")
    M = 100
    order = torch.randperm(B * M + 50, generator=g, device="cuda").to(torch.int32)
    table = order[:B * M].view(B, M).clone()
    k, v = pools(B * M + 50, 2, page, D, g, poison=False)
    q = torch.randn((B, S, 8, D), generator=g, device="cuda").bfloat16()
    return q, r.to(torch.int32), table, k, v


@pytest.mark.parametrize("schedule", [-1, 0, 3])
def test_results_do_not_depend_on_timing(schedule):
    q, pos, table, k, v = _state(4)
    ws = ga.paged_workspace(40, 1, 8, 2, 128)
    ga.attn_test_force_schedule(schedule)
    try:
        first = ga.attn_decode_step_paged(q, pos, table, k, v, 0.1, workspace=ws)
        for _ in range(20):
            assert torch.equal(first, ga.attn_decode_step_paged(q, pos, table, k, v, 0.1,
                                                                workspace=ws))
    finally:
        ga.attn_test_force_schedule(-1)


def test_captured_and_replayed():
    """One graph of a whole step, replayed while positions, tables and lengths change; a second
    graph with its own workspaces runs beside it on another stream."""
    graphs = []
    for seed in (5, 6):
        s = Server(4, 8, 2, 128, 16, 200, 40, 4, seed)
        s.lengths = i32([4, 2, 0, 1])
        s.new = torch.zeros((4, 4, 12, 128), dtype=torch.bfloat16, device="cuda")
        s.out = torch.empty((4, 4, 8, 128), dtype=torch.bfloat16, device="cuda")
        s.q = torch.empty_like(s.out)
        s.taken = torch.empty(4, dtype=torch.int32, device="cuda")

        def run(s=s):
            s.q.copy_(s.new[:, :, :8])
            ga.attn_pages_reserve(s.table, s.refs, s.pos, s.k, s.v, 4, lengths=s.lengths,
                                  taken=s.taken, workspace=s.pages_ws)
            ga.attn_paged_append(s.new[:, :, 8:10], s.new[:, :, 10:], s.pos, s.table, s.k, s.v,
                                 lengths=s.lengths)
            ga.attn_decode_step_paged(s.q, s.pos, s.table, s.k, s.v, 0.09, lengths=s.lengths,
                                      out=s.out, workspace=s.ws)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            run()
            ga.attn_pages_fork(s.table, s.refs, 16, lengths=torch.zeros_like(s.pos),
                               workspace=s.pages_ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graphs.append((s, graph, side))
    for k in range(8):
        for s, graph, side in graphs:
            s.new.copy_(torch.randn(s.new.shape, generator=s.g, device="cuda"))
            s.lengths.copy_(i32([4, k % 3, 1, 4 - k % 5]))
        torch.cuda.synchronize()
        for s, graph, side in graphs:
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for s, graph, side in graphs:
            check_decode(s.out, s.q, s.k, s.v, i64(s.pos), i64(s.lengths), s.table, 0.09)
            assert (s.taken >= 0).all()
            s.pos += s.lengths
            assert ga.attn_read_device_status(s.ws) == 0
            assert ga.attn_read_device_status(s.pages_ws) == 0


def test_calls_from_several_threads():
    """Four threads, each with its own stream, workspace and state; the same bits as alone."""
    states = [_state(10 + i, B=7 + i, S=1 + i) for i in range(4)]

    def step(i, **kw):
        q, pos, table, k, v = states[i]
        out = ga.attn_decode_step_paged(q, pos, table, k, v, 0.1, **kw)
        t, refs = table.clone(), torch.ones(k.shape[0], dtype=torch.int32, device="cuda")
        ga.attn_pages_fork(t, refs, 16, parents=torch.zeros_like(pos), **kw)
        return out, t, refs

    want = [step(i) for i in range(4)]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got[i] = step(i, stream=stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_call_on_a_given_stream_makes_its_memory_there():
    """Outputs and workspaces made by a call belong to the stream it runs on, not to the busy
    current one, whose freed memory holds ones."""
    q, pos, table, k, v = _state(20, B=5)
    refs = torch.ones(k.shape[0], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()

    def calls(stream):
        t, c = table.clone(), refs.clone()
        torch.cuda.synchronize()
        return t, c, lambda: (
            ga.attn_decode_step_paged(q, pos, table, k, v, 0.1, stream=stream),
            ga.attn_pages_reserve(t, c, pos, k, v, 1, stream=stream),
            ga.attn_pages_fork(t, c, 16, lengths=pos, stream=stream),
            ga.attn_pages_compact(t, c, k, v, stream=stream))

    calls(s)[2]()  # kernels loaded and the stream's first memory made
    torch.cuda.synchronize()
    for handle in (s, s.cuda_stream):
        t, c, run = calls(handle)
        want_k, want_v, want_t, want_c = k.clone(), v.clone(), i64(table), i64(refs)
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in
                (ga.attn_paged_workspace_size(5, 1, 8, 2, 128),
                 ga.attn_pages_workspace_size(5, 1, k.shape[0], 16), 256, 512, 4096)]
        torch.cuda.synchronize()
        del junk
        torch.cuda._sleep(50_000_000)
        busy = torch.cuda.Event()
        busy.record()
        out, taken, _, page_map = run()
        s.synchronize()
        assert not busy.query()  # nothing above waited for the current stream
        check_decode(out, q, want_k, want_v, i64(pos), None, table, 0.1)
        want_taken, _ = paged.reserve(want_t, want_c, i64(pos), None, 1, 16)
        paged.fork(want_t, want_c, None, i64(pos), 16)
        want_map, _ = paged.compact(want_t, want_c)
        assert (i64(taken) == want_taken).all() and (i64(page_map) == want_map).all()
        assert (i64(t) == want_t).all() and (i64(c) == want_c).all()
        k.copy_(want_k)
        v.copy_(want_v)


def test_the_binding_refuses_what_does_not_fit():
    q, pos, table, k, v = _state(21, B=3)
    refs = torch.ones(k.shape[0], dtype=torch.int32, device="cuda")
    ok = dict(q=q, pos=pos, table=table, k=k, v=v)

    def decode(**kw):
        c = dict(ok, **kw)
        return ga.attn_decode_step_paged(c["q"], c["pos"], c["table"], c["k"], c["v"], 0.1,
                                         lengths=c.get("lengths"), out=c.get("out"),
                                         workspace=c.get("workspace"))
    for bad in (dict(pos=pos[:2]), dict(table=table[:2]), dict(table=table[:, ::2]),
                dict(v=v[1:]), dict(v=v.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(k=k[..., ::2], v=v[..., ::2]), dict(lengths=pos[:1]), dict(out=q[:, 0]),
                dict(q=q[:, :, ::2]), dict(workspace=torch.zeros(64, device="cuda")[::2])):
        with pytest.raises(ValueError):
            decode(**bad)
    for bad in (dict(q=q.float()), dict(pos=pos.long()), dict(table=table.long()),
                dict(k=k.half(), v=v.half()), dict(lengths=pos.float()), dict(workspace=7)):
        with pytest.raises(TypeError):
            decode(**bad)
    with pytest.raises(ga.AttnError, match="workspace"):
        decode(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ga.AttnError, match="unsupported"):
        decode(k=k[:, :, :8], v=v[:, :, :8])
    with pytest.raises(ga.AttnError, match="invalid"):
        ga.attn_paged_append(q[:, 0, :2], q[:, 0, :2], pos, table, k, k)
    with pytest.raises(ValueError):
        ga.attn_pages_reserve(table, refs[1:], pos, k, v, 1)
    with pytest.raises(ValueError):
        ga.attn_pages_compact(table, refs[:-1], k, v)
    with pytest.raises(ga.AttnError):
        ga.attn_pages_reserve(table, refs, pos, k, v, 0)
    with pytest.raises(ValueError):
        ga.attn_pages_fork(table, refs, 16, parents=pos[:2])
    decode()


CAPTURE_FIRST = """
import torch, gqa_decode_attention_place_gb300 as ga
g = torch.Generator(device="cuda").manual_seed(9)
for B, S, P in ((3, 2, 200), (1100, 1, 20000)):  # calls of one launch, and of two
    k, v = (torch.randn((P, 2, 16, 64), generator=g, device="cuda").bfloat16() for _ in "kv")
    new = torch.randn((B, S, 12, 64), generator=g, device="cuda").bfloat16()
    q, pos = new[:, :, :8].contiguous(), torch.full((B,), 15, dtype=torch.int32, device="cuda")
    first = torch.full((B * 8 + P,), -1, dtype=torch.int32, device="cuda")
    first[B * 8:] = 0
    first[:B * 8:8] = torch.arange(B, device="cuda") // 2 + P // 2
    first[B * 8:] += torch.bincount(first[:B * 8:8], minlength=P).int()
    live = first.clone()
    table, refs = live[:B * 8].view(B, 8), live[B * 8:]
    parents = torch.arange(B, device="cuda").flip(0).int()
    ws, pws = ga.paged_workspace(B, S, 8, 2, 64), ga.pages_workspace(B, S, P, 16)
    out, taken = torch.empty_like(q), torch.empty_like(pos)
    page_map = torch.empty(P, dtype=torch.int32, device="cuda")
    kept = k.clone(), v.clone()
    def step():
        k.copy_(kept[0])
        v.copy_(kept[1])
        live.copy_(first)
        ga.attn_pages_reserve(table, refs, pos, k, v, S, taken=taken, workspace=pws)
        ga.attn_paged_append(new[:, :, 8:10], new[:, :, 10:], pos, table, k, v)
        ga.attn_pages_fork(table, refs, 16, parents=parents, workspace=pws)
        ga.attn_pages_fork(table, refs, 16, lengths=pos + S, workspace=pws)
        ga.attn_pages_compact(table, refs, k, v, page_map=page_map, workspace=pws)
        ga.attn_decode_step_paged(q, pos, table, k, v, 0.1, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (out.view(torch.int16), live, taken, page_map)]
    out.zero_()
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (out.view(torch.int16), live, taken, page_map)))
    assert torch.isfinite(out).all() and (taken > 0).all() and ga.attn_read_device_status(pws) == 0
print("same")
"""


def test_a_process_whose_first_calls_are_captured():
    """Nothing has to run before a capture, and a replay does what the calls do."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CAPTURE_FIRST], capture_output=True, text=True,
                       cwd=root, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr
