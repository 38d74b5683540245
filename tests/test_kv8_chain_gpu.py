"""The operators in a row as a decoding program uses them: norm and rotation,
8-bit append with bounds, block scores, selection and the decode; eagerly, on
another stream, captured in a CUDA graph and replayed, and after a prefill."""

import numpy as np
import pytest
import torch

import gqa_decode_attention_place_gb300 as ga
from oracle import kv8
from _kv8 import D, check_decode, f64

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5


class Stream:
    """A small program's state: 8-bit caches, bounds, tables, weights, workspaces."""

    def __init__(self, B, Hq, Hkv, L, block, count, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        nb = -(-L // block)
        self.B, self.Hq, self.Hkv, self.L, self.block, self.count = B, Hq, Hkv, L, block, count
        self.kc, self.vc = (torch.zeros((B, Hkv, L, D), dtype=torch.uint8, device="cuda")
                            .view(torch.float8_e4m3fn) for _ in "kv")
        self.ks, self.vs = (torch.ones((B, Hkv, nb), device="cuda") for _ in "kv")
        self.bounds = torch.zeros((B, Hkv, nb, 2, D), dtype=torch.bfloat16, device="cuda")
        a = torch.arange(L, device="cuda")[:, None] * \
            10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D)
        self.cos, self.sin = torch.cos(torch.cat([a, a], 1)), torch.sin(torch.cat([a, a], 1))
        self.w = (torch.randn((2, D), generator=g, device="cuda") * 0.1 + 1).bfloat16()
        self.ws = ga.kv8_sparse_workspace(B, Hq, Hkv, L, D, block, count)
        self.out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device="cuda")
        self.q_out = torch.empty_like(self.out)
        self.k_out = torch.empty((B, Hkv, D), dtype=torch.bfloat16, device="cuda")

    def prompt(self, qkv):
        """qkv [B, S, Hq + 2 Hkv, D]: the prompt's rows into the cache."""
        B, S = qkv.shape[:2]
        rows = qkv.reshape(B * S, -1, D)
        pos = torch.arange(S, dtype=torch.int32, device="cuda").repeat(B)
        _, k = ga.attn_qk_norm_rope(rows[:, :self.Hq], rows[:, self.Hq:self.Hq + self.Hkv],
                                    self.w[0], self.w[1], 1e-6, pos, self.cos, self.sin)
        zero = torch.zeros(B, dtype=torch.int32, device="cuda")
        ga.attn_kv8_append(k.view(B, S, self.Hkv, D),
                           qkv[:, :, self.Hq + self.Hkv:], zero, self.kc, self.vc,
                           self.ks, self.vs, self.block, k_bounds=self.bounds)

    def step(self, qkv, v, pos, stream=None):
        """One token per sequence: qkv [B, Hq + Hkv, D], v [B, Hkv, D]."""
        ga.attn_qk_norm_rope(qkv[:, :self.Hq], qkv[:, self.Hq:], self.w[0], self.w[1], 1e-6, pos,
                             self.cos, self.sin, q_out=self.q_out, k_out=self.k_out,
                             stream=stream)
        ga.attn_kv8_append(self.k_out, v, pos, self.kc, self.vc, self.ks, self.vs, self.block,
                           k_bounds=self.bounds, stream=stream)
        ga.attn_decode_step_kv8_sparse(self.q_out, pos, self.kc, self.vc, self.ks, self.vs,
                                       self.bounds, self.block, self.count, SCALE, first=1,
                                       recent=2, out=self.out, workspace=self.ws, stream=stream)
        return self.out

    def check(self, positions, what=""):
        """The last step's output, over the blocks that the scores of the state's bounds choose,
        and the step's own list against them."""
        torch.cuda.synchronize()
        pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
        scores = ga.attn_block_scores(self.q_out, pos, self.bounds, self.L, self.block)
        index = ga.attn_block_select(scores, pos, self.L, self.block, self.count, 1, 2)
        s, got = scores.cpu().numpy(), index.cpu().numpy()
        for b, p in enumerate(positions):
            for h in range(self.Hkv):
                assert np.array_equal(got[b, h], kv8.block_select(
                    s[b, h], p, self.L, self.block, self.count, 1, 2))
        check_decode(self.out, self.q_out, positions, self.kc, self.vc, self.ks, self.vs, self.L,
                     self.block, SCALE, index=got.tolist(), what=what)
        assert ga.attn_read_device_status(self.ws) == 0


def _rows(n, B, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((n, B, H, D), generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("block,count", [(16, 8), (64, 4)])
def test_prompt_then_steps(block, count):
    B, Hq, Hkv, L, S = 2, 8, 2, 700, 600
    st = Stream(B, Hq, Hkv, L, block, count, seed=80)
    g = torch.Generator(device="cuda").manual_seed(81)
    prompt = torch.randn((B, S, Hq + 2 * Hkv, D), generator=g, device="cuda").bfloat16()
    st.prompt(prompt)
    qk, v = _rows(20, B, Hq + Hkv, 82), _rows(20, B, Hkv, 83)
    for t in range(20):
        pos = torch.full((B,), S + t, dtype=torch.int32, device="cuda")
        st.step(qk[t], v[t], pos)
        if t % 6 == 0:
            st.check([S + t] * B, f"step {t}")
    # the cache's bounds are those of the exact keys it was given
    p = torch.arange(S, dtype=torch.int32, device="cuda").repeat(B)
    rows = prompt.reshape(B * S, -1, D)
    _, k = ga.attn_qk_norm_rope(rows[:, :Hq], rows[:, Hq:Hq + Hkv], st.w[0], st.w[1], 1e-6, p,
                                st.cos, st.sin)
    first = k.view(B, S, Hkv, D)[:, :block].amax(1)
    assert torch.equal(st.bounds[:, :, 0, 0], first)


def test_captured_graphs_on_two_streams():
    """Two streams' steps, each captured once with its own state and replayed from a position that
    advances on the device; replays of both in flight together."""
    progs = []
    for i in range(2):
        s = torch.cuda.Stream()
        st = Stream(1, 16, 8, 300, 16, 6, seed=84 + i)
        qkv, v = _rows(1, 1, 24, 86 + i)[0], _rows(1, 1, 8, 88 + i)[0]
        pos = torch.zeros(1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            st.step(qkv, v, pos)  # warm-up, repeated by the first replay
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            st.step(qkv, v, pos)
            pos += 1
        progs.append((s, st, graph, pos, qkv, v))
    for t in range(260):
        for s, st, graph, pos, qkv, v in progs:
            with torch.cuda.stream(s):
                qkv.mul_(-1.01 if t % 50 else 0.6)
                v.mul_(-0.99)
                graph.replay()
    torch.cuda.synchronize()
    for s, st, graph, pos, qkv, v in progs:
        assert int(pos) == 260
        st.check([259], "after 260 replays")


def test_stream_argument():
    """The calls run on the stream given, after work queued there."""
    st = Stream(2, 8, 2, 200, 32, 3, seed=90)
    st.prompt(torch.randn((2, 150, 12, D), device="cuda").bfloat16())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    qk, v = torch.zeros((2, 10, D), dtype=torch.bfloat16, device="cuda"), _rows(1, 2, 2, 91)[0]
    src = _rows(1, 2, 10, 92)[0]
    pos = torch.full((2,), 150, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        qk.copy_(src)
    st.step(qk, v, pos, stream=s)
    s.synchronize()
    st.check([150, 150])


def test_full_decode_of_a_prefilled_prompt_is_near_the_bf16_one():
    """A prompt through the causal prefill and the 8-bit cache: the next token's decode differs
    from the bf16 cache's by the codes' rounding (half an e4m3 step, 2^-4, of each value)."""
    Hq, Hkv, S, L = 8, 2, 500, 512
    g = torch.Generator(device="cuda").manual_seed(93)
    q, k, v = (torch.randn((S, h, D), generator=g, device="cuda").bfloat16()
               for h in (Hq, Hkv, Hkv))
    ga.attn_prefill_causal(q, k, v, 0, SCALE)
    kc, vc = (torch.zeros((1, Hkv, L, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    kc[0, :, :S], vc[0, :, :S] = k.transpose(0, 1), v.transpose(0, 1)
    st = Stream(1, Hq, Hkv, L, 64, 4, seed=94)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    ga.attn_kv8_append(k[None], v[None], zero, st.kc, st.vc, st.ks, st.vs, 64)
    pos = torch.full((1,), S - 1, dtype=torch.int32, device="cuda")
    qd = torch.randn((1, Hq, D), generator=g, device="cuda").bfloat16()
    want = f64(ga.attn_decode_step(qd, pos, kc, vc, SCALE))
    got = f64(ga.attn_decode_step_kv8(qd, pos, st.kc, st.vc, st.ks, st.vs, 64, SCALE))
    # the keys' rounding moves a score by 2^-4 sum|q k| at most, and each weight by e to that;
    # in the mean over 128 dims and 500 rows far less: what is checked is a gross error
    assert np.linalg.norm(got - want) <= 0.25 * np.linalg.norm(want)
