"""Cases and plain forms of the query/key norm with rotation, the 8-bit KV
cache and the block-sparse decode.

Each case names one operator and its sizes.  ``run`` makes one pass: in
elementary torch operations, or through the framework's entry points where
``own`` is true.  ``exact`` states the same operators in 64 bits.

Conventions: token-major [tokens, heads, D] or [B, S, heads, D] rows, caches
[B, Hkv, L, D]; the 8-bit cache holds e4m3 codes and a power-of-two scale per
block of ``block`` tokens, KV head and operand; ``k_bounds`` [B, Hkv, blocks,
2, D] holds the largest and the smallest key value of each block and channel.
"""

import math
import random

import torch

own = False

D8 = 128             # head dim of the 8-bit cache
E_MIN, E_MAX = -60, 60
EPS = 1e-6


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # a prompt's projections, q and k as views of one fused qkv buffer
        dict(name="norm_rope_prompt_8191", op="norm_rope", N=8191, Hq=32, Hkv=8, D=128, L=8192,
             fused=True),
        # one streaming token: norm, rotation and the cache write in one call
        dict(name="norm_rope_append_b1", op="norm_rope_append", B=1, S=1, Hq=16, Hkv=8, D=128,
             L=8192, fill="ragged"),
        # one decode step of a batch into the 8-bit cache (an odd cache length)
        dict(name="kv8_append_token_b64", op="kv8_append", B=64, S=1, Hkv=8, L=1000, block=64,
             bounds=True, fill="ragged"),
        # two prompts into the 8-bit cache, starting inside a block
        dict(name="kv8_append_prompt_8190", op="kv8_append", B=2, S=8190, Hkv=8, L=8192, block=64,
             bounds=True, fill="end"),
        # a single stream far into its cache: latency, work split over a long axis
        dict(name="decode_kv8_b1_8001", op="decode_kv8", B=1, Hq=16, Hkv=8, L=8001, block=64,
             fill="end"),
        # the largest batch: bandwidth
        dict(name="decode_kv8_b256_g8", op="decode_kv8", B=256, Hq=64, Hkv=8, L=8192, block=128,
             fill="end"),
        # scoring the blocks of one long context
        dict(name="block_scores_b1_128k", op="block_scores", B=1, Hq=16, Hkv=8, L=131072, block=64,
             fill="end"),
        # scoring the blocks of a ragged batch
        dict(name="block_scores_b32_64k", op="block_scores", B=32, Hq=32, Hkv=8, L=65535, block=32,
             fill="ragged"),
        # choosing 64 of 2048 blocks for one stream
        dict(name="block_select_b1_2048", op="block_select", B=1, Hkv=8, L=131072, block=64,
             count=64, first=1, recent=2, fill="end"),
        # choosing among the finest blocks for a ragged batch
        dict(name="block_select_b64_8192", op="block_select", B=64, Hkv=8, L=131072, block=16,
             count=512, first=4, recent=16, fill="ragged"),
        # attending 64 blocks of one long context
        dict(name="decode_blocks_b1_128k", op="decode_blocks", B=1, Hq=16, Hkv=8, L=131072,
             block=64, count=64, fill="end"),
        # attending an eighth of a batch's caches, 16 query heads to a KV head
        dict(name="decode_blocks_b32_g16", op="decode_blocks", B=32, Hq=128, Hkv=8, L=32768,
             block=32, count=128, fill="ragged"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_append", "kv8_append", "decode_kv8", "block_scores",
                     "block_select", "decode_blocks"])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    block = rng.choice([16, 32, 64, 128])
    fill = rng.choice(["ragged", "end"])
    if op == "norm_rope":
        return dict(op=op, N=_log(rng, 1, 8191), Hq=Hkv * min(g, 4), Hkv=Hkv,
                    D=rng.choice([64, 80, 96, 128, 256]) if Hkv < 5 else 128, L=8192,
                    fused=rng.random() < 0.5)
    if op == "norm_rope_append":
        B = _log(rng, 1, 256)
        S = _log(rng, 1, max(1, min(2000, 8191 // B)))
        return dict(op=op, B=B, S=S, Hq=Hkv * min(g, 4), Hkv=Hkv, D=rng.choice([64, 128]),
                    L=S + _log(rng, 1, 2000), fill=fill)
    if op == "kv8_append":
        B = _log(rng, 1, 256)
        S = _log(rng, 1, max(1, 16380 // B))
        return dict(op=op, B=B, S=S, Hkv=Hkv, L=S + _log(rng, 1, 1000), block=block,
                    bounds=rng.random() < 0.7, fill=fill)
    if op == "decode_kv8":
        B = _log(rng, 1, 256)
        L = _log(rng, 1, min(131072, 256 * 8192 // B))
        return dict(op=op, B=B, Hq=Hkv * g, Hkv=Hkv, L=L, block=block, fill=fill)
    if op == "block_scores":
        B = _log(rng, 1, 64)
        L = _log(rng, block, min(262144, 2048 * 32 * block // B))
        return dict(op=op, B=B, Hq=Hkv * g, Hkv=Hkv, L=L, block=block, fill=fill)
    if op == "block_select":
        B = _log(rng, 1, 64)
        L = _log(rng, block, 131072)
        count = _log(rng, 1, 512)
        first = rng.randint(0, min(4, count))
        return dict(op=op, B=B, Hkv=Hkv, L=L, block=block, count=count, first=first,
                    recent=rng.randint(0, min(16, count - first)), fill=fill)
    B = _log(rng, 1, 32)
    L = _log(rng, 1, min(131072, 32 * 32768 // B))
    return dict(op=op, B=B, Hq=Hkv * g, Hkv=Hkv, L=L, block=block,
                count=_log(rng, 1, max(1, 4096 // block)), fill=fill)


def _positions(c):
    """First (or only) position of each sequence, fixed by the sizes."""
    B, last = c["B"], c["L"] - c.get("S", 1)
    if c["fill"] == "end":
        return [last] * B
    r = random.Random(B * 1000003 + c["L"])
    return [r.randint(0, last) for _ in range(B)]


# ----------------------------------------------------------------- inputs --

def _randn(shape, g, dtype=torch.bfloat16, gain=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * gain).to(dtype)


def _tables(L, D):
    a = torch.arange(L, dtype=torch.float64, device="cuda")[:, None] * \
        10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    a = torch.cat([a, a], dim=1)
    return torch.cos(a).float().contiguous(), torch.sin(a).float().contiguous()


def _codes(B, Hkv, L, g):
    """e4m3 codes of normal values, about a quarter of the code range at one sigma."""
    out = torch.empty(B, Hkv, L, D8, dtype=torch.float8_e4m3fn, device="cuda")
    per = max(1, (1 << 26) // (Hkv * L * D8))
    for i in range(0, B, per):
        n = min(per, B - i)
        x = torch.randn((n, Hkv, L, D8), generator=g, device="cuda")
        out[i:i + n] = (x * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return out


def _scales(B, Hkv, nb, g):
    e = torch.randint(-8, -5, (B, Hkv, nb), generator=g, device="cuda")
    return torch.ldexp(torch.ones((), device="cuda"), e).float().contiguous()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": c}
    op = c["op"]
    if op in ("norm_rope", "norm_rope_append"):
        Hq, Hkv, D, L = c["Hq"], c["Hkv"], c["D"], c["L"]
        s["q_weight"] = _randn((D,), g, gain=0.1) + 1
        s["k_weight"] = _randn((D,), g, gain=0.1) + 1
        s["cos"], s["sin"] = _tables(L, D)
    if op == "norm_rope":
        N = c["N"]
        qkv = _randn((N, Hq + 2 * Hkv, D), g, gain=2.0)
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
        if not c["fused"]:
            s["q"], s["k"] = s["q"].contiguous(), s["k"].contiguous()
        s["positions"] = torch.randint(0, L, (N,), generator=g, device="cuda", dtype=torch.int32) \
            if N <= 256 else torch.arange(N, device="cuda", dtype=torch.int32) % L
        s["q_out"] = torch.empty(N, Hq, D, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty(N, Hkv, D, dtype=torch.bfloat16, device="cuda")
        return s
    B, L, Hkv = c["B"], c["L"], c["Hkv"]
    s["positions"] = torch.tensor(_positions(c), dtype=torch.int32, device="cuda")
    if op == "norm_rope_append":
        S = c["S"]
        s["q"] = _randn((B, S, Hq, D), g, gain=2.0)
        s["k_new"], s["v_new"] = _randn((B, S, Hkv, D), g, gain=2.0), _randn((B, S, Hkv, D), g)
        s["k_cache"], s["v_cache"] = _randn((B, Hkv, L, D), g), _randn((B, Hkv, L, D), g)
        s["q_out"] = torch.empty_like(s["q"])
        return s
    block = c["block"]
    nb = -(-L // block)
    if op in ("kv8_append", "decode_kv8", "decode_blocks"):
        s["k_cache"], s["v_cache"] = _codes(B, Hkv, L, g), _codes(B, Hkv, L, g)
        s["k_scale"], s["v_scale"] = _scales(B, Hkv, nb, g), _scales(B, Hkv, nb, g)
    if op in ("kv8_append", "block_scores") and c.get("bounds", True):
        s["k_bounds"] = torch.empty(B, Hkv, nb, 2, D8, dtype=torch.bfloat16, device="cuda")
        mid = _randn((B, Hkv, nb, D8), g)
        s["k_bounds"][:, :, :, 0] = mid + _randn((B, Hkv, nb, D8), g).abs()
        s["k_bounds"][:, :, :, 1] = mid - _randn((B, Hkv, nb, D8), g).abs()
    if op == "kv8_append":
        shape = (B, c["S"], Hkv, D8)
        s["k_new"], s["v_new"] = _randn(shape, g, gain=1.5), _randn(shape, g)
    if op in ("decode_kv8", "block_scores", "decode_blocks"):
        s["q"] = _randn((B, c["Hq"], D8), g)
    if op in ("decode_kv8", "decode_blocks"):
        s["out"] = torch.empty_like(s["q"])
        s["workspace"] = torch.zeros((1 << 20) + (2048 + B * Hkv) * (c["Hq"] // Hkv) * 1024,
                                     dtype=torch.uint8, device="cuda")
    if op == "block_scores":
        s["out"] = torch.empty(B, Hkv, nb, dtype=torch.float32, device="cuda")
    if op in ("block_select", "decode_blocks"):
        count = c["count"]
        blocks = torch.arange(nb, device="cuda")
        last = (s["positions"].long() // block)[:, None, None]
        # scores of few bits, so that some are alike
        scores = _randn((B, Hkv, nb), g, gain=20.0).float()
        scores = scores.masked_fill(blocks > last, -math.inf)
        if op == "block_select":
            s["scores"] = scores
            s["out"] = torch.empty(B, Hkv, count, dtype=torch.int32, device="cuda")
        else:  # the last block and random others, ascending, -1 behind them
            i = scores.masked_fill(blocks == last, math.inf).topk(min(count, nb), dim=2).indices
            i = torch.where(i <= last, i, nb).sort(dim=2).values
            i = torch.nn.functional.pad(i, (0, count - i.shape[2]), value=nb)
            s["block_index"] = torch.where(i < nb, i, -1).to(torch.int32).contiguous()
    return s


# ------------------------------------------------------------ plain forms --

def _norm_rope(x, w, cos, sin):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    half = x.shape[-1] // 2
    turned = torch.cat([-y[..., half:], y[..., :half]], dim=-1)
    return (y * cos + turned * sin).to(torch.bfloat16)


def _softmax_out(scores, seen, v, eq):
    """Softmax over the last axis of scores where `seen`, times v; zeros where nothing is seen."""
    scores = scores.masked_fill(~seen, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - m.masked_fill(m == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    return torch.einsum(eq, p, v) / total.masked_fill(total == 0, 1.0)


def _exponent(amax):
    m, x = torch.frexp(amax)
    e = torch.where(m > 0.875, x - 8, x - 9)  # 448 = 0.875 * 2^9
    return torch.where(amax > 0, e, E_MIN).clamp(E_MIN, E_MAX)


def _append_plain(new, pos, codes, scale, block, bounds=None):
    B, S, H, D = new.shape
    L, dev = codes.shape[2], new.device
    nt = (S + block - 2) // block + 1
    j = torch.minimum(pos[:, None] // block + torch.arange(nt, device=dev),
                      (pos[:, None] + S - 1) // block)                      # [B, nt]
    r = (j[:, :, None] * block + torch.arange(block, device=dev)).clamp(max=L - 1)
    at = r - pos[:, None, None]
    fresh = ((at >= 0) & (at < S))[..., None, None]                         # [B, nt, block, 1, 1]
    older = (at < 0)[..., None, None]
    bi = torch.arange(B, device=dev)
    x = new[bi[:, None, None], at.clamp(0, S - 1)].float()                  # [B, nt, block, H, D]
    ax = x.abs().masked_fill(~fresh, 0.0)
    e = _exponent(ax.amax(dim=(2, 4)))                                      # [B, nt, H]
    had = (j * block < pos[:, None])[..., None]
    old_scale = scale[bi[:, None], :, j]                                    # [B, nt, H]
    s = torch.ldexp(torch.ones((), device=dev), e)
    s = torch.where(had, torch.maximum(old_scale, s), s)
    raw = codes.view(torch.uint8)
    kept = raw[bi[:, None, None], :, r]                                     # [B, nt, block, H, D]
    cast = lambda y: y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
    moved = cast(kept.view(torch.float8_e4m3fn).float() * (old_scale / s)[:, :, None, :, None])
    put = torch.where(fresh, cast(x / s[:, :, None, :, None]), torch.where(older, moved, kept))
    raw[bi[:, None, None], :, r] = put
    scale[bi[:, None], :, j] = s
    if bounds is not None:
        was = bounds[bi[:, None], :, j].float()                             # [B, nt, H, 2, D]
        hi = x.masked_fill(~fresh, -math.inf).amax(2)
        lo = x.masked_fill(~fresh, math.inf).amin(2)
        hi = torch.where(had[..., None], torch.maximum(hi, was[..., 0, :]), hi)
        lo = torch.where(had[..., None], torch.minimum(lo, was[..., 1, :]), lo)
        bounds[bi[:, None], :, j] = torch.stack([hi, lo], dim=3).to(bounds.dtype)


def _plain(s):
    c = s["case"]
    op = c["op"]
    pos = s["positions"].long()
    if op == "norm_rope":
        cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
        return {"q": _norm_rope(s["q"], s["q_weight"], cos, sin),
                "k": _norm_rope(s["k"], s["k_weight"], cos, sin)}
    if op == "norm_rope_append":
        rows = pos[:, None] + torch.arange(c["S"], device=pos.device)
        cos, sin = s["cos"][rows][:, :, None], s["sin"][rows][:, :, None]
        b = torch.arange(c["B"], device=pos.device)[:, None]
        s["k_cache"][b, :, rows] = _norm_rope(s["k_new"], s["k_weight"], cos, sin)
        s["v_cache"][b, :, rows] = s["v_new"]
        return {"q": _norm_rope(s["q"], s["q_weight"], cos, sin), "k_cache": s["k_cache"],
                "v_cache": s["v_cache"]}
    B, Hkv, L, block = c["B"], c["Hkv"], c["L"], c["block"]
    if op == "kv8_append":
        _append_plain(s["k_new"], pos, s["k_cache"], s["k_scale"], block, s.get("k_bounds"))
        _append_plain(s["v_new"], pos, s["v_cache"], s["v_scale"], block)
        return [s[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale", "k_bounds") if k in s]
    if op == "decode_kv8":
        at = torch.arange(L, device=pos.device)
        q = s["q"].float().view(B, Hkv, -1, D8)
        k = s["k_cache"].float() * s["k_scale"][:, :, at // block, None]
        scores = torch.einsum("bhgd,bhld->bhgl", q, k) * D8 ** -0.5
        del k
        v = s["v_cache"].float() * s["v_scale"][:, :, at // block, None]
        out = _softmax_out(scores, at <= pos[:, None, None, None], v, "bhgl,bhld->bhgd")
        return out.reshape(B, -1, D8).to(torch.bfloat16)
    if op == "block_scores":
        q = s["q"].float().view(B, Hkv, -1, D8)
        both = torch.stack([q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)], dim=2)
        scores = torch.einsum("bhcd,bhjcd->bhj", both, s["k_bounds"].float())
        seen = torch.arange(scores.shape[2], device=pos.device) <= (pos // block)[:, None, None]
        return scores.masked_fill(~seen, -math.inf)
    if op == "block_select":
        scores = s["scores"]
        j = torch.arange(scores.shape[2], device=pos.device)
        last = (pos // block)[:, None, None]
        kind = (j <= last).int() + ((j <= last) & ((j < c["first"]) | (j > last - c["recent"])))
        order = scores.nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf) \
            .sort(dim=2, descending=True, stable=True).indices
        kind = kind.expand_as(order).gather(2, order)
        kind, by = kind.sort(dim=2, descending=True, stable=True)
        i = torch.where(kind > 0, order.gather(2, by), len(j))[:, :, :c["count"]]
        i = torch.nn.functional.pad(i, (0, c["count"] - i.shape[2]), value=len(j)).sort(2).values
        return torch.where(i < len(j), i, -1).to(torch.int32)
    i = s["block_index"].long()
    q = s["q"].float().view(B, Hkv, -1, D8)
    rows = (i[..., None] * block + torch.arange(block, device=pos.device)).flatten(2)
    seen = ((rows >= 0) & (rows <= pos[:, None, None]))[:, :, None]
    b = torch.arange(B, device=pos.device)[:, None, None]
    h = torch.arange(Hkv, device=pos.device)[:, None]
    at = rows.clamp(0, L - 1)
    k = s["k_cache"].view(torch.uint8)[b, h, at].view(torch.float8_e4m3fn).float() * \
        s["k_scale"][b, h, at // block, None]
    scores = torch.einsum("bhgd,bhld->bhgl", q, k) * D8 ** -0.5
    v = s["v_cache"].view(torch.uint8)[b, h, at].view(torch.float8_e4m3fn).float() * \
        s["v_scale"][b, h, at // block, None]
    v = v.masked_fill(~seen[:, :, 0, :, None], 0.0)
    return _softmax_out(scores, seen, v, "bhgl,bhld->bhgd").reshape(B, -1, D8).to(torch.bfloat16)


def run(state):
    if not own:
        return _plain(state)
    import gqa_decode_attention_place_gb300 as ga
    s = state
    c = s["case"]
    op = c["op"]
    if op == "norm_rope":
        q, k = ga.attn_qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], EPS,
                                    s["positions"], s["cos"], s["sin"], q_out=s["q_out"],
                                    k_out=s["k_out"])
        return {"q": q, "k": k}
    if op == "norm_rope_append":
        q = ga.attn_qk_norm_rope_append(s["q"], s["k_new"], s["v_new"], s["q_weight"],
                                        s["k_weight"], EPS, s["positions"], s["k_cache"],
                                        s["v_cache"], s["cos"], s["sin"], q_out=s["q_out"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "kv8_append":
        ga.attn_kv8_append(s["k_new"], s["v_new"], s["positions"], s["k_cache"], s["v_cache"],
                           s["k_scale"], s["v_scale"], c["block"], k_bounds=s.get("k_bounds"))
        return [s[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale", "k_bounds") if k in s]
    if op == "decode_kv8":
        return ga.attn_decode_step_kv8(s["q"], s["positions"], s["k_cache"], s["v_cache"],
                                       s["k_scale"], s["v_scale"], c["block"], D8 ** -0.5,
                                       out=s["out"], workspace=s["workspace"])
    if op == "block_scores":
        return ga.attn_block_scores(s["q"], s["positions"], s["k_bounds"], c["L"], c["block"],
                                    out=s["out"])
    if op == "block_select":
        return ga.attn_block_select(s["scores"], s["positions"], c["L"], c["block"], c["count"],
                                    c["first"], c["recent"], out=s["out"])
    return ga.attn_decode_step_kv8_blocks(s["q"], s["positions"], s["k_cache"], s["v_cache"],
                                          s["k_scale"], s["v_scale"], c["block"],
                                          s["block_index"], D8 ** -0.5, out=s["out"],
                                          workspace=s["workspace"])


# ------------------------------------------------------------------- work --

def work(case):
    c = case
    op = c["op"]
    if op in ("norm_rope", "norm_rope_append"):
        tokens = c["N"] if op == "norm_rope" else c["B"] * c["S"]
        heads = c["Hq"] + c["Hkv"] * (1 if op == "norm_rope" else 2)
        rows = min(tokens, c["L"])
        return {"bytes": tokens * heads * c["D"] * 4 + rows * c["D"] * 8 + 4 * c["D"],
                "flops": tokens * (c["Hq"] + c["Hkv"]) * c["D"] * 8}
    pos, Hkv, block = _positions(c), c["Hkv"], c["block"]
    if op == "kv8_append":
        S = c["S"]
        blocks = sum((p + S - 1) // block - p // block + 1 for p in pos) * Hkv
        values = c["B"] * S * Hkv * D8
        return {"bytes": 2 * values * 3 + 8 * blocks + (4 * D8 * blocks if c["bounds"] else 0),
                "flops": 2 * values * 3}
    if op == "block_scores":
        g, nb = c["Hq"] // Hkv, -(-c["L"] // block)
        blocks = sum(p // block + 1 for p in pos) * Hkv
        return {"bytes": blocks * 4 * D8 + c["B"] * (c["Hq"] * 2 * D8 + 4 * Hkv * nb),
                "flops": blocks * 4 * D8 + c["B"] * Hkv * g * 2 * D8}
    if op == "block_select":
        blocks = sum(p // block + 1 for p in pos) * Hkv
        return {"bytes": 4 * blocks + 4 * c["B"] * Hkv * c["count"], "flops": blocks}
    if op == "decode_kv8":
        rows, blocks = sum(p + 1 for p in pos), sum(p // block + 1 for p in pos)
    else:
        blocks = sum(min(c["count"], p // block + 1) for p in pos)
        rows = sum((min(c["count"], p // block + 1) - 1) * block + p % block + 1 for p in pos)
    return {"bytes": Hkv * (rows * 2 * D8 + blocks * 8) + c["B"] * c["Hq"] * D8 * 4,
            "flops": 4 * c["Hq"] * rows * D8}


# ------------------------------------------------------------ 64-bit form --

def _rotate64(x, w, pos, cos, sin):
    """[n, heads, D] rows at positions [n], each half written out."""
    x, w = x.double(), w.double()
    D = x.shape[-1]
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * w
    a, b = y[..., :D // 2], y[..., D // 2:]
    c, s = cos[pos].double()[:, None], sin[pos].double()[:, None]
    out = torch.empty_like(y)
    out[..., :D // 2] = a * c[..., :D // 2] - b * s[..., :D // 2]
    out[..., D // 2:] = b * c[..., D // 2:] + a * s[..., D // 2:]
    return out


def _attend64(q, k, v):
    """[g, D] queries over [n, D] rows."""
    if not len(k):
        return torch.zeros_like(q)
    t = q @ k.T / math.sqrt(D8)
    w = torch.exp(t - t.max(dim=1, keepdim=True).values)
    return (w @ v) / w.sum(dim=1, keepdim=True)


def _append64(new, p, codes, scale, block):
    """One (sequence, KV head): new [S, D] rows at p; the codes' values before rounding, and the scales."""
    values, scales = codes.double(), scale.double()
    for j in range(p // block, (p + len(new) - 1) // block + 1):
        lo, hi = max(p, j * block), min(p + len(new), (j + 1) * block)
        x = new[lo - p:hi - p].double()
        top = float(x.abs().max())
        e = E_MIN if top == 0 else max(E_MIN, min(E_MAX, math.ceil(math.log2(top / 448))))
        if j * block < p:
            was = float(scales[j])
            e = max(e, round(math.log2(was)))
            values[j * block:p] *= was / 2.0 ** e
        scales[j] = 2.0 ** e
        values[lo:hi] = x / 2.0 ** e
    return values, scales


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    if op == "norm_rope":
        p = s["positions"].long()
        return {"q": _rotate64(s["q"], s["q_weight"], p, s["cos"], s["sin"]),
                "k": _rotate64(s["k"], s["k_weight"], p, s["cos"], s["sin"])}
    if op == "block_select":
        return None
    pos = _positions(c)
    B, Hkv, L = c["B"], c["Hkv"], c["L"]
    if op == "norm_rope_append":
        S = c["S"]
        q, k, v = s["q"].double(), s["k_cache"].double(), s["v_cache"].double()
        for b in range(B):
            p = torch.arange(pos[b], pos[b] + S, device="cuda")
            q[b] = _rotate64(s["q"][b], s["q_weight"], p, s["cos"], s["sin"])
            turned = _rotate64(s["k_new"][b], s["k_weight"], p, s["cos"], s["sin"])
            k[b, :, pos[b]:pos[b] + S] = turned.transpose(0, 1)
            v[b, :, pos[b]:pos[b] + S] = s["v_new"][b].double().transpose(0, 1)
        return {"q": q, "k_cache": k, "v_cache": v}
    block = c["block"]
    if op == "kv8_append":
        S = c["S"]
        touched = B * Hkv * (S // block + 2)
        if touched > 40000:
            return None
        out = [s["k_cache"].double(), s["v_cache"].double(), s["k_scale"].double(),
               s["v_scale"].double()]
        for b in range(B):
            for h in range(Hkv):
                for n, new in ((0, s["k_new"]), (1, s["v_new"])):
                    out[n][b, h], out[n + 2][b, h] = _append64(
                        new[b, :, h], pos[b], s[("k_cache", "v_cache")[n]][b, h],
                        s[("k_scale", "v_scale")[n]][b, h].cpu(), block)
        if "k_bounds" in s:
            bounds = s["k_bounds"].double()
            for b in range(B):
                for j in range(pos[b] // block, (pos[b] + S - 1) // block + 1):
                    x = s["k_new"][b, max(0, j * block - pos[b]):(j + 1) * block - pos[b]].double()
                    top, low = x.max(dim=0).values, x.min(dim=0).values
                    if j * block < pos[b]:
                        top = torch.maximum(top, bounds[b, :, j, 0])
                        low = torch.minimum(low, bounds[b, :, j, 1])
                    bounds[b, :, j, 0], bounds[b, :, j, 1] = top, low
            out.append(bounds)
        return out
    g = c["Hq"] // Hkv
    if op == "block_scores":
        out = torch.full((B, Hkv, s["k_bounds"].shape[2]), -math.inf, dtype=torch.float64,
                         device="cuda")
        for b in range(B):
            n = pos[b] // block + 1
            hi, lo = s["k_bounds"][b, :, :n, 0].double(), s["k_bounds"][b, :, :n, 1].double()
            q = s["q"][b].double().view(Hkv, g, 1, D8)
            total = 0
            for i in range(g):
                total = total + torch.maximum(q[:, i] * hi, q[:, i] * lo).sum(-1)
            out[b, :, :n] = total
        return out
    out = torch.zeros(B, c["Hq"], D8, dtype=torch.float64, device="cuda")
    if op == "decode_blocks":
        index = s["block_index"].cpu().tolist()
    for b in range(B):
        for h in range(Hkv):
            if op == "decode_kv8":
                rows = torch.arange(pos[b] + 1, device="cuda")
            else:
                rows = [torch.arange(j * block, min((j + 1) * block, pos[b] + 1), device="cuda")
                        for j in index[b][h] if j >= 0]
                rows = torch.cat(rows) if rows else torch.empty(0, dtype=torch.long, device="cuda")
            at = rows // block
            k = s["k_cache"][b, h].view(torch.uint8)[rows].view(torch.float8_e4m3fn).double() * \
                s["k_scale"][b, h][at, None].double()
            v = s["v_cache"][b, h].view(torch.uint8)[rows].view(torch.float8_e4m3fn).double() * \
                s["v_scale"][b, h][at, None].double()
            out[b, h * g:(h + 1) * g] = _attend64(s["q"][b, h * g:(h + 1) * g].double(), k, v)
    return out
