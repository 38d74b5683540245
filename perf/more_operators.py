"""Cases and plain forms of the paged KV cache: the append, the decode step and
the calls that give out, share, free and move pages.

Each case names one operator and its sizes.  ``run`` makes one pass: in
elementary torch operations, or through the framework's entry points where
``own`` is true.  ``exact`` states the same operators in 64 bits.

Conventions: a pool of P pages of ``page`` rows, k_pages and v_pages
[P, Hkv, page, D] (any strides with dense rows); page_table [B, M] int32, the
page of rows j*page .. of sequence b, -1 for none; page_refs [P] int32, how
many table entries name a page, 0 for a free one.  New tokens of sequence b are
rows positions[b] .. positions[b] + n - 1, with n = lengths[b] of S or S.

The calls that change the table and the counts start from the same ones in
every pass: ``run`` puts them back first, with one copy for both.
"""

import math
import random

import torch

own = False


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decode step's rows of a batch, into pages of 16
        dict(name="paged_append_token_b64", op="append", B=64, S=1, Hkv=8, D=128, page=16, L=1000,
             layout="heads", fill="ragged", padded=False),
        # prompts of different lengths in one padded batch, starting inside a page
        dict(name="paged_append_prompt_8190", op="append", B=2, S=8190, Hkv=8, D=128, page=64,
             L=8192, layout="heads", fill="end", padded=True),
        # a single stream far into its cache: latency, work split over a long axis
        dict(name="decode_paged_b1_8001", op="decode", B=1, S=1, Hq=16, Hkv=8, D=128, page=64,
             L=8001, layout="heads", fill="end", padded=False),
        # a ragged batch over the finest pages
        dict(name="decode_paged_b64_ragged", op="decode", B=64, S=1, Hq=32, Hkv=8, D=128, page=16,
             L=8192, layout="heads", fill="ragged", padded=False),
        # the largest batch, keys and values token-major: bandwidth
        dict(name="decode_paged_b128_g8", op="decode", B=128, S=1, Hq=64, Hkv=8, D=128, page=128,
             L=8192, layout="rows", fill="end", padded=False),
        # four drafted tokens of each sequence at once, 8 query heads to a KV head
        dict(name="decode_paged_drafts_b32", op="decode", B=32, S=4, Hq=64, Hkv=8, D=128, page=32,
             L=16384, layout="heads", fill="ragged", padded=True),
        # a decode step's pages: one sequence in 16 starts a new one
        dict(name="reserve_step_b256", op="reserve", B=256, S=1, Hkv=8, D=128, page=16, L=1024,
             beams=1, spare=4096, layout="heads", fill="ragged", padded=False),
        # beams just forked: every one gets its own copy of the page they share
        dict(name="reserve_copies_b64", op="reserve", B=64, S=1, Hkv=8, D=128, page=128, L=8192,
             beams=4, spare=256, layout="heads", fill="ragged", padded=False),
        # beams change places after a step
        dict(name="fork_beams_b256", op="fork", B=256, page=16, L=8192, beams=4, spare=1000,
             order=True, cut=False),
        # a large batch drops rejected tokens and finished sequences
        dict(name="fork_cut_b512", op="fork", B=512, page=16, L=131072, beams=1, spare=1000,
             order=False, cut=True),
        # a small pool, a third of it free
        dict(name="compact_1024", op="compact", B=33, P=1024, used=0.66, Hkv=8, D=128, page=16,
             layout="heads"),
        # a large pool, half of it free
        dict(name="compact_32768", op="compact", B=256, P=32768, used=0.5, Hkv=8, D=128, page=16,
             layout="heads"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "reserve", "fork", "compact"])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8])
    D = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    layout = rng.choice(["heads", "rows", "pair"])
    fill = rng.choice(["ragged", "end"])
    if op == "append":
        B = _log(rng, 1, 256)
        S = _log(rng, 1, max(1, 16380 // B))
        return dict(op=op, B=B, S=S, Hkv=Hkv, D=D, page=page, L=S + _log(rng, 1, 1000),
                    layout=layout, fill=fill, padded=rng.random() < 0.5)
    if op == "decode":
        g = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        S = rng.choice([1, 1, 2, 3, 4, 5, 8])
        S = min(S, 32 // g)
        B = _log(rng, 1, 256)
        return dict(op=op, B=B, S=S, Hq=Hkv * g, Hkv=Hkv, D=D, page=page,
                    L=S + _log(rng, 1, min(131072, 128 * 8000 // B)), layout=layout, fill=fill,
                    padded=rng.random() < 0.5)
    if op == "reserve":
        beams = rng.choice([1, 1, 2, 4, 5])
        B = beams * _log(rng, 1, 1024 // beams)
        S = _log(rng, 1, max(1, 16384 // B))
        # a pool that may be too small for the last sequences
        return dict(op=op, B=B, S=S, Hkv=Hkv, D=D, page=page, L=S + _log(rng, 1, 400), beams=beams,
                    spare=_log(rng, 1, 65536 // page), layout=layout, fill=fill,
                    padded=rng.random() < 0.5)
    if op == "fork":
        beams = rng.choice([1, 2, 4, 5])
        B = beams * _log(rng, 1, 1024 // beams)
        order = rng.random() < 0.6
        return dict(op=op, B=B, page=page, L=_log(rng, 1, min(131072, (1 << 22) * page // B)),
                    beams=beams, spare=_log(rng, 1, 20000), order=order,
                    cut=not order or rng.random() < 0.5)
    P = _log(rng, 1, 262144 // page)
    return dict(op=op, B=_log(rng, 1, 256), P=P, used=rng.uniform(0.0, 1.0), Hkv=Hkv, D=D,
                page=page, layout=layout)


def _positions(c):
    """First new position of each sequence, fixed by the sizes; beams of a group stand alike."""
    B, last, beams = c["B"], c["L"] - c.get("S", 1), c.get("beams", 1)
    if c.get("fill") == "end":
        return [last] * B
    r = random.Random(B * 1000003 + c["L"])
    return [p for _ in range(B // beams) for p in [r.randint(0, last)] * beams]


def _lengths(c):
    """How many of the S new tokens each sequence has, fixed by the sizes."""
    if not c["padded"]:
        return [c["S"]] * c["B"]
    r = random.Random(c["B"] * 7919 + c["S"])
    return [r.randint(max(0, c["S"] // 2), c["S"]) for _ in range(c["B"])]


def _kept(c):
    """Rows of each sequence that stay, fixed by the sizes: most drop a few, some all."""
    r = random.Random(c["B"] * 104729 + c["L"])
    return [0 if r.random() < 0.1 else max(0, p - r.randint(0, 40)) for p in _positions(c)]


# ----------------------------------------------------------------- inputs --

def _randn(shape, g, gain=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * gain).to(torch.bfloat16)


def _pools(P, c, g):
    """k_pages and v_pages [P, Hkv, page, D] in one of the layouts that caches come in."""
    Hkv, page, D = c["Hkv"], c["page"], c["D"]
    shape = {"heads": (2, P, Hkv, page, D), "rows": (2, P, page, Hkv, D),
             "pair": (P, 2, Hkv, page, D)}[c["layout"]]
    both = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = both.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda", dtype=torch.bfloat16))
    if c["layout"] == "pair":
        return both[:, 0], both[:, 1]
    if c["layout"] == "rows":
        return both[0].transpose(1, 2), both[1].transpose(1, 2)
    return both[0], both[1]


def _table(counts, beams, M, spare, g, private=False):
    """Pages for groups of `beams` sequences that share theirs, `counts` pages each, given out in
    random order; with `private` the last of each sequence is its own.  (table, refs)"""
    n = torch.tensor(counts, device="cuda")
    B = len(counts)
    b, j = torch.arange(B, device="cuda")[:, None], torch.arange(M, device="cuda")
    mine = (b % beams == 0) | (private & (j == n[:, None] - 1))
    names = ((j < n[:, None]) & mine).flatten()
    P = int(names.sum()) + spare
    pages = torch.randperm(P, generator=g, device="cuda", dtype=torch.int32)
    table = pages[(names.cumsum(0) - 1).clamp(min=0)].view(B, M)
    table = torch.where(mine, table, table[b // beams * beams, j])
    table = torch.where(j < n[:, None], table, -1)
    refs = torch.bincount(table[table >= 0], minlength=P).to(torch.int32)
    return table, refs


def _kept_state(s, table, refs):
    """The table and the counts side by side, and what a pass starts from."""
    B, M = table.shape
    s["first"] = torch.cat([table.flatten(), refs])
    s["live"] = s["first"].clone()
    s["page_table"] = s["live"][:B * M].view(B, M)
    s["page_refs"] = s["live"][B * M:]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": c}
    op, B, page = c["op"], c["B"], c["page"]
    if op == "compact":
        P = c["P"]
        used = (torch.rand(P, generator=g, device="cuda") < c["used"]).nonzero()[:, 0]
        used = used[torch.randperm(len(used), generator=g, device="cuda")].to(torch.int32)
        M = -(-P // B) + 1
        table = torch.full((B * M,), -1, dtype=torch.int32, device="cuda")
        at = torch.randperm(B * M, generator=g, device="cuda")[:len(used)]
        table[at] = used
        refs = torch.bincount(used, minlength=P).to(torch.int32)
        _kept_state(s, table.view(B, M), refs)
        s["k_pages"], s["v_pages"] = _pools(P, c, g)
        s["page_map"] = torch.empty(P, dtype=torch.int32, device="cuda")
        s["workspace"] = torch.zeros(8192 + 16 * P, dtype=torch.uint8, device="cuda")
        return s
    pos = _positions(c)
    s["positions"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
    M = -(-c["L"] // page)
    if op == "fork":
        table, refs = _table([-(-(p + 1) // page) for p in pos], c["beams"], M, c["spare"], g,
                             private=True)
        _kept_state(s, table, refs)
        r = torch.randint(0, c["beams"], (B,), generator=g, device="cuda")
        lead = torch.arange(B, device="cuda") // c["beams"] * c["beams"]
        s["parents"] = (lead + r).to(torch.int32) if c["order"] else None
        s["kept"] = torch.tensor(_kept(c), dtype=torch.int32, device="cuda") if c["cut"] else None
        s["workspace"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        return s
    s["lengths"] = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda") \
        if c["padded"] else None
    if op == "reserve":
        table, refs = _table([-(-p // page) for p in pos], c["beams"], M, c["spare"], g)
        _kept_state(s, table, refs)
        s["k_pages"], s["v_pages"] = _pools(len(refs), c, g)
        s["taken"] = torch.empty(B, dtype=torch.int32, device="cuda")
        per = -(-(c["S"] - 1) // page) + 1
        s["workspace"] = torch.zeros(8192 + 24 * B + 8 * B * per, dtype=torch.uint8,
                                     device="cuda")
        return s
    S, Hkv, D = c["S"], c["Hkv"], c["D"]
    s["page_table"], refs = _table([-(-(p + n) // page) for p, n in zip(pos, _lengths(c))], 1, M,
                                   3, g)
    s["k_pages"], s["v_pages"] = _pools(len(refs), c, g)
    if op == "append":
        s["k_new"], s["v_new"] = _randn((B, S, Hkv, D), g), _randn((B, S, Hkv, D), g)
        return s
    s["q"] = _randn((B, S, c["Hq"], D), g)
    s["out"] = torch.empty_like(s["q"])
    s["workspace"] = torch.zeros(4096 + 4 * B * Hkv + 400 * S * (c["Hq"] // Hkv) * (D + 4) * 4,
                                 dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------ plain forms --

def _append_plain(s, c):
    B, S, page = c["B"], c["S"], c["page"]
    dev = s["positions"].device
    t = torch.arange(S, device=dev)
    n = s["lengths"][:, None] if c["padded"] else S
    b, t = (t < n).expand(B, S).nonzero(as_tuple=True)
    row = s["positions"].long()[b] + t
    at = s["page_table"].long()[b, row // page]
    s["k_pages"][at, :, row % page] = s["k_new"][b, t]
    s["v_pages"][at, :, row % page] = s["v_new"][b, t]


def _decode_plain(s, c):
    B, S, Hkv, D, page = c["B"], c["S"], c["Hkv"], c["D"], c["page"]
    table = s["page_table"].long().clamp(min=0)
    rows = torch.arange(table.shape[1] * page, device=table.device)
    t = torch.arange(S, device=table.device)
    last = s["positions"].long()[:, None] + t                               # [B, S]
    n = s["lengths"][:, None] if c["padded"] else S
    seen = ((rows <= last[..., None]) & (t < n)[..., None])[:, None, :, None]  # [B, 1, S, 1, rows]
    q = s["q"].float().view(B, S, Hkv, -1, D).permute(0, 2, 1, 3, 4)
    k = s["k_pages"][table].transpose(1, 2).reshape(B, Hkv, -1, D).float()
    x = torch.einsum("bhtgd,bhld->bhtgl", q, k) * D ** -0.5
    del k
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.masked_fill(m == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    del x
    v = s["v_pages"][table].transpose(1, 2).reshape(B, Hkv, -1, D).float()
    out = torch.einsum("bhtgl,bhld->bhtgd", p, v) / total.masked_fill(total == 0, 1.0)
    return out.permute(0, 2, 1, 3, 4).reshape(B, S, -1, D).to(torch.bfloat16)


def _reserve_plain(s, c):
    table, refs, page, S = s["page_table"], s["page_refs"], c["page"], c["S"]
    dev = table.device
    pos = s["positions"].long()
    n = s["lengths"].long() if c["padded"] else torch.full_like(pos, S)
    per = -(-(S - 1) // page) + 1
    j = pos[:, None] // page + torch.arange(per, device=dev)                # [B, per]
    wanted = j * page < (pos + n)[:, None]
    j = j.clamp(max=table.shape[1] - 1)
    b = torch.arange(len(pos), device=dev)[:, None].expand_as(j)
    was = table[b, j].long()
    shared = wanted & (was >= 0) & (refs[was.clamp(min=0)] > 1)
    need = wanted & ((was < 0) | shared)
    need &= (n > 0)[:, None]
    shared &= need
    free = (refs == 0).nonzero()[:, 0]
    ends = need.sum(1).cumsum(0)                                            # pages up to each sequence
    given = ends <= len(free)
    s["taken"].copy_(torch.where(given | ~need.any(1), need.sum(1), -1))
    rank = need.flatten().cumsum(0).view_as(need) - 1
    put = need & given[:, None]
    page_of = free[rank[put]]
    table[b[put], j[put]] = page_of.to(torch.int32)
    refs[page_of] = 1
    left = shared & given[:, None]
    refs -= torch.bincount(was[left], minlength=len(refs)).to(torch.int32)
    # the rows that a shared page holds before the new ones
    first = left[:, 0]
    src, dst = was[first, 0], table[b[first, 0], j[first, 0]].long()
    r = torch.arange(page, device=dev)
    m, r = (r < (pos % page)[first][:, None]).nonzero(as_tuple=True)
    s["k_pages"][dst[m], :, r] = s["k_pages"][src[m], :, r]
    s["v_pages"][dst[m], :, r] = s["v_pages"][src[m], :, r]


def _fork_plain(s, c):
    table, refs = s["page_table"], s["page_refs"]
    new = table.clone()
    if c["order"]:
        p = s["parents"].long()
        new = torch.where((p >= 0)[:, None], table[p.clamp(min=0)], -1)
    if c["cut"]:
        j = torch.arange(table.shape[1], device=table.device)
        new = torch.where(j * c["page"] < s["kept"][:, None], new, -1)
    count = torch.bincount(new[new >= 0], minlength=len(refs)) - \
        torch.bincount(table[table >= 0], minlength=len(refs))
    refs += count.to(torch.int32)
    table.copy_(new)


def _compact_plain(s, c):
    table, refs = s["page_table"], s["page_refs"]
    P = len(refs)
    i = torch.arange(P, device=table.device)
    used = refs > 0
    n = used.sum()
    src = (used & (i >= n)).nonzero()[:, 0]
    dst = (~used & (i < n)).nonzero()[:, 0]
    to = torch.where(used, i, -1)
    to[src] = dst
    s["k_pages"][dst] = s["k_pages"][src]
    s["v_pages"][dst] = s["v_pages"][src]
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, to[table.long().clamp(min=0)], -1))
    s["page_map"].copy_(to)


def _outputs(s):
    op = s["case"]["op"]
    names = {"append": ("k_pages", "v_pages"), "decode": ("out",),
             "reserve": ("page_table", "page_refs", "taken", "k_pages", "v_pages"),
             "fork": ("page_table", "page_refs"),
             "compact": ("page_table", "page_refs", "page_map", "k_pages", "v_pages")}[op]
    return {k: s[k] for k in names}


def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if "live" in s:
        s["live"].copy_(s["first"])
    if not own:
        if op == "decode":
            return {"out": _decode_plain(s, c)}
        {"append": _append_plain, "reserve": _reserve_plain, "fork": _fork_plain,
         "compact": _compact_plain}[op](s, c)
        return _outputs(s)
    import gqa_decode_attention_place_gb300 as ga
    if op == "append":
        ga.attn_paged_append(s["k_new"], s["v_new"], s["positions"], s["page_table"],
                             s["k_pages"], s["v_pages"], lengths=s["lengths"])
    elif op == "decode":
        ga.attn_decode_step_paged(s["q"], s["positions"], s["page_table"], s["k_pages"],
                                  s["v_pages"], c["D"] ** -0.5, lengths=s["lengths"],
                                  out=s["out"], workspace=s["workspace"])
    elif op == "reserve":
        ga.attn_pages_reserve(s["page_table"], s["page_refs"], s["positions"], s["k_pages"],
                              s["v_pages"], c["S"], lengths=s["lengths"], taken=s["taken"],
                              workspace=s["workspace"])
    elif op == "fork":
        ga.attn_pages_fork(s["page_table"], s["page_refs"], c["page"], parents=s["parents"],
                           lengths=s["kept"], workspace=s["workspace"])
    else:
        ga.attn_pages_compact(s["page_table"], s["page_refs"], s["k_pages"], s["v_pages"],
                              page_map=s["page_map"], workspace=s["workspace"])
    return _outputs(s)


# ------------------------------------------------------------------- work --

def work(case):
    c = case
    op, B, page = c["op"], c["B"], c["page"]
    if op == "compact":
        # half of what lies above the used count moves, on average
        pages = c["P"] * c["used"] * (1 - c["used"])
        moved = pages * c["Hkv"] * page * c["D"] * 2
        return {"bytes": 4 * moved + 8 * c["P"] + 8 * c["P"], "flops": c["P"]}
    pos = _positions(c)
    M = -(-c["L"] // page)
    if op == "fork":
        return {"bytes": 4 * B * M + 8 * B, "flops": B * M}
    n = _lengths(c)
    if op == "append":
        return {"bytes": sum(n) * c["Hkv"] * c["D"] * 8 + 8 * B, "flops": sum(n)}
    if op == "decode":
        g = c["Hq"] // c["Hkv"]
        rows = sum(p + k for p, k in zip(pos, n) if k)
        pairs = sum(p + t + 1 for p, k in zip(pos, n) for t in range(k)) * c["Hq"]
        return {"bytes": rows * (c["Hkv"] * c["D"] * 4 + 4 / page) +
                B * c["S"] * c["Hkv"] * g * c["D"] * 4, "flops": 4 * pairs * c["D"]}
    # reserve: the counts, one table entry for each page, the rows of copied pages
    used = sum(-(-p // page) for p in pos[::c["beams"]])
    rows = sum(p % page for p, k in zip(pos, n) if k and p % page) if c["beams"] > 1 else 0
    pages = sum(-(-(p + k) // page) - p // page for p, k in zip(pos, n) if k)
    return {"bytes": 4 * (used + c["spare"]) + 16 * pages + 8 * B + rows * c["Hkv"] * c["D"] * 8,
            "flops": used + c["spare"]}


# ------------------------------------------------------------ 64-bit form --

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op, page = c["op"], c["page"]
    if op == "fork":
        return None
    k, v = s["k_pages"], s["v_pages"]
    table = s["page_table"].cpu().tolist()
    if op == "decode":
        return {"out": _decode64(s, c, table)}
    if op == "append":
        k, v = k.double(), v.double()
        for b, (p, n) in enumerate(zip(_positions(c), _lengths(c))):
            for j in range(p // page, -(-(p + n) // page) if n else 0):
                lo, hi = max(p, j * page), min(p + n, (j + 1) * page)
                at = slice(lo - j * page, hi - j * page)
                k[table[b][j], :, at] = s["k_new"][b, lo - p:hi - p].transpose(0, 1).double()
                v[table[b][j], :, at] = s["v_new"][b, lo - p:hi - p].transpose(0, 1).double()
        return {"k_pages": k, "v_pages": v}
    refs = s["page_refs"].cpu().tolist()
    k, v = k.double(), v.double()
    if op == "compact":
        n = sum(r > 0 for r in refs)
        high = [p for p in range(n, len(refs)) if refs[p] > 0]
        low = [p for p in range(n) if refs[p] == 0]
        if high:
            src, dst = torch.tensor(high, device="cuda"), torch.tensor(low, device="cuda")
            k[dst], v[dst] = k[src], v[src]
        return {"page_table": None, "page_refs": None, "page_map": None, "k_pages": k,
                "v_pages": v}
    free = [p for p in range(len(refs)) if refs[p] == 0]
    copies, at = [], 0
    for b, (p, n) in enumerate(zip(_positions(c), _lengths(c))):
        js = range(p // page, -(-(p + n) // page)) if n else []
        js = [j for j in js if table[b][j] < 0 or refs[table[b][j]] > 1]
        if at + len(js) > len(free):
            break
        if js and js[0] == p // page and table[b][js[0]] >= 0 and p % page:
            copies.append((table[b][js[0]], free[at], p % page))
        at += len(js)
    for src, dst, rows in copies:
        k[dst, :, :rows], v[dst, :, :rows] = k[src, :, :rows], v[src, :, :rows]
    return {"page_table": None, "page_refs": None, "taken": None, "k_pages": k, "v_pages": v}


def _decode64(s, c, table):
    """Sequence by sequence and token by token, over exactly the rows that it sees."""
    page, Hkv, D, g = c["page"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (p, n) in enumerate(zip(_positions(c), _lengths(c))):
        if not n:
            continue
        names = torch.tensor(table[b][:-(-(p + n) // page)], device="cuda")
        k, v = ([x[names, h].reshape(-1, D).double() for h in range(Hkv)]
                for x in (s["k_pages"], s["v_pages"]))
        for h in range(Hkv):
            for t in range(n):
                q = s["q"][b, t, h * g:(h + 1) * g].double()
                x = q @ k[h][:p + t + 1].T / math.sqrt(D)
                w = torch.exp(x - x.max(dim=1, keepdim=True).values)
                out[b, t, h * g:(h + 1) * g] = (w @ v[h][:p + t + 1]) / w.sum(1, keepdim=True)
    return out
