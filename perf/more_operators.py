"""Operators beside the paged KV cache as they are measured: the table of a position rotation, storing
new tokens with their keys and queries rotated on the way, and attention of sequences that share a
prefix.

Each case is one call of one operator on synthetic data.  ``run`` computes it in plain torch
operations, or, with ``own`` set, through this package.

A pool is bf16 [n_pages, kv_heads, page, dim]: page ``table[b, j]`` holds positions j*page ..
j*page+page-1 of sequence b, -1 is no page.  A rotation table is fp32 [positions, rot]: the cosines
of its rot / 2 angles, then their sines; pair i is elements (i, i + rot / 2) of a head, or (2 i, 2 i + 1)
where pairs are interleaved, and elements from rot on are not rotated.  The query at position t
keeps the keys at positions s <= t with s > t - window (window 0: all) or s < sinks.
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # the table of a short context, made when a server starts
        dict(name="table_short", kind="table", positions=4096, rot=64, base=10000.0, scale=1.0),
        # that of 131072 positions, the angles of far positions among them, with a magnitude of its own
        dict(name="table_long", kind="table", positions=131072, rot=128, base=500000.0, scale=1.1386),
        # one new token of one sequence, Mistral-7B heads: the latency of a chat's step
        dict(name="rotate_one", kind="rotate", batch=1, heads=32, kv_heads=8, dim=128, page=16, rot=128,
             interleaved=False, new=1, single=0.0, history=900, mix=1),
        # one decode step of 64 sequences up to 131072 tokens long
        dict(name="rotate_decode", kind="rotate", batch=64, heads=32, kv_heads=8, dim=128, page=64, rot=128,
             interleaved=False, new=1, single=0.0, history=130000, mix=2),
        # a serving step that mixes prompts' chunks with single tokens, small heads of which half turns, pairs
        # side by side
        dict(name="rotate_mixed", kind="rotate", batch=33, heads=12, kv_heads=12, dim=64, page=32, rot=32,
             interleaved=True, new=701, single=0.7, history=9000, mix=3),
        # two long chunks, Gemma-3 heads
        dict(name="rotate_chunks", kind="rotate", batch=2, heads=16, kv_heads=8, dim=256, page=64, rot=256,
             interleaved=False, new=8192, single=0.0, history=24576, mix=4),
        # four answers to one short question: latency
        dict(name="shared_few", kind="shared", groups=1, members=4, heads=32, kv_heads=8, dim=128, page=16, window=0,
             sinks=0, prefix=900, tail=60, new=1, single=0.0, append=False, mix=5),
        # one decode step of 64 sequences that share a system prompt and a document; the new tokens are stored
        # in the same call
        dict(name="shared_decode", kind="shared", groups=1, members=64, heads=32, kv_heads=8, dim=128, page=64,
             window=0, sinks=0, prefix=32768, tail=700, new=1, single=0.0, append=True, mix=6),
        # several prompts, each continued by up to 24 beams, in a layer with the Mistral-7B window and four sinks
        dict(name="shared_window", kind="shared", groups=9, members=24, heads=32, kv_heads=8, dim=128, page=16,
             window=4096, sinks=4, prefix=12000, tail=500, new=1, single=0.0, append=False, mix=7),
        # many small groups, head dim 64
        dict(name="shared_groups", kind="shared", groups=31, members=13, heads=12, kv_heads=12, dim=64, page=32,
             window=0, sinks=0, prefix=6000, tail=300, new=1, single=0.0, append=False, mix=8),
        # drafts of up to eight tokens to be verified, head dim 256
        dict(name="shared_drafts", kind="shared", groups=2, members=32, heads=16, kv_heads=8, dim=256, page=64,
             window=0, sinks=0, prefix=16384, tail=400, new=8, single=0.2, append=True, mix=9),
        # questions of up to 120 tokens about one long document
        dict(name="shared_questions", kind="shared", groups=1, members=48, heads=32, kv_heads=8, dim=128, page=128,
             window=0, sinks=0, prefix=50000, tail=0, new=120, single=0.0, append=True, mix=10),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


_HEADS = [(32, 8, 128), (16, 8, 256), (12, 12, 64), (8, 1, 128), (24, 8, 64), (20, 4, 128)]


def draw(rng):
    mix = rng.randrange(1 << 30)
    kind = rng.choice(["table", "rotate", "rotate", "shared", "shared", "shared"])
    if kind == "table":
        return dict(kind=kind, positions=_spread(rng, 1, 131072), rot=rng.choice([16, 32, 48, 64, 128]),
                    base=rng.choice([10000.0, 500000.0, 1000000.0]), scale=rng.choice([1.0, 1.1386]))
    heads, kv_heads, dim = rng.choice(_HEADS)
    if kind == "rotate":
        new = _spread(rng, 1, 4000) if rng.random() < 0.7 else 1
        batch = _spread(rng, 1, 400)
        while batch * new > 12000:
            batch = max(1, batch // 2)
        return dict(kind=kind, batch=batch, heads=heads, kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128]),
                    rot=rng.choice([dim, dim, dim // 2, 16, 48]), interleaved=rng.random() < 0.4, new=new,
                    single=rng.choice([0.0, 0.5, 0.9]) if new > 1 else 0.0, history=_spread(rng, 1, 60000), mix=mix)
    new = _spread(rng, 2, 100) if rng.random() < 0.4 else 1
    groups, members = _spread(rng, 1, 40), _spread(rng, 1, 70)
    prefix, tail = _spread(rng, 16, 40000), _spread(rng, 1, 1000)
    # (at most about a sixth of the largest listed case's products, and a pool of a few GB)
    while groups * members * new * prefix > 48 * 120 * 50000 // 6:
        groups, members, new = max(1, groups * 2 // 3), max(1, members * 2 // 3), max(1, new * 2 // 3)
    while groups * (prefix + members * (tail + new)) > 400000:
        groups, tail = max(1, groups * 2 // 3), max(1, tail * 2 // 3)
    window = rng.choice([0, 0, 257, 1024, 4096])
    return dict(kind=kind, groups=groups, members=members, heads=heads, kv_heads=kv_heads, dim=dim,
                page=rng.choice([16, 32, 64, 128]), window=window, sinks=rng.choice([0, 1, 4, 37]) if window else 0,
                prefix=prefix, tail=tail, new=new, single=rng.choice([0.0, 0.5]) if new > 1 else 0.0,
                append=rng.random() < 0.5, mix=mix)


# ---------------------------------------------------------------------------------------------
# the lengths of a case: the same for every seed
# ---------------------------------------------------------------------------------------------
def _new_tokens(case, rng):
    if case["new"] == 1 or rng.random() < case["single"]:
        return 1
    return _spread(rng, max(1, case["new"] // 8), case["new"])


def _rows(case):
    """(tokens stored before the call, new tokens) of each sequence of a rotation; the first has the most."""
    rng = random.Random(case["mix"])
    out = [(case["history"], case["new"])]
    for _ in range(case["batch"] - 1):
        out.append((rng.randint(0, case["history"]), _new_tokens(case, rng)))
    return out


def _families(case):
    """For each group the tokens that its sequences share, and (tokens stored, new tokens) of each of them."""
    rng = random.Random(case["mix"])
    out = []
    for g in range(case["groups"]):
        size = case["members"] if g == 0 else _spread(rng, max(1, case["members"] // 4), case["members"])
        prefix = case["prefix"] if g == 0 else rng.randint(case["prefix"] // 3, case["prefix"])
        # an odd length: the prompt's last page is not full, and each sequence has a copy of it
        seqs = [(prefix + rng.randint(0, case["tail"]), _new_tokens(case, rng)) for _ in range(size)]
        out.append((prefix // case["page"] * case["page"], seqs))
    return out


def _kept_entries(case, p0, n):
    """Table entries of one sequence that still have a page (sinks, and what the window reaches)."""
    last = (p0 + n - 1) // case["page"]
    first = max(0, p0 - case["window"] + 1) // case["page"] if case["window"] else 0
    return list(range(0, min(first, -(-case["sinks"] // case["page"])))) + list(range(first, last + 1))


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _starts(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def _frequencies(rot, base, rng):
    """64-bit frequencies; a long context's are stretched by a factor (here one that the seed moves a little)."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    return (base ** (-2.0 * i / rot) / (1.0 + rng.random())).cuda()


def _batch(case, g, seqs):
    """What an attention or an append is given of its new tokens: views of one fused projection's output."""
    H, K = case["heads"], case["kv_heads"]
    start = _starts(n for _, n in seqs)
    qkv = _normal(g, start[-1], H + 2 * K, case["dim"])
    return {"case": case, "q": qkv[:, :H], "k_new": qkv[:, H:H + K], "v_new": qkv[:, H + K:],
            "p0": _i32([p for p, _ in seqs]), "start": _i32(start)}


def prepare(case, seed):
    rng = random.Random(seed)
    g = _gen(seed)
    if case["kind"] == "table":
        return {"case": case, "inv_freq": _frequencies(case["rot"], case["base"], rng)}
    P = case["page"]
    if case["kind"] == "rotate":
        seqs = _rows(case)
        s = _batch(case, g, seqs)
        # the pages of the new tokens and of some tokens before them
        kept = [list(range(max(0, p // P - 2), (p + n - 1) // P + 1)) for p, n in seqs]
        entries = [(i, j) for i, e in enumerate(kept) for j in e]
        n_pages = len(entries) + 3
        table = torch.full((len(seqs), max(j for _, j in entries) + 1), -1, dtype=torch.int32)
        at = torch.tensor(entries)
        table[at[:, 0], at[:, 1]] = torch.tensor(rng.sample(range(n_pages), len(entries)), dtype=torch.int32)
        angle = torch.arange(max(p + n for p, n in seqs), device="cuda").double()[:, None] * \
            _frequencies(case["rot"], 10000.0, rng)
        return {**s, "k_pages": _normal(g, n_pages, case["kv_heads"], P, case["dim"]),
                "v_pages": _normal(g, n_pages, case["kv_heads"], P, case["dim"]), "table": table.cuda(),
                "rope": torch.cat([angle.cos(), angle.sin()], 1).float(),
                "q_out": torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")}
    families = _families(case)
    seqs = [x for _, f in families for x in f]
    s = _batch(case, g, seqs)
    # pages that some sequence of the group keeps, those of the prefix once for all of them
    names, rows, b = {}, [], 0
    for i, (prefix, f) in enumerate(families):
        for p, n in f:
            rows.append([(j, names.setdefault((i, j) if j < prefix // P else (-1 - b, j), len(names)))
                         for j in _kept_entries(case, p, n)])
            b += 1
    n_pages = len(names) + 1 + len(names) // 8
    place = rng.sample(range(n_pages), len(names))  # pages come from all over the pool
    table = torch.full((len(seqs), max(j for r in rows for j, _ in r) + 1), -1, dtype=torch.int32)
    at = torch.tensor([(i, j, place[x]) for i, r in enumerate(rows) for j, x in r])
    table[at[:, 0], at[:, 1]] = at[:, 2].to(torch.int32)
    return {**s, "k_pages": _normal(g, n_pages, case["kv_heads"], P, case["dim"]),
            "v_pages": _normal(g, n_pages, case["kv_heads"], P, case["dim"]), "table": table.cuda(),
            "groups": _i32(_starts(len(f) for _, f in families)),
            # what the host knows of the batch: its longest chunk, and (for the plain form) its lengths
            "most": max(n for _, n in seqs), "families": families}


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"table": _own_table, "rotate": _own_rotate, "shared": _own_shared}[kind](state)
    return {"table": _table, "rotate": _rotate, "shared": _shared}[kind](state)


def _own_table(s):
    import sliding_window_attention_swa_gb300 as swa

    return swa.swa_rope_table(s["inv_freq"], s["case"]["positions"], s["case"]["scale"])


def _own_rotate(s):
    import sliding_window_attention_swa_gb300 as swa

    c = s["case"]
    q = swa.swa_paged_rope_append(s["q"], s["k_pages"], s["v_pages"], s["table"], s["k_new"], s["v_new"], s["p0"],
                                  s["rope"], q_start=None if c["new"] == 1 else s["start"],
                                  interleaved=c["interleaved"], q_out=s["q_out"])
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_shared(s):
    import sliding_window_attention_swa_gb300 as swa

    c = s["case"]
    o, lse, counts = swa.swa_paged_attend_shared(
        s["q"], s["k_pages"], s["v_pages"], s["table"], s["p0"], s["groups"], c["window"], n_sink=c["sinks"],
        q_start=None if c["new"] == 1 else s["start"], max_q=s["most"], k_new=s["k_new"] if c["append"] else None,
        v_new=s["v_new"] if c["append"] else None, want_counts=True)
    out = {"o": o, "lse": lse, "counts": counts}
    return {**out, "k_pages": s["k_pages"], "v_pages": s["v_pages"]} if c["append"] else out


def _table(s):
    c = s["case"]
    # (64 bits: an angle of 131071 radians has an error of a hundredth in 32)
    angle = torch.arange(c["positions"], device="cuda").double()[:, None] * s["inv_freq"]
    return torch.cat([angle.cos() * c["scale"], angle.sin() * c["scale"]], 1).float()


def _places(s):
    """(sequence, position) of every new token."""
    n = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["start"].long(), n, right=True) - 1
    return b, s["p0"].long()[b] + n - s["start"].long()[b]


def _turned(x, cos_sin, interleaved):
    rot = cos_sin.shape[1]
    cos, sin = cos_sin[:, None, :rot // 2], cos_sin[:, None, rot // 2:]
    x = x.to(cos_sin.dtype)
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _store(s, k):
    seq, at = _places(s)
    page, P = s["table"].long()[seq, at // s["case"]["page"]], s["case"]["page"]
    s["k_pages"][page, :, at % P] = k
    s["v_pages"][page, :, at % P] = s["v_new"]


def _rotate(s):
    c = s["case"]
    cos_sin = s["rope"][_places(s)[1]]
    s["q_out"].copy_(_turned(s["q"], cos_sin, c["interleaved"]))
    _store(s, _turned(s["k_new"], cos_sin, c["interleaved"]).to(torch.bfloat16))
    return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _shared(s):
    c = s["case"]
    H, K, D, P, W, ns = c["heads"], c["kv_heads"], c["dim"], c["page"], c["window"], c["sinks"]
    G, N = H // K, s["q"].shape[0]
    if c["append"]:
        _store(s, s["k_new"])
    seq, at = _places(s)
    table = s["table"].long()
    o = torch.empty(N, H, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(N, H, device="cuda")
    counts = torch.empty(N, H, dtype=torch.int32, device="cuda")
    b0 = n0 = 0
    for prefix, f in s["families"]:
        B, R, C = len(f), sum(n for _, n in f), max(n for _, n in f)
        # the prefix, once for the rows of all sequences (the first one's table may lack pages that lie behind its
        # own window: the highest entry is the page)
        keep = torch.arange(prefix, device="cuda")
        page = table[b0:b0 + B].amax(0)[keep // P].clamp(min=0)
        keys, vals = (s[x][page, :, keep % P].float() for x in ("k_pages", "v_pages"))  # [S, K, D]
        q = s["q"][n0:n0 + R].float()
        t = at[n0:n0 + R]
        kept = torch.ones(R, prefix, dtype=torch.bool, device="cuda")
        if W:
            kept = (keep > t[:, None] - W) | (keep < ns)
        x = torch.matmul(q.view(R, K, G, D).permute(1, 2, 0, 3).reshape(K, G * R, D), keys.permute(1, 2, 0))
        x = x.view(K, G, R, prefix).mul_(D ** -0.5).masked_fill_(~kept, -math.inf)
        # each sequence's own tokens, and its rows, padded to the longest
        span = max(p + n for p, n in f) - prefix
        pos = prefix + torch.arange(span, device="cuda")
        page = table[b0:b0 + B][:, (pos // P).clamp(max=table.shape[1] - 1)].clamp(min=0)
        end = torch.tensor([p + n for p, n in f], device="cuda")
        keys2, vals2 = (s[z][page, :, pos % P].float() for z in ("k_pages", "v_pages"))  # [B, S2, K, D]
        vals2 = torch.where((pos < end[:, None])[:, :, None, None], vals2, 0.0)
        first = s["start"][:-1].long()
        i = torch.arange(n0, n0 + R, device="cuda") - first[seq[n0:n0 + R]]
        j = seq[n0:n0 + R] - b0
        q2 = torch.zeros(B, C, H, D, device="cuda")
        q2[j, i] = q
        x2 = torch.matmul(q2.view(B, C, K, G, D).permute(0, 2, 3, 1, 4).reshape(B, K, G * C, D),
                          keys2.permute(0, 2, 3, 1)).view(B, K, G, C, span).mul_(D ** -0.5)
        t2 = torch.zeros(B, C, dtype=torch.long, device="cuda")
        t2[j, i] = t
        kept2 = pos <= t2[:, :, None]
        if W:
            kept2 &= (pos > t2[:, :, None] - W) | (pos < ns)
        x2.masked_fill_(~kept2[:, None, None], -math.inf)
        # one softmax over both
        m = x2.amax(-1)[j, :, :, i].permute(1, 2, 0)  # [K, G, R]
        if prefix:
            m = torch.maximum(m, x.amax(-1))
        x.sub_(m[..., None]).exp_()
        m2 = torch.zeros(B, K, G, C, device="cuda")
        m2[j, :, :, i] = m.permute(2, 0, 1)
        x2.sub_(m2[..., None]).exp_()
        total = x.sum(-1) + x2.sum(-1)[j, :, :, i].permute(1, 2, 0)
        y = torch.matmul(x.view(K, G * R, prefix), vals.permute(1, 0, 2)).view(K, G, R, D)
        y2 = torch.matmul(x2.view(B, K, G * C, span), vals2.permute(0, 2, 1, 3)).view(B, K, G, C, D)
        y = (y + y2[j, :, :, i].permute(1, 2, 0, 3)) / total[..., None]
        o[n0:n0 + R] = y.permute(2, 0, 1, 3).reshape(R, H, D).to(torch.bfloat16)
        lse[n0:n0 + R] = (m + total.log()).permute(2, 0, 1).reshape(R, H)
        counts[n0:n0 + R] = (kept.sum(-1) + kept2.sum(-1)[j, i])[:, None].to(torch.int32)
        b0, n0 = b0 + B, n0 + R
    out = {"o": o, "lse": lse, "counts": counts}
    return {**out, "k_pages": s["k_pages"], "v_pages": s["v_pages"]} if c["append"] else out


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without, and its result in 64 bits
# ---------------------------------------------------------------------------------------------
def work(case):
    if case["kind"] == "table":
        return {"bytes": 4 * case["positions"] * case["rot"] + 4 * case["rot"],
                "flops": 2 * case["positions"] * case["rot"]}
    H, K, D = case["heads"], case["kv_heads"], case["dim"]
    if case["kind"] == "rotate":
        seqs = _rows(case)
        n = sum(x for _, x in seqs)
        places = len({t for p, x in seqs for t in range(p, p + x)})  # table rows, each once
        return {"bytes": n * (H + 2 * K) * D * 4 + places * case["rot"] * 4 + 8 * len(seqs),
                "flops": 3 * n * (H + K) * case["rot"]}
    W, ns = case["window"], case["sinks"]
    read = pairs = new = entries = 0
    for prefix, f in _families(case):
        low = prefix  # the first position of the prefix that a window of the group reaches
        for p, n in f:
            lo = max(0, p - W + 1) if W else 0
            low = min(low, lo)
            read += p + n - max(lo, prefix) + max(0, min(ns, lo) - prefix)
            pairs += sum(min(t + 1, W) + min(max(0, t - W + 1), ns) if W else t + 1 for t in range(p, p + n))
            entries += len(_kept_entries(case, p, n))
            new += n
        read += prefix - low + min(ns, low)
    moved = new * K * D * 2 * 2 * (1 if case["append"] else 0)
    return {"bytes": read * K * D * 2 * 2 + moved + new * H * (D * 2 * 2 + 8) + 4 * entries, "flops": 4 * D * H * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "table":
        p, f = torch.arange(case["positions"], dtype=torch.float64, device="cuda"), s["inv_freq"]
        return torch.cat([torch.cos(torch.outer(p, f)), torch.sin(torch.outer(p, f))], 1) * case["scale"]
    H, K, D, P, W, ns = (case[x] if x in case else 0 for x in ("heads", "kv_heads", "dim", "page", "window", "sinks"))
    if case["kind"] == "rotate":
        # every pair (x, y) as the complex number x + iy, turned by cos + i sin
        half = case["rot"] // 2
        q, k, v = s["q"].double(), s["k_new"].double(), s["v_new"].double()
        k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
        n0 = 0
        for b, (p, n) in enumerate(_rows(case)):
            turn = torch.complex(s["rope"][p:p + n, :half].double(), s["rope"][p:p + n, half:].double())[:, None]
            for x in (q, k):
                part = x[n0:n0 + n, :, :2 * half]
                if case["interleaved"]:
                    z = torch.view_as_complex(part.reshape(n, -1, half, 2).contiguous()) * turn
                    x[n0:n0 + n, :, :2 * half] = torch.view_as_real(z).reshape(n, -1, 2 * half)
                else:
                    z = torch.complex(part[..., :half], part[..., half:]) * turn
                    x[n0:n0 + n, :, :2 * half] = torch.cat([z.real, z.imag], -1)
            for t in range(p - p % P, p + n, P):  # page by page
                i, j = max(t, p), min(t + P, p + n)
                page = int(s["table"][b, t // P])
                k_pages[page, :, i - t:j - t] = k[n0 + i - p:n0 + j - p].transpose(0, 1)
                v_pages[page, :, i - t:j - t] = v[n0 + i - p:n0 + j - p].transpose(0, 1)
            n0 += n
        return {"q": q, "k_pages": k_pages, "v_pages": v_pages}
    # the attention of each sequence by itself, from its definition
    q, kn, vn = (s[x].double() for x in ("q", "k_new", "v_new"))
    o = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
    n0 = b = 0
    for _, f in s["families"]:
        for p, n in f:
            lo = max(0, p - W + 1) if W else 0
            where = torch.cat([torch.arange(min(ns, lo)), torch.arange(lo, p + n)]).cuda()
            page, row = s["table"][b].long()[where // P], where % P
            k, v = s["k_pages"][page, :, row].double(), s["v_pages"][page, :, row].double()
            if case["append"]:  # the last n positions are the call's own rows
                k[-n:], v[-n:] = kn[n0:n0 + n], vn[n0:n0 + n]
            t = torch.arange(p, p + n, device="cuda")[:, None]
            ok = where <= t
            if W:
                ok &= (t - where < W) | (where < ns)
            for h in range(K):
                heads = slice(h * (H // K), (h + 1) * (H // K))
                dots = torch.einsum("ngd,sd->gns", q[n0:n0 + n, heads], k[:, h]) / math.sqrt(D)
                dots.masked_fill_(~ok, -math.inf)
                lse[n0:n0 + n, heads] = torch.logsumexp(dots, 2).T
                o[n0:n0 + n, heads] = torch.einsum("gns,sd->ngd", torch.softmax(dots, 2), v[:, h])
            n0, b = n0 + n, b + 1
    return {"o": o, "lse": lse, "counts": None, **({"k_pages": None, "v_pages": None} if case["append"] else {})}
