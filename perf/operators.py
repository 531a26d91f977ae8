"""The paged KV cache's operators as they are measured: attention of new tokens over a paged cache
(one token a sequence, a chunk, or a ragged batch of both), forking sequences, compacting the pool
and freeing pages.

Each case is one call of one operator on synthetic data.  ``run`` computes it in plain torch
operations, or, with ``own`` set, through this package.

A pool is bf16 [n_pages, kv_heads, page, dim] ([layers, ...] where pages are moved): page
``table[b, j]`` holds positions j*page .. j*page+page-1 of sequence b, -1 is no page.  The query at
position t keeps the keys at positions s <= t with s > t - window (window 0: all) or s < sinks.
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
        # one sequence, one new token, a short history: the latency of a chat's first answers
        dict(name="decode_one", kind="attend", batch=1, heads=32, kv_heads=8, dim=128, page=16, window=4096, sinks=0,
             new=1, single=0.0, history=900, append=False, mix=1),
        # one decode step of 64 sequences up to 131072 tokens long with the Mistral-7B window, the
        # new token's keys and values stored in the same call
        dict(name="decode_batch", kind="attend", batch=64, heads=32, kv_heads=8, dim=128, page=64, window=4096,
             sinks=0, new=1, single=0.0, history=131071, append=True, mix=2),
        # a 512-token chunk of one long prompt, Mistral-7B heads and window, stored in the same call
        dict(name="chunk_one", kind="attend", batch=1, heads=32, kv_heads=8, dim=128, page=16, window=4096, sinks=0,
             new=512, single=0.0, history=12345, append=True, mix=3),
        # a serving step that mixes prompts' chunks with single tokens, small heads, four sinks
        dict(name="step_mixed", kind="attend", batch=33, heads=12, kv_heads=12, dim=64, page=32, window=1024, sinks=4,
             new=701, single=0.7, history=9000, append=True, mix=4),
        # Gemma-3 local layers: two long chunks, head dim 256, window 1024
        dict(name="chunk_wide_heads", kind="attend", batch=2, heads=16, kv_heads=8, dim=256, page=64, window=1024,
             sinks=0, new=8192, single=0.0, history=24576, append=False, mix=5),
        # chunks over the whole of a long history (a layer without a window): the largest products
        dict(name="chunk_full", kind="attend", batch=2, heads=32, kv_heads=8, dim=128, page=128, window=0, sinks=0,
             new=2048, single=0.0, history=30000, append=False, mix=6),
        # one reorder of a beam search of 32 beams
        dict(name="fork_beams", kind="fork", rows=32, layers=4, kv_heads=8, dim=128, page=16, length=4000, parents=11,
             mix=7),
        # 48 prompts, each continued by several samples
        dict(name="fork_samples", kind="fork", rows=400, layers=4, kv_heads=8, dim=256, page=64, length=2000,
             parents=48, mix=8),
        # a small pool whose live pages move to its low end
        dict(name="compact_small", kind="compact", rows=24, layers=2, kv_heads=8, dim=128, page=16, pages=700,
             live=0.55, mix=9),
        # the same for a pool of gigabytes
        dict(name="compact_large", kind="compact", rows=200, layers=4, kv_heads=8, dim=128, page=64, pages=4001,
             live=0.5, mix=10),
        # pages behind the window of a few sequences go back to the pool
        dict(name="free_window_small", kind="free", rows=16, width=256, page=16, window=1024, sinks=4, mix=11),
        # the same for 1024 sequences of up to 65536 tokens, some of which have ended
        dict(name="free_window_large", kind="free", rows=1024, width=4096, page=16, window=4096, sinks=0, mix=12),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    mix = rng.randrange(1 << 30)
    kind = rng.choice(["attend", "attend", "attend", "fork", "compact", "free"])
    if kind == "attend":
        heads, kv_heads, dim = rng.choice([(32, 8, 128), (16, 8, 256), (12, 12, 64), (8, 1, 128), (24, 8, 64), (20, 4, 128)])
        new = _spread(rng, 1, 2000) if rng.random() < 0.6 else 1
        batch = _spread(rng, 1, 64)
        while batch * new > 4096:
            batch = max(1, batch // 2)
        window = rng.choice([0, 257, 1000, 1024, 4096])
        history = _spread(rng, 1, 131071 if window else 30000)
        if not window:
            while batch * new * history > 2 * 2048 * 30000 or batch * history > 400000:
                batch, history = max(1, batch // 2), max(1, history * 2 // 3)
        return dict(kind=kind, batch=batch, heads=heads, kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128]),
                    window=window, sinks=rng.choice([0, 0, 1, 4, 37]) if window else 0, new=new,
                    single=rng.choice([0.0, 0.5, 0.9]) if new > 1 else 0.0, history=history,
                    append=rng.random() < 0.5, mix=mix)
    if kind == "fork":
        rows = _spread(rng, 2, 256)
        return dict(kind=kind, rows=rows, layers=rng.randint(1, 4), kv_heads=rng.choice([1, 8, 12]),
                    dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]), length=_spread(rng, 1, 3000),
                    parents=rng.randint(1, rows), mix=mix)
    if kind == "compact":
        return dict(kind=kind, rows=_spread(rng, 1, 200), layers=rng.randint(1, 4), kv_heads=rng.choice([1, 8, 12]),
                    dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64]), pages=_spread(rng, 20, 3001),
                    live=rng.uniform(0.05, 0.95), mix=mix)
    return dict(kind=kind, rows=_spread(rng, 1, 1000), width=_spread(rng, 1, 4000), page=rng.choice([16, 32, 64, 128]),
                window=rng.choice([257, 1024, 4096]), sinks=rng.choice([0, 4, 37]), mix=mix)


# ---------------------------------------------------------------------------------------------
# the lengths and tables of a case: the same for every seed but for which page holds what
# ---------------------------------------------------------------------------------------------
def _lengths(case):
    """(tokens stored before the call, new tokens) of each sequence; the first has the most."""
    rng = random.Random(case["mix"])
    out = [(case["history"], case["new"])]
    for _ in range(case["batch"] - 1):
        if case["new"] == 1:  # a decode batch: lengths anywhere up to the longest
            out.append((rng.randint(0, case["history"]), 1))
        else:
            n = 1 if rng.random() < case["single"] else _spread(rng, max(1, case["new"] // 8), case["new"])
            out.append((rng.randint(case["history"] // 3, case["history"]), n))
    return out


def _kept_entries(case, p0, n):
    """Table entries of one sequence that still have a page (sinks, and what the window reaches)."""
    last = (p0 + n - 1) // case["page"]
    first = max(0, p0 - case["window"] + 1) // case["page"] if case["window"] else 0
    sink = range(0, min(first, -(-case["sinks"] // case["page"])))
    return list(sink) + list(range(first, last + 1))


def _row_lengths(case):
    """Tokens of each row of a fork."""
    rng = random.Random(case["mix"])
    return [rng.randint(max(1, case["length"] // 2), case["length"]) for _ in range(case["rows"])]


def _sources(case):
    """The row that each row of a fork continues (-1: the row ends)."""
    rng = random.Random(case["mix"] + 1)
    parents = rng.sample(range(case["rows"]), case["parents"])
    return [-1 if rng.random() < 0.03 else rng.choice(parents) for _ in range(case["rows"])]


def _freed(case):
    """Tokens of each row, and the position below which its pages are given up (-1: the row ends)."""
    rng = random.Random(case["mix"])
    span = case["width"] * case["page"]
    lens = [rng.randint(1, span) for _ in range(case["rows"])]
    lens[0] = span
    return lens, [-1 if rng.random() < 0.1 else max(0, n - case["window"] + 1) for n in lens]


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


def prepare(case, seed):
    rng = random.Random(seed)
    g = _gen(seed)
    if case["kind"] == "attend":
        seqs = _lengths(case)
        width = max(-(-(p + n) // case["page"]) for p, n in seqs)
        kept = [_kept_entries(case, p, n) for p, n in seqs]
        n_pages = sum(map(len, kept)) + 1 + sum(map(len, kept)) // 8
        pages = rng.sample(range(n_pages), sum(map(len, kept)))  # pages come from all over the pool
        table = torch.full((len(seqs), width), -1, dtype=torch.int32)
        b = torch.tensor([i for i, e in enumerate(kept) for _ in e])
        table[b, torch.tensor([j for e in kept for j in e])] = torch.tensor(pages, dtype=torch.int32)
        start = [0]
        for _, n in seqs:
            start.append(start[-1] + n)
        # the heads of one fused projection's output: views with its row stride
        qkv = _normal(g, start[-1], case["heads"] + 2 * case["kv_heads"], case["dim"])
        H, K = case["heads"], case["kv_heads"]
        return {"case": case, "q": qkv[:, :H], "k_new": qkv[:, H:H + K], "v_new": qkv[:, H + K:],
                "k_pages": _normal(g, n_pages, K, case["page"], case["dim"]),
                "v_pages": _normal(g, n_pages, K, case["page"], case["dim"]), "table": table.cuda(),
                "p0": _i32([p for p, _ in seqs]), "start": _i32(start),
                # what the host knows of the batch: its longest chunk and farthest position
                "most": max(n for _, n in seqs), "end": max(p + n for p, n in seqs)}
    if case["kind"] == "fork":
        lens, src = _row_lengths(case), _sources(case)
        need = [-(-n // case["page"]) for n in lens]
        width = max(need)
        n_pages = sum(need) + case["rows"] + 7
        pages = rng.sample(range(n_pages), sum(need))
        table = torch.full((case["rows"], width), -1, dtype=torch.int32)
        b = torch.tensor([i for i, n in enumerate(need) for _ in range(n)])
        table[b, torch.tensor([j for n in need for j in range(n)])] = torch.tensor(pages, dtype=torch.int32)
        ref = torch.zeros(n_pages, dtype=torch.int32)
        ref[torch.tensor(pages)] = 1
        shape = (case["layers"], n_pages, case["kv_heads"], case["page"], case["dim"])
        return {"case": case, "k_pages": _normal(g, *shape), "v_pages": _normal(g, *shape), "table": table.cuda(),
                "ref": ref.cuda(), "src": _i32(src), "lens": _i32(lens),
                "out_table": torch.empty(case["rows"], width, dtype=torch.int32, device="cuda"),
                "out_ref": torch.empty(n_pages, dtype=torch.int32, device="cuda")}
    if case["kind"] == "compact":
        n = case["pages"]
        live = rng.sample(range(n), max(1, int(n * case["live"])))
        # rows of about the same length; a tenth of the entries are pages that another row has too
        width = max(1, -(-len(live) // case["rows"])) + 2
        table = torch.full((case["rows"], width), -1, dtype=torch.int64)
        at = torch.arange(len(live))
        table[at % case["rows"], torch.div(at, case["rows"], rounding_mode="floor")] = torch.tensor(live)
        for b in range(1, case["rows"], 5):
            table[b, 0] = table[b - 1, 0]
        ref = torch.bincount(table[table >= 0], minlength=n).to(torch.int32)
        shape = (case["layers"], n, case["kv_heads"], case["page"], case["dim"])
        return {"case": case, "k_pages": _normal(g, *shape), "v_pages": _normal(g, *shape),
                "table": table.to(torch.int32).cuda(), "ref": ref.cuda(),
                "out_table": torch.empty(case["rows"], width, dtype=torch.int32, device="cuda"),
                "out_ref": torch.empty(n, dtype=torch.int32, device="cuda")}
    lens, below = _freed(case)
    need = torch.tensor([-(-x // case["page"]) for x in lens])
    total = int(need.sum())
    n_pages = total + 5
    # a third of the pages of the first half of the rows are shared with a neighbour
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed))[:total].to(torch.int32)
    j = torch.arange(case["width"])
    used = j[None, :] < need[:, None]
    table = torch.full((case["rows"], case["width"]), -1, dtype=torch.int32)
    table[used] = perm
    half = case["rows"] // 2 // 2 * 2
    both = used[0:half:2] & used[1:half:2] & (j % 3 == 0)
    table[1:half:2][both] = table[0:half:2][both]
    ref = torch.bincount(table[table >= 0].long(), minlength=n_pages).to(torch.int32)
    return {"case": case, "table": table.cuda(), "ref": ref.cuda(), "below": _i32(below),
            "out_table": torch.empty_like(table, device="cuda"), "out_ref": torch.empty_like(ref, device="cuda")}


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"attend": _own_attend, "fork": _own_fork, "compact": _own_compact, "free": _own_free}[kind](state)
    return {"attend": _attend, "fork": _fork, "compact": _compact, "free": _free}[kind](state)


def _own_attend(s):
    import sliding_window_attention_swa_gb300 as swa

    c = s["case"]
    o, lse, counts = swa.swa_paged_attend(
        s["q"], s["k_pages"], s["v_pages"], s["table"], s["p0"], c["window"], n_sink=c["sinks"],
        q_start=None if c["new"] == 1 else s["start"], max_q=s["most"], k_new=s["k_new"] if c["append"] else None,
        v_new=s["v_new"] if c["append"] else None, want_counts=True)
    out = {"o": o, "lse": lse, "counts": counts}
    return {**out, "k_pages": s["k_pages"], "v_pages": s["v_pages"]} if c["append"] else out


def _own_fork(s):
    import sliding_window_attention_swa_gb300 as swa

    table, ref = swa.swa_pages_fork(s["k_pages"], s["v_pages"], s["table"], s["ref"], s["src"], s["lens"],
                                    out_table=s["out_table"], out_ref=s["out_ref"])
    return {"table": table, "ref": ref, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_compact(s):
    import sliding_window_attention_swa_gb300 as swa

    table, ref, n_live = swa.swa_pages_compact(s["k_pages"], s["v_pages"], s["table"], s["ref"],
                                               out_table=s["out_table"], out_ref=s["out_ref"])
    return {"table": table, "ref": ref, "n_live": n_live, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_free(s):
    import sliding_window_attention_swa_gb300 as swa

    table, ref = swa.swa_pages_free(s["table"], s["ref"], s["below"], s["case"]["page"], n_sink=s["case"]["sinks"],
                                    out_table=s["out_table"], out_ref=s["out_ref"])
    return {"table": table, "ref": ref}


def _places(s):
    """(sequence, position) of every new token."""
    n = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["start"].long(), n, right=True) - 1
    return b, s["p0"].long()[b] + n - s["start"].long()[b]


def _attend(s):
    c = s["case"]
    H, K, D, P, W, ns = c["heads"], c["kv_heads"], c["dim"], c["page"], c["window"], c["sinks"]
    G, N, B, C = H // K, s["q"].shape[0], s["table"].shape[0], s["most"]
    seq, at = _places(s)
    table, p0 = s["table"].long(), s["p0"].long()
    new = (s["start"][1:] - s["start"][:-1]).long()
    if c["append"]:
        page = table[seq, at // P]
        s["k_pages"][page, :, at % P] = s["k_new"]
        s["v_pages"][page, :, at % P] = s["v_new"]
    # the key positions that a sequence's new tokens can reach: the sinks, then the window's
    lo = (p0 - (W - 1)).clamp(min=0) if W else torch.zeros_like(p0)
    span = min(s["end"], W - 1 + C) if W else s["end"]
    band = lo[:, None] + torch.arange(span, device="cuda")
    pos = torch.cat([torch.arange(ns, device="cuda").expand(B, ns), band], 1)
    there = pos < (p0 + new)[:, None]
    there[:, ns:] &= band >= ns
    page = table.gather(1, (pos // P).clamp(max=table.shape[1] - 1)).clamp(min=0)
    keys = s["k_pages"][page, :, pos % P].float()  # [B, S, K, D]
    vals = torch.where(there[:, :, None, None], s["v_pages"][page, :, pos % P].float(), 0.0)
    q = torch.zeros(B, C, H, D, device="cuda")
    first = s["start"][:-1].long()
    q[seq, torch.arange(N, device="cuda") - first[seq]] = s["q"].float()
    t = p0[:, None] + torch.arange(C, device="cuda")
    kept = there[:, None, :] & (pos[:, None, :] <= t[:, :, None])
    if W:
        kept &= (pos[:, None, :] > t[:, :, None] - W) | (pos[:, None, :] < ns)
    x = torch.matmul(q.view(B, C, K, G, D).permute(0, 2, 3, 1, 4).reshape(B, K, G * C, D), keys.permute(0, 2, 3, 1))
    x = x.view(B, K, G, C, -1).mul_(D ** -0.5)
    x.masked_fill_(~kept[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, K, G * C, -1), vals.permute(0, 2, 1, 3)).view(B, K, G, C, D) / total
    lse = (m + total.log()).squeeze(-1)
    i = torch.arange(N, device="cuda") - first[seq]
    out = {"o": o.permute(0, 3, 1, 2, 4).reshape(B, C, H, D)[seq, i].to(torch.bfloat16),
           "lse": lse.permute(0, 3, 1, 2).reshape(B, C, H)[seq, i].contiguous(),
           "counts": kept.sum(-1)[seq, i][:, None].expand(N, H).to(torch.int32)}
    return {**out, "k_pages": s["k_pages"], "v_pages": s["v_pages"]} if c["append"] else out


def _lowest_free(ref, n):
    """The n free pages of lowest index (the pool has as many)."""
    free = ref == 0
    rank = torch.cumsum(free, 0) - 1
    n_pages = ref.shape[0]
    slot = torch.where(free & (rank < n), rank, n)
    return torch.full((n + 1,), -1, device="cuda").scatter_(0, slot, torch.arange(n_pages, device="cuda"))[:n]


def _histogram(entries, n_pages):
    e = entries.reshape(-1)
    return torch.zeros(n_pages + 1, dtype=torch.int32, device="cuda").index_add_(
        0, torch.where(e >= 0, e, n_pages), torch.ones_like(e, dtype=torch.int32))[:n_pages]


def _fork(s):
    c, P = s["case"], s["case"]["page"]
    table, src, n_pages = s["table"].long(), s["src"].long(), s["ref"].shape[0]
    rows, width = table.shape
    j, i = torch.arange(width, device="cuda"), torch.arange(rows, device="cuda")
    lens = torch.where(src >= 0, s["lens"].long()[src.clamp(min=0)], 0)
    out = torch.where((src >= 0)[:, None] & (j < ((lens + P - 1) // P)[:, None]), table[src.clamp(min=0)], -1)
    # of the rows that continue one row, the first keeps its last page if that is not full
    first = torch.full((rows + 1,), rows, device="cuda").scatter_reduce_(0, torch.where(src >= 0, src, rows), i, "amin")
    part = lens % P
    copy = (src >= 0) & (part > 0) & (first[src.clamp(min=0)] != i)
    last = (lens // P).clamp(max=width - 1)
    old = out.gather(1, last[:, None])[:, 0]
    out = torch.where(copy[:, None] & (j == last[:, None]), -1, out)
    ref = s["ref"] - _histogram(table, n_pages) + _histogram(out, n_pages)
    rank = torch.cumsum(copy, 0) - 1
    fresh = _lowest_free(ref, rows)[rank.clamp(min=0)]
    out = torch.where(copy[:, None] & (j == last[:, None]), fresh[:, None], out)
    ref = ref + _histogram(torch.where(copy, fresh, -1), n_pages)
    # the rows that the parent has of its last page, in every layer
    i = copy.nonzero()[:, 0]
    rows_kept = (torch.arange(P, device="cuda") < part[i, None])[:, None, :, None]
    for pool in (s["k_pages"], s["v_pages"]):
        pool[:, fresh[i]] = torch.where(rows_kept, pool[:, old[i]], pool[:, fresh[i]])
    s["out_table"].copy_(out)
    s["out_ref"].copy_(ref)
    return {"table": s["out_table"], "ref": s["out_ref"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _compact(s):
    table, ref, n = s["table"].long(), s["ref"], s["ref"].shape[0]
    p = torch.arange(n, device="cuda")
    live = ref > 0
    count = live.sum()
    hole, mover = ~live & (p < count), live & (p >= count)
    # the k-th hole takes the k-th page above the count
    hole_rank, mover_rank = torch.cumsum(hole, 0) - 1, torch.cumsum(mover, 0) - 1
    at = torch.full((n + 1,), n, device="cuda").scatter_(0, torch.where(hole, hole_rank, n), p)
    to = torch.where(mover, at[mover_rank.clamp(min=0)], p)
    i = mover.nonzero()[:, 0]
    for pool in (s["k_pages"], s["v_pages"]):
        pool[:, to[i]] = pool[:, i]
    s["out_table"].copy_(torch.where(table >= 0, to[table.clamp(min=0)], -1))
    s["out_ref"].copy_(torch.where(p < count, ref, 0).scatter_(0, to[i], ref[i]))
    return {"table": s["out_table"], "ref": s["out_ref"], "n_live": count.to(torch.int32).reshape(1),
            "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _free(s):
    c, table = s["case"], s["table"].long()
    j = torch.arange(table.shape[1], device="cuda")
    below = s["below"].long()[:, None]
    gone = (below < 0) | (((j + 1) * c["page"] <= below) & (j * c["page"] >= c["sinks"]))
    gone &= table >= 0
    s["out_ref"].copy_(s["ref"] - _histogram(torch.where(gone, table, -1), s["ref"].shape[0]))
    s["out_table"].copy_(torch.where(gone, -1, table))
    return {"table": s["out_table"], "ref": s["out_ref"]}


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without, and its result in 64 bits
# ---------------------------------------------------------------------------------------------
def work(case):
    if case["kind"] == "attend":
        H, K, D, W = case["heads"], case["kv_heads"], case["dim"], case["window"]
        pairs = read = new = entries = 0
        for p, n in _lengths(case):
            lo = max(0, p - W + 1) if W else 0
            sinks = min(case["sinks"], lo)
            new += n
            read += p + n - lo + sinks
            entries += len(_kept_entries(case, p, n))
            full = sum(min(t + 1, W) if W else t + 1 for t in range(p, p + n))
            pairs += full + sum(max(0, min(case["sinks"], t - W + 1)) if W else 0 for t in range(p, p + n))
        # with the new rows stored in the same call they are read from the call's arguments and written once
        moved = new * K * D * 2 * 2 * (1 if case["append"] else 0)
        return {"bytes": read * K * D * 2 * 2 + moved + new * H * (D * 2 * 2 + 8) + entries * 4 + 8 * case["batch"],
                "flops": 4 * D * H * pairs}
    row = case.get("kv_heads", 0) * case.get("dim", 0) * 2 * 2 * case.get("layers", 0)  # one position of both pools
    if case["kind"] == "fork":
        lens, src = _row_lengths(case), _sources(case)
        seen, copied, pages = set(), 0, sum(-(-n // case["page"]) for n in lens)
        read = {}
        for s in src:
            if s >= 0 and s in seen:
                copied += lens[s] % case["page"]
                read[s] = lens[s] % case["page"]
            seen.add(s)
        table = case["rows"] * max(-(-n // case["page"]) for n in lens) * 4 * 2
        return {"bytes": (copied + sum(read.values())) * row + table + (pages + case["rows"] + 7) * 4 * 2 + 8 * case["rows"],
                "flops": 0}
    if case["kind"] == "compact":
        n, live = case["pages"], max(1, int(case["pages"] * case["live"]))
        moved = live * (n - live) // n  # of live pages placed at random, as many lie above the count
        width = max(1, -(-live // case["rows"])) + 2
        return {"bytes": 2 * moved * case["page"] * row + case["rows"] * width * 4 * 2 + n * 4 * 2, "flops": 0}
    lens, _ = _freed(case)
    pages = sum(-(-x // case["page"]) for x in lens) + 5
    return {"bytes": case["rows"] * case["width"] * 4 * 2 + pages * 4 * 2 + 4 * case["rows"], "flops": 0}


def exact(case, seed):
    """The attention of each sequence from its definition, in 64 bits (the other operators move values and count)."""
    if case["kind"] != "attend":
        return None
    s = prepare(case, seed)
    H, K, D, P, W, ns = case["heads"], case["kv_heads"], case["dim"], case["page"], case["window"], case["sinks"]
    q, kn, vn = (s[x].double() for x in ("q", "k_new", "v_new"))
    o = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
    n0 = 0
    for b, (p, n) in enumerate(_lengths(case)):
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
        for h in range(H):
            dots = (q[n0:n0 + n, h] @ k[:, h // (H // K)].T) / math.sqrt(D)
            dots[~ok] = -math.inf
            lse[n0:n0 + n, h] = torch.logsumexp(dots, 1)
            o[n0:n0 + n, h] = torch.softmax(dots, 1) @ v[:, h // (H // K)]
        n0 += n
    return {"o": o, "lse": lse, "counts": None, **({"k_pages": None, "v_pages": None} if case["append"] else {})}
