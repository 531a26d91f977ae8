"""Plain 64-bit reference of the paged cache's operators, and batches to run them on.

``attend`` computes one sequence's new tokens from the definition; the page operations are
modelled on Python lists, one page at a time.
"""
from __future__ import annotations

import math

import numpy as np
import torch


class Batch:
    """A paged batch on the host: seqs = [(tokens stored before, new tokens), ...].

    The pool's pages are dealt at random; whatever no token lies in holds `junk` (NaN unless
    given).  freed: pages behind the window (and not holding sinks) are given up.  lead, tail:
    rows of q before the first and behind the last sequence.
    """

    def __init__(self, seed, seqs, Hq, Hkv, D, ps, window=0, n_sink=0, junk=float("nan"), freed=True, lead=0, tail=0,
                 width=None, spare=3):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.Hq, self.Hkv, self.D, self.ps, self.window, self.n_sink = seqs, Hq, Hkv, D, ps, window, n_sink
        ends = [p + n for p, n in seqs]
        self.width = width or max(1, max(-(-e // ps) for e in ends))
        entries = []
        for b, (p, n) in enumerate(seqs):
            for j in range(-(-(p + n) // ps)):
                lo = max(0, p - window + 1) if window else 0
                if freed and (j + 1) * ps <= lo and j * ps >= n_sink:
                    continue
                entries.append((b, j))
        self.n_pages = len(entries) + spare
        perm = torch.randperm(self.n_pages, generator=g)[:len(entries)].tolist()
        self.table = torch.full((len(seqs), self.width), -1, dtype=torch.int32)
        for (b, j), page in zip(entries, perm):
            self.table[b, j] = page
        starts = [lead]
        for _, n in seqs:
            starts.append(starts[-1] + n)
        self.N = starts[-1] + tail
        self.q_start = torch.tensor(starts, dtype=torch.int32)
        self.p0 = torch.tensor([p for p, _ in seqs], dtype=torch.int32)
        rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
        self.q = rnd(self.N, Hq, D)
        self.keys = [rnd(e, Hkv, D) for e in ends]
        self.vals = [rnd(e, Hkv, D) for e in ends]
        self.k_pages = torch.full((self.n_pages, Hkv, ps, D), junk, dtype=torch.bfloat16)
        self.v_pages = self.k_pages.clone()
        for (b, j), page in zip(entries, perm):
            n = min(ps, ends[b] - j * ps)
            self.k_pages[page, :, :n] = self.keys[b][j * ps:j * ps + n].transpose(0, 1)
            self.v_pages[page, :, :n] = self.vals[b][j * ps:j * ps + n].transpose(0, 1)
        self.k_new = torch.full((self.N, Hkv, D), float("nan"), dtype=torch.bfloat16)
        self.v_new = self.k_new.clone()
        for b, (p, n) in enumerate(seqs):
            self.k_new[starts[b]:starts[b] + n] = self.keys[b][p:]
            self.v_new[starts[b]:starts[b] + n] = self.vals[b][p:]

    def without_new(self):
        """The pools before the new tokens are stored (their rows hold junk)."""
        k, v = self.k_pages.clone(), self.v_pages.clone()
        for b, (p, n) in enumerate(self.seqs):
            for t in range(p, p + n):
                page = int(self.table[b, t // self.ps])
                k[page, :, t % self.ps] = float("nan")
                v[page, :, t % self.ps] = float("nan")
        return k, v

    def rows(self):
        """(sequence, first row, rows) of every sequence with new tokens."""
        return [(b, int(self.q_start[b]), n) for b, (_, n) in enumerate(self.seqs) if n]

    def reference(self, b):
        p, n = self.seqs[b]
        q0 = int(self.q_start[b])
        args = self.q[q0:q0 + n], self.keys[b], self.vals[b]
        if n * (p + n) * self.Hq > 1 << 25:  # the larger ones on the GPU, in 64 bits too
            return tuple(x.cpu() for x in attend(*(x.cuda() for x in args), p, self.window, self.n_sink))
        return attend(*args, p, self.window, self.n_sink)


def attend(q, k, v, p0, window, n_sink, scale=None):
    """(o, lse, counts, mass, size) of new rows q [n,Hq,D] at positions p0 + i over k, v [p0 + n,Hkv,D]:
    mass = sum of p |v| (what a relative error of p can move o by), size = the largest scaled
    sum of |q||k| (what errors of the dot products scale with)."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    q, k, v = q.double(), k.double().repeat_interleave(G, 1), v.double().repeat_interleave(G, 1)
    t, s = (torch.arange(a, b, device=q.device) for a, b in ((p0, p0 + n), (0, k.shape[0])))
    t = t[:, None]
    keep = s <= t
    if window:
        keep &= (s > t - window) | (s < n_sink)
    x = torch.einsum("nhd,shd->nhs", q, k) * scale
    x = x.masked_fill(~keep[:, None, :], -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[..., None])
    o = torch.einsum("nhs,shd->nhd", p, v)
    mass = torch.einsum("nhs,shd->nhd", p, v.abs())
    size = torch.einsum("nhd,shd->nhs", q.abs(), k.abs()).amax(-1) * scale
    counts = keep.sum(-1)[:, None].expand(n, Hq)
    return o, lse, counts, mass, size


def check(o, lse, counts, ref, what=""):
    """Against attend()'s result.

    o: the weights p are rounded to bf16 once and the result once, each by at most 2^-8 of its
    value, so |error| <= 2^-8 (mass + |o|); the fp32 products, exponentials and sums add some
    2^-20 of the same quantities times the scores' size, below a twentieth of that.
    lse: a dot product of fp32 sums is off by at most 2^-20 of the sum of its terms' sizes
    (256 terms, each rounded by 2^-24, with room for truncating adders); the sum of weights
    and the logarithm add 2^-20 each.
    """
    o_ref, lse_ref, cnt_ref, mass, size = ref
    if counts is not None:
        assert torch.equal(counts.cpu().long(), cnt_ref.long()), f"{what}: counts differ"
    o, lse = o.cpu().double(), lse.cpu().double()
    assert torch.isfinite(o).all() and torch.isfinite(lse).all(), f"{what}: not finite"
    err, bound = (o - o_ref).abs(), 1.05 * 2.0 ** -8 * (mass + o_ref.abs()) + 1e-9
    assert (err <= bound).all(), f"{what}: o is off by up to {(err / bound).max():.3f} of its bound"
    err, bound = (lse - lse_ref).abs(), 2.0 ** -20 * (size + lse_ref.abs() + 2)
    assert (err <= bound).all(), f"{what}: lse is off by up to {(err / bound).max():.3f} of its bound"


# ---------------------------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------------------------
def free_pages(ref):
    return [p for p, r in enumerate(ref) if r == 0]


def reserve(table, ref, first, end, ps):
    table, ref = [list(r) for r in table], list(ref)
    for b, row in enumerate(table):
        for j in range(first[b] // ps, -(-end[b] // ps)) if end[b] > first[b] else ():
            if row[j] < 0:
                free = free_pages(ref)
                if free:
                    row[j] = free[0]
                    ref[free[0]] = 1
    return table, ref


def free(table, ref, below, ps, n_sink):
    table, ref = [list(r) for r in table], list(ref)
    for b, row in enumerate(table):
        for j, e in enumerate(row):
            if e >= 0 and (below[b] < 0 or ((j + 1) * ps <= below[b] and j * ps >= n_sink)):
                ref[e] -= 1
                row[j] = -1
    return table, ref


def fork(table, ref, src, lens, ps, pools):
    """pools: arrays [L, n_pages, H, ps, D], changed in place."""
    ref = list(ref)
    out = [[-1] * len(r) for r in table]
    for r in table:
        for e in r:
            if e >= 0:
                ref[e] -= 1
    own = []  # rows that need a page of their own
    for i, s in enumerate(src):
        if s < 0:
            continue
        full, part = divmod(lens[s], ps)
        for j in range(full):
            out[i][j] = table[s][j]
        if part:
            if s in src[:i]:
                own.append((i, s, full, part))
            else:
                out[i][full] = table[s][full]
        for j in out[i]:
            if j >= 0:
                ref[j] += 1
    for i, s, full, part in own:
        page = free_pages(ref)[0] if free_pages(ref) else -1
        out[i][full] = page
        if page >= 0:
            ref[page] = 1
            for a in pools:
                a[:, page, :, :part] = a[:, table[s][full], :, :part]
    return out, ref


def compact(table, ref, pools):
    n = len(ref)
    live = sum(r > 0 for r in ref)
    holes = [p for p in range(live) if ref[p] <= 0]
    movers = [p for p in range(live, n) if ref[p] > 0]
    to = dict(zip(movers, holes))
    ref = list(ref)
    for s, d in to.items():
        ref[d] = ref[s]
        for a in pools:
            a[:, d] = a[:, s]
    for p in range(live, n):
        ref[p] = 0
    return [[to.get(e, e) for e in r] for r in table], ref, live


def bits(t):
    """bf16 tensor as integers (NaN compares)."""
    return t.detach().cpu().contiguous().view(torch.int16).numpy().copy()


def i32(x, device="cuda"):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=device)
