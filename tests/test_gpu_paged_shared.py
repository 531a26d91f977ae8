"""Attention of sequences that share leading pages: every row against a plain 64-bit computation of each
sequence by itself (see paged_reference.check for the bounds), and against swa_paged_attend."""
import random

import pytest
import torch

import paged_reference as R
from test_gpu_paged import verify

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def swa():
    import sliding_window_attention_swa_gb300 as m

    m.load_library()
    return m


class Shared(R.Batch):
    """A batch of groups [(tokens shared, [(tokens stored before, new tokens), ...]), ...]: the first tokens
    of a group's sequences are the same, and the pages that lie within them are shared.  Whatever no query
    keeps holds `junk`."""

    def __init__(self, seed, groups, Hq, Hkv, D, ps, window=0, n_sink=0, junk=float("nan"), freed=True, lead=0, tail=0,
                 before=(), behind=()):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
        # (sequences of no group ahead of the groups and behind them)
        families = [(0, [s]) for s in before] + list(groups) + [(0, [s]) for s in behind]
        self.seqs = seqs = [s for _, f in families for s in f]
        self.Hq, self.Hkv, self.D, self.ps, self.window, self.n_sink = Hq, Hkv, D, ps, window, n_sink
        ends = [p + n for p, n in seqs]
        self.width = max(1, max(-(-e // ps) for e in ends))
        names, rows, self.keys, self.vals, b = {}, [], [], [], 0
        for i, (prefix, f) in enumerate(families):
            common = rnd(prefix, Hkv, D), rnd(prefix, Hkv, D)
            for p, n in f:
                own = max(0, p + n - prefix)
                for x, c in zip((self.keys, self.vals), common):
                    x.append(torch.cat([c[:p + n], rnd(own, Hkv, D)]))
                # new rows are no other sequence's
                for x in (self.keys[-1], self.vals[-1]):
                    x[p:] = rnd(n, Hkv, D)
                lo = max(0, p - window + 1) if window else 0
                rows.append([(j, names.setdefault((i, j) if (j + 1) * ps <= min(prefix, p) else (-1 - b, j), len(names)))
                             for j in range(-(-(p + n) // ps))
                             if not (freed and (j + 1) * ps <= lo and j * ps >= n_sink)])
                b += 1
        self.n_pages = len(names) + 3
        place = torch.randperm(self.n_pages, generator=g).tolist()
        self.table = torch.full((len(seqs), self.width), -1, dtype=torch.int32)
        for b, r in enumerate(rows):
            for j, x in r:
                self.table[b, j] = place[x]
        starts = [lead]
        for _, n in seqs:
            starts.append(starts[-1] + n)
        self.N = starts[-1] + tail
        self.q_start = torch.tensor(starts, dtype=torch.int32)
        self.p0 = torch.tensor([p for p, _ in seqs], dtype=torch.int32)
        self.q = rnd(self.N, Hq, D)
        self.k_pages = torch.full((self.n_pages, Hkv, ps, D), junk, dtype=torch.bfloat16)
        self.v_pages = self.k_pages.clone()
        self.k_new = torch.full((self.N, Hkv, D), float("nan"), dtype=torch.bfloat16)
        self.v_new = self.k_new.clone()
        for b, (p, n) in enumerate(seqs):
            self.k_new[starts[b]:starts[b] + n] = self.keys[b][p:]
            self.v_new[starts[b]:starts[b] + n] = self.vals[b][p:]
            lo = max(0, p - window + 1) if window else 0
            for j, x in rows[b]:
                end = min((j + 1) * ps, p + n)
                for t0, t1 in [(j * ps, end)] if junk == 0 else [(max(j * ps, lo), end), (j * ps, min(end, n_sink))] if n else []:
                    if t0 < t1:
                        self.k_pages[place[x], :, t0 - j * ps:t1 - j * ps] = self.keys[b][t0:t1].transpose(0, 1)
                        self.v_pages[place[x], :, t0 - j * ps:t1 - j * ps] = self.vals[b][t0:t1].transpose(0, 1)
        first, at = len(before), []
        for _, f in groups:
            at.append(first)
            first += len(f)
        self.groups = torch.tensor(at + [first], dtype=torch.int32)


def call(swa, x, append=False, groups=None, want_counts=True, **kw):
    """(o, lse, counts, k_pages, v_pages) of the call on batch x."""
    k, v = (t.cuda() for t in (x.without_new() if append else (x.k_pages, x.v_pages)))
    o = torch.full((x.N, x.Hq, x.D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((x.N, x.Hq), 7.0, device="cuda")
    cnt = torch.full((x.N, x.Hq), 7, dtype=torch.int32, device="cuda") if want_counts else None
    if append:
        kw.update(k_new=x.k_new.cuda(), v_new=x.v_new.cuda())
    kw.setdefault("q_start", x.q_start.cuda())
    swa.swa_paged_attend_shared(x.q.cuda(), k, v, x.table.cuda(), x.p0.cuda(),
                                (x.groups if groups is None else groups).cuda(), x.window, n_sink=x.n_sink, o=o, lse=lse,
                                row_counts=cnt, **kw)
    return o, lse, cnt, k, v


def run(swa, x, append=False, **kw):
    o, lse, cnt, k, v = call(swa, x, append, **kw)
    swa.swa_check_device_error()
    verify(x, o, lse, cnt)
    assert (R.bits(k) == R.bits(x.k_pages)).all() and (R.bits(v) == R.bits(x.v_pages)).all()
    return o, lse, cnt


# prefixes that end in and with a page, shorter and longer than a tile; one sequence, none; sequences that hold
# less than the others; lengths of zero
ONES = [(300, [(300, 1), (301, 1), (555, 1)]), (64, [(64, 1)]), (0, [(5, 1), (0, 1), (17, 1)]),
        (1000, [(1000 + 3 * i, 1) for i in range(21)]), (128, [(128, 1), (129, 1)]), (256, [(256, 1), (257, 1)]), (500, [(200, 1), (900, 1), (450, 1)]),
        (2048, [(2050, 1)] * 40)]
MIXED = [(300, [(300, 5), (301, 1), (555, 33)]), (64, [(64, 70)]), (0, [(5, 3), (0, 0), (0, 9)]),
         (1000, [(1000 + 3 * i, 1 + i % 4) for i in range(21)]), (256, [(256, 0), (257, 2), (268, 1), (256, 0)]),
         (700, [(100, 3), (900, 1), (0, 0), (450, 7)]), (2048, [(2050, 0), (2048, 200), (2049, 40), (2100, 1)])]
SHAPES = [
    # Hq, Hkv, D, page, window, sinks
    (8, 2, 128, 16, 0, 0), (8, 2, 128, 64, 100, 4), (4, 4, 64, 32, 0, 0), (32, 2, 64, 16, 357, 37), (7, 1, 128, 128, 1200, 0),
    (6, 2, 256, 64, 1000, 1), (16, 1, 256, 16, 0, 0), (3, 3, 256, 128, 700, 130), (5, 1, 64, 128, 450, 0),
    (12, 1, 128, 32, 400, 3), (16, 1, 64, 64, 1, 0), (2, 2, 128, 128, 2000, 300), (4, 4, 64, 16, 900, 250), (16, 2, 256, 32, 333, 20),
]


@pytest.mark.parametrize("append", [False, True], ids=["stored", "append"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_one_token_a_sequence(swa, shape, append):
    x = Shared(1, ONES, *shape)
    run(swa, x, append, q_start=None)


@pytest.mark.parametrize("hint", [0, 1, 16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_ragged_groups(swa, shape, hint):
    x = Shared(2, MIXED, *shape, lead=3, tail=5, before=[(9, 1), (40, 2)], behind=[(100, 3), (0, 1)])
    run(swa, x, hint == 0, max_q=hint)


@pytest.mark.parametrize("D,ps", [(64, 16), (128, 32), (256, 64)])
def test_same_as_each_by_itself(swa, D, ps):
    """Nothing of the groups shows: one group of all, none shared, groups that overlap what is shared."""
    x = Shared(3, MIXED, 8, 2, D, ps, 500, 2)
    B = len(x.seqs)
    for groups in ([0, B], [0, 1], [B, B], [0, 0, 0, B, B], list(range(B + 1)), [2, 7, 11, 30], [5, 6]):
        run(swa, x, groups=torch.tensor(groups, dtype=torch.int32))
    y = R.Batch(4, [(300, 2), (500, 1), (20, 9)] * 5, 8, 2, D, ps)
    y.groups = torch.tensor([0, 15], dtype=torch.int32)
    run(swa, y)
    run(swa, y, max_q=2)


def random_tree(rng, D):
    ps = rng.choice([16, 32, 64, 128])
    groups = []
    for _ in range(rng.randrange(1, 7)):
        prefix = rng.choice([0, rng.randrange(1, 400), rng.randrange(200, 4000)])
        longest = rng.choice([1, 1, 4, 90])
        groups.append((prefix, [(rng.choice([prefix, prefix + rng.randrange(300), rng.randrange(prefix + 1)]),
                                 rng.choice([0, 1, 1, rng.randrange(longest + 1)])) for _ in range(rng.randrange(1, 30))]))
    G = rng.choice([1, 2, 3, 5, 8, 16])
    H = rng.choice([1, 2, 3])
    window = rng.choice([0, 0, 1, 64, 300, 700, 1500])
    return groups, G * H, H, ps, window, rng.choice([0, 1, 40, 200]) if window else 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("seed", range(12))
def test_drawn_batches(swa, seed, D):
    rng = random.Random(1000 * D + seed)
    groups, Hq, Hkv, ps, window, sinks = random_tree(rng, D)
    x = Shared(seed, groups, Hq, Hkv, D, ps, window, sinks, freed=rng.random() < 0.5)
    if x.N == 0:
        return
    run(swa, x, rng.random() < 0.5, max_q=rng.choice([0, 0, 1, max(n for _, n in x.seqs)]))


@pytest.mark.parametrize("D,ps", [(64, 64), (128, 16), (256, 128)])
def test_long_prefixes_and_many_groups(swa, D, ps):
    # prefixes spread over every CTA and joined again; many groups, more than the kernels' lists hold at a time
    run(swa, Shared(5, [(20000, [(20000 + i, 1) for i in range(9)])], 4, 1, D, ps), q_start=None)
    run(swa, Shared(6, [(12000, [(12000 + 7 * i, 3 + i) for i in range(33)])], 4, 1, D, ps))
    run(swa, Shared(7, [(300 + i % 70, [(370 + i % 9, 1)] * (1 + i % 3)) for i in range(700)], 4, 1, D, ps), q_start=None)
    run(swa, Shared(8, [(500, [(500, 2)] * 2)] * 300, 4, 1, D, ps, 377, 3))


def test_units_of_two_query_tiles(swa):
    # head dim 128 and many rows: pairs of query tiles in the prefix part, and in the own part
    for Hq, Hkv, window, most in ((16, 16, 700, 2000), (32, 8, 0, 900)):
        x = Shared(9, [(900, [(900 + i, 100 + 7 * i) for i in range(most // 90)]), (300, [(300, most), (310, most // 2)])], Hq,
                   Hkv, 128, 32, window, 2 if window else 0)
        assert x.N // (2 * (128 // (Hq // Hkv))) * Hkv >= 2 * 152  # (pairs in the own part, too)
        run(swa, x, want_counts=False)


@pytest.mark.parametrize("append", [False, True], ids=["stored", "append"])
@pytest.mark.parametrize("shape", [(8, 2, 64, 16, 0, 0), (8, 2, 64, 64, 5500, 200), (4, 1, 128, 128, 0, 0), (7, 1, 128, 32, 7000, 3),
                                   (4, 2, 256, 64, 0, 0), (8, 1, 256, 128, 6500, 1), (16, 16, 128, 64, 6000, 40)], ids=str)
def test_chunks_behind_long_prefixes(swa, shape, append):
    # prefixes long enough for chunks to share them; sequences that hold less or have nothing new
    Hq, Hkv = shape[:2]
    per_tile = 128 // (Hq // Hkv)
    lists = [(9000, [(9000 + 3 * i, 1 + i % 7) for i in range(24)] + [(9000, 0), (9111, per_tile + 3)]), (300, [(300, 9)] * 3),
             (7777, [(7777, 2)] * 3 + [(8000 + i, 1 + 9 * (i % 2)) for i in range(30)])]
    if Hq == 16 == Hkv:  # pairs of query tiles
        lists = [(9000, [(9000 + i, 30) for i in range(96)])]
    for prefix, f in lists[::2]:
        own = sum(-(-n // per_tile) for _, n in f)
        assert (own + -sum(n for _, n in f) // per_tile) * min(prefix, (shape[4] or prefix) - 600) > 3600 * own
    run(swa, Shared(24, lists, *shape, lead=2, tail=3), append)


def test_as_many_sequences_and_groups_as_a_call_takes(swa):
    x = Shared(10, [(208, [(208 + i % 9, 1 if j % 3 else 0) for i in range(2)]) for j in range(4096)], 2, 1, 64, 16)
    assert len(x.seqs) == 8192
    run(swa, x)
    run(swa, x, groups=torch.tensor([0, 8192], dtype=torch.int32))
    x.groups = torch.cat([torch.zeros(8192 - 4096, dtype=torch.int32), x.groups])  # (empty groups)
    run(swa, x)
    with pytest.raises(swa.SwaError):
        call(swa, x, groups=torch.zeros(8194, dtype=torch.int32))


@pytest.mark.parametrize("case", [(8, 2, 128, 16, 400, 4), (4, 4, 64, 64, 300, 130), (6, 2, 256, 32, 365, 37),
                                  (2, 1, 64, 128, 1000, 0)], ids=str)
def test_positions_that_no_query_keeps_may_hold_anything(swa, case):
    # pages that are there all the same, with NaN between the sinks and every window
    for seqs in ([(1500, 1), (1510, 1), (1601, 1)], [(1500, 40), (1510, 1), (1601, 3)]):
        run(swa, Shared(11, [(1500, seqs)] * 3, *case, freed=False))


def test_rows_that_keep_nothing_of_the_prefix(swa):
    # windows of some sequences end behind what is shared, of others they do not
    for D, ps in ((64, 16), (128, 64), (256, 128)):
        for sinks in (0, 5):
            x = Shared(12, [(1024, [(1024, 1), (1100, 1), (1500, 1), (3000, 1)])] * 4, 8, 2, D, ps, 300, sinks)
            run(swa, x, q_start=None)
            run(swa, x)


def test_values_of_the_extremes(swa):
    x = Shared(13, [(700, [(700 + i, 1) for i in range(20)])], 8, 2, 128, 16)
    # scores of some hundreds: one key takes all the weight, in the prefix for some rows and behind it for others
    x.q = (x.q.float() * 60).to(torch.bfloat16)
    run(swa, x, q_start=None)
    x.q.zero_()
    run(swa, x, q_start=None)
    x.v_pages = (x.v_pages.float() * 1e30).to(torch.bfloat16)
    x.vals = [(v.float() * 1e30).to(torch.bfloat16) for v in x.vals]
    run(swa, x, q_start=None)


def test_layouts(swa):
    x = Shared(14, MIXED, 8, 2, 128, 32)
    o, lse, cnt = run(swa, x)
    wide_q = torch.zeros(x.N, 12, 136, dtype=torch.bfloat16, device="cuda")
    wide_q[:, 2:10, :128] = x.q.cuda()
    wide_o = torch.full((x.N, 9, 144), 7.0, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    args = x.k_pages.cuda(), x.v_pages.cuda(), x.table.cuda(), x.p0.cuda(), x.groups.cuda()
    torch.cuda.synchronize()
    got = swa.swa_paged_attend_shared(wide_q[:, 2:10, :128], *args, q_start=x.q_start.cuda(), o=wide_o[:, 1:, :128],
                                      stream=side, want_counts=True, scale=128 ** -0.5)
    side.synchronize()
    assert torch.equal(got[0], o) and torch.equal(got[1], lse) and torch.equal(got[2], cnt)
    assert (wide_o[:, 0] == 7).all() and (wide_o[:, :, 128:] == 7).all()
    # a workspace of the caller's, whatever it holds
    size = 1 << 28
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        again = swa.swa_paged_attend_shared(x.q.cuda(), *args, q_start=x.q_start.cuda(), workspace=ws)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    swa.swa_check_device_error()


def test_broken_device_data(swa):
    x = Shared(15, [(300, [(300, 1), (310, 2), (333, 1)]), (100, [(100, 1), (120, 1)])], 4, 2, 64, 16)
    bad_position = {"prefill": 0, "split": 0, "cache": swa.DEVERR_BAD_POSITION}
    # groups out of range or in disorder: computed alone, and reported
    for groups in ([0, 3, 6], [-1, 3, 5], [3, 0, 5], [0, 1 << 30, 5]):
        for hint in (0, 2):
            o, lse, cnt, *_ = call(swa, x, groups=torch.tensor(groups, dtype=torch.int32), max_q=hint)
            st, words = swa.swa_read_device_errors()
            assert st == 1 and words == bad_position, words
            verify(x, o, lse, cnt)
    # a sequence out of range: skipped, the rest of its group computed alone
    for wrong in (-1, x.width * 16, (1 << 31) - 1):
        for hint in (0, 2):
            x.p0[1], p = wrong, int(x.p0[1])
            o, lse, cnt, *_ = call(swa, x, max_q=hint)
            x.p0[1] = p
            st, words = swa.swa_read_device_errors()
            assert st == 1 and words == bad_position, words
            assert (o[1:3] == 7).all() and (lse[1:3] == 7).all() and (cnt[1:3] == 7).all()
            for b, q0, n in x.rows():
                if b != 1:
                    R.check(o[q0:q0 + n], lse[q0:q0 + n], cnt[q0:q0 + n], x.reference(b), f"sequence {b}")
    # a page that is missing in every row of the group counts as rows of zeros
    for entry in (-1, x.n_pages, -(1 << 31)):
        table = x.table.clone()
        x.table[:3, 4] = entry
        keys, vals = x.keys, x.vals
        x.keys, x.vals = [k.clone() for k in keys], [v.clone() for v in vals]
        for b in range(3):
            x.keys[b][64:80] = 0
            x.vals[b][64:80] = 0
        for hint in (0, 2):
            o, lse, cnt, *_ = call(swa, x, max_q=hint)
            st, words = swa.swa_read_device_errors()
            assert st == 1 and words == {"prefill": 0, "split": 0, "cache": swa.DEVERR_BAD_PAGE}, words
            verify(x, o, lse, cnt)
        x.table, x.keys, x.vals = table, keys, vals
    run(swa, x)


def test_refusals(swa):
    x = Shared(16, [(64, [(64, 2), (70, 1)])], 4, 2, 64, 16)
    args = [t.cuda() for t in (x.q, x.k_pages, x.v_pages, x.table, x.p0)]
    groups, start = x.groups.cuda(), x.q_start.cuda()
    for bad in (groups.long(), groups.cpu(), groups[None], groups[:1], groups.repeat(2)[::2]):
        with pytest.raises(ValueError):
            swa.swa_paged_attend_shared(*args, bad, q_start=start)
    with pytest.raises(ValueError):
        swa.swa_paged_attend_shared(*args, groups)  # three rows, two sequences
    with pytest.raises(ValueError):
        swa.swa_paged_attend_shared(*args, groups, q_start=start, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(swa.SwaError):
        swa.swa_paged_attend_shared(*args, groups, q_start=start,
                                    workspace=torch.empty(1 << 10, dtype=torch.uint8, device="cuda"))
    with pytest.raises(swa.SwaError):
        swa.swa_paged_attend_shared(*args, groups, -1, q_start=start)
    empty = args[0][:0]
    o, lse, _ = swa.swa_paged_attend_shared(empty, *args[1:], groups, q_start=torch.zeros_like(start))
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_calls_repeat_bit_for_bit(swa, D):
    x = Shared(17, [(9000, [(9000 + 31 * i, 1 + i % 3) for i in range(40)]), (700, [(701, 1)] * 9)], 8, 2, D, 32)
    first = call(swa, x, max_q=0)
    few = call(swa, x, max_q=3)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(call(swa, x, max_q=0)[:3], first))
        assert all(torch.equal(a, b) for a, b in zip(call(swa, x, max_q=3)[:3], few))
    swa.swa_check_device_error()


def test_two_streams_at_once(swa):
    xs = [Shared(18 + i, [(4000, [(4000 + 11 * j, 1 + i) for j in range(30)])], 8, 2, 128, 16) for i in range(2)]
    want = [call(swa, x, max_q=1 + i) for i, x in enumerate(xs)]
    dev = [[t.cuda() for t in (x.q, x.k_pages, x.v_pages, x.table, x.p0, x.groups, x.q_start)] for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(swa.swa_paged_attend_shared(*dev[i][:6], q_start=dev[i][6], max_q=1 + i, stream=s))
    torch.cuda.synchronize()
    swa.swa_check_device_error()
    for i in range(2):
        assert all(torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1]) for o, lse, _ in got[i])


def test_captured_and_replayed_with_other_groups(swa):
    """One decode step of samples -- their rows forked, their keys and queries rotated and stored, their attention
    with the prefix read once -- captured, then replayed for other lengths, tables and groups."""
    Hq, Hkv, D, ps, B = 8, 2, 128, 16, 12
    rope = swa.swa_rope_table(10000.0 ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64), 2000)
    cases = [Shared(30, [(400, [(400, 1)] * 7), (900, [(901, 1), (930, 1), (905, 1), (900, 1), (950, 1)])], Hq, Hkv, D, ps,
                    junk=0.0),
             Shared(31, [(600, [(601 + i, 1) for i in range(4)]), (77, [(100, 1), (80, 1)]), (333, [(340, 1)] * 6)], Hq, Hkv, D,
                    ps, junk=0.0)]
    n_pages = max(x.n_pages for x in cases)
    width = max(x.width for x in cases)

    def padded(x):
        pools = [torch.cat([t, torch.zeros(n_pages - x.n_pages, *t.shape[1:], dtype=t.dtype)]) for t in x.without_new()]
        pools = [torch.nan_to_num(t.float()).to(torch.bfloat16) for t in pools]
        table = torch.cat([x.table, torch.full((B, width - x.width), -1, dtype=torch.int32)], 1)
        groups = torch.cat([x.groups, x.groups[-1:].expand(4 - len(x.groups))])
        return [t.cuda() for t in (x.q, x.k_new, x.v_new, *pools, table, x.p0, groups)]

    def step(q, kn, vn, k, v, table, p0, groups):
        turned = swa.swa_paged_rope_append(q, k, v, table, kn, vn, p0, rope)
        o, lse, cnt = swa.swa_paged_attend_shared(turned, k, v, table, p0, groups, want_counts=True)
        plain = swa.swa_paged_attend(turned, k, v, table, p0, want_counts=True)
        return turned, o, lse, cnt, *plain

    state = padded(cases[0])
    step(*state)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*state)
    for x in (cases[1], cases[0], cases[1]):
        new = padded(x)
        for dst, src in zip(state, new):
            dst.copy_(src)
        graph.replay()
        want = step(*new)
        swa.swa_check_device_error()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(state, new))
        # the queries and keys as they lie there, each sequence by itself
        q, k, v = out[0].cpu(), new[3].cpu(), new[4].cpu()
        for b, (p, _) in enumerate(x.seqs):
            at = torch.arange(p + 1)
            page, row = new[5].cpu()[b].long()[at // ps], at % ps
            ref = R.attend(q[b:b + 1], k[page, :, row], v[page, :, row], p, 0, 0)
            R.check(out[1][b:b + 1], out[2][b:b + 1], out[3][b:b + 1], ref, f"sequence {b}")
            R.check(out[4][b:b + 1], out[5][b:b + 1], out[6][b:b + 1], ref, f"sequence {b}, alone")


def test_samples_of_one_prompt(swa):
    """A prompt is forked into samples, which go on for some tokens each: every step against the unshared call."""
    Hq, Hkv, D, ps, B, prompt = 8, 2, 64, 16, 6, 203
    g = torch.Generator(device="cuda").manual_seed(40)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    k, v = rnd(200, Hkv, ps, D), rnd(200, Hkv, ps, D)
    table = torch.full((B, 20), -1, dtype=torch.int32, device="cuda")
    held = torch.zeros(200, dtype=torch.int32, device="cuda")
    rope = swa.swa_rope_table(10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32), 400)
    length = R.i32([prompt] + [0] * (B - 1))
    swa.swa_pages_reserve(table, held, R.i32([0] * B), length, ps)
    rows = rnd(prompt, Hq, D), rnd(prompt, Hkv, D), rnd(prompt, Hkv, D)
    start = R.i32([0] + [prompt] * B)
    q = swa.swa_paged_rope_append(rows[0], k, v, table, rows[1], rows[2], R.i32([0] * B), rope, q_start=start)
    swa.swa_paged_attend(q, k, v, table, R.i32([0] * B), q_start=start)
    table, held = swa.swa_pages_fork(k, v, table, held, R.i32([0] * B), length)
    p0 = R.i32([prompt] * B)
    groups = R.i32([0, B])
    for step in range(20):
        swa.swa_pages_reserve(table, held, p0, p0 + 1, ps)
        q = swa.swa_paged_rope_append(rnd(B, Hq, D), k, v, table, rnd(B, Hkv, D), rnd(B, Hkv, D), p0, rope)
        o, lse, cnt = swa.swa_paged_attend_shared(q, k, v, table, p0, groups, want_counts=True)
        for b in range(B):
            p = prompt + step
            at = torch.arange(p + 1, device="cuda")
            page, row = table[b].long()[at // ps], at % ps
            ref = R.attend(q[b:b + 1], k[page, :, row], v[page, :, row], p, 0, 0)
            R.check(o[b:b + 1], lse[b:b + 1], cnt[b:b + 1], [t.cpu() for t in ref], f"step {step}, sample {b}")
        p0 = p0 + 1
    swa.swa_check_device_error()


@pytest.mark.parametrize("hint", [0, 1])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_sequences_that_overlap(swa, D, hint):
    """A q_start that goes up and down gives sequences rows that others have, too: work that ends, reported, nothing
    outside the call's buffers, and the next call is right."""
    x = Shared(50, [(300, [(300, 4)] * 60)], 4, 2, D, 16, lead=2, tail=3)
    good = x.q_start.clone()
    for wrong in (0, 1, 17, 100, x.N):
        x.q_start[1::3] = wrong
        o, lse, cnt, *_ = call(swa, x, max_q=hint)
        st, words = swa.swa_read_device_errors()
        assert st in (0, 1) and words["prefill"] == words["split"] == 0, words
        assert (o[-3:] == 7).all() or wrong == x.N
        x.q_start = good.clone()
    run(swa, x, max_q=hint)


@pytest.mark.parametrize("hint", [0, 1])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_nothing_is_read_that_the_call_has_not_written(swa, shape, hint):
    # a workspace of NaN: a value of it would show even with a weight of zero
    ws = torch.empty(1 << 31, dtype=torch.uint8, device="cuda").fill_(0xff)
    run(swa, Shared(25, MIXED, *shape, lead=3, tail=5, before=[(9, 1), (40, 2)], behind=[(100, 3), (0, 1)]), max_q=hint, workspace=ws)
    long = [(9000, [(9000 + 3 * i, 1 + i % 7) for i in range(24)] + [(9111, 128 // (shape[0] // shape[1]) + 3)])]
    run(swa, Shared(26, long, *shape[:4], 0, 0), max_q=hint, workspace=ws.fill_(0xff))


def test_one_workspace_for_many_calls(swa):
    """Calls one after the other in one workspace, whatever the last one left there: shapes, parts and hints change."""
    ws = torch.empty(1 << 29, dtype=torch.uint8, device="cuda").fill_(0x5a)
    xs = [(Shared(60, ONES, 8, 2, 128, 16), 1), (Shared(61, MIXED, 8, 2, 64, 32, 300, 5), 0),
          (Shared(62, MIXED, 4, 2, 256, 64), 1), (Shared(63, ONES[2:3], 8, 2, 128, 16), 0), (Shared(64, MIXED, 16, 1, 128, 16), 0)]
    for _ in range(2):
        for x, hint in xs:
            run(swa, x, max_q=hint, workspace=ws)


@pytest.mark.parametrize("hint", [0, 1])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_calls_in_a_row_with_cold_and_warm_caches(swa, D, hint):
    """Two batches in turn in one workspace, without a wait between the calls, their pages in L2 or not: what a call
    leaves in the workspace (lengths, lists, results) is never taken for the next one's, and copies may land
    late: every result is bit for bit the first one, which is checked."""
    ps = 16 if D == 128 else 64
    xs = [Shared(80, [(3000, [(3000 + 17 * i, 1) for i in range(40)]), (500, [(500 + i, 1) for i in range(3)])], 8, 2, D, ps),
          Shared(81, [(700, [(700 + i, 1) for i in range(9)]), (2500, [(2500 + 5 * i, 1) for i in range(30)]),
                      (64, [(300, 1)] * 4)], 8, 2, D, ps)]
    assert len(xs[0].seqs) == len(xs[1].seqs)
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda").fill_(0x77)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")  # more than L2
    dev = [[t.cuda() for t in (x.q, x.k_pages, x.v_pages, x.table, x.p0, x.groups)] for x in xs]
    start = xs[0].q_start.cuda()
    first, got = [], [[], []]
    for i, x in enumerate(xs):
        first.append(call(swa, x, q_start=None if hint else start, workspace=ws)[:2])
        swa.swa_check_device_error()
        verify(x, *first[i], None)
    for turn in range(30):
        if turn % 3 == 0:
            flush.fill_(turn)
        for i in (0, 1, 1, 0):
            got[i].append(swa.swa_paged_attend_shared(*dev[i], q_start=None if hint else start, workspace=ws)[:2])
    swa.swa_check_device_error()
    for i in range(2):
        for turn, (o, lse) in enumerate(got[i]):
            assert torch.equal(o, first[i][0]) and torch.equal(lse, first[i][1]), f"batch {i}, call {turn}"
