"""Attention of shared prefixes with many new tokens a sequence, in batches that the release build shares: each test says by
the plan's own rule, read from its source, that its groups are no groups of single sequences there."""
import os
import re

import pytest
import torch

import paged_reference as R
from test_gpu_paged import verify
from test_gpu_paged_shared import Shared, call

pytestmark = pytest.mark.gpu

SOURCE = os.path.join(os.path.dirname(__file__), "..", "sliding_window_attention_swa_gb300", "csrc", "swa_paged_shared.cu")


@pytest.fixture(scope="module", params=["release", "debug"])
def swa(request):
    import sliding_window_attention_swa_gb300 as m

    if request.param == "release":
        m.load_library()
        yield m
        return
    prev = m.use_library(m.load_library(m.build(debug=True)))
    try:
        yield m
        assert m.load_library()._name.endswith("libswa_debug.so")
    finally:
        m.use_library(prev)


def constants():
    text = open(SOURCE).read()
    release = text.index("#else", text.index("#ifdef SWA_DEBUG"))
    one = lambda name, at: int(re.compile(rf"constexpr int {name} = (\d+);").search(text, at).group(1))  # noqa: E731
    return one("kLeastSaved", release), one("kLeastShared", 0), one("kTileRows", 0)


def shares(seqs, prefix, G, page):
    """Whether a group of sequences [(tokens stored before, new tokens)] without a window is computed as one: positions
    saved by each of its sequences' query tiles."""
    least_saved, least_shared, tile = constants()
    TQ, tokens = tile // G, sum(n for _, n in seqs)
    used = min(prefix, min(p for p, _ in seqs)) // page * page
    own, pre = sum(-(-n // TQ) for _, n in seqs), -(-tokens // TQ)
    return pre < own and used >= least_shared and used * (own - pre) >= least_saved * own


def test_the_rule_is_read_from_the_source():
    assert constants()[0] > 100 and constants()[1] > 16 and constants()[2] == 128


@pytest.mark.parametrize("D,ps", [(64, 64), (128, 16), (256, 128)])
def test_calls_in_a_row_with_cold_and_warm_caches(swa, D, ps):
    """Two batches in turn in one workspace, without a wait between the calls, their pages in L2 or not: what a call
    leaves in the workspace -- lengths, units, lists, results of both parts -- is never taken for the next one's, and
    copies may land late: every result is bit for bit the first one, which is checked."""
    lists = [[(9000, [(9000 + 17 * i, 1 + i % 5) for i in range(40)]), (5000, [(5000 + i, 1) for i in range(30)])],
             [(7000, [(7000 + i, 1 + i % 3) for i in range(25)]), (8500, [(8500 + 5 * i, 1 + i % 4) for i in range(44)]),
              (64, [(300, 7)])]]
    for x in lists:
        for prefix, f in x:
            assert len(f) == 1 or shares(f, prefix, 4, ps), (prefix, len(f))
    more = sum(n for _, f in lists[0] for _, n in f) - sum(n for _, f in lists[1] for _, n in f)
    xs = [Shared(120 + i, x, 8, 2, D, ps, tail=max(0, more if i else -more)) for i, x in enumerate(lists)]
    assert xs[0].N == xs[1].N and len(xs[0].seqs) == len(xs[1].seqs)
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda").fill_(0x77)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")  # more than L2
    dev = [[t.cuda() for t in (x.q, x.k_pages, x.v_pages, x.table, x.p0, x.groups)] for x in xs]
    start = [x.q_start.cuda() for x in xs]
    out = lambda x: (torch.full((x.N, 8, D), 7.0, dtype=torch.bfloat16, device="cuda"),  # noqa: E731
                     torch.full((x.N, 8), 7.0, device="cuda"))
    first, got = [], [[], []]
    for i, x in enumerate(xs):
        first.append(call(swa, x, workspace=ws)[:2])
        swa.swa_check_device_error()
        verify(x, *first[i], None)
    for turn in range(30):
        if turn % 3 == 0:
            flush.fill_(turn)
        for i in (0, 1, 1, 0):
            o, lse = out(xs[i])
            got[i].append(swa.swa_paged_attend_shared(*dev[i], q_start=start[i], workspace=ws, o=o, lse=lse)[:2])
    swa.swa_check_device_error()
    for i in range(2):
        for turn, (o, lse) in enumerate(got[i]):
            assert torch.equal(o, first[i][0]) and torch.equal(lse, first[i][1]), f"batch {i}, call {turn}"


@pytest.mark.parametrize("Hq,Hkv,window,sinks", [(16, 2, 0, 0), (16, 1, 0, 0), (16, 2, 6800, 70)])
def test_pairs_of_query_tiles_in_both_parts(swa, Hq, Hkv, window, sinks):
    """Head dim 128 and so many rows that units are pairs of query tiles, in the prefix part and in the own part; every
    row against 64 bits.  (Sequences that hold a little more than the prefix, their pages made on the GPU.)"""
    D, ps, G = 128, 64, Hq // Hkv
    prefix, n = 7040, 128 // G // 2 - 1 + G // 16
    B = -(-304 * 256 // (Hq * n)) + 5
    seqs = [(prefix + 3 * (i % 40), n) for i in range(B)]
    N, TQ = B * n, 128 // G
    assert N // (2 * TQ) * Hkv >= 2 * 152 and shares(seqs, window - 100 if window else prefix, G, ps)
    g = torch.Generator(device="cuda").manual_seed(130)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    own = -(-(3 * 39 + n) // ps)
    width, n_pages = prefix // ps + own, prefix // ps + own * B
    k, v, q = rnd(n_pages, Hkv, ps, D), rnd(n_pages, Hkv, ps, D), rnd(N, Hq, D)
    place = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.cat([place[:prefix // ps].expand(B, -1), place[prefix // ps:].view(B, own)], 1).contiguous()
    p0 = R.i32([p for p, _ in seqs])
    start = R.i32([n * i for i in range(B + 1)])
    o, lse, cnt = swa.swa_paged_attend_shared(q, k, v, table, p0, R.i32([0, B]), window, q_start=start, n_sink=sinks,
                                              want_counts=True)
    swa.swa_check_device_error()
    for b, (p, _) in enumerate(seqs):
        at = torch.arange(p + n, device="cuda")
        page, row = table[b].long()[at // ps], at % ps
        ref = R.attend(q[b * n:(b + 1) * n], k[page, :, row], v[page, :, row], p, window, sinks)
        R.check(o[b * n:(b + 1) * n], lse[b * n:(b + 1) * n], cnt[b * n:(b + 1) * n], [t.cpu() for t in ref], f"sequence {b}")
