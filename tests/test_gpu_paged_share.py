"""How the paged attention kernels share their work out, by the code that they run (paged_share.cu writes
down every CTA's share and pieces): every tile of every unit goes to exactly one CTA, the pieces of a
shared unit name its owner, their number and slots of their own, the shares are even, and what the
few-row kernel's join reads names exactly a unit's pieces.  All ways of sharing are drawn: one
warp's plan of a small batch and the general one, units dealt whole, in waves with a tail, and cut up."""
import ctypes
import importlib
import os
import random
import subprocess

import pytest
import torch

from paged_reference import i32
from test_paged_share_cpu import units

pytestmark = pytest.mark.gpu

JOIN_TILES = 12  # a CTA may lie this much above the mean where all units are dealt whole
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    B = importlib.import_module("sliding_window_attention_swa_gb300.build")
    out = str(tmp_path_factory.mktemp("share") / "paged_share.so")
    subprocess.check_call([B.nvcc(), *B.flags(), "-shared", "-o", out, os.path.join(HERE, "paged_share.cu")])
    return ctypes.CDLL(out)


def shares_of(lib, kind, grid, TT, min_tiles, seqs, H, window, n_sink, most):
    """Each CTA's (share, pieces)."""
    starts = [0]
    for _, n in seqs:
        starts.append(starts[-1] + n)
    p0, q_start = i32([p for p, _ in seqs]), i32(starts)
    width = max(1, max(-(-(p + n) // 16) for p, n in seqs))
    shares = torch.full((grid, 8), -7, dtype=torch.int32, device="cuda")
    pieces = torch.full((grid, most, 10), -7, dtype=torch.int32, device="cuda")
    err = i32([0])
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    assert lib.paged_shares(kind, grid, TT, min_tiles, most, ptr(p0), ptr(q_start), starts[-1], len(seqs), width, 4, H,
                            window, n_sink, ptr(shares), ptr(pieces), ptr(err)) == 0
    assert err.item() == 0
    pieces = pieces.tolist()
    return [(dict(first=s[0] + (s[1] << 31), waves=s[2], tiles=s[3], left=s[4], turn=s[5]), [x[:9] for x in pieces[c][:s[6]]])
            for c, s in enumerate(shares.tolist())]


def draw(rng, want):
    """A batch; want: the way of sharing that it is drawn for."""
    kind = rng.choice([0, 1, 2]) if want in ("few", "cut") else rng.choice([1, 2])
    TT, grid = rng.choice([1, 4, 16]) if kind == 0 else rng.choice([8, 21, 64, 128]), rng.choice([3, 31, 152, 200])
    H = rng.choice([1, 2, 8])
    if kind == 0:
        grid *= 2
    if want == "few":  # at most four units a sequence; with waves no more than the CTAs
        seqs = [(rng.choice([0, rng.randrange(9000)]), rng.randrange(4 * TT + 1)) for _ in range(rng.randrange(1, 33))]
    elif want == "cut":  # few long units
        seqs = [(rng.randrange(20000), rng.choice([0, TT, 5 * TT])) for _ in range(rng.randrange(1, 60))]
    elif want == "whole":
        seqs = [(rng.randrange(700), rng.choice([0, 1, rng.randrange(6 * TT)])) for _ in range(rng.randrange(33, 200))]
    else:  # some units far longer than the others
        seqs = [(rng.choice([0, 3, 20000]), rng.choice([0, 1, rng.randrange(30 * TT)])) for _ in range(rng.randrange(1, 120))]
    return kind, grid, TT, H, seqs, rng.choice([0, 0, 1, 100, 1000]), rng.choice([0, 1, 37, 200])


@pytest.mark.parametrize("want", ["few", "cut", "whole", "waves"])
def test_every_tile_once_and_evenly(lib, want):
    rng = random.Random(want)
    seen_ways = {}
    for _ in range(60):
        kind, grid, TT, H, seqs, window, n_sink = draw(rng, want)
        BN, min_tiles = (128 if kind == 1 else 64), (1 if kind == 0 else 4)
        us = units(seqs, H, TT, BN, window or 1 << 31, n_sink if window else 0)
        total, what = sum(u[3] for u in us), (kind, grid, TT, H, seqs, window, n_sink)
        if total == 0:
            continue
        got = shares_of(lib, kind, grid, TT, min_tiles, seqs, H, window, n_sink, len(us) + 2)
        tiles, shared, load = {}, {}, [0] * grid
        number = {u[:3]: i for i, u in enumerate(us)}
        for c, (share, pieces) in enumerate(got):
            for b, h, ut, j0, j1, n, slot, owner, count in pieces:
                u = number[b, h, ut]
                assert us[u][3] == n and 0 <= j0 < j1 <= n, what
                for j in range(j0, j1):
                    assert tiles.setdefault((u, j), c) == c and (j == j0 or tiles[u, j - 1] == c), what
                load[c] += j1 - j0
                if j1 - j0 < n:
                    shared.setdefault(u, []).append((j0, slot, owner, count, c))
                else:
                    assert kind == 0 or count == 0, what
            assert kind == 0 or share["tiles"] == load[c], what
        assert len(tiles) == total and sum(load) == total, what  # (each once: none has two CTAs)
        for u, ps in shared.items():
            ps.sort()
            cs = [x[4] for x in ps]
            assert len(set(cs)) == len(cs), what
            owner = cs[0] if kind == 0 else ps[0][2]
            assert [x[1] for x in ps] == [2 * owner + 1] + [2 * (owner + k) for k in range(1, len(ps))], what
            if kind:
                assert {x[2:4] for x in ps} == {(owner, len(ps))} and 2 * (owner + len(ps)) <= 2 * grid, what
            else:  # what the join finds: the CTAs whose stretches start before the unit's end
                end = sum(x[3] for x in us[:u + 1])
                assert cs == list(range(owner, owner + len(cs))), what
                assert sum(s["first"] < end for s, _ in got[owner + 1:]) + 1 == len(cs), what
        slots = [s for ps in shared.values() for _, s, *_ in ps]
        assert len(set(slots)) == len(slots), what
        # evenness, against the mean and what whole units alone come to
        mean, waves = max(-(-total // grid), min_tiles), max((s["waves"] for s, _ in got), default=0)
        if waves and not any(s["left"] for s, _ in got):
            way = "whole"
            assert max(load) <= mean + JOIN_TILES, what
        elif waves:
            way = "waves"
            assert len(us) // grid - 1 == waves, what
            alone = [0] * grid
            for i, u in enumerate(us[:waves * grid]):
                w, c = divmod(i, grid)
                alone[grid - 1 - c if w & 1 else c] += u[3]
            assert all(x <= max(-(-total // grid), y) for x, y in zip(load, alone)), what
        else:
            way = "cut"
            assert max(load) <= mean, what
        few = len(seqs) <= 32 and all(-(-n // TT) <= 4 for _, n in seqs) and (kind == 0 or len(us) <= grid)
        seen_ways[way, few] = seen_ways.get((way, few), 0) + 1
    # the ways that the draws stand for were taken
    for way in {"few": [("whole", True), ("cut", True)], "cut": [("cut", False)], "whole": [("whole", False)],
                "waves": [("waves", False)]}[want]:
        assert seen_ways.get(way, 0) >= 5, seen_ways


def test_as_many_sequences_as_a_call_takes(lib):
    seqs = [(i % 40, 1 if i % 31 == 0 else 0) for i in range(8192)]
    seqs[77] = (1000, 200)
    for kind, grid, TT in ((0, 456, 8), (1, 152, 64), (2, 152, 64)):
        us = units(seqs, 1, TT, 128 if kind == 1 else 64, 20, 1)
        got = shares_of(lib, kind, grid, TT, 1 if kind == 0 else 4, seqs, 1, 20, 1, len(us) + 2)
        assert sum(x[4] - x[3] for _, ps in got for x in ps) == sum(u[3] for u in us)
