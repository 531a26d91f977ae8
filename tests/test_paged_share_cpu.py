"""How the paged attention shares its work out (swa_paged.cuh), modelled on the host: every tile of
every unit goes to exactly one CTA, the shares are even, a CTA leaves at most one unit open and
takes over at most one, and the records the merge reads name exactly the pieces of each shared
unit.  The tiles of a unit cover every key its tokens keep, each once."""
import random

import pytest


def unit_tiles(p0, n, ut, TT, BN, window, n_sink):
    t0, t1 = p0 + ut * TT, p0 + min(n, (ut + 1) * TT) - 1
    lo = (t0 - window + 1) // BN if t0 >= window else 0
    sink = min(lo, -(-min(n_sink, t0 + 1) // BN)) if n_sink else 0
    return list(range(sink)) + list(range(lo, t1 // BN + 1))


def units(seqs, H, TT, BN, window, n_sink):
    return [(b, h, ut, len(unit_tiles(p0, n, ut, TT, BN, window, n_sink)))
            for b, (p0, n) in enumerate(seqs) for h in range(H) for ut in range(-(-n // TT))]


def walk(us, share):
    """(unit index, j0, j1) of a share that starts at (unit, tile) with `left` tiles."""
    u, j, left = share
    while left > 0 and u < len(us):
        j1 = min(us[u][3], j + left)
        yield u, j, j1
        left -= j1 - j
        u, j = u + 1, 0


@pytest.mark.parametrize("seed", range(40))
def test_every_tile_once(seed):
    rng = random.Random(seed)
    BN, TT = rng.choice([(64, 1), (64, 4), (128, 64), (64, 21), (128, 256)])
    window, n_sink = rng.choice([1 << 31, 1, 100, 1000]), rng.choice([0, 1, 37, 200])
    H, grid, min_tiles = rng.choice([1, 2, 8]), rng.choice([1, 3, 152, 304, 456]), rng.choice([1, 2, 4])
    seqs = [(rng.choice([0, rng.randrange(5000)]), rng.choice([0, 1, 1, rng.randrange(1, 700)]))
            for _ in range(rng.randrange(1, 60))]
    us = units(seqs, H, TT, BN, window, n_sink)
    starts = [0]
    for u in us:
        starts.append(starts[-1] + u[3])
    total = starts[-1]
    if total == 0:
        return
    R = max(-(-total // grid), min_tiles)
    seen, opened, slots = {}, {}, {}
    for c in range(grid):
        X = c * R
        if X >= total:
            continue
        u = next(i for i in range(len(us)) if starts[i + 1] > X)
        n_open = n_begun = 0
        for u, j0, j1 in walk(us, (u, X - starts[u], min(R, total - X))):
            assert j1 > j0
            for j in range(j0, j1):
                assert (u, j) not in seen
                seen[u, j] = c
            begun, is_open = j0 > 0, j1 < us[u][3]
            n_begun += begun
            if begun:
                slots[u].append(2 * c)
            elif is_open:
                n_open += 1
                slots[u] = [2 * c + 1]
                # what the merge finds: the CTAs whose stretches start before the unit's end
                end = X + min(R, total - X) + us[u][3] - j1
                assert end == starts[u + 1]
                opened[c] = (1 + sum(min(x * R, total) < end for x in range(c + 1, grid)), u)
        assert n_open <= 1 and n_begun <= 1
    assert len(seen) == total
    for c, (pieces, u) in opened.items():
        assert slots[u] == [2 * c + 1] + [2 * (c + k) for k in range(1, pieces)]
        # what the tile kernel's pieces carry: the owner and the number of pieces, from the unit's tiles
        assert starts[u] // R == c and (starts[u + 1] - 1) // R - c + 1 == pieces
    assert sorted(u for _, u in opened.values()) == sorted(slots)


@pytest.mark.parametrize("seed", range(20))
def test_tiles_cover_the_kept_keys(seed):
    rng = random.Random(100 + seed)
    BN, TT = rng.choice([64, 128]), rng.choice([1, 5, 32, 64])
    window, n_sink = rng.choice([1, 50, 300, 1 << 31]), rng.choice([0, 1, 40, 400])
    p0, n = rng.randrange(1500), rng.randrange(1, 200)
    for ut in range(-(-n // TT)):
        tiles = unit_tiles(p0, n, ut, TT, BN, window, n_sink)
        assert len(set(tiles)) == len(tiles) and tiles == sorted(tiles)
        for t in range(p0 + ut * TT, p0 + min(n, (ut + 1) * TT)):
            kept = [s for s in range(t + 1) if s > t - window or s < n_sink]
            assert {s // BN for s in kept} <= set(tiles)
            # the count that the kernels compute
            behind = t - window + 1 if t >= window else 0
            assert len(kept) == t + 1 - behind + min(behind, n_sink)


@pytest.mark.parametrize("seed", range(40))
def test_waves_and_tail(seed):
    """The tile kernel's sharing from two units a CTA: whole units in waves of alternating direction,
    the rest cut into stretches that fill every CTA up to one level."""
    rng = random.Random(200 + seed)
    BN, TT, grid = rng.choice([(64, 64, 7), (128, 64, 152), (128, 20, 31), (64, 128, 16)])
    window, n_sink, H = rng.choice([1 << 31, 100, 1000]), rng.choice([0, 37]), rng.choice([1, 2, 8])
    seqs = [(rng.choice([0, rng.randrange(5000)]), rng.choice([0, 1, rng.randrange(1, 2000)]))
            for _ in range(rng.randrange(1, 60))]
    us = units(seqs, H, TT, BN, window, n_sink)
    waves = max(0, len(us) // grid - 1)
    if waves == 0:
        return
    starts = [0]
    for u in us:
        starts.append(starts[-1] + u[3])
    total, bulk = starts[-1], waves * grid

    def dealt_to(u):
        w, c = divmod(u, grid)
        return grid - 1 - c if w & 1 else c

    loads = [0] * grid
    for u in range(bulk):
        loads[dealt_to(u)] += us[u][3]
    mine = [[w * grid + (grid - 1 - c if w & 1 else c) for w in range(waves)] for c in range(grid)]
    assert sorted(u for m in mine for u in m) == list(range(bulk))
    assert [sum(us[u][3] for u in m) for m in mine] == loads
    tail = total - sum(loads)
    lo = -(-total // grid)
    hi = max(loads) + -(-tail // grid) if max(loads) > lo else lo
    while lo < hi:
        mid = (lo + hi) // 2
        if sum(max(0, mid - x) for x in loads) >= tail:
            hi = mid
        else:
            lo = mid + 1
    at, first, left = sum(loads), [], []
    for x in loads:
        q = max(0, lo - x)
        first.append(at)
        left.append(max(0, min(q, total - at)))
        at += q
    assert sum(left) == tail
    # no CTA has more than the level, unless its waves alone have
    assert all(x + q <= max(lo, x) for x, q in zip(loads, left))
    seen, slots, opened, carried = set(), {}, {}, {}

    def turn_of(X):
        return sum(n > 0 and f + n <= X for f, n in zip(first, left))

    for c in range(grid):
        if not left[c]:
            continue
        u = next(i for i in range(len(us)) if starts[i + 1] > first[c])
        assert u >= bulk
        for u, j0, j1 in walk(us, (u, first[c] - starts[u], left[c])):
            for j in range(j0, j1):
                assert (u, j) not in seen
                seen.add((u, j))
            if j0 > 0:
                slots[u].append(c)
            elif j1 < us[u][3]:
                slots[u] = [c]
                opened[c] = u
            # what the piece carries: turns count the CTAs with a stretch
            if j0 > 0 or j1 < us[u][3]:
                owner, end = turn_of(starts[u]), turn_of(starts[u + 1] - 1)
                carried.setdefault(u, set()).add((owner, end - owner + 1))
    assert len(seen) == tail
    for c, u in opened.items():
        (owner, pieces), = carried[u]
        turns = [sum(left[x] > 0 for x in range(y)) for y in slots[u]]
        assert turns == list(range(owner, owner + pieces))
