"""How swa_paged_attend_shared cuts a unit's keys into stretches (swa_paged_shared.cuh), modelled on the host: the
stretches of a unit's own part and of its group's prefix cover every key that its tokens keep, each once, no more of
them than there are planes; and what the plan finds to be shared is what every sequence can take from one row of
the page table."""
import random

import pytest

LEAST = 64


def split_keys(lo, end, sink0, sink1, planes):
    first = lo & ~15
    n, most = end - first, planes - 1
    keys = max(LEAST, (-(-n // most) + 15) & ~15)
    out = [(max(lo, first + i * keys), min(end, first + (i + 1) * keys)) for i in range(-(-n // keys))]
    assert len(out) <= most
    return out + ([(sink0, sink1)] if sink1 > sink0 else [])


def own_keys(p0, n, base, ut, TT, window, sinks, planes):
    t0, t1 = p0 + ut * TT, p0 + min(n, (ut + 1) * TT) - 1
    lo = max(base, t0 - window + 1 if window and t0 >= window else 0)
    return split_keys(lo, t1 + 1, base, min(sinks, lo), planes)


def prefix_keys(p0, end, window, sinks, planes):
    lo = p0 - window + 1 if window and p0 >= window else 0
    return split_keys(lo, end, 0, min(sinks, lo), planes)


@pytest.mark.parametrize("seed", range(60))
def test_stretches_cover_the_kept_keys_once(seed):
    rng = random.Random(seed)
    window, sinks = rng.choice([0, 1, 50, 300, 1000]), rng.choice([0, 1, 40, 400])
    if not window:
        sinks = 0
    ps, TT = rng.choice([16, 32, 64, 128]), rng.choice([1, 4, 16])
    least = rng.randrange(0, 3000)  # the least p0 of a group
    base = rng.choice([0, rng.randrange(0, least // ps + 1) * ps])
    lo = max(0, least - window + 1) if window else 0
    if base <= lo:
        base = 0
    for _ in range(4):
        p0, n, planes = least + rng.choice([0, rng.randrange(900)]), rng.randrange(1, 40), rng.randrange(3, 20)
        prefix = prefix_keys(least, base, window, sinks, planes) if base else []
        for ut in range(-(-n // TT)):
            parts = prefix + own_keys(p0, n, base, ut, TT, window, sinks, planes)
            seen = [s for a, b in parts for s in range(a, b)]
            assert len(seen) == len(set(seen)) and all(a < b for a, b in parts)
            for t in range(p0 + ut * TT, p0 + min(n, (ut + 1) * TT)):
                kept = {s for s in range(t + 1) if not window or s > t - window or s < sinks}
                assert kept <= set(seen), (t, sorted(kept - set(seen))[:5])


def plan(tables, p0s, ps, window, sinks):
    """Shared positions of a group as the plan finds them, and the row whose pages serve."""
    leader = min(range(len(p0s)), key=lambda b: (p0s[b], b))
    p0 = p0s[leader]
    lo = max(0, p0 - window + 1) if window else 0
    e_sink = -(-sinks // ps)
    entries = list(range(min(lo // ps, e_sink))) + list(range(lo // ps, p0 // ps))
    shared = len(entries)
    for b, row in enumerate(tables):
        my_lo = max(0, p0s[b] - window + 1) if window else 0
        for i, j in enumerate(entries):
            if ((j + 1) * ps > my_lo or j < e_sink) and row[j] != tables[leader][j]:
                shared = min(shared, i)
                break
    n_sinks = min(lo // ps, e_sink)
    return (0 if shared < n_sinks else (lo // ps + shared - n_sinks) * ps), leader


@pytest.mark.parametrize("seed", range(60))
def test_what_is_shared_serves_every_sequence(seed):
    rng = random.Random(100 + seed)
    ps, window = rng.choice([16, 32]), rng.choice([0, 40, 300])
    sinks = rng.choice([0, 1, 50]) if window else 0
    p0s = [rng.randrange(0, 700) for _ in range(rng.randrange(2, 6))]
    width = max(p0s) // ps + 1
    page = lambda b, j: j if rng.random() < 0.97 else 1000 * (b + 1) + j  # noqa: E731  (mostly the same page)
    tables = []
    for b, p in enumerate(p0s):
        lo = max(0, p - window + 1) if window else 0
        tables.append([-1 if (j + 1) * ps <= lo and j * ps >= sinks and rng.random() < 0.5 else page(b, j) for j in range(width)])
    base, leader = plan(tables, p0s, ps, window, sinks)
    assert base % ps == 0 and base <= min(p0s)
    for b, p in enumerate(p0s):  # every key below base that the first new token keeps lies in the leader's page
        for s in range(base):
            if not window or s > p - window or s < sinks:
                assert tables[b][s // ps] == tables[leader][s // ps], (b, s)
