"""Attention of shared prefixes where q_start goes up and down: what that makes of the groups and the sequences,
and that it is reported."""
import random
import time

import pytest
import torch

import paged_reference as R
from test_gpu_paged_shared import Shared, call, run, swa  # noqa: F401  (swa: the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 256])
def test_groups_of_the_same_rows_are_none(swa, D):  # noqa: F811
    """Pairs of sequences that have all rows of the batch between them, each pair a group, and behind each pair a
    sequence that goes back to the first row.  If they shared, the batch's rows would be computed once a group.  A
    prefix in tiles waits for its producers, which are planted to stop: no wait may run out."""
    pairs, half = 40, 20
    x = Shared(90, [(700, [(700, half), (700, half), (700, 0)])] * pairs, 4, 2, D, 16)
    good, groups = x.q_start, x.groups
    x.N = 2 * half
    x.q = x.q[:x.N]
    x.q_start = torch.tensor([0] + [half, x.N, 0] * pairs, dtype=torch.int32)
    x.groups = torch.tensor([y for i in range(pairs) for y in (3 * i, 3 * i + 2)] + [3 * pairs], dtype=torch.int32)
    swa.swa_debug_set_faults(band_stop_fill=0)
    try:
        t0 = time.time()
        call(swa, x, max_q=1)
        st, words = swa.swa_read_device_errors()
        waited = time.time() - t0
    finally:
        swa.swa_debug_set_faults()
    assert st == 1 and words == {"prefill": 0, "split": 0, "cache": swa.DEVERR_BAD_POSITION}, words
    assert waited < 5.0
    # and so with many new tokens a sequence; the same sequences in order share as before
    call(swa, x)
    st, words = swa.swa_read_device_errors()
    assert st == 1 and words["split"] == 0 and words["cache"] == swa.DEVERR_BAD_POSITION, words
    x = Shared(90, [(700, [(700, half), (700, half), (700, 0)])] * pairs, 4, 2, D, 16)
    assert torch.equal(good, x.q_start) and torch.equal(groups, x.groups)
    run(swa, x, max_q=1)


def test_a_list_that_goes_down_at_its_end(swa):  # noqa: F811
    """As many sequences as a call takes, the last of which goes down: seen by every block, and there is no group."""
    x = Shared(91, [(300, [(300, 1)] * 4095), (300, [(301, 1)] * 4097)], 2, 1, 64, 64)
    x.q_start[-1] -= 2
    swa.swa_debug_set_faults(band_stop_fill=0)
    try:
        call(swa, x, max_q=1)
        st, words = swa.swa_read_device_errors()
    finally:
        swa.swa_debug_set_faults()
    assert st == 1 and words == {"prefill": 0, "split": 0, "cache": swa.DEVERR_BAD_POSITION}, words


def check_rows(swa, x, got, kept):  # noqa: F811
    """Rows of the sequences `kept` hold their results, all others are as they were."""
    o, lse, cnt, *_ = got
    mine = torch.zeros(x.N, dtype=torch.bool)
    for b in kept:
        q0, n = int(x.q_start[b]), x.seqs[b][1]
        mine[q0:q0 + n] = True
        R.check(o[q0:q0 + n], lse[q0:q0 + n], cnt[q0:q0 + n], x.reference(b), f"sequence {b}")
    assert (o.cpu()[~mine] == 7).all() and (lse.cpu()[~mine] == 7).all() and (cnt.cpu()[~mine] == 7).all()


@pytest.mark.parametrize("hint", [0, 4])
@pytest.mark.parametrize("D,B", [(64, 9), (128, 300), (256, 40)])
def test_sequences_beside_broken_ones(swa, D, B, hint):  # noqa: F811
    """An entry of q_start that is too small or too large breaks the two sequences that it parts; all the others have
    their results, whatever their number."""
    good = Shared(92, [(260, [(260 + i % 5, 1 + i % 4) for i in range(B)])], 4, 2, D, 16)
    for entry in sorted({1, 2, B // 2, B - 2}):
        for wrong in (-3, good.N + 1, (1 << 31) - 1):
            start = good.q_start.clone()
            good.q_start[entry] = wrong
            got = call(swa, good, max_q=hint)
            good.q_start = start
            st, words = swa.swa_read_device_errors()
            assert st == 1 and words == {"prefill": 0, "split": 0, "cache": swa.DEVERR_BAD_POSITION}, words
            check_rows(swa, good, got, [b for b in range(B) if b not in (entry - 1, entry)])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_of_sequences_with_rows_in_common_none_is_taken(swa, D):  # noqa: F811
    """Few new tokens: rows that two sequences have stay as they were, the others hold their results."""
    x = Shared(93, [(300, [(300, 4)] * 30 + [(400, 4)])], 4, 2, D, 16, lead=2, tail=3)  # (room for 16 more in a row)
    start = x.q_start.clone()
    # sequence 4 ends where 2 begins, and 5 begins there: it has the rows of 2 to 5
    x.q_start[5] = start[2]
    x.seqs[5] = (300, int(start[6] - start[2]))
    got = call(swa, x, max_q=4)
    st, words = swa.swa_read_device_errors()
    assert st == 1 and words == {"prefill": 0, "split": 0, "cache": swa.DEVERR_BAD_POSITION}, words
    check_rows(swa, x, got, [b for b in range(31) if b not in (2, 3, 4, 5)])


@pytest.mark.parametrize("hint", [0, 1])
def test_as_many_sequences_as_a_call_takes_have_all_rows_each(swa, hint):  # noqa: F811
    x = Shared(94, [(64, [(64, 1)] * 8191 + [(700, 1)])], 16, 1, 64, 16)  # (room for 600 in a row)
    x.N = 600
    x.q = x.q[:600]
    x.q_start = torch.tensor([0, 600] * 4096 + [0], dtype=torch.int32)
    t0 = time.time()
    o, lse, *_ = call(swa, x, max_q=hint)
    st, words = swa.swa_read_device_errors()
    assert time.time() - t0 < 20.0
    assert st == 1 and words == {"prefill": 0, "split": 0, "cache": swa.DEVERR_BAD_POSITION}, words
    assert hint == 0 or ((o == 7).all() and (lse == 7).all())
    y = Shared(95, [(260, [(260, 1)] * 64)], 16, 1, 64, 16)
    run(swa, y, max_q=hint)


@pytest.mark.parametrize("library", ["release", "debug"])
@pytest.mark.parametrize("seed", range(10))
def test_drawn_lists_in_disorder(swa, seed, library):  # noqa: F811
    """Some entries of q_start are anything: with few new tokens exactly the sequences in range that have no row in
    common with another have their results, and all other rows stay as they were; no check of the bounds-checking build
    fires."""
    prev = swa.use_library(swa.load_library(swa.build(debug=True))) if library == "debug" else None
    try:
        rng = random.Random(seed)
        B = rng.choice([3, 12, 40, 200])
        seqs = [(400 + rng.randrange(60), rng.randrange(5)) for _ in range(B)] + [(900, 1)]  # (room in the table's rows)
        x = Shared(96 + seed, [(400, seqs)], 4, 2, rng.choice([64, 128]), 16, lead=rng.randrange(3), tail=rng.randrange(4))
        good = x.q_start.clone()
        for _ in range(6):
            for _ in range(rng.randrange(1, 5)):
                x.q_start[rng.randrange(B + 2)] = rng.choice([-1, 0, x.N, x.N + 1, rng.randrange(x.N + 1), int(good[rng.randrange(B)])])
            start = x.q_start.tolist()
            ok = [a >= 0 and a <= b <= x.N for a, b in zip(start, start[1:])]
            down = any(a > b for a, b in zip(start, start[1:]))
            spans = [(a, b) if y else (0, 0) for a, b, y in zip(start, start[1:], ok)]
            common = lambda s, t: s[0] < s[1] and t[0] < t[1] and s[0] < t[1] and t[0] < s[1]  # noqa: E731
            kept = [b for b in range(B + 1) if ok[b] and spans[b][1] - spans[b][0] == x.seqs[b][1] > 0
                    and not any(common(spans[b], s) for c, s in enumerate(spans) if c != b)]
            # (others in range whose number of rows is not their own: computed, of keys that the batch does not have)
            loose = [b for b in range(B + 1) if ok[b] and b not in kept and spans[b][0] < spans[b][1]
                     and not any(common(spans[b], s) for c, s in enumerate(spans) if c != b)]
            o, lse, cnt, *_ = call(swa, x, max_q=4)
            st, words = swa.swa_read_device_errors()
            assert words["prefill"] == words["split"] == 0, words
            assert words["cache"] & ~(swa.DEVERR_BAD_POSITION | swa.DEVERR_BAD_PAGE) == 0, words
            assert bool(words["cache"] & swa.DEVERR_BAD_POSITION) == (down or not all(ok)), words
            mine = torch.zeros(x.N, dtype=torch.bool)
            for b in kept:
                q0, q1 = spans[b]
                mine[q0:q1] = True
                R.check(o[q0:q1], lse[q0:q1], cnt[q0:q1], x.reference(b), f"sequence {b}")
            for b in loose:
                mine[spans[b][0]:spans[b][1]] = True
            assert (o.cpu()[~mine] == 7).all() and (lse.cpu()[~mine] == 7).all() and (cnt.cpu()[~mine] == 7).all()
            x.q_start = good.clone()
    finally:
        if prev is not None:
            swa.use_library(prev)
