"""Attention of shared prefixes where q_start goes up and down: what that makes of the groups and the sequences,
and that it is reported."""
import time

import pytest
import torch

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
