"""Attention of shared prefixes whose producers stop: waits that run out are reported, and the next call is
right (swa_debug_set_faults; nothing faults or hangs)."""
import time

import pytest
import torch

from test_gpu_paged_shared import Shared, call, run, swa  # noqa: F401  (swa: the module's fixture)

pytestmark = pytest.mark.gpu

SWA_ERR_TIMEOUT = 4
FEW = [(2000, [(2000 + i, 1) for i in range(30)]), (500, [(500, 1)] * 3)]
MANY = [(8000, [(8000 + i, 7) for i in range(30)]), (500, [(500, 90)] * 3)]


@pytest.mark.parametrize("groups,D,hint,fault,word", [
    pytest.param(FEW, 64, 1, dict(split_stop_stage=0), "split", id="stretches-first-step"),
    pytest.param(FEW, 128, 1, dict(split_stop_stage=3), "split", id="stretches-d128"),
    pytest.param(FEW, 256, 1, dict(split_stop_stage=2), "split", id="stretches-d256"),
    pytest.param(FEW, 64, 1, dict(band_stop_fill=0), "prefill", id="prefix-first-fill"),
    pytest.param(FEW, 128, 1, dict(band_stop_fill=3), "prefill", id="prefix-d128"),
    pytest.param(FEW, 256, 1, dict(band_stop_fill=3), "prefill", id="prefix-d256"),
    pytest.param(MANY, 128, 0, dict(band_stop_fill=2), "prefill", id="both-parts-d128"),
    pytest.param(MANY, 256, 0, dict(band_stop_fill=2), "prefill", id="both-parts-d256"),
])
def test_producer_stop_times_out_and_recovers(swa, groups, D, hint, fault, word):  # noqa: F811
    x = Shared(70, groups, 8, 2, D, 16)
    swa.swa_debug_set_faults(**fault)
    try:
        t0 = time.time()
        call(swa, x, max_q=hint)
        st, words = swa.swa_read_device_errors()
        waited = time.time() - t0
    finally:
        swa.swa_debug_set_faults()
    assert st == SWA_ERR_TIMEOUT, (st, words)
    assert words == {**{"prefill": 0, "split": 0, "cache": 0}, word: swa.DEVERR_WAIT_TIMEOUT}, words
    assert waited < 30.0
    run(swa, x, max_q=hint)
    torch.cuda.synchronize()


@pytest.mark.parametrize("what,shared", [("same", True), ("window", True), ("freed", True), ("sinks", True),
                                         ("other", False), ("behind", False), ("short", False)])
def test_what_is_shared(swa, what, shared):  # noqa: F811
    """A group whose prefix goes to the many-row kernel waits for its producers, one that shares nothing does not."""
    seqs = [(2000 + i, 1) for i in range(30)]
    window, sinks = {"window": (700, 0), "freed": (700, 0), "sinks": (700, 40), "behind": (300, 0)}.get(what, (0, 0))
    if what == "freed":  # (a page that the first sequence needs and the others have given up)
        seqs = [(2000, 1)] + [(2300 + i, 1) for i in range(29)]
    if what == "behind":  # (all but the first look behind what they share)
        seqs = [(2250, 1)] + [(2700 + i, 1) for i in range(29)]
    x = Shared(71, [(150 if what == "short" else 2000, seqs)], 8, 2, 64, 16, window, sinks)
    if what == "other":  # one sequence has a page of its own at the start, with the same tokens
        free = [p for p in range(x.n_pages) if p not in x.table.unique().tolist()][0]
        x.k_pages[free], x.v_pages[free] = x.k_pages[int(x.table[3, 0])], x.v_pages[int(x.table[3, 0])]
        x.table[3, 0] = free
    swa.swa_debug_set_faults(band_stop_fill=0)
    try:
        call(swa, x, q_start=None)
        st, words = swa.swa_read_device_errors()
    finally:
        swa.swa_debug_set_faults()
    assert (st == SWA_ERR_TIMEOUT) == shared and words["prefill"] == (swa.DEVERR_WAIT_TIMEOUT if shared else 0), words
    run(swa, x, q_start=None)
