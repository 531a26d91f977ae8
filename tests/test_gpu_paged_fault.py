"""Paged attention whose producers stop: waits that run out are reported, and the next call is right.

swa_debug_set_faults lets a producer stop issuing copies at a chosen fill or stage, so the other
roles' waits, each bounded (about 2.1 s), run out; the CTA drains what it did issue and
returns.  Nothing faults or hangs.
"""
import time

import pytest
import torch

import paged_reference as R
from test_gpu_paged import run, swa  # noqa: F401  (swa: the module's fixture)

pytestmark = pytest.mark.gpu

SWA_ERR_TIMEOUT = 4

# (a CTA's share of these: at least four tiles, two fills each, and at head dim 256 two of the query tile)
STOPS = [
    # Hq, Hkv, D, (history, new tokens) of each sequence, window, fault, word that reports it
    pytest.param(8, 2, 64, [(900, 70), (30, 5)], 0, dict(band_stop_fill=0), "prefill", id="d64-first-fill"),
    pytest.param(8, 2, 64, [(3000, 70), (30, 5)], 0, dict(band_stop_fill=5), "prefill", id="d64"),
    pytest.param(8, 2, 128, [(3000, 70), (30, 5)], 0, dict(band_stop_fill=4), "prefill", id="d128-one-tile"),
    pytest.param(16, 16, 128, [(40, 5000)], 200, dict(band_stop_fill=3), "prefill", id="d128-two-tiles"),
    pytest.param(4, 2, 256, [(3000, 70), (30, 5)], 0, dict(band_stop_fill=1), "prefill", id="d256-query-tile"),
    pytest.param(4, 2, 256, [(3000, 70), (30, 5)], 0, dict(band_stop_fill=6), "prefill", id="d256"),
    pytest.param(8, 2, 128, [(3000, 1), (30, 1)], 0, dict(split_stop_stage=0), "split", id="few-rows-first-stage"),
    pytest.param(8, 2, 128, [(40000, 1), (9000, 1)], 0, dict(split_stop_stage=2), "split", id="few-rows"),
]


@pytest.mark.parametrize("Hq,Hkv,D,seqs,window,fault,word", STOPS)
def test_producer_stop_times_out_and_recovers(swa, Hq, Hkv, D, seqs, window, fault, word):  # noqa: F811
    x = R.Batch(70, seqs, Hq, Hkv, D, 16, window)
    q, k, v = x.q.cuda(), x.k_pages.cuda(), x.v_pages.cuda()
    table, p0 = x.table.cuda(), x.p0.cuda()
    start = x.q_start.cuda() if word == "prefill" else None
    swa.swa_debug_set_faults(**fault)
    try:
        t0 = time.time()
        swa.swa_paged_attend(q, k, v, table, p0, window, q_start=start)
        st, words = swa.swa_read_device_errors()
        waited = time.time() - t0
    finally:
        swa.swa_debug_set_faults()
    assert st == SWA_ERR_TIMEOUT, (st, words)
    assert words == {**{"prefill": 0, "split": 0, "cache": 0}, word: swa.DEVERR_WAIT_TIMEOUT}, words
    assert waited < 30.0
    run(swa, x, q_start=start)


@pytest.mark.parametrize("stop", [9, 12])
@pytest.mark.parametrize("Hq,Hkv,D,seqs,window", [
    pytest.param(8, 2, 64, [(3000, 70)] * 24, 0, id="d64"),
    pytest.param(8, 2, 128, [(3000, 70)] * 24, 0, id="d128-one-tile"),
    pytest.param(16, 16, 128, [(900, 5000)], 700, id="d128-two-tiles"),
    pytest.param(4, 2, 256, [(1500, 70)] * 24, 0, id="d256"),
    pytest.param(4, 2, 256, [(i % 40, 3) for i in range(600)], 0, id="d256-pieces-of-a-tile"),
])
def test_producers_that_stop_late(swa, Hq, Hkv, D, seqs, window, stop):  # noqa: F811
    """... when both producers have been through every slot of the ring: only the waits behind the missing
    fills run out, not the producers' own for their copies."""
    x = R.Batch(72, seqs, Hq, Hkv, D, 16, window)
    q, k, v, table, p0, start = (t.cuda() for t in (x.q, x.k_pages, x.v_pages, x.table, x.p0, x.q_start))
    swa.swa_debug_set_faults(band_stop_fill=stop)
    try:
        t0 = time.time()
        swa.swa_paged_attend(q, k, v, table, p0, window, q_start=start)
        st, words = swa.swa_read_device_errors()
        waited = time.time() - t0
    finally:
        swa.swa_debug_set_faults()
    assert st == SWA_ERR_TIMEOUT, (st, words)
    assert words == {"prefill": swa.DEVERR_WAIT_TIMEOUT, "split": 0, "cache": 0}, words
    assert waited < 4.0, waited  # one limit of about 2.1 s, at the same time everywhere
    if stop == 12:
        run(swa, x)


@pytest.mark.parametrize("heads", [(16, 16, 128), (32, 8, 128)], ids=str)
def test_units_of_two_query_tiles(swa, heads):  # noqa: F811
    # head dim 128 and many tokens: pairs of tiles, a last pair of one tile, pairs whose second tile has
    # a few rows, and pairs that several CTAs share
    Hq, Hkv, D = heads
    for seqs, w in (([(5, 2600), (700, 2617), (0, 33), (64, 129)], 300), ([(9, 4990), (6000, 130)], 0 if Hkv == 8 else 700)):
        run(swa, R.Batch(71, seqs, Hq, Hkv, D, 32, w, 2 if w else 0), want_counts=False)
