"""Attention of shared prefixes whose producers stop: waits that run out are reported, and the next call is
right (swa_debug_set_faults; nothing faults or hangs)."""
import time

import pytest
import torch

from test_gpu_paged_shared import Shared, call, run, swa  # noqa: F401  (swa: the module's fixture)

pytestmark = pytest.mark.gpu

SWA_ERR_TIMEOUT = 4
FEW = [(2000, [(2000 + i, 1) for i in range(30)]), (500, [(500, 1)] * 3)]
MANY = [(2000, [(2000 + i, 7) for i in range(30)]), (500, [(500, 90)] * 3)]


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
