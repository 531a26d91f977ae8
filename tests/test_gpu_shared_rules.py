"""What swa_paged_attend_shared takes for shared, at the least number of positions of use that it shares: a prefix that is computed
as one, of more rows than a stretch takes, waits for producers, which are planted to stop; one that is not does not."""
import os
import re

import pytest

from test_gpu_paged_shared import Shared, call, run, swa  # noqa: F401  (swa: the module's fixture)

pytestmark = pytest.mark.gpu

SOURCE = os.path.join(os.path.dirname(__file__), "..", "sliding_window_attention_swa_gb300", "csrc", "swa_paged_shared.cu")
LEAST = int(re.search(r"constexpr int kLeastShared = (\d+);", open(SOURCE).read()).group(1))
SWA_ERR_TIMEOUT = 4


def of_use(seqs, prefix, window, page):
    """Positions below the prefix's last whole page that two sequences at least have a use for."""
    p0 = sorted(p for p, _ in seqs)
    base = min(prefix, p0[0]) // page * page
    return base - (max(0, p0[1] - window + 1) if window else 0)


@pytest.mark.parametrize("name,prefix,seqs,window", [
    ("least", LEAST, [(LEAST + i, 1) for i in range(30)], 0),
    ("one less", LEAST + 15 - 16, [(LEAST + i, 1) for i in range(30)], 0),
    ("all but one hold less", LEAST + 400, [(LEAST - 1 + 16 * (i == 0), 1) for i in range(30)], 0),
    ("the least p0 decides", LEAST + 400, [(LEAST + 100 * (i > 0), 1) for i in range(30)], 0),
    # (1008 positions, the second window starts at 1008 - LEAST)
    ("a window's", 1008, [(1008, 1)] + [(1008 + 299 - LEAST, 1)] * 29, 300),
    ("one less in a window", 1008, [(1008, 1)] + [(1008 + 300 - LEAST, 1)] * 29, 300),
])
def test_the_least_that_is_shared(swa, name, prefix, seqs, window):  # noqa: F811
    x = Shared(140, [(prefix, seqs)], 8, 2, 64, 16, window)
    shared = of_use(seqs, prefix, window, 16) >= LEAST
    assert shared == (name in ("least", "the least p0 decides", "a window's")), of_use(seqs, prefix, window, 16)
    swa.swa_debug_set_faults(band_stop_fill=0)
    try:
        call(swa, x, q_start=None)
        st, words = swa.swa_read_device_errors()
    finally:
        swa.swa_debug_set_faults()
    assert (st == SWA_ERR_TIMEOUT) == shared and words["prefill"] == (swa.DEVERR_WAIT_TIMEOUT if shared else 0), words
    run(swa, x, q_start=None)


@pytest.mark.parametrize("sinks", [0, 5, 130])
@pytest.mark.parametrize("D,ps", [(64, 16), (128, 64), (256, 128)])
def test_rows_of_a_tile_that_keep_nothing_of_the_prefix(swa, D, ps, sinks):  # noqa: F811
    """Two sequences look at what all share, the windows of the others begin behind it (their sinks do not): a tile's
    rows of both kinds, in two tiles of rows."""
    seqs = [(2048, 1), (2058, 1)] + [(2600 + 7 * i, 1) for i in range(60)]
    assert of_use(seqs, 2048, 300, ps) >= LEAST and len(seqs) * 4 > 128
    for order in (seqs, seqs[::-1], seqs[30:] + seqs[:30]):
        x = Shared(141, [(2048, order)], 8, 2, D, ps, 300, sinks)
        run(swa, x, q_start=None)
        run(swa, x, True, q_start=None)
