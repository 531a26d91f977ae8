"""The paged cache's operators through the debug build of the library (libswa_debug.so), whose kernels
check every index they compute -- page boxes, query tiles, rows of o, lse and counts -- against
the tensor it addresses before the access.  The results must match the references as before, and
no check may fire."""
import pytest

import test_gpu_pages as PAGES
import test_gpu_paged as PAGED

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def swa():
    import sliding_window_attention_swa_gb300 as m

    prev = m.use_library(m.load_library(m.build(debug=True)))
    try:
        yield m
    finally:
        m.use_library(prev)


@pytest.fixture(autouse=True)
def clean(swa):
    yield
    assert swa.load_library()._name.endswith("libswa_debug.so")
    st, words = swa.swa_read_device_errors()
    assert st == 0 and words == {"prefill": 0, "split": 0, "cache": 0}, words


@pytest.mark.parametrize("append", [False, True], ids=["stored", "append"])
@pytest.mark.parametrize("case", PAGED.DECODE, ids=str)
def test_one_token_a_sequence(swa, case, append):
    PAGED.test_one_token_a_sequence(swa, case, append)


@pytest.mark.parametrize("case", PAGED.CHUNK, ids=str)
def test_ragged_batch(swa, case):
    PAGED.test_ragged_batch(swa, case, True)


@pytest.mark.parametrize("heads", [(16, 1, 128), (16, 1, 256)], ids=str)
def test_more_units_than_two_waves(swa, heads):
    PAGED.test_more_units_than_two_waves(swa, heads)


@pytest.mark.parametrize("heads", [(12, 4, 128), (5, 5, 64), (6, 2, 256)], ids=str)
def test_shared_units_with_rows_missing(swa, heads):
    PAGED.test_shared_units_with_rows_missing(swa, heads)


def test_layouts_and_sizes(swa):
    PAGED.test_strided_rows(swa)
    PAGED.test_append_alone(swa)
    for hint in (0, 1):
        PAGED.test_broken_device_data(swa, hint)


@pytest.mark.parametrize("hint", [0, 1])
def test_positions_that_no_query_keeps(swa, hint):
    for case in ((16, 16, 128, 128, 130, 0), (4, 4, 64, 64, 300, 130), (6, 2, 256, 32, 65, 37)):
        PAGED.test_positions_that_no_query_keeps_may_hold_anything(swa, case, hint)


def test_pages(swa):
    PAGES.test_reserve_when_the_pool_runs_out(swa)
    PAGES.test_free(swa, 40, 90, 4000, 32, 0, True)
    PAGES.test_fork(swa, 6, 200, (3, 2, 32, 128))
    PAGES.test_compact(swa, 30, 9, 400, (1, 2, 32, 64), False)
    PAGES.test_serving_run(swa)


@pytest.mark.parametrize("inplace", [True, False])
def test_pages_of_every_plan(swa, inplace):
    # one cluster's plan of a fork and the grids', tables and pools of several scan steps
    PAGES.test_forks_of_forks(swa, 40, 30, 4, inplace)
    PAGES.test_forks_of_forks(swa, 300, 400, 8, inplace)
    PAGES.test_compact(swa, 9, 4000, 50000, (1, 1, 1, 8), inplace)
    PAGES.test_free(swa, 700, 33, 20000, 1, 3, inplace)
    PAGES.test_reserve(swa, 1500, 4, 20000, 128)
    PAGES.test_copy(swa, 3)


def test_tiles_from_hbm_and_pairs(swa):
    PAGED.test_tiles_that_come_from_hbm(swa, 1024, 400, 32)
    PAGED.test_pairs_of_one_key_tile_behind_single_query_tiles(swa, (32, 8, 128))
    PAGED.test_sequences_that_overlap_are_no_work(swa, 64, 0)
