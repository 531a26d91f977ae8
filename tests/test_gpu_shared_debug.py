"""The rotation and the attention of shared prefixes through the debug build of the library (libswa_debug.so),
whose kernels check every index they compute before the access, and which shares prefixes of chunks however
short.  The results must match the references as before, and no check may fire."""
import pytest

import test_gpu_paged_shared as SHARED
import test_gpu_rope as ROPE

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


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", ROPE.SHAPES, ids=str)
def test_rotation(swa, shape, interleaved):
    ROPE.test_append(swa, shape, interleaved)


def test_rotation_of_parts_and_broken_data(swa):
    for D in (64, 128, 256):
        ROPE.test_parts_and_layouts(swa, D)
    ROPE.test_broken_device_data(swa)
    ROPE.test_table(swa, 96, 1000)


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("shape", SHARED.SHAPES, ids=str)
def test_one_token_a_sequence(swa, shape, append):
    SHARED.test_one_token_a_sequence(swa, shape, append)


@pytest.mark.parametrize("hint", [0, 1])
@pytest.mark.parametrize("shape", SHARED.SHAPES, ids=str)
def test_ragged_groups(swa, shape, hint):
    SHARED.test_ragged_groups(swa, shape, hint)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("seed", range(12))
def test_drawn_batches(swa, seed, D):
    SHARED.test_drawn_batches(swa, seed, D)


def test_many_groups_and_broken_data(swa):
    SHARED.test_as_many_sequences_and_groups_as_a_call_takes(swa)
    SHARED.test_broken_device_data(swa)


@pytest.mark.parametrize("hint", [0, 1])
def test_lists_in_disorder(swa, hint):
    SHARED.test_sequences_that_overlap(swa, 64, hint)


@pytest.mark.parametrize("D,ps", [(64, 16), (128, 32), (256, 64)])
def test_groups_and_long_prefixes(swa, D, ps):
    SHARED.test_same_as_each_by_itself(swa, D, ps)
    SHARED.test_long_prefixes_and_many_groups(swa, D, ps)


def test_chunks(swa):
    SHARED.test_units_of_two_query_tiles(swa)
    SHARED.test_rows_that_keep_nothing_of_the_prefix(swa)
    SHARED.test_chunks_behind_long_prefixes(swa, (8, 2, 64, 64, 5500, 200), True)
    for case in ((8, 2, 128, 16, 400, 4), (4, 4, 64, 64, 300, 130), (6, 2, 256, 32, 365, 37)):
        SHARED.test_positions_that_no_query_keeps_may_hold_anything(swa, case)
