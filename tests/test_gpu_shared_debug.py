"""The rotation and the attention of shared prefixes through the debug build of the library (libswa_debug.so),
whose kernels check every index they compute before the access.  The results must match the references as
before, and no check may fire."""
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
@pytest.mark.parametrize("seed", range(4))
def test_drawn_batches(swa, seed, D):
    SHARED.test_drawn_batches(swa, seed, D)


def test_many_groups_and_broken_data(swa):
    SHARED.test_as_many_sequences_and_groups_as_a_call_takes(swa)
    SHARED.test_broken_device_data(swa)


@pytest.mark.parametrize("hint", [0, 1])
def test_lists_in_disorder(swa, hint):
    SHARED.test_sequences_that_overlap(swa, 64, hint)
