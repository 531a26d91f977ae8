"""The rotation in place on the host: rows that would lie elsewhere than they lay are refused before anything is launched
(no GPU needed)."""
import ctypes

import pytest

import sliding_window_attention_swa_gb300 as swa
from test_paged_abi_cpu import FAKE, pair, valid_paged


@pytest.fixture(scope="module")
def lib():
    swa.build()
    return swa.load_library()


@pytest.mark.parametrize("N,heads,strides,status", [
    (9, 8, (2048, 128), 1), (9, 8, (1024, 256), 1), (9, 2, (512, 64), 1), (1, 8, (1024, 64), 1), (2, 2, (1032, 128), 1),
    (0, 8, (2048, 128), 0), (0, 8, (1024, 128), 0),  # (of no rows nothing lies elsewhere)
])
def test_strides_of_queries_in_place(lib, N, heads, strides, status):
    p, c = valid_paged()
    p.q = p.o = FAKE
    p.N, p.H_q, c.B = N, heads, 4
    p.o_strides = pair(*strides)
    assert lib.swa_paged_rope_append(ctypes.byref(p), ctypes.byref(c), ctypes.byref(swa.SwaRope(FAKE, 1000, 64, 0)), None) == status
