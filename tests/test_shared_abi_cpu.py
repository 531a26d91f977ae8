"""The C entry points of the attention of shared prefixes on the host: invalid arguments refused before anything is
launched, and what the workspace depends on (no GPU needed)."""
import ctypes

import pytest

import sliding_window_attention_swa_gb300 as swa
from test_paged_abi_cpu import BIG, FAKE, pair, valid_paged


@pytest.fixture(scope="module")
def lib():
    swa.build()
    return swa.load_library()


@pytest.mark.parametrize("mutate,status", [
    (lambda p, c, g: setattr(p, "q", None), 1),
    (lambda p, c, g: setattr(p, "lse", None), 1),
    (lambda p, c, g: setattr(p, "p0", None), 1),
    (lambda p, c, g: setattr(p, "q_start", None), 1),
    (lambda p, c, g: setattr(p, "N", -1), 1),
    (lambda p, c, g: setattr(p, "H_q", 34), 2),
    (lambda p, c, g: setattr(p, "window", -1), 1),
    (lambda p, c, g: setattr(p, "n_sink", -1), 1),
    (lambda p, c, g: setattr(p, "k_new", FAKE), 1),
    (lambda p, c, g: setattr(p, "o_strides", pair(0, 128)), 2),
    (lambda p, c, g: setattr(c, "page_size", 24), 2),
    (lambda p, c, g: setattr(c, "d_h", 96), 2),
    (lambda p, c, g: g.update(start=None), 1),
    (lambda p, c, g: g.update(start=FAKE + 2), 2),
    (lambda p, c, g: g.update(n=0), 1),
    (lambda p, c, g: g.update(n=-3), 1),
    (lambda p, c, g: g.update(n=8193), 2),
    (lambda p, c, g: g.update(ws=None), 5),
    (lambda p, c, g: g.update(ws=FAKE + 64), 5),
    (lambda p, c, g: g.update(bytes=1000), 5),
])
def test_attend_shared_rejects(lib, mutate, status):
    p, c = valid_paged()
    g = dict(start=FAKE, n=3, ws=FAKE, bytes=BIG)
    mutate(p, c, g)
    refs = ctypes.byref(p), ctypes.byref(c)
    assert lib.swa_paged_attend_shared(*refs, g["start"], g["n"], g["ws"], g["bytes"], None) == status
    if status != 5 and g["start"] == FAKE:
        assert lib.swa_paged_shared_workspace_size(*refs, g["n"]) == 0


def test_null_structures_and_nothing_to_do(lib):
    p, c = valid_paged()
    assert lib.swa_paged_attend_shared(None, ctypes.byref(c), FAKE, 1, FAKE, BIG, None) == 1
    assert lib.swa_paged_attend_shared(ctypes.byref(p), None, FAKE, 1, FAKE, BIG, None) == 1
    p.N = 0
    need = lib.swa_paged_shared_workspace_size(ctypes.byref(p), ctypes.byref(c), 1)
    assert need > 0
    assert lib.swa_paged_attend_shared(ctypes.byref(p), ctypes.byref(c), FAKE, 1, FAKE, need, None) == 0


def test_workspace_grows_with_the_rows(lib):
    """... and is the same for any device data: N, the groups, the heads and the hint decide."""
    p, c = valid_paged()

    def size(N, groups=3, max_q=0):
        p.N, p.max_q, c.B = N, max_q, 40
        return lib.swa_paged_shared_workspace_size(ctypes.byref(p), ctypes.byref(c), groups)

    for hint in (0, 1):
        sizes = [size(N, max_q=hint) for N in (1, 2, 16, 17, 40, 41, 300, 5000, 100000, 1 << 20)]
        # both parts' results of every row, fp32 (with a hint of few rows in planes, of which few rows have more)
        for N, now in zip((1, 2, 16, 17, 40, 41, 300, 5000, 100000, 1 << 20), sizes):
            assert now >= 2 * N * p.H_q * c.d_h * 4, (N, now)
        assert hint or sizes == sorted(sizes)
        assert hint or size(40, 8192) >= size(40, 1)
    p.q_start, p.N = None, c.B
    assert lib.swa_paged_shared_workspace_size(ctypes.byref(p), ctypes.byref(c), 3) > 0
