"""The size of swa_paged_attend_shared's workspace: bounded by the results, whatever the number of groups, and never
smaller for a larger call (no GPU needed)."""
import ctypes

import pytest

import sliding_window_attention_swa_gb300 as swa
from test_paged_abi_cpu import FAKE, valid_paged

MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    swa.build()
    return swa.load_library()


def size(lib, N, groups, heads=(32, 8, 128), B=None, max_q=0):
    """B None: one token a sequence."""
    p, c = valid_paged()
    p.q_start = None if B is None else FAKE
    p.N, c.B, p.max_q = N, N if B is None else B, max_q
    p.H_q, c.H_kv, c.d_h = heads
    return lib.swa_paged_shared_workspace_size(ctypes.byref(p), ctypes.byref(c), groups)


@pytest.mark.parametrize("N,groups,B,max_q,heads,most", [
    (4, 1, None, 0, (32, 8, 128), 32), (64, 1, None, 0, (32, 8, 128), 100), (256, 1, None, 0, (32, 8, 128), 120),
    (1024, 1, None, 0, (32, 8, 128), 180), (2048, 1, None, 0, (32, 8, 128), 300), (8192, 1, None, 0, (32, 8, 128), 900),
    (8192, 4096, None, 0, (32, 8, 128), 1200), (1024, 1, 256, 4, (32, 8, 128), 200), (160, 2, 50, 8, (16, 8, 256), 160),
    (8192, 1, None, 0, (8, 8, 64), 160),
])
def test_bounded(lib, N, groups, B, max_q, heads, most):
    assert 0 < size(lib, N, groups, heads, B, max_q) <= most * MB


@pytest.mark.parametrize("heads", [(32, 8, 128), (16, 1, 64), (8, 1, 128), (12, 12, 64), (6, 2, 256), (20, 4, 128)])
def test_a_few_times_the_results(lib, heads):
    """Own parts in three planes, the prefix's in one of tiles and, for the groups' tokens, three of stretches; the
    stretches for every resident warp (2432 at most; eight a warp, of up to 16 / G tokens), the two kernels' slots."""
    Hq, H, D = heads
    TT = 16 // (Hq // H)
    row = Hq * (4 * D + 8)
    slots = 2 * 2 * 152 * 2 * 128 * (4 * D + 8)
    for N in (1, 2, 3, 7, 16, 33, 100, 777, 5000, 8192):
        for groups in (1, 2, 5, 40, 300, 8192):
            few = min(N + TT, groups * TT)
            every = min(128 * N, 8 * 2432 // H * TT)
            lists = 32 * (6 * N + 8 * 2432) + 100 * (N + 8192)
            assert size(lib, N, groups, heads) <= (4 * N + 3 * few + every + 8) * row + slots + lists + MB, (N, groups)


@pytest.mark.parametrize("heads", [(32, 8, 128), (16, 1, 64), (8, 1, 128), (12, 12, 64), (6, 2, 256), (20, 4, 128), (32, 2, 128)])
def test_more_groups_never_need_less(lib, heads):
    for N, B, max_q in ((1, None, 0), (7, None, 0), (8, None, 0), (100, None, 0), (4001, None, 0), (37, 12, 1), (500, 300, 1),
                        (500, 300, 0), (60, 5, 1)):
        sizes = [size(lib, N, g, heads, B, max_q) for g in [*range(1, 200), 500, 1000, 2000, 8192]]
        assert sizes == sorted(sizes) and sizes[0] > 0, (N, B, max_q)


@pytest.mark.parametrize("heads", [(32, 8, 128), (16, 1, 64), (8, 1, 128), (12, 12, 64), (6, 2, 256)])
def test_more_sequences_of_one_token_never_need_less(lib, heads):
    for groups in (1, 2, 31, 300):
        sizes = [size(lib, N, groups, heads) for N in [*range(1, 300), 1000, 5000, 8192]]
        assert sizes == sorted(sizes) and sizes[0] > 0, groups
