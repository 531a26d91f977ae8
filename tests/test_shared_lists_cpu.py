"""The lists of stretches that swa_paged_attend_shared makes for few new tokens, by the kernels' own functions on the
host (shared_stretches.cu; no GPU needed)."""
import ctypes
import importlib
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    B = importlib.import_module("sliding_window_attention_swa_gb300.build")
    out = str(tmp_path_factory.mktemp("stretches") / "shared_stretches.so")
    subprocess.check_call([B.nvcc(), *B.flags(), "-shared", "-o", out, os.path.join(HERE, "shared_stretches.cu")])
    return ctypes.CDLL(out)


def counted(lib, q_start, p0, N, TT, planes):
    B = len(p0)
    ints = lambda x: (ctypes.c_int * len(x))(*x)  # noqa: E731
    out = ctypes.c_longlong(), ctypes.c_longlong()
    lib.count_stretches(ints(q_start), ints(p0), B, N, TT, planes, *(ctypes.byref(x) for x in out))
    return out[0].value, out[1].value


def room(N, B, TT, planes):
    return min(N, N // TT + B) * planes


def test_sequences_that_all_have_all_rows_are_not_counted(lib):
    """0, N, 0, N, ...: half of the sequences are in range and each has all rows.  Together their stretches are more than
    32 bits count at the sizes of a call (here 1/256 of its sequences, and 1/16 of the rows); none of them is taken."""
    B, N, TT, planes = 32, 17000, 1, 3
    every, taken = counted(lib, [0, N] * (B // 2) + [0], [1000] * B, N, TT, planes)
    assert every * 256 * 16 > 1 << 31 and every > room(N, B, TT, planes)
    assert taken == 0


@pytest.mark.parametrize("seed", range(80))
def test_no_list_has_more_than_there_is_room_for(lib, seed):
    rng = random.Random(seed)
    B, N, TT, planes = rng.randrange(1, 60), rng.randrange(1, 200), rng.choice([1, 2, 5, 16]), rng.randrange(3, 20)
    q_start = sorted(rng.randrange(N + 1) for _ in range(B + 1))
    p0 = [rng.randrange(3000) for _ in range(B)]
    every, taken = counted(lib, q_start, p0, N, TT, planes)
    assert taken == every <= room(N, B, TT, planes)  # (a list in order: all are)
    for _ in range(rng.randrange(1, 10)):
        q_start[rng.randrange(B + 1)] = rng.choice([rng.randrange(N + 1), -3, N + 1, 0, N])
    every, taken = counted(lib, q_start, p0, N, TT, planes)
    assert taken <= min(every, room(N, B, TT, planes))
