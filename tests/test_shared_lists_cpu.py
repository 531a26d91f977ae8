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


# ---------------------------------------------------------------------------------------------
# how a unit's keys are cut
# ---------------------------------------------------------------------------------------------
def own(lib, p0, n, base, ut, TT, window, sinks, planes):
    out = (ctypes.c_int * (2 * planes))()
    count = lib.own_stretches(p0, n, base, ut, TT, window, sinks, planes, out)
    return [tuple(out[2 * i:2 * i + 2]) for i in range(count)]


def prefix(lib, p0, end, window, sinks, planes):
    out = (ctypes.c_int * (2 * planes))()
    count = lib.prefix_stretches(p0, end, window, sinks, planes, out)
    return [tuple(out[2 * i:2 * i + 2]) for i in range(count)]


@pytest.mark.parametrize("seed", range(120))
def test_the_kernels_stretches_cover_the_kept_keys_once(lib, seed):
    """A unit's own stretches and its group's: every key that a token of it keeps lies in exactly one, and they are no
    more than there are planes, the sinks' among them."""
    rng = random.Random(seed)
    window, sinks = rng.choice([0, 1, 50, 300, 1000]), rng.choice([0, 1, 40, 400])
    ps, TT = rng.choice([16, 32, 64, 128]), rng.choice([1, 4, 16])
    least = rng.choice([rng.randrange(0, 3000), (1 << 30) - 4000])  # the least p0 of a group
    base = rng.choice([0, rng.randrange(0, least // ps + 1) * ps])
    if least > 4000:
        window, base = window or 700, rng.choice([0, (least - 300) // ps * ps])
    lo = max(0, least - window + 1) if window else 0
    if base <= lo:
        base = 0
    for _ in range(4):
        p0, n, planes = least + rng.choice([0, rng.randrange(900)]), rng.randrange(1, 40), rng.randrange(3, 20)
        shared = prefix(lib, least, base, window, sinks, planes) if base else []
        assert len(shared) <= planes
        for ut in range(-(-n // TT)):
            mine = own(lib, p0, n, base, ut, TT, window, sinks, planes)
            assert 0 < len(mine) <= planes
            parts = sorted(shared + mine)
            assert all(a < b for a, b in parts) and all(x[1] <= y[0] for x, y in zip(parts, parts[1:]))
            for t in range(p0 + ut * TT, p0 + min(n, (ut + 1) * TT)):
                first = max(0, t - window + 1) if window else 0
                for a, b in ([(0, min(sinks, first))] if min(sinks, first) > 0 else []) + [(first, t + 1)]:
                    # [a, b) lies in the stretches
                    for x, y in parts:
                        if x <= a < y:
                            a = y
                    assert a >= b, (t, a, b, parts)
