"""The C entry points of the rotation on the host: invalid arguments refused before anything is launched (no
GPU needed)."""
import ctypes
import os
import subprocess

import pytest

import sliding_window_attention_swa_gb300 as swa
from test_paged_abi_cpu import FAKE, ROOT, pair, valid_paged

NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    swa.build()
    return swa.load_library()


def test_struct_layout_matches_header(tmp_path):
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    fields = [f for f, _ in swa.SwaRope._fields_]
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "swa.h"\nint main(void) {'
                   + "".join(f'printf("%zu ", offsetof(swa_rope, {f}));' for f in fields)
                   + 'printf("%zu", sizeof(swa_rope)); return 0; }')
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    assert got == [getattr(swa.SwaRope, f).offset for f in fields] + [ctypes.sizeof(swa.SwaRope)]
    packed = swa.SwaRope.from_buffer_copy(swa._ROPE.pack(1, 2, 3, 4) + bytes(4))
    assert [getattr(packed, f) for f in fields] == [1, 2, 3, 4]


@pytest.mark.parametrize("args,status", [
    ((None, 64, 10, 1.0, FAKE), 1),
    ((FAKE, 64, 10, 1.0, None), 1),
    ((FAKE, 0, 10, 1.0, FAKE), 1),
    ((FAKE, -16, 10, 1.0, FAKE), 1),
    ((FAKE, 64, -1, 1.0, FAKE), 1),
    ((FAKE, 64, 10, NAN, FAKE), 1),
    ((FAKE, 64, 10, float("inf"), FAKE), 1),
    ((FAKE, 24, 10, 1.0, FAKE), 2),
    ((FAKE, 272, 10, 1.0, FAKE), 2),
    ((FAKE, 64, (1 << 30) + 1, 1.0, FAKE), 2),
    ((FAKE + 4, 64, 10, 1.0, FAKE), 2),
    ((FAKE, 64, 10, 1.0, FAKE + 8), 2),
    ((FAKE, 64, 0, 1.0, FAKE), 0),  # nothing to do
])
def test_table_rejects(lib, args, status):
    assert lib.swa_rope_table(*args, None) == status


def valid_rope():
    p, c = valid_paged()
    p.lse = None
    p.k_new = p.v_new = FAKE
    return p, c, swa.SwaRope(FAKE, 1000, 64, 0)


@pytest.mark.parametrize("mutate,status", [
    (lambda p, c, r: setattr(r, "table", None), 1),
    (lambda p, c, r: setattr(r, "n_pos", 0), 1),
    (lambda p, c, r: setattr(r, "rot_dim", 0), 1),
    (lambda p, c, r: setattr(r, "rot_dim", 144), 1),      # more than the head
    (lambda p, c, r: setattr(r, "rot_dim", 40), 2),
    (lambda p, c, r: setattr(r, "interleaved", 2), 2),
    (lambda p, c, r: setattr(r, "interleaved", -1), 2),
    (lambda p, c, r: setattr(r, "table", FAKE + 4), 2),
    (lambda p, c, r: (setattr(p, "q", None), setattr(p, "k_new", None), setattr(p, "v_new", None)), 1),
    (lambda p, c, r: setattr(p, "v_new", None), 1),
    (lambda p, c, r: setattr(p, "o", None), 1),
    (lambda p, c, r: setattr(p, "H_q", 7), 1),
    (lambda p, c, r: setattr(p, "H_q", 0), 1),
    (lambda p, c, r: setattr(p, "p0", None), 1),
    (lambda p, c, r: setattr(p, "q_start", None), 1),     # N rows, B sequences
    (lambda p, c, r: setattr(p, "N", -1), 1),
    (lambda p, c, r: setattr(p, "q", FAKE + 8), 2),
    (lambda p, c, r: setattr(p, "o_strides", pair(1024, 4)), 2),
    (lambda p, c, r: setattr(p, "q_strides", pair(-8, 128)), 2),
    (lambda p, c, r: setattr(p, "kn_strides", pair(12, 128)), 2),
    (lambda p, c, r: setattr(p, "k_new", FAKE + 2), 2),
    (lambda p, c, r: setattr(c, "d_h", 96), 2),
    (lambda p, c, r: setattr(c, "page_size", 24), 2),
    (lambda p, c, r: setattr(c, "k_pages", None), 1),
])
def test_append_rejects(lib, mutate, status):
    p, c, r = valid_rope()
    mutate(p, c, r)
    assert lib.swa_paged_rope_append(ctypes.byref(p), ctypes.byref(c), ctypes.byref(r), None) == status


def test_nothing_to_do_launches_nothing(lib):
    p, c, r = valid_rope()
    p.N = 0
    refs = ctypes.byref(p), ctypes.byref(c)
    assert lib.swa_paged_rope_append(*refs, ctypes.byref(r), None) == 0
    assert lib.swa_paged_rope_append(*refs, None, None) == 1
    p.q = None
    assert lib.swa_paged_rope_append(*refs, ctypes.byref(r), None) == 0
