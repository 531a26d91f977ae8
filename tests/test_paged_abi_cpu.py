"""The paged cache's C entry points on the host: struct layouts, and invalid arguments refused before
anything is launched (no GPU needed)."""
import ctypes
import os
import subprocess

import pytest

import sliding_window_attention_swa_gb300 as swa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, BIG = 0x10000, 1 << 62


@pytest.fixture(scope="module")
def lib():
    swa.build()
    return swa.load_library()


def test_struct_layout_matches_header(tmp_path):
    structs = {"swa_paged_cache": swa.SwaPagedCache, "swa_paged_params": swa.SwaPagedParams,
               "swa_page_tables": swa.SwaPageTables, "swa_page_pool": swa.SwaPagePool}
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "swa.h"', "int main(void) {"]
    for cname, py in structs.items():
        lines.append(f'printf("{cname} size %zu\\n", sizeof({cname}));')
        for f, _ in py._fields_:
            lines.append(f'printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));')
    lines.append("return 0; }")
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    for line in subprocess.check_output([str(exe)]).decode().splitlines():
        cname, field, val = line.split()
        py = structs[cname]
        got = ctypes.sizeof(py) if field == "size" else getattr(py, field).offset
        assert got == int(val), (cname, field, got, val)


def valid_paged():
    c = swa.SwaPagedCache(FAKE, FAKE, FAKE, 100, 16, 2, 128, 4, 50)
    p = swa.SwaPagedParams()
    p.q = p.p0 = p.q_start = p.o = p.lse = FAKE
    for name in ("q_strides", "o_strides", "kn_strides", "vn_strides"):
        setattr(p, name, (1024, 128))
    p.N, p.H_q, p.window, p.scale = 9, 8, 100, 0.1
    return p, c


def pair(x, y):
    return (ctypes.c_int64 * 2)(x, y)


@pytest.mark.parametrize("mutate,status", [
    (lambda p, c: setattr(p, "q", None), 1),
    (lambda p, c: setattr(p, "lse", None), 1),
    (lambda p, c: setattr(p, "p0", None), 1),
    (lambda p, c: setattr(p, "q_start", None), 1),          # N rows, B sequences
    (lambda p, c: setattr(p, "N", -1), 1),
    (lambda p, c: setattr(p, "H_q", 7), 1),
    (lambda p, c: setattr(p, "H_q", 0), 1),
    (lambda p, c: setattr(p, "H_q", 34), 2),                # 17 heads a group
    (lambda p, c: setattr(p, "window", -1), 1),
    (lambda p, c: setattr(p, "n_sink", -1), 1),
    (lambda p, c: setattr(p, "max_q", -1), 1),
    (lambda p, c: setattr(p, "scale", float("inf")), 1),
    (lambda p, c: setattr(p, "scale", 0.0), 2),
    (lambda p, c: setattr(p, "k_new", FAKE), 1),            # without v_new
    (lambda p, c: (setattr(p, "k_new", FAKE), setattr(p, "v_new", FAKE + 2)), 2),
    (lambda p, c: (setattr(p, "k_new", FAKE), setattr(p, "v_new", FAKE), setattr(p, "vn_strides", pair(100, 12))), 2),
    (lambda p, c: setattr(p, "q", FAKE + 8), 2),
    (lambda p, c: setattr(p, "q_strides", pair(1024, 4)), 2),
    (lambda p, c: setattr(p, "o_strides", pair(0, 128)), 2),
    (lambda p, c: setattr(p, "q_start", FAKE + 2), 2),
    (lambda p, c: setattr(p, "row_counts", FAKE + 1), 2),
    (lambda p, c: setattr(c, "k_pages", None), 1),
    (lambda p, c: setattr(c, "page_table", None), 1),
    (lambda p, c: setattr(c, "B", 0), 1),
    (lambda p, c: setattr(c, "table_width", 0), 1),
    (lambda p, c: setattr(c, "n_pages", 0), 1),
    (lambda p, c: setattr(c, "page_size", 24), 2),
    (lambda p, c: setattr(c, "page_size", 256), 2),
    (lambda p, c: setattr(c, "d_h", 96), 2),
    (lambda p, c: setattr(c, "table_width", 1 << 28), 2),   # positions past 2^31
    (lambda p, c: setattr(c, "table_width", (1 << 30) // c.page_size + 1), 2),  # positions past 2^30
    (lambda p, c: setattr(c, "B", 8193), 2),
    (lambda p, c: setattr(c, "n_pages", 1 << 29), 2),       # 2^31 groups of eight rows
    (lambda p, c: setattr(c, "v_pages", FAKE + 4), 2),
])
def test_attend_rejects(lib, mutate, status):
    p, c = valid_paged()
    mutate(p, c)
    assert lib.swa_paged_attend(ctypes.byref(p), ctypes.byref(c), FAKE, BIG, None) == status
    assert lib.swa_paged_workspace_size(ctypes.byref(p), ctypes.byref(c)) == 0


@pytest.mark.parametrize("group", [1, 3, 4, 8, 16])
def test_the_hint_chooses_the_kernel_at_any_size(lib, group):
    """The workspace is the chosen kernel's: few rows up to 16 rows a group, many above, whatever the
    number of tokens named."""
    p, c = valid_paged()
    c.H_kv, p.H_q = 2, 2 * group

    def size(max_q):
        p.max_q = max_q
        return lib.swa_paged_workspace_size(ctypes.byref(p), ctypes.byref(c))

    many, few = size(0), size(1)
    assert 0 < few != many > 0
    for t in range(1, 40):
        assert size(t) == (few if t * group <= 16 else many)
    for t in (1 << 27, 1 << 28, 1 << 29, 1 << 30, (1 << 32) // group // 2 + 1, (1 << 31) - 1):
        assert size(min(t, (1 << 31) - 1)) == many, t


def test_null_structures_are_refused(lib):
    p, c = valid_paged()
    assert lib.swa_paged_attend(ctypes.byref(p), None, FAKE, BIG, None) == 1
    assert lib.swa_paged_attend(None, ctypes.byref(c), FAKE, BIG, None) == 1
    assert lib.swa_paged_append(None, ctypes.byref(c), None) == 1
    assert lib.swa_pages_free(None, FAKE, 0, None) == 1


def test_nothing_to_do_launches_nothing(lib):
    p, c = valid_paged()
    p.N = 0
    need = lib.swa_paged_workspace_size(ctypes.byref(p), ctypes.byref(c))
    assert lib.swa_paged_attend(ctypes.byref(p), ctypes.byref(c), FAKE, need, None) == 0
    p.k_new = p.v_new = FAKE
    assert lib.swa_paged_append(ctypes.byref(p), ctypes.byref(c), None) == 0
    p.k_new = p.v_new = None
    assert lib.swa_paged_append(ctypes.byref(p), ctypes.byref(c), None) == 1
    pool = swa.SwaPagePool(FAKE, FAKE, 0, 1, 10, 2, 16, 64)
    assert lib.swa_pages_copy(ctypes.byref(pool), None, None, 0, None) == 0


def valid_tables():
    return swa.SwaPageTables(FAKE, FAKE, 2 * FAKE, 2 * FAKE, 4, 50, 100, 16)


def valid_pool():
    return swa.SwaPagePool(FAKE, FAKE, 100 * 2 * 16 * 64, 3, 100, 2, 16, 64)


def in_place(t):
    t.out_table, t.out_ref = t.table, t.ref


@pytest.mark.parametrize("mutate,status", [
    (lambda t: setattr(t, "table", None), 1),
    (lambda t: setattr(t, "ref", None), 1),
    (lambda t: setattr(t, "out_table", None), 1),
    (lambda t: setattr(t, "out_ref", None), 1),
    (lambda t: setattr(t, "B", 0), 1),
    (lambda t: setattr(t, "width", 0), 1),
    (lambda t: setattr(t, "n_pages", 0), 1),
    (lambda t: setattr(t, "page_size", 0), 1),
    (lambda t: setattr(t, "width", 1 << 28), 2),
    (lambda t: (setattr(t, "B", 1 << 20), setattr(t, "width", 1 << 12)), 2),
])
def test_tables_reject(lib, mutate, status):
    for ip in (False, True):
        t = valid_tables()
        if ip:
            in_place(t)
        mutate(t)
        pool = valid_pool()
        pool.n_pages, pool.page_size = t.n_pages, t.page_size
        b, bp = ctypes.byref(t), ctypes.byref(pool)
        assert lib.swa_pages_workspace_size(b) == 0
        if not ip:
            assert lib.swa_pages_fork(b, bp, FAKE, FAKE, FAKE, BIG, None) == status
        else:
            assert lib.swa_pages_reserve(b, FAKE, FAKE, FAKE, BIG, None) in (1, status)
        assert lib.swa_pages_free(b, FAKE, 0, None) in (1, status)
        assert lib.swa_pages_compact(b, bp, FAKE, FAKE, BIG, None) in (1, status)


def test_in_place_or_not(lib):
    t, pool = valid_tables(), valid_pool()
    b, bp = ctypes.byref(t), ctypes.byref(pool)
    assert lib.swa_pages_reserve(b, FAKE, FAKE, FAKE, BIG, None) == 1       # in place only
    t.out_table = t.table                                                   # one of the two in place
    assert lib.swa_pages_free(b, FAKE, 0, None) == 1
    assert lib.swa_pages_compact(b, bp, FAKE, FAKE, BIG, None) == 1
    assert lib.swa_pages_fork(b, bp, FAKE, FAKE, FAKE, BIG, None) == 1      # never in place
    in_place(t)
    assert lib.swa_pages_fork(b, bp, FAKE, FAKE, FAKE, BIG, None) == 1


def test_pages_arguments_reject(lib):
    t, pool = valid_tables(), valid_pool()
    b, bp = ctypes.byref(t), ctypes.byref(pool)
    need = lib.swa_pages_workspace_size(b)
    assert need > 0
    assert lib.swa_pages_free(b, None, 0, None) == 1
    assert lib.swa_pages_free(b, FAKE, -1, None) == 1
    assert lib.swa_pages_free(b, FAKE + 1, 0, None) == 2
    assert lib.swa_pages_fork(b, bp, None, FAKE, FAKE, need, None) == 1
    assert lib.swa_pages_fork(b, bp, FAKE, FAKE + 2, FAKE, need, None) == 2
    assert lib.swa_pages_fork(b, bp, FAKE, FAKE, FAKE, need - 1, None) == 5
    assert lib.swa_pages_fork(b, bp, FAKE, FAKE, None, need, None) == 5
    assert lib.swa_pages_fork(b, bp, FAKE, FAKE, FAKE + 128, need, None) == 5
    assert lib.swa_pages_fork(b, None, FAKE, FAKE, FAKE, need, None) == 1
    assert lib.swa_pages_compact(b, bp, None, FAKE, need, None) == 1
    assert lib.swa_pages_compact(b, bp, FAKE, FAKE, need - 1, None) == 5
    assert lib.swa_pages_copy(bp, None, FAKE, 1, None) == 1
    assert lib.swa_pages_copy(bp, FAKE, FAKE, -1, None) == 1
    assert lib.swa_pages_copy(bp, FAKE, FAKE + 1, 1, None) == 2
    in_place(t)
    assert lib.swa_pages_reserve(b, None, FAKE, FAKE, need, None) == 1
    assert lib.swa_pages_reserve(b, FAKE, FAKE, FAKE, need - 1, None) == 5


@pytest.mark.parametrize("mutate,status", [
    (lambda p: setattr(p, "k_pages", None), 1),
    (lambda p: setattr(p, "n_layers", 0), 1),
    (lambda p: setattr(p, "d_h", 0), 1),
    (lambda p: setattr(p, "d_h", 12), 2),
    (lambda p: setattr(p, "layer_stride", 100 * 2 * 16 * 64 - 8), 1),   # layers overlap
    (lambda p: setattr(p, "layer_stride", 100 * 2 * 16 * 64 + 4), 2),
    (lambda p: setattr(p, "v_pages", FAKE + 8), 2),
    (lambda p: (setattr(p, "H_kv", 1 << 15), setattr(p, "d_h", 1 << 12)), 2),
])
def test_pool_rejects(lib, mutate, status):
    t, pool = valid_tables(), valid_pool()
    mutate(pool)
    assert lib.swa_pages_copy(ctypes.byref(pool), FAKE, FAKE, 1, None) == status
    assert lib.swa_pages_fork(ctypes.byref(t), ctypes.byref(pool), FAKE, FAKE, FAKE, BIG, None) == status


def test_pool_has_to_match_the_tables(lib):
    t, pool = valid_tables(), valid_pool()
    for name in ("n_pages", "page_size"):
        p = valid_pool()
        setattr(p, name, getattr(p, name) // 2)
        assert lib.swa_pages_fork(ctypes.byref(t), ctypes.byref(p), FAKE, FAKE, FAKE, BIG, None) == 1
        assert lib.swa_pages_compact(ctypes.byref(t), ctypes.byref(p), FAKE, FAKE, BIG, None) == 1
    assert pool.n_pages == t.n_pages


def test_packed_layouts_match_the_structures():
    # the Python calls pack these structures in one go: every field at its offset
    for packed, struct in ((swa._PAGED_PARAMS, swa.SwaPagedParams), (swa._PAGED_CACHE, swa.SwaPagedCache),
                           (swa._PAGE_TABLES, swa.SwaPageTables), (swa._PAGE_POOL, swa.SwaPagePool)):
        fields = [(name, getattr(struct, name).offset + 8 * i) for name, t in struct._fields_
                  for i in range(2 if t is swa._c_i64x2 else 1)]
        data = packed.pack(*range(1, len(fields) + 1))
        assert packed.size <= ctypes.sizeof(struct) < packed.size + 8
        got = struct.from_buffer_copy(data + bytes(8))
        want = 1
        for name, t in struct._fields_:
            for v in getattr(got, name) if t is swa._c_i64x2 else [getattr(got, name)]:
                assert v == want, name
                want += 1
