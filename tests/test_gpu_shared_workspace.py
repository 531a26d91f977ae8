"""Attention of shared prefixes in a workspace of exactly the size that is asked for: nothing behind it is written, and
the places of the prefixes' results are those that are read, however many groups and tokens there are."""
import ctypes

import pytest
import torch

import sliding_window_attention_swa_gb300 as m
from test_gpu_paged_shared import MIXED, ONES, Shared, run, swa  # noqa: F401  (swa: the module's fixture)

pytestmark = pytest.mark.gpu


def exactly(x, n_groups, one_each, hint):
    """A workspace of the call's size at the front of a larger buffer of 0xee, and the buffer."""
    p, c = m.SwaPagedParams(), m.SwaPagedCache()
    fake = 4096
    p.q = p.o = p.lse = p.p0 = fake
    p.q_start = None if one_each else fake
    p.N, p.H_q, p.max_q, p.window, p.n_sink, p.scale = x.N, x.Hq, hint, x.window, x.n_sink, x.D ** -0.5
    for st in (p.q_strides, p.o_strides):
        st[0], st[1] = x.Hq * x.D, x.D
    c.k_pages = c.v_pages = c.page_table = fake
    c.n_pages, c.page_size, c.H_kv, c.d_h, c.B, c.table_width = x.n_pages, x.ps, x.Hkv, x.D, len(x.seqs), x.width
    size = m.load_library().swa_paged_shared_workspace_size(ctypes.byref(p), ctypes.byref(c), n_groups)
    assert size > 0
    whole = torch.full((size + (1 << 20),), 0xee, dtype=torch.uint8, device="cuda")
    return whole[:size], whole


def run_exactly(swa, x, one_each=False, hint=0):  # noqa: F811
    ws, whole = exactly(x, len(x.groups) - 1, one_each, hint)
    run(swa, x, max_q=hint, workspace=ws, **(dict(q_start=None) if one_each else {}))
    assert (whole[len(ws):] == 0xee).all()


@pytest.mark.parametrize("shape", [(8, 2, 128, 16), (4, 4, 64, 32), (8, 1, 128, 16), (6, 2, 256, 64), (16, 1, 64, 16)], ids=str)
def test_all_kinds_of_groups(swa, shape):  # noqa: F811
    run_exactly(swa, Shared(110, ONES, *shape), one_each=True)
    run_exactly(swa, Shared(111, MIXED, *shape, lead=3, tail=5, before=[(9, 1)], behind=[(100, 3)]))
    run_exactly(swa, Shared(111, MIXED, *shape, lead=3, tail=5, before=[(9, 1)], behind=[(100, 3)]), hint=1)


@pytest.mark.parametrize("D,ps", [(64, 16), (128, 32), (256, 64)])
@pytest.mark.parametrize("G", [1, 2, 5, 8])
def test_groups_as_large_as_a_stretch(swa, G, D, ps):  # noqa: F811
    """Groups of 16 / G tokens or fewer, so that their prefixes are stretches, up to the last row of the batch; fewer of
    them than have all tokens, as many, and more."""
    most = 16 // G
    for sizes in ([1, 2, 2, 2], [most] * 3, [1] * (2 * most + 1) + [most], [2] * 40, [most] * 200, [1, most]):
        # (every size a group; sequences that hold a little more than the prefix)
        x = Shared(112, [(4000 if len(sizes) < 10 else 300, [(4000 + i if len(sizes) < 10 else 300 + i, 1) for i in range(n)])
                         for n in sizes], G, 1, D, ps)
        run_exactly(swa, x, one_each=True)
    # one group behind many sequences of none
    x = Shared(113, [(3000, [(3000 + i, 1) for i in range(most)])], G, 1, D, ps, before=[(40, 1)] * 77)
    run_exactly(swa, x, one_each=True)
    # drafts: groups of sequences with two tokens each
    if most >= 4:
        x = Shared(114, [(2000, [(2000 + i, 2) for i in range(most // 2)])] * 9, G, 1, D, ps, lead=1, tail=2)
        run_exactly(swa, x, hint=2)
