"""Reserving, giving back, forking, compacting and copying the pages of a paged cache, against models
on Python lists (tables, counts and page contents equal), and a run of them together with the
attention that reads the pages."""
import numpy as np
import pytest
import torch

import paged_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def swa():
    import sliding_window_attention_swa_gb300 as m

    m.load_library()
    return m


def tables(seed, B, width, n_pages, fill=0.7, shared=0.2):
    """A random table with its counts (and some pages held by someone else)."""
    rng = np.random.default_rng(seed)
    free = list(rng.permutation(n_pages))
    table = np.full((B, width), -1, dtype=np.int32)
    for b in range(B):
        for j in range(width):
            if rng.random() < fill and free:
                table[b, j] = free.pop()
    for b in range(1, B):
        m = (rng.random(width) < shared) & (table[b - 1] >= 0)
        table[b, m] = table[b - 1, m]
    ref = np.bincount(table[table >= 0], minlength=n_pages).astype(np.int32)
    others = rng.random(n_pages) < 0.05
    ref[others] += 1
    return table, ref


def same(got, want):
    np.testing.assert_array_equal(got.cpu().numpy(), np.asarray(want))


@pytest.mark.parametrize("B,width,n_pages,ps", [(1, 1, 1, 16), (3, 7, 40, 16), (40, 9, 700, 1), (5, 3000, 40000, 16),
                                                (1500, 4, 20000, 128)])
def test_reserve(swa, B, width, n_pages, ps):
    table, ref = tables(1, B, width, n_pages, fill=0.4)
    rng = np.random.default_rng(2)
    first = rng.integers(0, width * ps + 1, B)
    end = np.minimum(width * ps, first + rng.integers(-3, width * ps + 1, B))
    first[0], end[0] = 0, width * ps
    if B > 1500 // 2 or width > 1000:  # keep the model's search short
        first, end = first // 2, np.minimum(end, first // 2 + 3 * ps)
    want = R.reserve(table.tolist(), ref.tolist(), first.tolist(), end.tolist(), ps)
    t, r = R.i32(table), R.i32(ref)
    swa.swa_pages_reserve(t, r, R.i32(first), R.i32(end), ps)
    st, words = swa.swa_read_device_errors()
    lacks = any(want[0][b][j] < 0 for b in range(B) if end[b] > first[b]
                for j in range(first[b] // ps, -(-end[b] // ps)))
    assert words["cache"] == (swa.DEVERR_NO_PAGE if lacks else 0)
    same(t, want[0])
    same(r, want[1])


def test_reserve_when_the_pool_runs_out(swa):
    t, r = R.i32([[-1, -1, -1], [-1, -1, -1]]), R.i32([0, 1, 0, 0])
    swa.swa_pages_reserve(t, r, R.i32([0, 0]), R.i32([33, 48]), 16)
    assert swa.swa_read_device_errors() == (1, {"prefill": 0, "split": 0, "cache": swa.DEVERR_NO_PAGE})
    same(t, [[0, 2, 3], [-1, -1, -1]])
    same(r, [1, 1, 1, 1])
    # a range outside the row: reported, the row left as it is
    t, r = R.i32([[-1, -1], [-1, -1], [-1, -1]]), R.i32([0, 0, 0])
    swa.swa_pages_reserve(t, r, R.i32([-1, 0, 5]), R.i32([3, 33, 6]), 16)
    assert swa.swa_read_device_errors()[1]["cache"] == swa.DEVERR_BAD_POSITION
    same(t, [[-1, -1], [-1, -1], [0, -1]])


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("B,width,n_pages,ps,ns", [(1, 1, 1, 16, 0), (3, 7, 40, 16, 4), (40, 90, 4000, 32, 0),
                                                   (700, 33, 20000, 1, 3)])
def test_free(swa, B, width, n_pages, ps, ns, inplace):
    table, ref = tables(3, B, width, n_pages)
    rng = np.random.default_rng(4)
    below = rng.integers(-1, width * ps + 2, B)
    below[::3] = -1
    want = R.free(table.tolist(), ref.tolist(), below.tolist(), ps, ns)
    t, r = R.i32(table), R.i32(ref)
    kw = {} if inplace else dict(out_table=torch.full_like(t, 99), out_ref=torch.full_like(r, 99))
    ot, orf = swa.swa_pages_free(t, r, R.i32(below), ps, n_sink=ns, **kw)
    swa.swa_check_device_error()
    same(ot, want[0])
    same(orf, want[1])
    assert (ot is t) == inplace
    if not inplace:
        same(t, table)
        same(r, ref)


def test_free_of_what_nobody_holds(swa):
    t, r = R.i32([[0, 1], [2, 9]]), R.i32([1, 0, 1])
    swa.swa_pages_free(t, r, R.i32([-1, -1]), 16)
    assert swa.swa_read_device_errors()[1]["cache"] == swa.DEVERR_BAD_REF | swa.DEVERR_BAD_PAGE
    same(t, [[-1, -1], [-1, -1]])
    same(r, [0, 0, 0])


def pools(seed, L, n_pages, H, ps, D):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(L, n_pages, H, ps, D, generator=g).to(torch.bfloat16) for _ in range(2)]


@pytest.mark.parametrize("shape", [(1, 1, 16, 64), (3, 2, 32, 128), (2, 5, 64, 8), (1, 3, 1, 24), (2, 1, 128, 256)],
                         ids=str)
@pytest.mark.parametrize("B,most", [(1, 40), (6, 200), (70, 130)])
def test_fork(swa, B, most, shape):
    L, H, ps, D = shape
    rng = np.random.default_rng(B + most)
    lens = rng.integers(0, most + 1, B)
    lens[0] = most
    if B > 2:
        lens[2] = lens[2] // ps * ps  # no page in part
    width = -(-most // ps) + 1
    n_pages = int(sum(-(-n // ps) for n in lens)) + 2 * B
    perm = rng.permutation(n_pages).tolist()
    table = np.full((B, width), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        for j in range(-(-int(n) // ps) + (b % 2)):  # some rows hold a page past their last token
            table[b, j] = perm.pop()
    ref = np.bincount(table[table >= 0], minlength=n_pages).astype(np.int32)
    for kind in ("random", "one", "same", "none"):
        src = {"random": rng.integers(-1, B, B), "one": np.zeros(B, int), "same": np.arange(B),
               "none": np.full(B, -1)}[kind]
        k, v = pools(7, L, n_pages, H, ps, D)
        wk, wv = R.bits(k), R.bits(v)
        want = R.fork(table.tolist(), ref.tolist(), src.tolist(), lens.tolist(), ps, (wk, wv))
        kd, vd, t, r = k.cuda(), v.cuda(), R.i32(table), R.i32(ref)
        out_ref = torch.full_like(r, 99) if kind == "random" else None
        ot, orf = swa.swa_pages_fork(kd, vd, t, r, R.i32(src), R.i32(lens), out_ref=out_ref)
        swa.swa_check_device_error()
        same(ot, want[0])
        same(orf, want[1])
        same(t, table)
        np.testing.assert_array_equal(R.bits(kd), wk)
        np.testing.assert_array_equal(R.bits(vd), wv)


@pytest.mark.parametrize("B,most,ps", [(300, 400, 8), (9, 3000, 1), (1500, 20, 4)])
def test_fork_of_a_large_table(swa, B, most, ps):
    # tables and pools that the grids plan, instead of one cluster
    test_fork(swa, B, most, (1, 1, ps, 8))


def fork_by_pages(table, ref, src, lens, ps):
    """The header's rule, page by page: (new table, new counts, [(from, to, tokens)])."""
    table, ref = np.array(table), np.array(ref)
    out = np.full_like(table, -1)
    full, last = {}, {}  # page -> rows that have it as a full one, as a last one that is not
    for i, s in enumerate(src):
        if s >= 0:
            n, part = divmod(int(lens[s]), ps)
            out[i, :n] = table[s, :n]
            for p in out[i, :n]:
                full.setdefault(int(p), []).append(i)
            if part:
                last.setdefault(int(table[s, n]), []).append((i, n, part))
    copies = []
    for p, rows in last.items():
        keeps = 0 if p in full else 1
        for i, n, _ in rows[:keeps]:
            out[i, n] = p
        copies += [(i, n, p, part) for i, n, part in rows[keeps:]]
    count = lambda t: np.bincount(t[t >= 0], minlength=len(ref))  # noqa: E731
    ref = ref - count(table) + count(out)
    free, moves = np.flatnonzero(ref == 0), []
    for (i, n, p, part), q in zip(sorted(copies), free):
        out[i, n] = q
        ref[q] = 1
        moves.append((p, int(q), part))
    return out, ref, moves


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("B,most,ps", [(2, 32, 16), (7, 90, 16), (40, 30, 4), (300, 400, 8)], ids=str)
def test_forks_of_forks(swa, B, most, ps, inplace):
    """Rows that share pages already, cut back to lengths inside them or on their borders, and forked
    again: no row may be left with a last page that it would write to and that another row has."""
    rng = np.random.default_rng(B)
    width = -(-most // ps)
    n_pages = 2 * B * width + B
    k, v = pools(14, 2, n_pages, 1, ps, 8)
    wk, wv = R.bits(k), R.bits(v)
    kd, vd = k.cuda(), v.cuda()
    table = rng.permutation(n_pages)[:B * width].reshape(B, width).astype(np.int32)
    ref = np.bincount(table.ravel(), minlength=n_pages).astype(np.int32)
    lens = np.full(B, most)
    for turn in range(6):
        src = rng.integers(0, max(1, B // 3), B) if turn % 2 == 0 else np.arange(B)
        if turn == 5:
            src = rng.integers(-1, B, B)
        wt, wr, moves = fork_by_pages(table, ref, src, lens, ps)
        for p, q, part in moves:
            for a in (wk, wv):
                a[:, q, :, :part] = a[:, p, :, :part]
        t, r = R.i32(table), R.i32(ref)
        ot, orf = swa.swa_pages_fork(kd, vd, t, r, R.i32(src), R.i32(lens), out_ref=None if inplace else torch.full_like(r, 9))
        swa.swa_check_device_error()
        same(ot, wt)
        same(orf, wr)
        np.testing.assert_array_equal(R.bits(kd), wk)
        np.testing.assert_array_equal(R.bits(vd), wv)
        table, ref, lens = wt, wr, np.where(src >= 0, lens[src], 0)
        for i in np.flatnonzero(lens % ps):
            page = table[i, lens[i] // ps]
            assert page >= 0 and (table == page).sum() == 1, f"turn {turn}: row {i} shares its last page"
        # rows cut back: anywhere, or by whole pages
        cut = rng.integers(0, 2 * ps + 1, B) if turn % 3 else rng.integers(0, 3, B) * ps
        lens = np.maximum(lens - cut, 0)


@pytest.mark.parametrize("lens,want,moves", [
    ([30, 30], [[0, 1], [0, 2]], [(1, 2, 14)]),
    ([17, 30], [[0, 1], [0, 2]], [(1, 2, 14)]),
    ([32, 30], [[0, 1], [0, 2]], [(1, 2, 14)]),  # a full page of row 0
    ([30, 32], [[0, 2], [0, 1]], [(1, 2, 14)]),  # of row 1
    ([16, 30], [[0, -1], [0, 1]], []),
    ([9, 30], [[2, -1], [0, 1]], [(0, 2, 9)]),
], ids=str)
@pytest.mark.parametrize("wide", [False, True], ids=["one-cluster", "grids"])
def test_rows_that_shared_a_page_and_were_cut_back(swa, lens, want, moves, wide):
    k, v = (x.cuda() for x in pools(15, 2, 4, 2, 16, 8))
    wk, wv = k.clone(), v.clone()
    for p, q, n in moves:
        for a in (wk, wv):
            a[:, q, :, :n] = a[:, p, :, :n]
    more = 16 * 1024 if wide else 0
    t, r = R.i32([[0, 1] + [-1] * more, [0, 1] + [-1] * more]), R.i32([2, 2, 0, 0])
    ot, orf = swa.swa_pages_fork(k, v, t, r, R.i32([0, 1]), R.i32(lens))
    swa.swa_check_device_error()
    same(ot[:, :2], want)
    same(orf, np.bincount([p for row in want for p in row if p >= 0], minlength=4))
    assert (ot[:, 2:] == -1).all() and torch.equal(k, wk) and torch.equal(v, wv)


def test_fork_refusals_and_broken_data(swa):
    k, v = (x.cuda() for x in pools(8, 1, 5, 1, 16, 8))
    t, r = R.i32([[0, 1], [2, -1], [3, 4]]), R.i32([1, 1, 1, 1, 1])
    lens = R.i32([20, 3, 32])
    with pytest.raises(swa.SwaError):
        swa.swa_pages_fork(k, v, t, r, R.i32([0, 1, 2]), lens, out_table=t)
    with pytest.raises(ValueError):
        swa.swa_pages_fork(k[:, :4], v[:, :4], t, r[:4].contiguous(), R.i32([0, 1]), lens)
    with pytest.raises(swa.SwaError):
        swa.swa_pages_fork(k[:, :4].contiguous(), v[:, :4].contiguous(), t, r, R.i32([0, 1, 2]), lens)
    # rows that do not exist, lengths that do not fit: empty rows, reported
    for src, ln in (([0, 7, -2], [20, 3, 32]), ([0, 1, 2], [20, -1, 33])):
        ot, orf = swa.swa_pages_fork(k, v, t, r.clone(), R.i32(src), R.i32(ln))
        assert swa.swa_read_device_errors()[1]["cache"] == swa.DEVERR_BAD_POSITION
        same(ot, [[0, 1], [-1, -1], [-1, -1]])
        same(orf, [1, 1, 0, 0, 0])
    # no page left for the second copy
    r2 = R.i32([1, 1, 2, 2, 2])
    k2 = k.clone()
    ot, orf = swa.swa_pages_fork(k2, v, t, r2, R.i32([0, 0, 0]), lens)
    assert swa.swa_read_device_errors()[1]["cache"] == swa.DEVERR_NO_PAGE
    same(ot, [[0, 1], [0, -1], [0, -1]])
    same(orf, [3, 1, 1, 1, 1])
    np.testing.assert_array_equal(R.bits(k2), R.bits(k))


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("B,width,n_pages,shape", [(1, 1, 1, (1, 1, 16, 64)), (4, 5, 30, (2, 3, 16, 8)),
                                                   (30, 9, 400, (1, 2, 32, 64)), (9, 4000, 50000, (1, 1, 1, 8))])
def test_compact(swa, B, width, n_pages, shape, inplace):
    L, H, ps, D = shape
    for fill in (0.0, 0.3, 0.95):
        table, ref = tables(9, B, width, n_pages, fill=fill)
        k, v = pools(10, L, n_pages, H, ps, D)
        wk, wv = R.bits(k), R.bits(v)
        wt, wr, live = R.compact(table.tolist(), ref.tolist(), (wk, wv))
        kd, vd, t, r = k.cuda(), v.cuda(), R.i32(table), R.i32(ref)
        kw = {} if inplace else dict(out_table=torch.full_like(t, 99), out_ref=torch.full_like(r, 99))
        ot, orf, n_live = swa.swa_pages_compact(kd, vd, t, r, **kw)
        swa.swa_check_device_error()
        assert n_live.item() == live
        same(ot, wt)
        same(orf, wr)
        np.testing.assert_array_equal(R.bits(kd), wk)
        np.testing.assert_array_equal(R.bits(vd), wv)
        if not inplace:
            same(t, table)
            same(r, ref)


def test_a_row_as_long_as_a_call_takes(swa):
    # 2^31 - 1 entries: the steps behind the last one pass 2^31
    last = (1 << 31) - 1
    k, v = (x.cuda() for x in pools(16, 1, 5, 1, 1, 8))
    table, ref = torch.full((1, last), -1, dtype=torch.int32, device="cuda"), R.i32([0, 1, 0, 0, 0])
    swa.swa_pages_reserve(table, ref, R.i32([last - 3]), R.i32([last]), 1)
    swa.swa_check_device_error()
    same(table[0, -4:], [-1, 0, 2, 3])
    same(ref, [1, 1, 1, 1, 0])
    out, _ = swa.swa_pages_fork(k, v, table, ref, R.i32([0]), R.i32([last]))
    swa.swa_check_device_error()
    assert torch.equal(out, table)
    same(ref, [1, 1, 1, 1, 0])
    swa.swa_pages_free(table, ref, R.i32([last - 1]), 1, n_sink=last - 2, out_table=out, out_ref=ref.clone())
    same(out[0, -4:], [-1, 0, -1, 3])
    swa.swa_pages_free(table, ref, R.i32([last - 2]), 1)
    swa.swa_check_device_error()
    same(table[0, -4:], [-1, -1, 2, 3])
    same(ref, [0, 1, 1, 1, 0])
    want = k[0, 3].clone()
    _, _, live = swa.swa_pages_compact(k, v, table, ref)
    swa.swa_check_device_error()
    same(table[0, -4:], [-1, -1, 2, 0])
    same(ref, [1, 1, 1, 0, 0])
    assert live.item() == 3 and torch.equal(k[0, 0], want) and int((table >= 0).sum()) == 2


@pytest.mark.parametrize("layers", [None, 3])
def test_copy(swa, layers):
    k, v = pools(11, layers or 1, 9, 2, 32, 64)
    if layers is None:
        k, v = k[0], v[0]
    kd, vd = k.cuda(), v.cuda()
    swa.swa_pages_copy(kd, vd, R.i32([0, 0, 8]), R.i32([3, 7, 1]))
    swa.swa_check_device_error()
    for a, d in ((k, kd), (v, vd)):
        w = a.clone()
        for s, t in ((0, 3), (0, 7), (8, 1)):
            (w[t] if layers is None else w[:, t]).copy_(a[s] if layers is None else a[:, s])
        np.testing.assert_array_equal(R.bits(d), R.bits(w))
    swa.swa_pages_copy(kd, vd, R.i32([]), R.i32([]))
    before = R.bits(kd)
    swa.swa_pages_copy(kd, vd, R.i32([0, -1, 9]), R.i32([9, 2, 2]))  # pairs outside the pool: skipped
    assert swa.swa_read_device_errors()[1]["cache"] == swa.DEVERR_BAD_PAGE
    np.testing.assert_array_equal(R.bits(kd), before)


def test_layers_apart(swa):
    # a pool whose layers lie further apart than their pages need: the rest is not touched
    big = torch.randn(2, 7, 2, 16, 8, device="cuda").to(torch.bfloat16)
    k, v = big[:, :5], big.clone()[:, :5]
    want = big.clone()
    want[:, 4] = want[:, 1]
    swa.swa_pages_copy(k, v, R.i32([1]), R.i32([4]))
    assert torch.equal(big, want)


def test_serving_run(swa):
    """Pages reserved, two prompts prefilled in chunks, forked, decoded, trimmed behind the window,
    compacted and decoded on, in two layers: every step's attention is that of the tokens
    themselves, and at the end the pool is empty again."""
    L, Hq, Hkv, D, ps, W, ns, B, width, n_pages = 2, 8, 2, 64, 16, 40, 2, 4, 12, 40
    g = torch.Generator().manual_seed(12)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    k_pool = torch.full((L, n_pages, Hkv, ps, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    v_pool = torch.full_like(k_pool, float("nan"))
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    ref = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    hist = [[(torch.empty(0, Hkv, D), torch.empty(0, Hkv, D)) for _ in range(B)] for _ in range(L)]  # tokens so far
    lens = [0] * B

    def step(new):
        nonlocal lens
        p0, end = R.i32(lens), R.i32([a + n for a, n in zip(lens, new)])
        swa.swa_pages_reserve(table, ref, p0, end, ps)
        start = R.i32([sum(new[:i]) for i in range(B + 1)])
        N = sum(new)
        for layer in range(L):
            q, k, v = rnd(N, Hq, D), rnd(N, Hkv, D), rnd(N, Hkv, D)
            o, lse, cnt = swa.swa_paged_attend(q.cuda(), k_pool[layer], v_pool[layer], table, p0, W, n_sink=ns,
                                               q_start=start, max_q=max(new), k_new=k.cuda(), v_new=v.cuda(),
                                               want_counts=True)
            swa.swa_check_device_error()
            for b, n in enumerate(new):
                if n:
                    a = sum(new[:b])
                    hk, hv = hist[layer][b]
                    hist[layer][b] = (torch.cat([hk, k[a:a + n]]), torch.cat([hv, v[a:a + n]]))
                    R.check(o[a:a + n], lse[a:a + n], cnt[a:a + n],
                            R.attend(q[a:a + n], *hist[layer][b], lens[b], W, ns), f"layer {layer}, row {b}")
        lens = [a + n for a, n in zip(lens, new)]
        # what lies behind the next token's window goes back
        swa.swa_pages_free(table, ref, R.i32([max(0, n - W + 1) for n in lens]), ps, n_sink=ns)

    step([37, 0, 0, 20])
    step([50, 0, 0, 1])
    new_table, _ = swa.swa_pages_fork(k_pool, v_pool, table, ref, R.i32([0, 0, 0, 3]), R.i32(lens))
    table.copy_(new_table)
    for layer in range(L):
        hist[layer] = [hist[layer][i] for i in (0, 0, 0, 3)]
    lens = [lens[i] for i in (0, 0, 0, 3)]
    for _ in range(3):
        step([1, 1, 1, 1])
    _, _, n_live = swa.swa_pages_compact(k_pool, v_pool, table, ref)
    assert int((ref > 0).sum()) == n_live.item() and (ref[n_live.item():] == 0).all()
    k_pool[:, n_live.item():] = float("nan")  # what no sequence holds may be overwritten
    v_pool[:, n_live.item():] = float("nan")
    for _ in range(3):
        step([1, 1, 2, 1])
    step([18, 1, 1, 0])
    swa.swa_pages_free(table, ref, R.i32([-1] * B), ps)
    swa.swa_check_device_error()
    assert (table == -1).all() and (ref == 0).all()


@pytest.mark.parametrize("few", [True, False], ids=["single-tokens", "chunks"])
def test_a_captured_step_is_the_called_one(swa, few):
    """Reserve, append and attend, free, fork and compact as one graph, replayed: the tables, counts,
    pages and rows are bit for bit those of the same calls made one by one."""
    Hq, Hkv, D, ps, W, B, width, n_pages = 8, 2, 128, 16, 100, 6, 30, 220
    n = 1 if few else 30
    g = torch.Generator().manual_seed(13)
    steps = [tuple(torch.randn(B * n, h, D, generator=g).to(torch.bfloat16).cuda() for h in (Hq, Hkv, Hkv))
             for _ in range(6)]

    def state():
        z = dict(dtype=torch.int32, device="cuda")
        s = dict(k=torch.zeros(n_pages, Hkv, ps, D, dtype=torch.bfloat16, device="cuda"),
                 table=torch.full((B, width), -1, **z), ref=torch.zeros(n_pages, **z), p0=torch.zeros(B, **z),
                 src=R.i32([0, 0, 2, 3, 3, 5]), start=R.i32([i * n for i in range(B + 1)]),
                 new_table=torch.zeros(B, width, **z), live=torch.zeros(1, **z),
                 o=torch.zeros(B * n, Hq, D, dtype=torch.bfloat16, device="cuda"), lse=torch.zeros(B * n, Hq, device="cuda"))
        s["v"] = torch.zeros_like(s["k"])
        s["q"], s["kn"], s["vn"] = (torch.zeros_like(x) for x in steps[0])
        return s

    def step(s):
        end = s["p0"] + n
        swa.swa_pages_reserve(s["table"], s["ref"], s["p0"], end, ps)
        swa.swa_paged_attend(s["q"], s["k"], s["v"], s["table"], s["p0"], W, q_start=None if few else s["start"],
                             k_new=s["kn"], v_new=s["vn"], o=s["o"], lse=s["lse"])
        swa.swa_pages_free(s["table"], s["ref"], (end - W).clamp(min=0), ps, n_sink=1)
        swa.swa_pages_fork(s["k"], s["v"], s["table"], s["ref"], s["src"], end, out_table=s["new_table"])
        s["table"].copy_(s["new_table"])
        swa.swa_pages_compact(s["k"], s["v"], s["table"], s["ref"], n_live=s["live"])
        s["p0"].copy_(end)

    a, b = state(), state()
    step(state())  # (one-time setup before the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for q, k, v in steps:
        for s in (a, b):
            for name, x in zip(("q", "kn", "vn"), (q, k, v)):
                s[name].copy_(x)
        step(a)
        graph.replay()
        swa.swa_check_device_error()
        for name in ("table", "ref", "p0", "live", "lse"):
            assert torch.equal(a[name], b[name]), name
        for name in ("o", "k", "v"):
            np.testing.assert_array_equal(R.bits(a[name]), R.bits(b[name]), err_msg=name)
