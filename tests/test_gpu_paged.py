"""Attention of ragged batches of new tokens over a paged cache, and the append that stores them,
against a plain 64-bit computation (every row; counts exact; see paged_reference.check for
the bounds)."""
import pytest
import torch

import paged_reference as R

pytestmark = pytest.mark.gpu


def run(swa, x, append=False, want_counts=True, **kw):
    """The call on batch x, checked against the reference; returns (o, lse, counts, k_pages, v_pages)."""
    k, v = x.without_new() if append else (x.k_pages, x.v_pages)
    k, v = k.cuda(), v.cuda()
    o = torch.full((x.N, x.Hq, x.D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((x.N, x.Hq), 7.0, device="cuda")
    cnt = torch.full((x.N, x.Hq), 7, dtype=torch.int32, device="cuda") if want_counts else None
    if append:
        kw.update(k_new=x.k_new.cuda(), v_new=x.v_new.cuda())
    kw.setdefault("q_start", x.q_start.cuda())
    swa.swa_paged_attend(x.q.cuda(), k, v, x.table.cuda(), x.p0.cuda(), x.window, n_sink=x.n_sink, o=o, lse=lse,
                         row_counts=cnt, **kw)
    swa.swa_check_device_error()
    verify(x, o, lse, cnt)
    return o, lse, cnt, k, v


def verify(x, o, lse, cnt, skip=()):
    mine = torch.zeros(x.N, dtype=torch.bool)
    for b, q0, n in x.rows():
        if b in skip:
            continue
        mine[q0:q0 + n] = True
        R.check(o[q0:q0 + n], lse[q0:q0 + n], None if cnt is None else cnt[q0:q0 + n], x.reference(b), f"sequence {b}")
    rest = ~mine
    assert (o.cpu()[rest] == 7).all() and (lse.cpu()[rest] == 7).all(), "rows of no sequence were written"
    assert cnt is None or (cnt.cpu()[rest] == 7).all()


@pytest.fixture(scope="module")
def swa():
    import sliding_window_attention_swa_gb300 as m

    m.load_library()
    return m


ONE = [(0, 1), (1, 1), (14, 1), (15, 1), (16, 1), (62, 1), (63, 1), (64, 1), (127, 1), (128, 1), (129, 1), (1000, 1),
       (3001, 1)]
RAGGED = [(0, 1), (5, 33), (0, 0), (130, 1), (64, 64), (0, 257), (0, 0), (1111, 7), (300, 129), (2000, 1)]
DECODE = [
    # Hq, Hkv, D, page, window, sinks
    (8, 2, 128, 16, 0, 0), (8, 2, 128, 64, 100, 4), (4, 4, 64, 32, 1, 0), (32, 2, 64, 16, 257, 37),
    (7, 1, 128, 128, 128, 0), (6, 2, 256, 64, 1000, 1), (16, 1, 256, 16, 0, 0), (3, 3, 256, 128, 2, 130),
    (5, 1, 64, 128, 64, 0),
]
CHUNK = DECODE + [(12, 1, 128, 32, 300, 3), (24, 8, 64, 64, 0, 0), (16, 8, 256, 16, 129, 5), (2, 2, 128, 16, 17, 0),
                  (16, 1, 128, 64, 0, 0)]


@pytest.mark.parametrize("append", [False, True], ids=["stored", "append"])
@pytest.mark.parametrize("case", DECODE, ids=str)
def test_one_token_a_sequence(swa, case, append):
    Hq, Hkv, D, ps, w, ns = case
    x = R.Batch(1, ONE, Hq, Hkv, D, ps, w, ns)
    *_, k, v = run(swa, x, append, q_start=None)
    assert (R.bits(k) == R.bits(x.k_pages)).all() and (R.bits(v) == R.bits(x.v_pages)).all()


@pytest.mark.parametrize("append", [False, True], ids=["stored", "append"])
@pytest.mark.parametrize("case", CHUNK, ids=str)
def test_ragged_batch(swa, case, append):
    Hq, Hkv, D, ps, w, ns = case
    x = R.Batch(2, RAGGED, Hq, Hkv, D, ps, w, ns, lead=3, tail=5)
    *_, k, v = run(swa, x, append)
    assert (R.bits(k) == R.bits(x.k_pages)).all() and (R.bits(v) == R.bits(x.v_pages)).all()


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 16, 17, 31, 63, 64, 65, 100, 128, 300])
@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 4, 64), (4, 2, 256)], ids=str)
def test_chunk_lengths(swa, heads, n):
    Hq, Hkv, D = heads
    for p0, w in ((0, 0), (777, 200), (127, 0)):
        run(swa, R.Batch(3, [(p0, n)], Hq, Hkv, D, 16, w), max_q=n)


@pytest.mark.parametrize("D,ps", [(64, 16), (128, 32), (256, 64)])
def test_the_hint_chooses_no_result(swa, D, ps):
    # a wrong or absent max_q: both kernels on batches of few and of many new tokens
    for seqs in (ONE, RAGGED):
        x = R.Batch(4, seqs, 8, 2, D, ps, 500, 2)
        for hint in (0, 1, 4, 100000):
            run(swa, x, max_q=hint)


@pytest.mark.parametrize("seqs", [[(20000, 1)], [(9000, 3), (100, 1)], [(12000, 40)], [(0, 1)], [(15, 1)] * 40,
                                  [(70, 2)] * 300, [(0, 0), (0, 0)]], ids=lambda s: f"{len(s)}x{s[0]}")
def test_long_histories_and_many_sequences(swa, seqs):
    # one sequence spread over every CTA, joined again; several sequences in one CTA's share
    for D, ps in ((64, 64), (128, 16), (256, 128)):
        run(swa, R.Batch(5, seqs, 4, 1, D, ps), want_counts=False)
        run(swa, R.Batch(6, seqs, 4, 1, D, ps), max_q=max(n for _, n in seqs))


def test_as_many_sequences_as_a_call_takes(swa):
    seqs = [(i % 40, 1 if i % 31 == 0 else 0) for i in range(8192)]
    seqs[77] = (1000, 200)
    run(swa, R.Batch(8, seqs, 2, 1, 64, 16, 20, 1))
    k = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    table, p0 = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in ((8193, 1), 8193))
    with pytest.raises(swa.SwaError):
        swa.swa_paged_attend(torch.zeros(8193, 1, 64, dtype=torch.bfloat16, device="cuda"), k, k.clone(), table, p0)
    # one token a sequence
    o, lse, _ = swa.swa_paged_attend(torch.ones(8192, 1, 64, dtype=torch.bfloat16, device="cuda"), k, k.clone(),
                                     table[:8192], p0[:8192])
    swa.swa_check_device_error()
    assert (o == 0).all() and (lse == 0).all()  # one key, its score 0


@pytest.mark.parametrize("heads", [(16, 1, 128), (16, 1, 64), (16, 1, 256)], ids=str)
def test_more_units_than_two_waves(swa, heads):
    # whole units dealt to the CTAs first: one long chunk, a batch of many, one whose first units are
    # far longer than the others (some CTAs are above the mean before the rest is shared out)
    Hq, Hkv, D = heads
    tokens = 16 if D < 256 else 8  # of a unit
    u = 304
    for seqs, w in (([(0, u * tokens + 5)], 300), ([(37 * i, 9 * tokens + i) for i in range(40)], 0),
                    ([(30000, 20 * tokens)] + [(0, 3)] * 330, 0), ([(5, 1)] * 200 + [(3, 2 * tokens + 1)] * 70, 0)):
        x = R.Batch(13, seqs, Hq, Hkv, D, 64, w, 3 if w else 0)
        run(swa, x, want_counts=False)


@pytest.mark.parametrize("heads", [(32, 8, 128), (16, 1, 128)], ids=str)
def test_pairs_of_one_key_tile_behind_single_query_tiles(swa, heads):
    # units of two query tiles that read one tile of keys, in turn with units of one query tile: dealt
    # whole, and behind long units that several CTAs share
    Hq, Hkv, D = heads
    pair = 2 * (128 // (Hq // Hkv))  # tokens of a unit of two query tiles
    few = 60 if Hkv > 1 else 240
    seqs = [(0, pair + pair // 4)] * few + [(9000, pair // 3), (0, pair)] * 6 + [(0, 3), (0, 2 * pair)] * 4
    run(swa, R.Batch(15, seqs, Hq, Hkv, D, 64), want_counts=False)


@pytest.mark.parametrize("heads", [(12, 4, 128), (5, 5, 64), (6, 2, 256)], ids=str)
def test_shared_units_with_rows_missing(swa, heads):
    # units spread over many CTAs whose last query tile is not full, in one and two query tiles
    Hq, Hkv, D = heads
    for n in (3, 40, 45, 70, 131):
        for p0 in (2000, 9000):
            run(swa, R.Batch(14, [(p0, n), (100, 1)], Hq, Hkv, D, 32), append=n == 45)


@pytest.mark.parametrize("hint", [0, 1])
@pytest.mark.parametrize("case", [(8, 2, 128, 16, 100, 4), (16, 16, 128, 128, 130, 0), (4, 4, 64, 64, 300, 130),
                                  (6, 2, 256, 32, 65, 37), (2, 1, 64, 128, 1, 1)], ids=str)
def test_positions_that_no_query_keeps_may_hold_anything(swa, case, hint):
    # rows between the sinks and the first new token's window, in pages that are there all the same
    Hq, Hkv, D, ps, w, sinks = case
    seqs = [(500, 1), (129, 1), (1000, 1), (0, 1)] if hint else [(500, 33), (129, 300), (1000, 1), (257, 140), (0, 9)]
    if Hq == 16 and not hint:
        seqs.append((600, 3000))  # (units of two query tiles)
    x = R.Batch(51, seqs, Hq, Hkv, D, ps, w, sinks, freed=False)
    for b, (p, _) in enumerate(seqs):
        for t in range(sinks, p - w + 1):
            page = int(x.table[b, t // ps])
            x.k_pages[page, :, t % ps] = float("nan")
            x.v_pages[page, :, t % ps] = float("inf") if t % 2 else float("nan")
    run(swa, x, max_q=hint, q_start=None if hint else x.q_start.cuda())


@pytest.mark.parametrize("ps", [32, 128])
@pytest.mark.parametrize("w,sinks", [(1024, 0), (0, 0), (1024, 400)], ids=str)
def test_tiles_that_come_from_hbm(swa, w, sinks, ps):
    """Single tokens in the many-row kernel at head dim 64, their keys and values out of L2 before each
    call, so that copies land late and unevenly; NaN in every tail and between sinks and window."""
    seqs = [(1000 + 8003 * i // 60 + i % 37, 1) for i in range(61)]
    x = R.Batch(52, seqs, 4, 4, 64, ps, w, sinks, freed=not sinks)
    if sinks:
        for b, (p, _) in enumerate(seqs):
            for j in range(x.width):
                lo, hi = max(sinks - j * ps, 0), min(p - w + 1 - j * ps, ps)
                if lo < hi:
                    for t in (x.k_pages, x.v_pages):
                        t[int(x.table[b, j]), :, lo:hi] = float("nan")
    q, k, v, table, p0, start = (t.cuda() for t in (x.q, x.k_pages, x.v_pages, x.table, x.p0, x.q_start))
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")  # more than L2
    first = None
    for turn in range(40):
        flush.fill_(turn)
        got = swa.swa_paged_attend(q, k, v, table, p0, w, n_sink=sinks, q_start=start, want_counts=True)
        if first is None:
            first = got
            swa.swa_check_device_error()
            verify(x, *first)
        assert all(torch.equal(a, b) for a, b in zip(got, first)), f"call {turn} differs from the first"
    swa.swa_check_device_error()


def test_values_of_the_extremes(swa):
    # scores of +-1000s: one key carries all the weight, and the running maximum jumps
    x = R.Batch(7, [(500, 70), (900, 1)], 8, 2, 128, 32)
    for t in (x.keys[0], x.keys[1]):
        t *= 100
    y = R.Batch(7, [(500, 70), (900, 1)], 8, 2, 128, 32)
    for b, (p, n) in enumerate(x.seqs):  # lay the scaled keys into the pages
        for t in range(p + n):
            y.k_pages[int(y.table[b, t // 32]), :, t % 32] = x.keys[b][t]
    y.keys = x.keys
    run(swa, y)
    run(swa, y, max_q=1)


def test_strided_rows(swa):
    # q, k_new, v_new as views of one fused projection, o as a view with rows apart
    x = R.Batch(8, RAGGED, 8, 2, 128, 16, 300, 4)
    qkv = torch.cat([x.q, x.k_new, x.v_new], 1).cuda()
    out = torch.full((x.N, 2, 8, 128 + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    o = out[:, 1, :, :128]
    k, v = (t.cuda() for t in x.without_new())
    _, lse, cnt = swa.swa_paged_attend(qkv[:, :8], k, v, x.table.cuda(), x.p0.cuda(), 300, n_sink=4,
                                       q_start=x.q_start.cuda(), k_new=qkv[:, 8:10], v_new=qkv[:, 10:], o=o,
                                       want_counts=True)
    swa.swa_check_device_error()
    verify(x, o, lse, cnt)
    assert (out[:, 0] == 7).all() and (out[:, 1, :, 128:] == 7).all()
    assert (R.bits(k) == R.bits(x.k_pages)).all() and (R.bits(v) == R.bits(x.v_pages)).all()


def test_scale(swa):
    x = R.Batch(9, [(40, 20), (3, 1)], 4, 2, 64, 16)
    o, lse, _ = swa.swa_paged_attend(x.q.cuda(), x.k_pages.cuda(), x.v_pages.cuda(), x.table.cuda(), x.p0.cuda(), 0,
                                     0.3, q_start=x.q_start.cuda())
    for b, q0, n in x.rows():
        p = x.seqs[b][0]
        R.check(o[q0:q0 + n], lse[q0:q0 + n], None,
                R.attend(x.q[q0:q0 + n], x.keys[b], x.vals[b], p, 0, 0, scale=0.3))


def test_append_alone(swa):
    x = R.Batch(10, RAGGED, 8, 4, 64, 32, lead=2, tail=2)
    k, v = (t.cuda() for t in x.without_new())
    swa.swa_paged_append(k, v, x.table.cuda(), x.k_new.cuda(), x.v_new.cuda(), x.p0.cuda(), q_start=x.q_start.cuda())
    swa.swa_check_device_error()
    assert (R.bits(k) == R.bits(x.k_pages)).all() and (R.bits(v) == R.bits(x.v_pages)).all()


def test_append_of_one_token_a_sequence(swa):
    x = R.Batch(16, [(i * 13, 1) for i in range(50)], 8, 4, 64, 32)
    k, v = (t.cuda() for t in x.without_new())
    graph = torch.cuda.CUDAGraph()
    a = x.table.cuda(), x.k_new.cuda(), x.v_new.cuda(), x.p0.cuda()
    with torch.cuda.graph(graph):
        swa.swa_paged_append(k, v, *a)
    graph.replay()
    swa.swa_check_device_error()
    assert (R.bits(k) == R.bits(x.k_pages)).all() and (R.bits(v) == R.bits(x.v_pages)).all()


def test_offsets_past_32_bits(swa):
    # the pages lie past element 2^31 of their pools
    x = R.Batch(11, [(70, 1), (10, 90)], 8, 8, 128, 64)
    per = 8 * 64 * 128
    first = (1 << 31) // per + 5
    k = torch.empty((first + x.n_pages, 8, 64, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    k[first:], v[first:] = x.k_pages.cuda(), x.v_pages.cuda()
    table = torch.where(x.table >= 0, x.table + first, x.table).cuda()
    for hint in (1, 0):
        o, lse, cnt = swa.swa_paged_attend(x.q.cuda(), k, v, table, x.p0.cuda(), q_start=x.q_start.cuda(), max_q=hint,
                                           k_new=x.k_new.cuda(), v_new=x.v_new.cuda(), want_counts=True)
        swa.swa_check_device_error()
        verify(x, o, lse, cnt)


def error_bits(swa):
    st, words = swa.swa_read_device_errors()
    return st, words


@pytest.mark.parametrize("hint", [0, 1])
def test_broken_device_data(swa, hint):
    """What the device finds broken is reported, its sequence skipped, and the others are right."""
    def call(x, table=None, p0=None, q_start=None):
        o = torch.full((x.N, x.Hq, x.D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((x.N, x.Hq), 7.0, device="cuda")
        swa.swa_paged_attend(x.q.cuda(), x.k_pages.cuda(), x.v_pages.cuda(), (x.table if table is None else table).cuda(),
                             (x.p0 if p0 is None else p0).cuda(), x.window, o=o, lse=lse, max_q=hint,
                             q_start=(x.q_start if q_start is None else q_start).cuda())
        return o, lse

    x = R.Batch(12, [(50, 9), (20, 3), (7, 1)], 4, 2, 64, 16)
    # a negative position, one past the table's end
    for p in (-1, 16 * x.width):
        p0 = x.p0.clone()
        p0[1] = p
        o, lse = call(x, p0=p0)
        assert error_bits(swa) == (1, {"prefill": 0, "split": 0, "cache": swa.DEVERR_BAD_POSITION})
        verify(x, o, lse, None, skip=(1,))
    # a row list that goes down, or past the rows
    for at, to in ((1, -3), (3, x.N + 1)):
        q_start = x.q_start.clone()
        q_start[at] = to
        o, lse = call(x, q_start=q_start)
        st, words = error_bits(swa)
        assert st == 1 and words["cache"] == swa.DEVERR_BAD_POSITION
        if at == 3:
            verify(x, o, lse, None, skip=(2,))
    # a page that is needed and missing, or not in the pool
    for e in (-1, x.n_pages, 2 ** 31 - 1, -2 ** 31):
        table = x.table.clone()
        table[0, 1] = e
        o, lse = call(x, table=table)
        assert error_bits(swa) == (1, {"prefill": 0, "split": 0, "cache": swa.DEVERR_BAD_PAGE})
        assert torch.isfinite(o).all()
        for b, q0, n in x.rows()[1:]:
            R.check(o[q0:q0 + n], lse[q0:q0 + n], None, x.reference(b))
    # ... which rows of zeros stand in for
    y = R.Batch(12, [(50, 9), (20, 3), (7, 1)], 4, 2, 64, 16)
    y.keys[0][16:32] = 0
    y.vals[0][16:32] = 0
    R.check(o[:9], lse[:9], None, y.reference(0))
    # an append to a missing page stores nothing there
    k, v = x.k_pages.cuda(), x.v_pages.cuda()
    table = torch.full_like(x.table, -1)
    swa.swa_paged_append(k, v, table.cuda(), x.k_new.cuda(), x.v_new.cuda(), x.p0.cuda(), q_start=x.q_start.cuda())
    assert error_bits(swa)[1]["cache"] == swa.DEVERR_BAD_PAGE
    assert (R.bits(k) == R.bits(x.k_pages)).all()
    # and the next call is clean
    run(swa, x)


@pytest.mark.parametrize("hint", [0, 1])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_sequences_that_overlap_are_no_work(swa, D, hint):
    # q_start goes up and down, so that every other sequence has all rows: reported, and not computed (the
    # units of many such sequences pass what 32 bits count)
    B, N = 80, 1280
    start = R.i32([N * (b % 2) for b in range(B + 1)])
    k = torch.zeros(N // 16, 1, 16, D, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(N // 16, dtype=torch.int32, device="cuda").repeat(B, 1)
    q = torch.zeros(N, 2, D, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.full_like(q, 7), torch.full((N, 2), 7.0, device="cuda")
    swa.swa_paged_attend(q, k, k.clone(), table, R.i32([0] * B), q_start=start, max_q=hint, o=o, lse=lse)
    assert error_bits(swa) == (1, {"prefill": 0, "split": 0, "cache": swa.DEVERR_BAD_POSITION})
    assert (o == 7).all() and (lse == 7).all()


@pytest.mark.parametrize("hint", [0, 1])
def test_captured_and_replayed(swa, hint):
    # two graphs with workspaces of their own, replayed in turn with other lengths and pages
    def batch(seed, seqs):
        return R.Batch(seed, seqs, 8, 2, 128, 16, 400, 2, width=80, spare=200 - 0)

    lens = {0: [(100, 5), (1200, 1), (0, 30)], 1: [(900, 20), (3, 15), (640, 1)]}
    graphs = []
    for g in range(2):
        x = batch(20 + g, lens[g])
        t = dict(q=x.q.cuda(), k=x.k_pages.cuda(), v=x.v_pages.cuda(), table=x.table.cuda(), p0=x.p0.cuda(),
                 start=x.q_start.cuda())
        o = torch.full((x.N, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((x.N, 8), 7.0, device="cuda")

        def call(t=t, o=o, lse=lse):
            swa.swa_paged_attend(t["q"], t["k"], t["v"], t["table"], t["p0"], 400, n_sink=2, q_start=t["start"],
                                 max_q=hint, o=o, lse=lse)

        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append((graph, t, o, lse))
    for turn in range(3):
        for g in range(2):
            graph, t, o, lse = graphs[g]
            # the same sizes of everything, other lengths: the tokens dealt another way
            seqs = {0: [(100 + turn, 5 + turn), (1200, 1), (7 * turn, 30 - turn)],
                    1: [(900 - turn, 20), (3, 15 - turn), (640, 1 + turn)]}[g]
            x = batch(30 + 2 * turn + g, seqs)
            assert x.N == o.shape[0]
            k = torch.full_like(t["k"], float("nan"))
            v = torch.full_like(k, float("nan"))
            n = min(k.shape[0], x.n_pages)
            assert int(x.table.max()) < n
            k[:n], v[:n] = x.k_pages[:n].cuda(), x.v_pages[:n].cuda()
            for name, val in dict(q=x.q, k=k, v=v, table=x.table, p0=x.p0, start=x.q_start).items():
                t[name].copy_(val)
            o.fill_(7)
            graph.replay()
            swa.swa_check_device_error()
            verify(x, o, lse, None)


def test_one_workspace_for_many_calls(swa):
    # whatever it holds: other calls' partial results and counters, of other shapes
    ws = torch.full((96 << 20,), 255, dtype=torch.uint8, device="cuda")
    xs = [R.Batch(45 + D, [(5000, 40), (9, 1), (700, 130)], 8, 2, D, 32) for D in (64, 128, 256)]
    xs += [R.Batch(46 + D, [(5000, 1), (9, 1), (12000, 1)], 8, 2, D, 32) for D in (64, 128, 256)]
    for turn in range(2):
        for x in xs[::1 - 2 * turn]:
            one = x.N == 3
            run(swa, x, append=turn == 1, workspace=ws, q_start=None if one else x.q_start.cuda())


def test_few_workspace_sizes_are_kept(swa):
    # a server whose longest chunk varies: the sizes looked up stay as few as the kernels' shapes
    x = R.Batch(48, [(5, 2), (3, 1)], 4, 2, 64, 16)
    a = x.q.cuda(), x.k_pages.cuda(), x.v_pages.cuda(), x.table.cuda(), x.p0.cuda()
    start, before = x.q_start.cuda(), len(swa._paged_ws_size)
    for most in [*range(2, 200), 1 << 20, (1 << 31) - 1]:
        swa.swa_paged_attend(*a, q_start=start, max_q=most)
    assert len(swa._paged_ws_size) - before <= 17
    swa.swa_check_device_error()


def test_two_streams_at_once(swa):
    xs = [R.Batch(40 + i, [(3000, 70), (10, 1), (900, 200)], 8, 2, 128, 32, 1000) for i in range(4)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    args = [(x.q.cuda(), x.k_pages.cuda(), x.v_pages.cuda(), x.table.cuda(), x.p0.cuda(), x.q_start.cuda()) for x in xs]
    torch.cuda.synchronize()
    outs = []
    for i, a in enumerate(args):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(swa.swa_paged_attend(*a[:5], 1000, q_start=a[5], max_q=[0, 1][i // 2], want_counts=True))
    torch.cuda.synchronize()
    swa.swa_check_device_error()
    for x, (o, lse, cnt) in zip(xs, outs):
        verify(x, o, lse, cnt)


def test_on_a_stream_that_is_not_the_current_one(swa):
    # the call's own memory belongs to its stream: the current stream's blocks come and go meanwhile
    side = torch.cuda.Stream()
    for seqs, hint in (([(3000, 70), (10, 1), (900, 200)], 0), ([(3000, 1), (10, 1), (9000, 1)], 1)):
        x = R.Batch(47, seqs, 8, 2, 128, 32, 1000)
        a = (x.q.cuda(), x.k_pages.cuda(), x.v_pages.cuda(), x.table.cuda(), x.p0.cuda())
        start = None if hint else x.q_start.cuda()
        want = swa.swa_paged_attend(*a, 1000, q_start=start, max_q=hint, want_counts=True)
        torch.cuda.synchronize()
        got = []
        for _ in range(20):
            for n in (1 << 20, 10 << 20, 40 << 20):
                torch.full((n,), 255, dtype=torch.uint8, device="cuda")
            got.append(swa.swa_paged_attend(*a, 1000, q_start=start, max_q=hint, want_counts=True, stream=side))
        torch.cuda.synchronize()
        swa.swa_check_device_error(side)
        for g in got:
            assert all(torch.equal(p, q) for p, q in zip(g, want))
    # the pages' calls take one, too
    table, ref = torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), torch.zeros(20, dtype=torch.int32, device="cuda")
    k = torch.randn(20, 2, 16, 64, device="cuda").to(torch.bfloat16)
    v, kn = k.clone(), torch.randn(2, 2, 64, device="cuda").to(torch.bfloat16)
    zero, end, src, one, last = R.i32([0, 0]), R.i32([20, 20]), R.i32([0, 0]), R.i32([0]), R.i32([19])
    torch.cuda.synchronize()
    swa.swa_pages_reserve(table, ref, zero, end, 16, stream=side)
    swa.swa_paged_append(k, v, table, kn, kn, zero, stream=side)
    t2, r2 = swa.swa_pages_fork(k, v, table, ref, src, end, stream=side)
    swa.swa_pages_compact(k, v, t2, r2, stream=side)
    swa.swa_pages_copy(k, v, one, last, stream=side)
    torch.cuda.synchronize()
    swa.swa_check_device_error(side)
    # (row 0's first page stays with it and its copy, both rows' others are their own)
    assert t2.tolist() == [[0, 1, -1, -1], [0, 2, -1, -1]] and r2.tolist()[:4] == [2, 1, 1, 0]
    assert torch.equal(k[19], k[0]) and torch.equal(k[0, :, 0], kn[0]) and torch.equal(k[1, :, :4], k[2, :, :4])
    swa.swa_pages_free(t2, r2, R.i32([-1, -1]), 16, stream=side)
    torch.cuda.synchronize()
    assert (t2 == -1).all() and (r2 == 0).all()


def test_same_call_same_bits(swa):
    x = R.Batch(50, [(5000, 300), (77, 1), (4000, 1)], 8, 2, 128, 16)
    for hint in (0, 1):
        a, b = (run(swa, x, max_q=hint) for _ in range(2))
        assert (R.bits(a[0]) == R.bits(b[0])).all() and torch.equal(a[1], b[1])


def test_refusals(swa):
    x = R.Batch(60, [(5, 2), (3, 1)], 4, 2, 64, 16)
    a = dict(q=x.q.cuda(), k_pages=x.k_pages.cuda(), v_pages=x.v_pages.cuda(), page_table=x.table.cuda(),
             p0=x.p0.cuda(), q_start=x.q_start.cuda())

    def refused(**kw):
        with pytest.raises((ValueError, swa.SwaError)):
            swa.swa_paged_attend(**{**a, **kw})

    refused(q=a["q"].float())
    refused(q=a["q"][:, :, :32])
    refused(q=a["q"].cpu())
    refused(q=a["q"][:, :3])                       # heads not a multiple of the kv heads
    refused(q=a["q"].expand(3, 4, 64)[:, :1].expand(3, 4, 64))  # a head stride of 0
    refused(k_pages=a["k_pages"].transpose(1, 2))
    refused(v_pages=a["v_pages"][:-1])
    refused(page_table=a["page_table"].long())
    refused(page_table=a["page_table"].cpu())
    refused(p0=a["p0"][:1])
    refused(q_start=a["q_start"][:2])
    refused(q_start=None)                          # three rows, two sequences
    refused(k_new=x.k_new.cuda())                  # without v_new
    refused(k_new=x.k_new.cuda()[:2], v_new=x.v_new.cuda()[:2])
    refused(window=-1)
    refused(n_sink=-1)
    refused(scale=float("nan"))
    refused(o=torch.empty(3, 4, 32, dtype=torch.bfloat16, device="cuda"))
    refused(lse=torch.empty(3, 4, dtype=torch.float64, device="cuda"))
    refused(row_counts=torch.empty(3, 4, device="cuda"))
    refused(k_pages=a["k_pages"][:, :, :8].contiguous(), v_pages=a["v_pages"][:, :, :8].contiguous())  # pages of 8
    refused(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))  # too small
    o, lse, _ = swa.swa_paged_attend(x.q[:0].cuda(), *(a[n] for n in ("k_pages", "v_pages", "page_table", "p0")),
                                     q_start=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    swa.swa_check_device_error()


def test_workspaces_of_another_kind_are_refused(swa):
    # (one in host memory would be written to by the kernels)
    x = R.Batch(61, [(5, 2), (3, 1)], 4, 2, 64, 16)
    a = [t.cuda() for t in (x.q, x.k_pages, x.v_pages, x.table, x.p0)]
    start, ref = x.q_start.cuda(), torch.zeros(x.n_pages, dtype=torch.int32, device="cuda")
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    for ws in (torch.empty(64 << 20, dtype=torch.uint8), torch.empty(64 << 20, dtype=torch.uint8).pin_memory(),
               torch.empty(64 << 20, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace"):
            swa.swa_paged_attend(*a, q_start=start, workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            swa.swa_pages_reserve(a[3], ref, zero, zero, 16, workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            swa.swa_pages_fork(*a[1:4], ref, zero, zero, workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            swa.swa_pages_compact(*a[1:4], ref, workspace=ws)
    swa.swa_check_device_error()


def test_numbers_that_32_bits_do_not_hold_are_refused(swa):
    x = R.Batch(62, [(5, 2), (3, 1)], 4, 2, 64, 16)
    a = [t.cuda() for t in (x.q, x.k_pages, x.v_pages, x.table, x.p0)]
    start, ref = x.q_start.cuda(), torch.ones(x.n_pages, dtype=torch.int32, device="cuda")
    for kw in (dict(window=1 << 31), dict(n_sink=1 << 32), dict(max_q=1 << 31), dict(scale=1e39)):
        with pytest.raises(swa.SwaError if "scale" in kw else ValueError):  # (packed as infinity)
            swa.swa_paged_attend(*a, q_start=start, **kw)
    below = torch.full((2,), 1 << 20, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        swa.swa_pages_free(a[3], ref, below, 16, n_sink=1 << 32)  # (its low 32 bits are 0)
    with pytest.raises(ValueError):
        swa.swa_pages_free(a[3], ref, below, 1 << 31)
    assert torch.equal(a[3].cpu(), x.table)
    swa.swa_check_device_error()
