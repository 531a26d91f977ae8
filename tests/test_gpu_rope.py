"""The table of a rotation, and the append that rotates keys and queries on their way into a paged cache,
against 64-bit computations."""
import math

import pytest
import torch

import paged_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def swa():
    import sliding_window_attention_swa_gb300 as m

    m.load_library()
    return m


def frequencies(rot, base=10000.0):
    return base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)


def host_table(rot, n_pos):
    angle = torch.arange(n_pos).double()[:, None] * frequencies(rot)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


# ---------------------------------------------------------------------------------------------
# table
# ---------------------------------------------------------------------------------------------
def check_table(got, f, n_pos, scale, first=0):
    """An entry is off by its angle's error (2^-33 turns of rounding and 2^-25 of at most an eighth of a turn:
    2.5e-8), sincospif's (two steps of at most 2^-24) and the product's rounding, 2^-24: below 2^-22 of
    the scale together.  The 64-bit reference adds p |f| 2^-53."""
    angle = torch.arange(first, first + n_pos, device="cuda").double()[:, None] * f.cuda()
    ref = torch.cat([angle.cos(), angle.sin()], 1) * scale
    bound = 2.0 ** -22 * abs(scale) + abs(scale) * (angle.abs().amax().item() * 2.0 ** -52)
    assert (got.double() - ref).abs().max().item() <= bound


@pytest.mark.parametrize("n_pos", [1, 2, 7, 8, 9, 1000, 4097])
@pytest.mark.parametrize("rot", [16, 32, 48, 96, 128, 256])
def test_table(swa, rot, n_pos):
    f = frequencies(rot)
    got = swa.swa_rope_table(f.cuda(), n_pos)
    assert got.shape == (n_pos, rot) and got.dtype == torch.float32
    check_table(got, f, n_pos, 1.0)


def test_table_of_far_positions_and_odd_frequencies(swa):
    check_table(swa.swa_rope_table(frequencies(64, 5e5).cuda(), 1 << 20, 1.25), frequencies(64, 5e5), 1 << 20, 1.25)
    # negative ones, whole turns, several turns a position, none
    f = torch.tensor([-1.0, 2 * math.pi, -0.37, 1000.5, 0.0, 1e-9, math.pi, -math.pi / 2], dtype=torch.float64)
    got = swa.swa_rope_table(f.cuda(), 3001, -0.5)
    check_table(got, f, 3001, -0.5)
    assert (got[:, 4] == -0.5).all() and (got[:, 12] == 0).all()
    assert (got[0, :8] == -0.5).all() and (got[0, 8:] == 0).all()


def test_table_layouts(swa):
    f = frequencies(32).cuda()
    whole = torch.full((60, 32), 7.0, device="cuda")
    out = whole[3:53]  # (rows of a larger buffer)
    assert swa.swa_rope_table(f, 50, out=out) is out
    check_table(out, f, 50, 1.0)
    assert (whole[:3] == 7).all() and (whole[53:] == 7).all()
    assert swa.swa_rope_table(f, 0).shape == (0, 32)
    bad = f.clone()
    bad[3], bad[5] = float("nan"), float("inf")
    got = swa.swa_rope_table(bad, 9)
    wrong = torch.zeros(32, dtype=torch.bool, device="cuda")
    wrong[[3, 5, 19, 21]] = True
    assert torch.equal(torch.isnan(got), wrong.expand(9, 32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = swa.swa_rope_table(f, 50, stream=side)
    side.synchronize()
    assert torch.equal(got, out)


def test_table_refusals(swa):
    f = frequencies(32).cuda()
    for bad in (f.float(), f.cpu(), f[None], frequencies(64).cuda()[::2]):
        with pytest.raises(ValueError):
            swa.swa_rope_table(bad, 10)
    for out in (torch.empty(10, 32), torch.empty(10, 31, device="cuda"), torch.empty(10, 64, device="cuda")[:, ::2],
                torch.empty(10, 32, dtype=torch.float64, device="cuda")):
        with pytest.raises(ValueError):
            swa.swa_rope_table(f, 10, out=out)
    for args in ((f[:7], 10), (frequencies(512).cuda(), 10), (f, -1), (f, 10, float("inf"))):
        with pytest.raises((swa.SwaError, RuntimeError)):
            swa.swa_rope_table(*args)
    with pytest.raises(ValueError):
        swa.swa_rope_table(f, 1 << 32)


# ---------------------------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------------------------
def turned(x, table, pos, interleaved):
    """(rotated x [n, heads, d], the size of what an fp32 computation rounds) in 64 bits."""
    half = table.shape[1] // 2
    c, s = (table[pos][:, None, a:a + half].double() for a in (0, half))
    x = x.double()
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y, size = x.clone(), x.abs()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    size[..., a], size[..., b] = (x[..., a] * c).abs() + (x[..., b] * s).abs(), (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, size


def close(got, ref, size):
    """One rounding to bf16 (2^-8 of the value), two products and a sum in fp32 (2^-24 each of at most size)."""
    got = got.cpu().double()
    return ((got - ref).abs() <= 2.0 ** -8 * (1 + 2.0 ** -20) * ref.abs() + 2.0 ** -22 * size).all()


def batch(x, rot, n_pos=None):
    pools = [t.cuda() for t in x.without_new()]
    return pools, host_table(rot, n_pos or max(p + n for p, n in x.seqs)), x.table.cuda(), x.p0.cuda(), x.q_start.cuda()


def verify(x, table, interleaved, q_out, k, v, before, skip=()):
    k_want, v_want = (R.bits(t).copy() for t in before)
    mine = torch.zeros(x.N, dtype=torch.bool)
    for b, q0, n in x.rows():
        if b in skip:
            continue
        p = x.seqs[b][0]
        pos = torch.arange(p, p + n)
        mine[q0:q0 + n] = True
        if q_out is not None:
            assert close(q_out[q0:q0 + n], *turned(x.q[q0:q0 + n], table, pos, interleaved)), f"queries of sequence {b}"
        if k is None:
            continue
        page, row = x.table[b].long()[pos // x.ps], pos % x.ps
        assert close(k.cpu()[page, :, row], *turned(x.keys[b][p:], table, pos, interleaved)), f"keys of sequence {b}"
        # (what of a key is not rotated, and every value, bit for bit)
        rot = table.shape[1]
        assert (R.bits(k)[page, :, row, rot:] == R.bits(x.keys[b][p:])[..., rot:]).all()
        k_want[page, :, row] = R.bits(k)[page, :, row]
        v_want[page, :, row] = R.bits(x.vals[b][p:])
    if q_out is not None:
        assert (q_out.cpu()[~mine] == 7).all(), "rows of no sequence were written"
    if k is not None:
        assert (R.bits(k) == k_want).all() and (R.bits(v) == v_want).all(), "other rows of the pages were written"


ONE = [(0, 1), (1, 1), (15, 1), (16, 1), (127, 1), (128, 1), (4001, 1)]
RAGGED = [(0, 1), (5, 33), (0, 0), (130, 1), (64, 64), (0, 257), (0, 0), (1111, 7), (300, 129)]
SHAPES = [
    # Hq, Hkv, D, page, rot
    (8, 2, 128, 16, 128), (32, 8, 128, 64, 64), (4, 4, 64, 32, 64), (12, 12, 64, 16, 32), (16, 8, 256, 64, 256),
    (6, 2, 256, 128, 48), (7, 1, 128, 128, 16), (1, 1, 64, 16, 48), (40, 2, 128, 32, 112), (5, 5, 256, 16, 240),
]


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_append(swa, shape, interleaved):
    Hq, Hkv, D, ps, rot = shape
    for seqs, lead, tail in ((ONE, 0, 0), (RAGGED, 3, 5)):
        x = R.Batch(21, seqs, Hq, Hkv, D, ps, lead=lead, tail=tail)
        (k, v), table, pages, p0, start = batch(x, rot)
        q_out = torch.full(x.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        got = swa.swa_paged_rope_append(x.q.cuda(), k, v, pages, x.k_new.cuda(), x.v_new.cuda(), p0, table.cuda(),
                                        q_start=None if seqs is ONE else start, interleaved=interleaved, q_out=q_out)
        swa.swa_check_device_error()
        assert got is q_out
        verify(x, table, interleaved, q_out, k, v, x.without_new())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_parts_and_layouts(swa, D):
    x = R.Batch(22, RAGGED, 6, 2, D, 16)
    (k, v), table, pages, p0, start = batch(x, 32)
    rope = table.cuda()
    both = torch.full(x.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    swa.swa_paged_rope_append(x.q.cuda(), k, v, pages, x.k_new.cuda(), x.v_new.cuda(), p0, rope, q_start=start, q_out=both)
    # keys and values alone, queries alone, queries in place
    k2, v2 = (t.cuda() for t in x.without_new())
    assert swa.swa_paged_rope_append(None, k2, v2, pages, x.k_new.cuda(), x.v_new.cuda(), p0, rope, q_start=start) is None
    assert (R.bits(k2) == R.bits(k)).all() and (R.bits(v2) == R.bits(v)).all()
    alone = swa.swa_paged_rope_append(x.q.cuda(), k2, v2, pages, None, None, p0, rope, q_start=start)
    assert torch.equal(alone, both) and (R.bits(k2) == R.bits(k)).all()
    q = x.q.cuda()
    assert swa.swa_paged_rope_append(q, k2, v2, pages, None, None, p0, rope, q_start=start, q_out=q) is q
    assert torch.equal(q, both)
    # the heads of one projection's output, on another stream, the output a view with strides of its own
    qkv = torch.cat([x.q, x.k_new, x.v_new], 1).cuda()
    wide = torch.full((x.N, 9, D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    k3, v3 = (t.cuda() for t in x.without_new())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    swa.swa_paged_rope_append(qkv[:, :6], k3, v3, pages, qkv[:, 6:8], qkv[:, 8:], p0, rope, q_start=start,
                              q_out=wide[:, 2:8, :D], stream=side)
    side.synchronize()
    assert torch.equal(wide[:, 2:8, :D], both)
    assert (wide[:, :2] == 7).all() and (wide[:, 8:] == 7).all() and (wide[..., D:] == 7).all()
    assert (R.bits(k3) == R.bits(k)).all() and (R.bits(v3) == R.bits(v)).all()
    swa.swa_check_device_error()


def test_many_tokens_and_sequences(swa):
    for seqs in ([(9, 9001)], [(i % 50, 1) for i in range(3001)], [(i % 40, i % 3) for i in range(8192)]):
        x = R.Batch(23, seqs, 4, 1, 64, 16)
        (k, v), table, pages, p0, start = batch(x, 64)
        q_out = torch.full(x.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        swa.swa_paged_rope_append(x.q.cuda(), k, v, pages, x.k_new.cuda(), x.v_new.cuda(), p0, table.cuda(),
                                  q_start=start, q_out=q_out)
        swa.swa_check_device_error()
        pos = torch.cat([torch.arange(p, p + n) for p, n in seqs])
        assert close(q_out, *turned(x.q, table, pos, False))
        seq = torch.repeat_interleave(torch.arange(len(seqs)), torch.tensor([n for _, n in seqs]))
        page, row = x.table[seq, pos // 16].long(), pos % 16
        assert close(k.cpu()[page, :, row], *turned(x.k_new[:len(pos)], table, pos, False))
        assert torch.equal(v.cpu()[page, :, row], x.v_new[:len(pos)])


def test_no_tokens(swa):
    x = R.Batch(24, [(3, 0), (5, 0)], 4, 2, 64, 16)
    (k, v), table, pages, p0, start = batch(x, 64)
    before = R.bits(k)
    got = swa.swa_paged_rope_append(x.q.cuda(), k, v, pages, x.k_new.cuda(), x.v_new.cuda(), p0, table.cuda(), q_start=start)
    assert got.shape == (0, 4, 64) and (R.bits(k) == before).all()


def test_infinities_stay_where_they_are(swa):
    # a pair with an infinity becomes infinities or NaN; the head's other elements do not see it
    x = R.Batch(25, [(7, 3)], 4, 2, 128, 16)
    x.q[1, 2, 5], x.q[2, 0, 70] = float("inf"), float("nan")
    (k, v), table, pages, p0, start = batch(x, 128)
    got = swa.swa_paged_rope_append(x.q.cuda(), k, v, pages, x.k_new.cuda(), x.v_new.cuda(), p0, table.cuda(),
                                    q_start=start).cpu()
    wild = ~torch.isfinite(got)
    assert wild[1, 2, [5, 69]].all() and wild[2, 0, [6, 70]].all() and wild.sum() == 4


def test_broken_device_data(swa):
    x = R.Batch(26, [(5, 3), (40, 2), (9, 4), (2, 1)], 4, 2, 64, 16, lead=1, tail=1)
    (k, v), table, pages, p0, start = batch(x, 64)
    rope = table.cuda()
    new = x.k_new.cuda(), x.v_new.cuda()

    def go(p0, pages, rope):
        pools = [t.cuda() for t in x.without_new()]
        q_out = torch.full(x.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        swa.swa_paged_rope_append(x.q.cuda(), *pools, pages, *new, p0, rope, q_start=start, q_out=q_out)
        return q_out, *pools, swa.swa_read_device_errors()

    # a position below 0 or past the table row: that sequence is left as it was
    for wrong in (-1, 3 * 16 + 14, (1 << 31) - 1):
        bad = p0.clone()
        bad[1] = wrong
        q_out, k, v, (st, words) = go(bad, pages, rope)
        assert st == 1 and words == {"prefill": 0, "split": 0, "cache": swa.DEVERR_BAD_POSITION}
        verify(x, table, False, q_out, k, v, x.without_new(), skip=(1,))
    # a rotation's table that ends before sequence 1's last token: that token is left as it was
    q_out, k, v, (st, words) = go(p0, pages, rope[:41])
    assert st == 1 and words["cache"] == swa.DEVERR_BAD_POSITION
    row = 1 + 3 + 1
    assert (q_out[row] == 7).all() and not (q_out[row - 1] == 7).all()
    assert torch.isnan(k[int(x.table[1, 2]), :, 41 % 16]).all()
    # no page, or one that the pool has not: the token is not stored, its query is there
    for entry in (-1, x.n_pages, -(1 << 31)):
        bad = pages.clone()
        bad[2, 0] = entry
        q_out, k, v, (st, words) = go(p0, bad, rope)
        assert st == 1 and words["cache"] == swa.DEVERR_BAD_PAGE
        verify(x, table, False, q_out, None, None, x.without_new())
        verify(x, table, False, None, k, v, x.without_new(), skip=(2,))
    # a start that goes down: rows in reach are rotated by some position, nothing else is written
    down = start.clone()
    down[2] = 0
    swa.swa_paged_rope_append(x.q.cuda(), k, v, pages, *new, p0, rope, q_start=down)
    st, words = swa.swa_read_device_errors()
    assert st == 1 and words["prefill"] == words["split"] == 0 and words["cache"]


def test_append_refusals(swa):
    x = R.Batch(27, [(5, 3), (40, 2)], 4, 2, 64, 16)
    (k, v), table, pages, p0, start = batch(x, 64)
    q, kn, vn, rope = x.q.cuda(), x.k_new.cuda(), x.v_new.cuda(), table.cuda()

    def refused(error, q=q, k=k, kn=kn, vn=vn, rope=rope, p0=p0, start=start, **kw):
        with pytest.raises(error):
            swa.swa_paged_rope_append(q, k, v, pages, kn, vn, p0, rope, q_start=start, **kw)

    refused(ValueError, q=None, kn=None, vn=None)
    refused(ValueError, vn=None)
    refused(ValueError, q=q.float())
    refused(ValueError, q=q[:, :, ::2])
    refused(ValueError, q=q.cpu())
    refused(ValueError, kn=kn[:4], vn=vn[:4])
    refused(ValueError, rope=rope.double())
    refused(ValueError, rope=rope[:, ::2])
    refused(ValueError, rope=rope.cpu())
    refused(ValueError, rope=rope[0])
    refused(ValueError, p0=p0.long())
    refused(ValueError, start=None)
    refused(ValueError, q_out=torch.empty(5, 3, 64, dtype=torch.bfloat16, device="cuda"))
    refused(ValueError, q=None, q_out=torch.empty_like(q))
    wide = torch.zeros(5, 4, 128, dtype=torch.bfloat16, device="cuda")
    refused(ValueError, q=wide[:, :, :64], q_out=torch.as_strided(wide, (5, 4, 64), (256, 64, 1)))
    refused(swa.SwaError, rope=rope[:, :40].contiguous())                     # no multiple of 16
    refused(swa.SwaError, rope=host_table(128, 50).cuda())                    # more than the head
    refused(swa.SwaError, rope=rope[:0])
    refused(swa.SwaError, rope=rope.view(-1)[1:-63].view(-1, 64))             # not aligned
    refused(swa.SwaError, q=torch.zeros(5, 3, 64, dtype=torch.bfloat16, device="cuda"))  # 3 heads for 2
    refused(swa.SwaError, q=torch.zeros(5, 4, 68, dtype=torch.bfloat16, device="cuda")[:, :, :64])


def test_captured_and_replayed(swa):
    # other positions, tokens and tables at each replay
    x = R.Batch(28, [(5, 30), (70, 2), (9, 1)], 4, 2, 128, 16)
    (k, v), table, pages, p0, start = batch(x, 128, 200)
    q, kn, vn, rope = x.q.cuda(), x.k_new.cuda(), x.v_new.cuda(), table.cuda()
    q_out = torch.full(x.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    swa.swa_paged_rope_append(q, k, v, pages, kn, vn, p0, rope, q_start=start, q_out=q_out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        swa.swa_paged_rope_append(q, k, v, pages, kn, vn, p0, rope, q_start=start, q_out=q_out)
    y = R.Batch(29, [(11, 25), (0, 7), (60, 1)], 4, 2, 128, 16, width=x.width, spare=4)
    assert y.n_pages == x.n_pages and y.N == x.N
    before = y.without_new()
    k.copy_(before[0])
    v.copy_(before[1])
    for dst, src in ((q, y.q), (kn, y.k_new), (vn, y.v_new), (pages, y.table), (p0, y.p0), (start, y.q_start)):
        dst.copy_(src)
    graph.replay()
    swa.swa_check_device_error()
    verify(y, table, False, q_out, k, v, before)
