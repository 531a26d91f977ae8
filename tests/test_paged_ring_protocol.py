"""Model check of the paged tile kernel's barriers (CPU only).

paged_tile_kernel streams a CTA's key and value tiles through a ring of NSLOT shared-memory slots
that two producer warps fill, computes scores in two or three tensor-memory slots, and hands
them to softmax warps that write P over them.  Every hand-over is an mbarrier, and a wait
names only the parity of the phase it waits for: it is right only if the phase before has completed
already, and the phase behind cannot.

The roles run here as coroutines in random orders and at random speeds: the planner (which hands the
pieces over and loads the query tiles), the producers of keys and of values, copies that land in any
order, the MMA warp, the tensor pipe (which completes MMAs and commits in order), and every
softmax and epilogue warp.  At every
wait that a parity lets pass, the phase counted must be the newest one completed.  Besides:
  * an MMA's tiles have landed and are still in their slots, until it completes;
  * a fill goes to a slot whose tile has been read by all its readers;
  * the value rows that are zeroed (in tiles where a sequence, its sinks or the part before its
    window ends) are those of a tile that has landed;
  * O is rescaled when the MMAs that write it are complete;
  * no order ends in a deadlock;
  * a producer that gives up returns when, and not before, its own copies have landed.
A model of the protocol, not of the kernel's code: the orders below restate the kernel's.  The ring
sizes are the source's.
"""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "sliding_window_attention_swa_gb300", "csrc", "swa_paged_tile.cu")


def ring_slots(D):
    """NSLOT of TileCfg<D>, by its line in the source."""
    with open(SOURCE) as f:
        line = re.search(r"static constexpr int NSLOT = D == 64 \? (\d+) : NSLOT_RAW;", f.read())
    assert line, "TileCfg's NSLOT is no longer what this test reads"
    if D == 64:
        return int(line.group(1))
    nqt, bn = (2, 128) if D == 128 else (1, 64)
    return (232448 - 512 - nqt * 128 * 8 - (nqt * 128 * D * 2 if nqt == 2 else 0)) // (bn * D * 2)


NP = 4  # pieces planned ahead


class Barrier:
    def __init__(self, name, count):
        self.name, self.count, self.arrived, self.done = name, count, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived, self.done = 0, self.done + 1

    def passes(self, phase):
        if (self.done & 1) == (phase & 1):  # what the hardware compares
            return False
        assert self.done == phase + 1, f"{self.name}: a wait for phase {phase} passes with {self.done} completed"
        return True


class Kernel:
    """pieces: [(tiles, single)]; nqt, ns: query tiles of a CTA, score slots."""

    waits_twice = False  # (a fault that the model catches)

    def __init__(self, pieces, nslot, nqt, ns, rng):
        self.pieces, self.nslot, self.nqt, self.ns, self.rng = pieces, nslot, nqt, ns, rng
        b = lambda name, n, count: [Barrier(f"{name}[{i}]", count) for i in range(n)]  # noqa: E731
        self.full, self.empty = b("full", nslot, 1), b("empty", nslot, 1)
        self.qf, self.qe = b("q_full", 2, 1), b("q_empty", 2, 4)
        self.sf, self.pf = b("s_full", 3, 1), b("p_full", 3, 4)
        self.od, self.of = b("o_done", 2, 1), b("o_free", 2, 4)
        self.meet = Barrier("meet", 4 * nqt)
        self.piece, self.used = b("piece_full", NP, 1), b("piece_empty", NP, 2 + nqt + 8)
        self.occupant, self.landed, self.in_flight, self.reads = {}, set(), [], {}
        self.stop = [1 << 30, 1 << 30]  # the producers' first fills that they do not issue
        self.fills = [0, 1]             # their next fills
        self.issued = [[], []]
        self.pipe = []   # MMAs and commits in issue order
        self.o_writes = [0, 0]  # MMAs into each accumulator that have not completed
        self.start = []  # tiles before each piece
        t = 0
        for n, _ in pieces:
            self.start.append(t)
            t += n
        # tiles whose value rows are zeroed: the last of a piece, and two at any place
        self.zeroed = set()
        for (n, _), J in zip(pieces, self.start):
            self.zeroed.add(J + n - 1)
            e = rng.randrange(-1, n)
            self.zeroed |= {J + i for i in (e, e + 1) if 0 <= i < n}

    # ---- fills: a piece's query tile first at one query tile a CTA (two), then K and V of its tiles
    def kfill(self, k, g):
        return (2 * (k + 1) if self.nqt == 1 else 0) + 2 * g

    def issue(self, p):
        prev = self.occupant.get(p % self.nslot)
        assert prev is None or (prev in self.landed and self.reads.get(prev) == 0), f"fill {p} over {prev}, still read"
        self.occupant[p % self.nslot] = p
        self.in_flight.append(p)

    def get_piece(self, k):
        return self.piece[k % NP], k // NP

    def give_back(self, k):
        self.used[k % NP].arrive()

    def producer(self, values):
        yield self.get_piece(0)
        self.give_back(0)
        for k, ((n, _), J) in enumerate(zip(self.pieces, self.start)):
            if k + 1 < len(self.pieces):  # the next piece's pages are looked up ahead
                yield self.get_piece(k + 1)
                self.give_back(k + 1)
            if self.nqt == 1:
                for p in (self.kfill(k, J) - 2, self.kfill(k, J) - 1):
                    if not values:
                        if p >= self.stop[0]:
                            return
                        yield self.empty[p % self.nslot], p // self.nslot - 1
                        self.reads[p] = 1
                        self.issue(p)
                        self.issued[0].append(p)
                    self.fills[values] += 1
            for g in range(J, J + n):
                p = self.kfill(k, g) + values
                assert p == self.fills[values]
                if p >= self.stop[values]:
                    return
                yield self.empty[p % self.nslot], p // self.nslot - 1
                self.reads[p] = 2 if self.nqt == 2 and not self.pieces[k][1] else 1
                self.issue(p)
                self.issued[values].append(p)
                self.fills[values] += 2

    # ---- the exit of a producer: may it return?
    def own(self, values, p):
        starts = [self.kfill(k, J) - 2 for k, J in enumerate(self.start)]
        if self.nqt == 1 and (p in starts or p - 1 in starts):
            return not values
        return p & 1 == values

    def tests(self, bar, phase):  # (a test of the parity, no claim about the phase)
        return (bar.done & 1) != (phase & 1)

    def drained(self, values):
        """As the kernel asks it: its fills among the last NSLOT + 2 up to its last one, the newest first.  One
        that was released has landed, and so have all before it; one whose full barrier names its phase has."""
        later, last = False, next((p for p in range(self.fills[values] - 1, -1, -1) if self.own(values, p)), -1)
        for p in range(last, max(last - self.nslot - 2, -1), -1):
            if not self.own(values, p):
                continue
            released = self.tests(self.empty[p % self.nslot], p // self.nslot)
            if not (later or released or self.tests(self.full[p % self.nslot], p // self.nslot)):
                return False
            later = later or released
        return True

    def drained_by_slot(self, values):
        """A fault that the model catches: the last own fill of every slot, whoever has filled it since."""
        newest = {p % self.nslot: p for p in self.issued[values]}
        return all(self.tests(self.full[x], p // self.nslot) for x, p in newest.items())

    def planner(self):
        k, kq, more, loads, y = 0, 0, True, [0, 0], 1
        while more or (self.nqt == 2 and kq < k):
            while more:
                if k >= NP:
                    bar, phase = self.used[k % NP], k // NP - 1
                    if self.nqt == 2 and kq < k:
                        if not bar.passes(phase):
                            break
                    else:
                        yield bar, phase
                more = k < len(self.pieces)
                self.piece[k % NP].arrive()
                k += more
            if self.nqt == 1 or kq >= k:
                continue
            single = self.pieces[kq][1]
            self.give_back(kq)
            y ^= single
            for x in ([y] if single else [0, 1]):
                if loads[x]:
                    yield self.qe[x], loads[x] - 1
                self.in_flight.append(("q", x))
                loads[x] += 1
            kq += 1

    # ---- the tensor pipe
    def mma(self, what, fill, acc=None):
        assert fill in self.landed, f"{what} reads fill {fill} before it lands"
        assert self.occupant[fill % self.nslot] == fill, f"{what} reads fill {fill} after its slot was refilled"
        if acc is not None:
            self.o_writes[acc] += 1
        self.pipe.append(("mma", fill, acc))

    def commit(self, bar):
        self.pipe.append(("commit", bar))

    def pipe_step(self):
        if not self.pipe:
            return False
        op = self.pipe.pop(0)
        if op[0] == "commit":
            op[1].arrive()
        else:
            self.reads[op[1]] -= 1
            assert self.reads[op[1]] >= 0
            if op[2] is not None:
                self.o_writes[op[2]] -= 1
        return True

    def land_step(self):
        if not self.in_flight:
            return False
        p = self.in_flight.pop(self.rng.randrange(len(self.in_flight)))
        if isinstance(p, tuple):
            self.qf[p[1]].arrive()
        else:
            self.landed.add(p)
            self.full[p % self.nslot].arrive()
        return True

    def has_landed(self, p):
        return self.full[p % self.nslot], p // self.nslot

    # ---- the MMA warp
    def mma_warp(self):
        ns, slot_of = self.ns, self.nslot
        nq, y, used, was_single = [0, 0], 1, [0, 0], False
        for k, ((n, single), J) in enumerate(zip(self.pieces, self.start)):
            yield self.get_piece(k)
            self.give_back(k)
            both = was_single or single

            def pv(slot, acc, first, phase, fv, wait_v=True):
                if wait_v:
                    yield self.has_landed(fv)
                yield self.pf[slot], phase
                if first and k >= 1:
                    yield self.of[acc], k - 1
                    if self.nqt == 2 and both and (acc == 0 or self.waits_twice):
                        yield self.of[acc ^ 1], k - 1
                self.mma("P V", fv, acc)

            def scores(slot, fill):
                self.mma("S", fill)
                self.commit(self.sf[slot])

            if self.nqt == 1:
                for h in (1, 2):
                    yield self.has_landed(self.kfill(k, J) - h)
                for p in (self.kfill(k, J) - 2, self.kfill(k, J) - 1):
                    self.mma("query copy", p)
                    self.commit(self.empty[p % slot_of])
                for g in range(J, J + n + 1):
                    if g < J + n:
                        f = self.kfill(k, g)
                        yield self.has_landed(f)
                        scores(g & 1, f)
                        self.commit(self.empty[f % slot_of])
                    if g > J:
                        fv = self.kfill(k, g - 1) + 1
                        yield from pv((g - 1) & 1, 0, g - 1 == J, (g - 1) >> 1, fv)
                        self.commit(self.empty[fv % slot_of])
                self.commit(self.od[0])
            elif not single:
                yield self.qf[0], nq[0]
                yield self.has_landed(2 * J)
                scores(0, 2 * J)
                yield self.qf[1], nq[1]
                scores(1, 2 * J)
                nq = [nq[0] + 1, nq[1] + 1]
                for i in range(n):
                    f = 2 * (J + i)
                    yield self.has_landed(f + 1)
                    if i + 1 < n:
                        yield self.has_landed(f + 2)
                    for x in (0, 1):
                        yield from pv(x, x, i == 0, used[x] + i, f + 1, wait_v=False)
                        if i + 1 < n:
                            scores(x, f + 2)
                        else:
                            self.commit(self.od[x])
                used = [used[0] + n, used[1] + n]
            else:
                y ^= 1
                s_slot = (lambda i: (J + i) % 3) if ns == 3 else (lambda i: i & 1)
                yield self.qf[y], nq[y]
                nq[y] += 1
                for i in range(min(n, ns - 1)):
                    yield self.has_landed(2 * (J + i))
                    scores(s_slot(i), 2 * (J + i))
                for i in range(n):
                    f, x = 2 * (J + i), i & 1
                    if i + ns - 1 < n:
                        fk = f + 2 * (ns - 1)
                        yield self.has_landed(fk)
                        scores(s_slot(i + ns - 1), fk)
                    if ns == 3:
                        phase = (J + i) // 3
                    else:
                        phase = used[x]
                        used[x] += 1
                    yield from pv(s_slot(i), x, i < 2, phase, f + 1)
                    self.commit(self.empty[(f + 1) % slot_of])
                self.commit(self.od[0])
                self.commit(self.od[1])
            was_single = single
        yield self.get_piece(len(self.pieces))

    # ---- a softmax warp (with two query tiles a CTA also its epilogue)
    def zero(self, k, g):
        fv = self.kfill(k, g) + 1
        yield self.has_landed(fv)
        assert fv in self.landed and self.occupant[fv % self.nslot] == fv, f"rows of fill {fv} are zeroed before it lands"

    def rescale(self, k, g, acc):
        if self.ns == 3 or self.nqt == 1:
            f = self.kfill(k, g - self.nqt) + 1
            yield self.empty[f % self.nslot], f // self.nslot
        assert self.o_writes[acc] == 0, f"O is rescaled at tile {g} under a P V"

    def softmax_warp(self, wg, quarter):
        n_s, n_meet, y = 0, 0, 1
        for k, ((n, single), J) in enumerate(zip(self.pieces, self.start)):
            yield self.get_piece(k)
            for i in range(wg if single and self.nqt == 2 else 0, n, 2 if single and self.nqt == 2 else 1):
                g = J + i
                slot = g % 3 if self.ns == 3 else wg if self.nqt == 2 else g & 1
                phase = g // 3 if self.ns == 3 else n_s if self.nqt == 2 else g >> 1
                if g in self.zeroed and (self.nqt == 1 or single or wg == 0):
                    yield from self.zero(k, g)
                yield self.sf[slot], phase
                n_s += 1
                if self.nqt == 2 and not single:
                    if i + 1 == n:
                        self.qe[wg].arrive()
                    if wg == 1 and quarter == 0:
                        self.empty[(2 * g) % self.nslot].arrive()
                        if i > 0:
                            self.empty[(2 * g - 1) % self.nslot].arrive()
                elif self.nqt == 2 and quarter == 0:
                    self.empty[(2 * g) % self.nslot].arrive()
                if i >= (2 if single and self.nqt == 2 else 1) and self.rng.random() < 0.5:
                    yield from self.rescale(k, g, wg)
                self.pf[slot].arrive()
            if self.nqt == 1:
                if k > 0:
                    yield self.of[0], k - 1
                self.meet.arrive()
                self.give_back(k)
                continue
            yield self.od[wg], k
            if single:
                yield self.od[wg ^ 1], k
            if not single and wg == 1 and quarter == 0:
                self.empty[(2 * (J + n) - 1) % self.nslot].arrive()
            if single:
                y ^= 1
                if wg == y:
                    self.qe[y].arrive()
                self.meet.arrive()
                yield self.meet, n_meet
                n_meet += 1
                assert self.o_writes == [0, 0]
            self.of[wg].arrive()
            for _ in range(self.rng.choice((0, 0, 0, 30))):  # (the join of a shared unit takes its time)
                yield self.piece[k % NP], k // NP
            self.give_back(k)
        yield self.get_piece(len(self.pieces))

    def epilogue_warp(self):  # one query tile a CTA: a warpgroup of its own
        for k in range(len(self.pieces)):
            yield self.get_piece(k)
            yield self.meet, k
            yield self.od[0], k
            assert self.o_writes[0] == 0
            self.of[0].arrive()
            self.give_back(k)
        yield self.get_piece(len(self.pieces))

    def run(self, stopping=False, drained="drained"):
        """stopping: the producers give up at random fills; the others run on as far as they can."""
        if stopping:
            total = sum(n for n, _ in self.pieces) * 2 + 2 * len(self.pieces) * (self.nqt == 1)
            at = self.rng.randrange(total)
            self.stop = [at, max(0, at + self.rng.choice((0, 0, 1, -2, 3)))]
        roles = [self.planner(), self.producer(0), self.producer(1), self.mma_warp()]
        roles += [self.softmax_warp(wg, q) for wg in range(self.nqt) for q in range(4)]
        roles += [self.epilogue_warp() for _ in range(4 * (2 - self.nqt))]
        waits = [next(r, None) for r in roles]
        # roles of very different speeds, so that each falls behind the others in some runs
        speed = [self.rng.choice((0.03, 0.3, 1.0)) for _ in range(len(roles) + 2)]
        while any(w is not None for w in waits) or self.pipe or self.in_flight:
            order = sorted(range(len(speed)), key=lambda a: -speed[a] * self.rng.random())
            for a in order:
                if a >= len(roles):
                    if (self.pipe_step if a == len(roles) else self.land_step)():
                        break
                elif waits[a] is not None and waits[a][0].passes(waits[a][1]):
                    waits[a] = next(roles[a], None)
                    break
            else:
                if stopping:
                    break
                stuck = [f"{w[0].name} phase {w[1]}" for w in waits if w]
                raise AssertionError(f"deadlock: {self.pieces}, waiting for {stuck}")
            if stopping and self.rng.random() < 0.2:
                for v in (0, 1):
                    if waits[1 + v] is None and getattr(self, drained)(v):
                        assert not set(self.issued[v]) & set(self.in_flight), "a producer returns before its copies"
        if stopping:
            for v in (0, 1):
                assert getattr(self, drained)(v), f"a drain that runs into its limit: {self.pieces}, stops {self.stop}"


# name: head dim, score slots, query tiles a CTA, kinds of pieces (whether of a single query tile)
FLAVOURS = {
    "d64": (64, 3, 2, (True,)),
    "d128-single": (128, 2, 2, (True,)),
    "d128-pairs": (128, 2, 2, (False,)),
    "d128-mixed": (128, 2, 2, (True, False)),
    "d256": (256, 2, 1, (False,)),
}


def runs(name, nslot, count):
    _, ns, nqt, kinds = FLAVOURS[name]
    for seed in range(count):
        rng = random.Random(f"{name} {seed}")
        pieces = [(rng.choice((1, 1, 2, 3, 5, 6, 8, 12, 17)), rng.choice(kinds)) for _ in range(rng.randint(1, 7))]
        yield Kernel(pieces, nslot, nqt, ns, rng)


@pytest.mark.parametrize("name", FLAVOURS)
def test_every_wait_names_its_phase(name):
    for kernel in runs(name, ring_slots(FLAVOURS[name][0]), 300):
        kernel.run()


@pytest.mark.parametrize("name", FLAVOURS)
def test_producers_that_stop_drain_their_copies(name):
    for kernel in runs(name, ring_slots(FLAVOURS[name][0]), 300):
        kernel.run(stopping=True)


@pytest.mark.parametrize("name", ["d128-single", "d128-pairs", "d256"])
def test_model_catches_a_drain_by_slot(name):
    """In an odd ring keys and values take turns in a slot: the other producer's later fill has overtaken the
    phase of this one's last."""
    caught = 0
    for kernel in runs(name, ring_slots(FLAVOURS[name][0]), 60):
        try:
            kernel.run(stopping=True, drained="drained_by_slot")
        except AssertionError as e:
            assert "runs into its limit" in str(e), e
            caught += 1
    assert caught > 0


def premature(name, nslot, count, what):
    """Runs of `count` in which a wait passes early (or what it guards is not so)."""
    n = 0
    for kernel in runs(name, nslot, count):
        try:
            kernel.run()
        except AssertionError as e:
            assert re.search(what, str(e)), e
            n += 1
    return n


def test_model_catches_a_ring_of_eight_slots():
    """With three score slots and eight ring slots the slot of V(g) held V(g - 4), which S(g - 2) does not
    wait for: the wait before V(g)'s rows are zeroed passes while that copy is in flight."""
    assert premature("d64", 8, 300, r"full\[\d+\]: a wait") > 0


def test_model_catches_a_ring_of_seven_slots():
    """... and with seven the slot of V(g - 2) is released once more, of K(g + 2), which does not wait for
    P(g): the rescaling's wait before that may miss its phase."""
    assert premature("d64", 7, 100, "deadlock") > 0


def test_model_catches_a_second_wait_for_an_accumulator(monkeypatch):
    """A unit of two query tiles and one key tile behind a piece of one query tile: the second product
    must not wait again until the first accumulator is free of the last piece, since by then
    the first warpgroup may be done with this one."""
    monkeypatch.setattr(Kernel, "waits_twice", True)
    assert premature("d128-mixed", ring_slots(128), 1500, r"deadlock.*'o_free\[0\]") > 0
