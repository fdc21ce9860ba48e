"""The barriers of the latent attention kernels (``latent_kernel`` in ``latent_attention.cu``, ``expanded_kernel`` in
``expanded_attention.cu``) as models whose warps run in random order over random item lists (no GPU).

As in ``test_page_chunk_protocol_host``: each warp is a generator with the kernel's loop bounds, slots and parities;
copies land and issued MMAs run later, those of one warp in order.  Checked at every step: a wait that ends has seen the
phase it is for, no one arrives twice in a phase, nothing is overwritten before its last read or read before its last
write, and all warps end."""
import random

import pytest

from test_page_chunk_protocol_host import Barrier


class Model:
    """Barriers, warps, and queues of things that happen later (a queue's in order)."""

    def __init__(self, counts):
        self.b = {name: Barrier(name, n) for name, n in counts.items()}
        self.queues = {}

    def wait(self, name, count):
        """Until phase number `count` of the barrier is over, as the kernels ask: by its parity."""
        bar = self.b[name]
        while not bar.passes(count & 1):
            yield
        assert bar.phase == count + 1, (name, "passed for phase", count, "at", bar.phase)

    def later(self, queue, act):
        self.queues.setdefault(queue, []).append(act)

    def run(self, rnd, warps):
        live, still = list(range(len(warps))), 0
        speed, pipe = [rnd.choice([1, 1, 3, 10]) for _ in warps], rnd.choice([1, 4, 12])
        while live or any(self.queues.values()):
            before = [(b.phase, len(b.here)) for b in self.b.values()], sum(map(len, self.queues.values())), len(live)
            for _ in range(len(warps)):
                busy = [q for q in self.queues.values() if q]
                if busy and rnd.randrange(16) < pipe:
                    rnd.choice(busy).pop(0)()
                if live:
                    i = rnd.choices(live, [speed[x] for x in live])[0]
                    try:
                        next(warps[i])
                    except StopIteration:
                        live.remove(i)
            after = [(b.phase, len(b.here)) for b in self.b.values()], sum(map(len, self.queues.values())), len(live)
            still = 0 if before != after else still + 1
            assert still < 3000, ("no warp goes on", live)


# ---------------------------------------------------------------------------
# Absorbed form
# ---------------------------------------------------------------------------

class Latent(Model):
    """`rows_here`: softmax warps with rows; `units`: slots of the ring; `buffers` of S; `items`: steps of each."""

    def __init__(self, rows_here, units, buffers, items, **counts):
        n = {("full", i): 3 for i in range(4)} | {("full3", i): 1 for i in range(4)}
        n |= {("unit_empty", i): 1 for i in range(units)} | {("rope_empty", i): 1 for i in range(2)}
        n |= {("s_full", i): 1 for i in range(buffers)} | {("s_read", i): rows_here for i in range(buffers)}
        n |= {"q_full": 4, "q_asked": 4, "p_full": 4, "o_free": 4, "pv_done": 1, "group": 4}
        n |= {k: v for k, v in counts.items() if k in n}
        super().__init__(n)
        self.rows_here, self.units, self.buffers, self.items = rows_here, units, buffers, items
        self.unit = [None] * units          # slot -> (step, unit) that it holds
        self.rope = [{}, {}]                # half -> {load warp: step}
        self.q, self.s, self.p = {}, [None] * buffers, {}
        self.s_done, self.pv_units, self.pv_steps = 0, 0, 0   # steps' S, units' and steps' PV executed
        self.s_units = self.rope_reads = 0  # units and position keys read by S
        self.s_got = {}                     # step -> warps that have read S
        self.o_item, self.o_got = None, {}  # item in O, item -> warps that have read it
        self.q_of = -1
        self.n_bar = [0] * 4

    def sync(self, w):
        """The softmax warps' vote: all meet."""
        mine = self.n_bar[w]
        self.n_bar[w] += 1
        self.b["group"].arrive((w, mine))
        while self.b["group"].phase <= mine:
            yield

    def load(self, w):
        slot, rnd, g = w, 0, 0
        yield from self.wait("q_asked", 0)
        for steps in self.items:
            for _ in range(steps):
                if rnd > 0:
                    yield from self.wait(("unit_empty", slot), rnd - 1)
                if w < 2 and g >= 2:
                    yield from self.wait(("rope_empty", g & 1), (g >> 1) - 1)
                old = self.unit[slot]
                if old is not None:
                    u = 4 * old[0] + old[1]
                    assert self.pv_units > u and self.s_units > u, ("unit overwritten", old)
                self.unit[slot] = None
                if w < 2:
                    assert g < 2 or self.rope_reads > g - 2, "position keys overwritten"
                    self.rope[g & 1][w] = None

                def land(slot=slot, g=g):
                    self.unit[slot] = (g, w)
                    if w < 2:
                        self.rope[g & 1][w] = g
                    self.b["full" if w < 3 else "full3", g & 3].arrive((w, g))

                self.later(("copies", w), land)
                slot += 4
                if slot >= self.units:
                    slot, rnd = slot - self.units, rnd + 1
                g += 1
                yield

    def scores(self):
        g, slot, n_item = 0, 0, 0
        for steps in self.items:
            yield from self.wait("q_full", n_item)
            for _ in range(steps):
                yield from self.wait(("full", g & 3), g >> 2)
                if g >= self.buffers:
                    yield from self.wait(("s_read", g % self.buffers), g // self.buffers - 1)

                def rope(g=g, n_item=n_item):
                    assert self.rope[g & 1] == {0: g, 1: g}, ("position keys", g, self.rope)
                    assert self.q == {w: n_item for w in range(self.rows_here)}, ("Q", n_item, self.q)
                    old = self.s[g % self.buffers]
                    assert old is None or self.s_got.get(old, 0) == self.rows_here, ("S overwritten", old)
                    self.s[g % self.buffers] = None
                    self.rope_reads += 1

                self.later("s", rope)
                self.later("s", lambda g=g: self.b["rope_empty", g & 1].arrive("commit"))
                yield
                for b in range(4):
                    if b == 3:
                        yield from self.wait(("full3", g & 3), g >> 2)

                    def unit(slot=slot, g=g, b=b):
                        assert self.unit[slot] == (g, b), ("S reads", (g, b), self.unit[slot])
                        self.s_units += 1

                    self.later("s", unit)
                    slot = (slot + 1) % self.units
                    yield

                def done(g=g):
                    self.s[g % self.buffers] = g
                    self.s_done += 1
                    self.b["s_full", g % self.buffers].arrive("commit")

                self.later("s", done)
                g += 1
            n_item += 1

    def outputs(self):
        g, slot, n_item = 0, 0, 0
        for steps in self.items:
            for s in range(steps):
                yield from self.wait("p_full", g)
                if s == 0 and n_item > 0:
                    yield from self.wait("o_free", n_item - 1)
                for b in range(4):
                    def unit(slot=slot, g=g, b=b, n_item=n_item, s=s):
                        assert self.unit[slot] == (g, b), ("PV reads", (g, b), self.unit[slot])
                        assert self.p == {w: g for w in range(self.rows_here)}, ("P", g, self.p)
                        if s == 0 and b == 0:
                            assert self.o_item is None or self.o_got.get(self.o_item, 0) == 4, "O overwritten"
                            self.o_item = n_item
                        assert self.o_item == n_item
                        self.pv_units += 1

                    self.later("pv", unit)
                    self.later("pv", lambda slot=slot: self.b["unit_empty", slot].arrive("commit"))
                    if b == 3:
                        def done():
                            self.pv_steps += 1
                            self.b["pv_done"].arrive("commit")
                        self.later("pv", done)
                    slot = (slot + 1) % self.units
                    yield
                g += 1
            n_item += 1

    def softmax(self, w, moved):
        here, g = w < self.rows_here, 0

        def write_q(item, first):
            if item < len(self.items):
                if here:
                    if first:
                        self.b["q_asked"].arrive(w)
                    assert item == 0 or self.s_done >= sum(self.items[:item]), "Q still to be read"
                    self.q[w] = item
                elif first:
                    self.b["q_asked"].arrive(w)
                self.b["q_full"].arrive(w)

        write_q(0, True)
        yield
        for item, steps in enumerate(self.items):
            for s in range(steps):
                if here:
                    yield from self.wait(("s_full", g % self.buffers), g // self.buffers)
                    assert self.s[g % self.buffers] == g
                    self.s_got[g] = self.s_got.get(g, 0) + 1
                    self.b["s_read", g % self.buffers].arrive(w)
                yield
                yield from self.sync(w)
                if moved(g) and s > 0:
                    yield from self.sync(w)
                    yield from self.wait("pv_done", g - 1)
                    assert self.pv_steps == g, "O rescaled beside a PV"
                elif g > 0:
                    yield from self.wait("pv_done", g - 1)
                assert self.pv_steps == g, "P overwritten"
                if here:
                    self.p[w] = g
                yield
                yield from self.sync(w)
                self.b["p_full"].arrive(w)
                g += 1
            write_q(item + 1, False)
            yield from self.wait("pv_done", g - 1)
            yield from self.sync(w)
            assert self.o_item == item and self.pv_steps == g
            yield
            self.o_got[item] = self.o_got.get(item, 0) + 1
            self.b["o_free"].arrive(w)
            yield from self.sync(w)

    def go(self, rnd):
        share, salt = rnd.choice([0, 2, 8]), rnd.random()
        moved = lambda g: random.Random((salt, g).__hash__()).randrange(8) < share
        self.run(rnd, [self.load(w) for w in range(4)] + [self.scores(), self.outputs()] +
                 [self.softmax(w, moved) for w in range(4)])


FORMS = [(1, 12, 2), (2, 12, 2), (4, 11, 1)]  # tiles of 16, 32 and 64 rows


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("seed", range(5))
def test_absorbed_item_lists(form, seed):
    rnd = random.Random(seed)
    for _ in range(12):
        Latent(*form, [rnd.choice([1, 1, 2, 3, 4, 7, 15]) for _ in range(rnd.randint(1, 6))]).go(rnd)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("wrong", [{"q_full": 3}, {"p_full": 3}, {"o_free": 3}])
def test_the_absorbed_model_sees_wrong_counts(form, wrong):
    rnd = random.Random(7)
    with pytest.raises(AssertionError):
        for _ in range(20):
            Latent(*form, [rnd.choice([1, 2, 3, 7]) for _ in range(4)], **wrong).go(rnd)


def test_the_absorbed_model_sees_a_ring_that_is_too_long_for_its_barriers():
    """A ring of six steps: keys may land for step g + 4 before anyone has waited for those of step g."""
    rnd = random.Random(8)
    with pytest.raises(AssertionError):
        for _ in range(40):
            Latent(4, 24, 1, [15, 15]).go(rnd)


# ---------------------------------------------------------------------------
# Expanded form
# ---------------------------------------------------------------------------

SLOTS = 8


def k_slots(t):
    return [(5 * t + s) % SLOTS for s in range(3)]


def v_slots(t):
    return [(5 * t + 3 + s) % SLOTS for s in range(2)]


class Expanded(Model):
    """An item is (KV tiles of group 0, of group 1, whether its last KV tile is a row's last and ragged)."""

    def __init__(self, items, **counts):
        n = {}
        for i in (0, 1):
            n |= {("k_full", i): 1, ("v_full", i): 1, ("k_empty", i): 2, ("v_empty", i): 2, ("s_full", i): 1,
                  ("p_full", i): 4, ("o_full", i): 1, ("o_free", i): 4}
        n |= {"tail": 1, "q_full": 1, "q_empty": 2}
        for k, v in counts.items():
            for name in n:
                if name == k or name[0] == k:
                    n[name] = v
        super().__init__(n)
        self.items = items
        self.slot = [None] * SLOTS                 # slot -> (kind, KV tile) whole, None on its way
        self.owner = [None] * SLOTS                # slot -> (kind, KV tile) asked for
        self.reads = {}                            # (kind, KV tile) -> groups done with it
        self.q_item, self.q_reads = None, {}       # item in Q, item -> groups done with it
        self.s, self.p = [None, None], [{}, {}]    # group -> KV tile in S; {warp: KV tile} of P
        self.pv = [0, 0]                           # PVs executed of each group
        self.o, self.o_got = [None, None], {}

    def ask(self, kind, t, slots):
        for s in slots:
            old = self.owner[s]
            assert old is None or self.reads.get(old, 0) == 2, ("overwritten", old, "by", (kind, t))
            self.owner[s], self.slot[s] = (kind, t), None

    def land(self, kind, t, slots, barrier):
        def act():
            for s in slots:
                self.slot[s] = (kind, t)
            self.b[barrier].arrive(("tma", kind, t))
        self.later(("copies", kind), act)

    def tma(self):
        t = n_item = 0
        last_tail = -2
        for a, b, tail in self.items:
            n = max(a, b)
            if n == 0:
                continue
            if n_item > 0:
                yield from self.wait("q_empty", n_item - 1)
                assert self.q_reads.get(n_item - 1, 0) == 2, "Q overwritten"

            def q(item=n_item):
                self.q_item = item
                self.b["q_full"].arrive(("q", item))

            self.q_item = None
            self.later("copies q", q)
            n_item += 1
            for j in range(n):
                if t >= 2:
                    yield from self.wait(("v_empty", t & 1), (t >> 1) - 1)
                self.ask("k", t, k_slots(t))
                self.land("k", t, k_slots(t), ("k_full", t & 1))
                yield
                is_tail = tail and j == n - 1
                if t >= 1:
                    yield from self.wait(("k_empty", (t - 1) & 1), (t - 1) >> 1)
                if is_tail and last_tail == t - 1 and t > 0:
                    yield from self.wait(("v_full", (t - 1) & 1), (t - 1) >> 1)
                self.ask("v", t, v_slots(t))
                if is_tail:
                    last_tail = t
                    self.land("raw", t, v_slots(t), "tail")
                else:
                    self.land("v", t, v_slots(t), ("v_full", t & 1))
                yield
                t += 1

    def zero(self):
        t = n_tail = 0
        for a, b, tail in self.items:
            n = max(a, b)
            t += n
            if n and tail:
                yield from self.wait("tail", n_tail)
                n_tail += 1
                yield
                for s in v_slots(t - 1):
                    assert self.slot[s] == ("raw", t - 1), ("zeroing", t - 1, self.slot[s])
                    self.slot[s] = ("v", t - 1)
                self.b["v_full", (t - 1) & 1].arrive("zero")

    def read(self, kind, t, slots):
        for s in slots:
            assert self.slot[s] == (kind, t), ("read", (kind, t), self.slot[s])

    def through(self, kind, t):
        self.reads[kind, t] = self.reads.get((kind, t), 0) + 1

    def mma(self, g):
        t = n_item = n_p = n_out = 0
        commit = lambda name: self.later(("mma", g), lambda: self.b[name].arrive(("commit", g)))
        for item in self.items:
            mine, n = item[g], max(item[:2])
            if n == 0:
                continue
            yield from self.wait("q_full", n_item)
            for j in range(n + 1):
                tv, tk = t + j - 1, t + j
                if j > 0:
                    yield from self.wait(("v_full", tv & 1), tv >> 1)
                    if j <= mine:
                        yield from self.wait(("p_full", g), n_p)
                        n_p += 1
                        if j == 1 and n_out > 0:
                            yield from self.wait(("o_free", g), n_out - 1)

                        def pv(tv=tv, first=j == 1, out=n_out):
                            self.read("v", tv, v_slots(tv))
                            assert self.p[g] == {w: tv for w in range(4)}, ("P", tv, self.p[g])
                            if first:
                                assert self.o[g] is None or self.o_got.get((g, self.o[g]), 0) == 4, "O overwritten"
                                self.o[g] = out
                            self.pv[g] += 1
                            self.through("v", tv)

                        self.later(("mma", g), pv)
                        commit(("v_empty", tv & 1))
                        if j == mine:
                            commit(("o_full", g))
                            n_out += 1
                    else:
                        self.through("v", tv)
                        self.b["v_empty", tv & 1].arrive(("skip", g))
                    yield
                if j < n:
                    yield from self.wait(("k_full", tk & 1), tk >> 1)
                    if j < mine:
                        def qk(tk=tk, n_item=n_item):
                            self.read("k", tk, k_slots(tk))
                            assert self.q_item == n_item, ("Q", n_item, self.q_item)
                            self.s[g] = tk
                            self.through("k", tk)

                        self.later(("mma", g), qk)
                        commit(("s_full", g))
                        commit(("k_empty", tk & 1))
                    else:
                        self.through("k", tk)
                        self.b["k_empty", tk & 1].arrive(("skip", g))
                    if j == n - 1:
                        def done(n_item=n_item):
                            self.q_reads[n_item] = self.q_reads.get(n_item, 0) + 1
                        self.later(("mma", g), done)
                        commit("q_empty")
                    yield
            t += n
            n_item += 1

    def softmax(self, g, w):
        t = n_s = n_o = 0
        for item in self.items:
            mine, n = item[g], max(item[:2])
            for j in range(mine):
                yield from self.wait(("s_full", g), n_s)
                assert self.s[g] == t + j, ("S", t + j, self.s[g])
                assert self.pv[g] == n_s, "O not complete behind S"  # (what a moved reference rescales)
                n_s += 1
                yield
                self.p[g][w] = t + j
                self.b["p_full", g].arrive(w)
                yield
            if mine:
                yield from self.wait(("o_full", g), n_o)
                assert self.o[g] == n_o and self.pv[g] == n_s
                yield
                self.o_got[g, n_o] = self.o_got.get((g, n_o), 0) + 1
                self.b["o_free", g].arrive(w)
                n_o += 1
            t += n

    def go(self, rnd):
        self.run(rnd, [self.tma(), self.zero(), self.mma(0), self.mma(1)] +
                 [self.softmax(g, w) for g in (0, 1) for w in range(4)])


def _item(rnd):
    a, b = rnd.choice([(1, 0), (1, 1), (1, 2), (0, 1), (2, 3), (4, 4), (5, 0), (6, 7), (9, 9), (0, 3), (0, 0), (3, 3)])
    return a, b, rnd.random() < 0.5


@pytest.mark.parametrize("seed", range(8))
def test_expanded_item_lists(seed):
    rnd = random.Random(seed)
    for _ in range(25):
        Expanded([_item(rnd) for _ in range(rnd.randint(1, 8))]).go(rnd)


def test_expanded_tails_next_to_one_another():
    rnd = random.Random(50)
    kinds = [(1, 0), (1, 1), (0, 1), (2, 2), (1, 2), (3, 3)]
    for x in kinds:
        for y in kinds:
            for tails in ((1, 1, 1, 1), (1, 0, 1, 1), (0, 1, 1, 0)):
                Expanded([(*k, bool(t)) for k, t in zip((x, y, x, y), tails)]).go(rnd)


@pytest.mark.parametrize("wrong", [{"k_empty": 1}, {"v_empty": 1}, {"p_full": 3}, {"q_empty": 1}, {"o_free": 3}, {"o_free": 5}])
def test_the_expanded_model_sees_wrong_counts(wrong):
    rnd = random.Random(9)
    with pytest.raises(AssertionError):
        for _ in range(40):
            Expanded([_item(rnd) for _ in range(5)], **wrong).go(rnd)
