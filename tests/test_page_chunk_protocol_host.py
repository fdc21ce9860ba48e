"""The barriers of a page-scaled chunk CTA (``page_chunk_cta`` in ``page_attention.cuh``) as a model
that runs its warps in random order over random tile lists (no GPU).

Each warp is a generator with the kernel's own loop bounds, buffer indexes and parities; the tensor
pipe takes the issued MMAs and commits in order, later.  Checked at every step: a wait that ends has
seen the phase it is for (a parity alone cannot tell phases two apart), no warp arrives twice in a phase,
no buffer is overwritten before its last read or read before its last write, and all warps end.

A tile is (two, n_kv, cut): whether both groups have rows of their own, its KV tiles, and whether it
is a piece of a cut tile."""
import random

import pytest


class Barrier:
    def __init__(self, name, n):
        self.name, self.n, self.phase, self.here = name, n, 0, set()

    def arrive(self, who):
        assert who not in self.here, (self.name, who, "arrives twice in a phase")
        self.here.add(who)
        if len(self.here) == self.n:
            self.here, self.phase = set(), self.phase + 1

    def passes(self, parity):
        return (self.phase & 1) != parity


class Cta:
    def __init__(self, tiles, **arrivals):
        n = dict(q_ready=4, p_ready=4, ml_ready=4, joined=4, k_ready=4, v_ready=3, qk_done=1, o_done=1, k_free=1, v_free=1)
        n.update(arrivals)
        self.tiles = tiles
        self.b = {}
        for name in n:
            for i in (0, 1):
                self.b[name, i] = Barrier((name, i), n[name])
        self.queue = []  # issued MMAs and commits
        self.k, self.v = [{}, {}], [{}, {}]  # buffer -> the KV tile that each warp's part holds
        self.terms = [{} for _ in range(4)]
        self.term_reads = {}  # KV tile -> softmax warps that have read its terms
        self.reads = {}  # (kind, KV tile) -> MMAs that have read it
        self.s = [None, None]  # group -> KV tile whose scores are in S
        self.p = [{}, {}]  # group -> {warp: KV tile whose P' it has written}
        self.q = [{}, {}]  # group -> {warp: tile whose queries it has written}
        self.o = [None, None]  # group -> tile whose sums are in O
        self.pv = [0, 0]  # PVs executed
        self.o_reads = {}  # (tile, group) -> warps that have read the group's O
        self.ml, self.ml_read = {}, {}
        self.first = []  # KV tiles before each tile
        at = 0
        for _, n_kv, _ in tiles:
            self.first.append(at)
            at += n_kv

    def wait(self, name, i, count):
        """Until phase number `count` of the barrier is over, as the kernel asks: by its parity."""
        bar = self.b[name, i]
        while not bar.passes(count & 1):
            yield
        assert bar.phase == count + 1, (bar.name, "passed for phase", count, "at", bar.phase)

    def takes_part(self, g, t):
        two, n_kv, _ = self.tiles[t]
        return g == 0 or two or n_kv > 1

    def groups_of(self, jt, t):
        """Groups that read KV tile jt (counted within tile t)."""
        return (0, 1) if self.tiles[t][0] else (jt & 1,)

    def used_up(self, kind, jg):
        t = max(i for i, f in enumerate(self.first) if f <= jg)
        return self.reads.get((kind, jg), 0) == len(self.groups_of(jg - self.first[t], t))

    def convert(self, is_v, w):
        jg, freed, ready, buf = 0, *(("v_free", "v_ready", self.v) if is_v else ("k_free", "k_ready", self.k))
        kind = "v" if is_v else "k"
        for _, n_kv, _ in self.tiles:
            for _ in range(n_kv):
                if jg > 1:
                    yield from self.wait(freed, jg & 1, (jg - 2) >> 1)
                old = buf[jg & 1].get(w)
                assert old is None or self.used_up(kind, old), (kind, "overwritten", old)
                buf[jg & 1][w] = jg
                if not is_v:
                    old = self.terms[jg & 3].get(w)
                    if old is not None:
                        t = max(i for i, f in enumerate(self.first) if f <= old)
                        assert self.term_reads.get(old, 0) == 4 * len(self.groups_of(old - self.first[t], t)), ("terms", old)
                    self.terms[jg & 3][w] = jg
                yield
                self.b[ready, jg & 1].arrive((kind, w))
                jg += 1
                yield

    def issue(self):
        seen = {"k": 0, "v": 0, ("p", 0): 0, ("p", 1): 0, ("q", 0): 0, ("q", 1): 0}

        def wait_for(what):
            # all of a step's barriers are polled together
            names = {"k": "k_ready", "v": "v_ready"}
            while True:
                done = True
                for x in what:
                    if x in names:
                        ok = self.b[names[x], seen[x] & 1].passes((seen[x] >> 1) & 1)
                    else:
                        ok = self.b[x[0] + "_ready", x[1]].passes(seen[x] & 1)
                    done = done and ok
                if done:
                    break
                yield
            for x in what:
                if x in names:
                    assert self.b[names[x], seen[x] & 1].phase == (seen[x] >> 1) + 1, (x, seen[x])
                else:
                    assert self.b[x[0] + "_ready", x[1]].phase == seen[x] + 1, (x, seen[x])
                seen[x] += 1

        jg0 = 0
        for t, (two, n_kv, _) in enumerate(self.tiles):
            dj, j, q = (1 if two else 2), 0, 0
            for _ in range(2 * (n_kv + 1) if two else n_kv + 2):
                has_k, has_v = j < n_kv, j >= dj and j - dj < n_kv
                last_q, first_q = not two or q == 1, not two or q == 0
                jg, jv = jg0 + j, jg0 + j - dj
                what = []
                if has_v:
                    what.append(("p", q))
                if has_k and j < dj:
                    what.append(("q", q))
                if first_q:
                    what += ["k"] * has_k + ["v"] * has_v
                yield from wait_for(what)
                if has_v:
                    self.queue.append(("pv", q, jv, t, j - dj < dj))
                if has_k:
                    self.queue.append(("qk", q, jg, t))
                yield
                if has_k:
                    self.queue.append(("commit", "qk_done", q))
                elif has_v:
                    self.queue.append(("commit", "o_done", q))
                if last_q:
                    if has_v:
                        self.queue.append(("commit", "v_free", jv & 1))
                    if has_k:
                        self.queue.append(("commit", "k_free", jg & 1))
                j += last_q
                q ^= 1
            jg0 += n_kv

    def tensor(self):
        """One step of the pipe, if something is issued."""
        if not self.queue:
            return False
        op, *a = self.queue.pop(0)
        if op == "commit":
            self.b[a[0], a[1]].arrive("commit")
        elif op == "qk":
            q, jg, t = a
            assert self.k[jg & 1] == {w: jg for w in range(4)}, ("K", jg, self.k[jg & 1])
            assert self.q[q] == {w: t for w in range(4)}, ("Q", t, self.q[q])
            self.s[q] = jg
            self.reads["k", jg] = self.reads.get(("k", jg), 0) + 1
        else:
            q, jv, t, first = a
            assert self.v[jv & 1] == {w: jv for w in range(3)}, ("V", jv, self.v[jv & 1])
            assert self.p[q] == {w: jv for w in range(4)}, ("P", jv, self.p[q])
            if first:
                assert self.o[q] is None or self.o_reads.get((self.o[q], q), 0) == 4, ("O overwritten", self.o[q])
                self.o[q] = t
            assert self.o[q] == t
            self.pv[q] += 1
            self.reads["v", jv] = self.reads.get(("v", jv), 0) + 1
        return True

    def softmax(self, g, w):
        mine = [t for t in range(len(self.tiles)) if self.takes_part(g, t)]
        n_qk = n_tile = n_join = n_pv = 0

        def write_q(t):
            assert self.s[g] is None or not any(op[0] == "qk" and op[1] == g for op in self.queue), "Q still to be read"
            self.q[g][w] = t
            self.b["q_ready", g].arrive(w)

        if mine:
            write_q(mine[0])
        for a, t in enumerate(mine):
            two, n_kv, cut = self.tiles[t]
            for j in range(0 if two else g, n_kv, 1 if two else 2):
                yield from self.wait("qk_done", g, n_qk)
                n_qk += 1
                jg = self.first[t] + j
                assert self.s[g] == jg and self.pv[g] == n_pv, "S or O not complete"
                yield
                assert self.terms[jg & 3] == {x: jg for x in range(4)}, ("terms", jg)
                self.term_reads[jg] = self.term_reads.get(jg, 0) + 1
                self.p[g][w] = jg
                n_pv += 1
                yield
                self.b["p_ready", g].arrive(w)
            if a + 1 < len(mine):
                write_q(mine[a + 1])
            yield from self.wait("o_done", g, n_tile)
            n_tile += 1
            assert self.o[g] == t and self.pv[g] == n_pv
            if not two and n_kv > 1:
                if g == 1:
                    assert self.ml.get(w) is None or self.ml_read.get(w) == self.ml[w], "(m, l) overwritten"
                    self.ml[w] = t
                    self.b["ml_ready", 0].arrive(w)
                    yield from self.wait("joined", 0, n_join)
                    n_join += 1
                else:
                    yield from self.wait("ml_ready", 0, n_join)
                    yield
                    assert self.ml.get(w) == t
                    self.ml_read[w] = t
                    for both in (0, 1):
                        self.o_reads[t, both] = self.o_reads.get((t, both), 0) + 1
                    self.b["joined", 0].arrive(w)
                    if cut:
                        yield from self.wait("joined", 0, n_join)
                    n_join += 1
            else:
                yield
                self.o_reads[t, g] = self.o_reads.get((t, g), 0) + 1

    def run(self, rnd):
        warps = [self.convert(False, w) for w in range(4)] + [self.convert(True, w) for w in range(3)] + [self.issue()]
        warps += [self.softmax(g, w) for g in (0, 1) for w in range(4)]
        live, speed, still = list(range(len(warps))), [rnd.choice([1, 1, 3, 10]) for _ in warps], 0
        pipe = rnd.choice([1, 4, 12])
        while live or self.queue:
            before = [(b.phase, len(b.here)) for b in self.b.values()], len(self.queue), len(live)
            for _ in range(len(warps)):
                if rnd.randrange(16) < pipe:
                    self.tensor()
                if live:
                    i = rnd.choices(live, [speed[x] for x in live])[0]
                    try:
                        next(warps[i])
                    except StopIteration:
                        live.remove(i)
            after = [(b.phase, len(b.here)) for b in self.b.values()], len(self.queue), len(live)
            still = 0 if before != after else still + 1
            assert still < 2000, ("no warp goes on", live, self.tiles)


def _tiles(rnd):
    tiles = []
    for _ in range(rnd.randint(1, 7)):
        cut = rnd.random() < 0.3
        tiles.append((rnd.random() < 0.5, rnd.randint(2, 6) if cut else rnd.choice([1, 1, 2, 3, 4, 5, 7, 9]), cut))
    return tiles


@pytest.mark.parametrize("seed", range(8))
def test_random_tile_lists(seed):
    rnd = random.Random(seed)
    for _ in range(25):
        Cta(_tiles(rnd)).run(rnd)


def test_short_tiles_in_every_order():
    rnd = random.Random(99)
    kinds = [(two, n, False) for two in (False, True) for n in (1, 2, 3)]
    for a in kinds:
        for b in kinds:
            Cta([a, b, a, a]).run(rnd)


@pytest.mark.parametrize("wrong", [dict(k_ready=3), dict(v_ready=2), dict(p_ready=3), dict(q_ready=5), dict(ml_ready=3)])
def test_the_model_sees_wrong_counts(wrong):
    """A barrier initialised with another count is found, as a missed buffer, a wrong phase or no progress."""
    rnd = random.Random(5)
    with pytest.raises(AssertionError):
        for _ in range(20):
            Cta(_tiles(rnd), **wrong).run(rnd)
