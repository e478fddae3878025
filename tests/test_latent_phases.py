"""The absorbed latent kernel's hand-overs, as a model run in random orders.

Copies, the two warps that issue MMAs, tensor cores and softmax warps run as in the kernel, each step whenever its
waits allow.  The model asks that no barrier gets an arrival or bytes that its phase does not
expect, that every product reads the tile, scores and weights that it should, that nothing is
overwritten before it is read, and that the walk always ends.
"""
import random

import pytest


class Bar:
    """An mbarrier: `count` arrivals and the bytes they announce end a phase."""

    def __init__(self, count):
        self.count, self.pending, self.tx, self.phase = count, count, 0, 0

    def _over(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def arrive(self, tx=0):
        assert self.pending > 0, "an arrival that the phase does not expect"
        self.pending -= 1
        self.tx += tx
        self._over()

    def bytes(self, n):
        self.tx -= n
        assert self.tx >= 0 or self.pending > 0, "bytes that the phase does not expect"
        self._over()

    def done(self, parity):     # what a wait by parity sees
        return (self.phase & 1) != parity


PARTS = 3       # of a key tile: one that only Q K^T reads, and two that P.V reads again


class Model:
    def __init__(self, segments, stages, rng, early_expect=False):
        self.seg, self.S, self.rng, self.early = segments, stages, rng, early_expect
        self.q_full, self.q_empty = Bar(1), Bar(1)
        self.k_full = [[Bar(1) for _ in range(PARTS)] for _ in range(stages)]
        self.k_empty = [[Bar(1) for _ in range(PARTS)] for _ in range(stages)]
        self.s_full, self.s_empty = [Bar(1), Bar(1)], [Bar(8), Bar(8)]
        self.p_full, self.pv_done, self.o_empty = Bar(8), Bar(1), Bar(8)
        self.flying, self.queues = [], [[], []]
        self.tile = [[None] * PARTS for _ in range(stages)]     # what each part holds
        self.q = self.o = self.p = None
        self.s = [None, None]
        self.read = 0       # tiles whose scores every softmax warp has read

    def copies(self, g):    # a warp a part; the first copies Q too
        it = 0
        for sg, nt in enumerate(self.seg):
            if g == 0:
                while sg > 0 and not self.q_empty.done((sg - 1) & 1):
                    yield
                self.q_full.arrive(1)
                self.flying.append(("q", sg))
            for _ in range(nt):
                st = it % self.S
                if self.early:
                    self.k_full[st][g].arrive(1)
                while it >= self.S and not self.k_empty[st][g].done((it // self.S - 1) & 1):
                    yield
                if not self.early:
                    self.k_full[st][g].arrive(1)
                self.flying.append(("k", st, g, it))
                yield
                it += 1

    def land(self):         # one copy in flight, in any order
        while True:
            if self.flying:
                x = self.flying.pop(self.rng.randrange(len(self.flying)))
                if x[0] == "q":
                    self.q = x[1]
                    self.q_full.bytes(1)
                else:
                    self.tile[x[1]][x[2]] = x[3]
                    self.k_full[x[1]][x[2]].bytes(1)
            yield

    def scores(self):       # the warp that issues Q K^T
        it = 0
        for sg, nt in enumerate(self.seg):
            while not self.q_full.done(sg & 1):
                yield
            for n in range(nt):
                st = it % self.S
                while it >= 2 and not self.s_empty[it & 1].done((it // 2 - 1) & 1):
                    yield
                for g in range(PARTS):
                    while not self.k_full[st][g].done((it // self.S) & 1):
                        yield
                    self.queues[0].append(("qk", it, st, g, sg))
                    if g == 0:
                        self.queues[0].append(("commit", self.k_empty[st][0]))
                    yield
                self.queues[0].append(("commit", self.s_full[it & 1]))
                if n == nt - 1:
                    self.queues[0].append(("commit", self.q_empty))
                it += 1

    def values(self):       # the warp that issues P.V
        it = 0
        for sg, nt in enumerate(self.seg):
            for n in range(nt):
                while not self.p_full.done(it & 1):
                    yield
                while n == 0 and sg > 0 and not self.o_empty.done((sg - 1) & 1):
                    yield
                for g in range(1, PARTS):
                    self.queues[1] += [("pv", it, it % self.S, g, n == 0 and g == 1, sg),
                                       ("commit", self.k_empty[it % self.S][g])]
                self.queues[1].append(("commit", self.pv_done))
                it += 1
                yield

    def tensor(self):       # what a warp issued runs in its order
        while True:
            queue = self.rng.choice(self.queues)
            if queue:
                x = queue.pop(0)
                if x[0] == "commit":
                    x[1].arrive()
                elif x[0] == "qk":
                    assert self.tile[x[2]][x[3]] == x[1] and self.q == x[4]
                    assert self.read >= x[1] - 1, "scores overwritten before they were read"
                    self.s[x[1] & 1] = x[1]
                else:
                    assert self.tile[x[2]][x[3]] == x[1] and self.p == [x[1]] * 8
                    if x[4]:
                        assert self.o is None or self.o == ["out", x[5] - 1, 8]
                        self.o = ["sum", x[5], 0]
                    assert self.o[:2] == ["sum", x[5]]
            yield

    def softmax(self, warp, seen):
        it = 0
        for sg, nt in enumerate(self.seg):
            for _ in range(nt):
                while not self.s_full[it & 1].done((it >> 1) & 1):
                    yield
                assert self.s[it & 1] == it
                seen[warp] = it + 1
                self.read = min(seen)
                self.s_empty[it & 1].arrive()
                yield
                while it > 0 and not self.pv_done.done((it - 1) & 1):
                    yield
                assert not any(x[0] == "pv" for x in self.queues[1]), "weights still read"
                self.p = self.p or [None] * 8
                self.p[warp] = it
                self.p_full.arrive()
                it += 1
                yield
            while not self.pv_done.done((it - 1) & 1):
                yield
            assert self.o[1] == sg
            self.o = ["out", sg, self.o[2] + 1 if self.o[0] == "out" else 1]
            self.o_empty.arrive()
            yield

    def run(self):
        seen = [0] * 8
        roles = [self.copies(g) for g in range(PARTS)] + \
            [self.scores(), self.values()] + [self.softmax(w, seen) for w in range(8)]
        live = roles + [self.land(), self.tensor()]
        weight = [self.rng.choice([1, 1, 3, 20]) for _ in live]
        for _ in range(200000):
            g = self.rng.choices(live, weight)[0]
            try:
                next(g)
            except StopIteration:
                i = live.index(g)
                del live[i], weight[i]
                if not any(r in live for r in roles):
                    return
        raise AssertionError("the walk does not end")


@pytest.mark.parametrize("stages", [2, 4])
def test_every_order_ends_and_reads_what_it_should(stages):
    for seed in range(100):
        rng = random.Random(seed)
        segments = [rng.randint(1, 7) for _ in range(rng.randint(1, 4))]
        Model(segments, stages, rng).run()


def test_announcing_a_tile_before_its_place_is_free_is_noticed():
    with pytest.raises(AssertionError, match="does not expect"):
        for seed in range(50):
            Model([6], 2, random.Random(seed), early_expect=True).run()
