"""The absorbed latent kernel's hand-overs, as a model run in random orders.

Copies, MMA issue, tensor cores and softmax warps run as in the kernel, each step whenever its
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


class Model:
    def __init__(self, segments, stages, rng, early_expect=False):
        self.seg, self.S, self.rng, self.early = segments, stages, rng, early_expect
        self.q_full, self.q_empty = Bar(1), Bar(1)
        self.k_full = [Bar(1) for _ in range(stages)]
        self.k_empty = [[Bar(1), Bar(1)] for _ in range(stages)]
        self.s_full = [Bar(1), Bar(1)]
        self.p_full, self.pv_done, self.o_empty = Bar(4), Bar(1), Bar(4)
        self.flying, self.queue = [], []
        self.tile = [[None, None] for _ in range(stages)]   # what each half holds
        self.q = self.o = self.p = None
        self.s = [None, None]
        self.read = 0       # tiles whose scores every softmax warp has read

    def copies(self):
        it = 0
        for sg, nt in enumerate(self.seg):
            while sg > 0 and not self.q_empty.done((sg - 1) & 1):
                yield
            self.q_full.arrive(1)
            self.flying.append(("q", sg))
            for _ in range(nt):
                st = it % self.S
                if self.early:
                    self.k_full[st].arrive(2)
                for half in range(2):
                    while it >= self.S and not self.k_empty[st][half].done((it // self.S - 1) & 1):
                        yield
                    if half == 0 and not self.early:
                        self.k_full[st].arrive(2)
                    self.flying.append(("k", st, half, it))
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
                    self.k_full[x[1]].bytes(1)
            yield

    def issue(self):
        qk, pv = [0, 0, 0], [0, 0, 0]       # segment, tile of it, tile
        while pv[0] < len(self.seg):
            if pv[2] < qk[2] and self.p_full.done(pv[2] & 1) and \
                    (pv[1] > 0 or pv[0] == 0 or self.o_empty.done((pv[0] - 1) & 1)):
                st = pv[2] % self.S
                for half in range(2):
                    self.queue.append(("pv", pv[2], st, half, pv[1] == 0 and half == 0, pv[0]))
                    if half == 0:
                        self.queue.append(("commit", self.k_empty[st][0]))
                self.queue += [("commit", self.pv_done), ("commit", self.k_empty[st][1])]
                at = pv
            elif qk[0] < len(self.seg) and qk[2] < pv[2] + 2 and \
                    self.k_full[qk[2] % self.S].done((qk[2] // self.S) & 1) and \
                    (qk[1] > 0 or self.q_full.done(qk[0] & 1)):
                self.queue += [("qk", qk[2], qk[2] % self.S, qk[0]),
                               ("commit", self.s_full[qk[2] & 1])]
                if qk[1] == self.seg[qk[0]] - 1:
                    self.queue.append(("commit", self.q_empty))
                at = qk
            else:
                yield
                continue
            at[1] += 1
            at[2] += 1
            if at[1] == self.seg[at[0]]:
                at[0], at[1] = at[0] + 1, 0
            yield

    def tensor(self):       # in order
        while True:
            if self.queue:
                x = self.queue.pop(0)
                if x[0] == "commit":
                    x[1].arrive()
                elif x[0] == "qk":
                    assert self.tile[x[2]] == [x[1], x[1]] and self.q == x[3]
                    assert self.read >= x[1] - 1, "scores overwritten before they were read"
                    self.s[x[1] & 1] = x[1]
                else:
                    assert self.tile[x[2]][x[3]] == x[1] and self.p == [x[1]] * 4
                    if x[4]:
                        assert self.o is None or self.o == ["out", x[5] - 1, 4]
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
                while it > 0 and not self.pv_done.done((it - 1) & 1):
                    yield
                assert not any(x[0] == "pv" for x in self.queue), "weights still read"
                self.p = self.p or [None] * 4
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
        seen = [0] * 4
        roles = [self.copies(), self.issue()] + [self.softmax(w, seen) for w in range(4)]
        live = roles + [self.land(), self.tensor()]
        weight = [self.rng.choice([1, 1, 3, 20]) for _ in live]
        for _ in range(20000):
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
    for seed in range(150):
        rng = random.Random(seed)
        segments = [rng.randint(1, 7) for _ in range(rng.randint(1, 4))]
        Model(segments, stages, rng).run()


def test_announcing_a_tile_before_its_place_is_free_is_noticed():
    with pytest.raises(AssertionError, match="does not expect"):
        for seed in range(50):
            Model([6], 2, random.Random(seed), early_expect=True).run()
