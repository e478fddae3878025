"""The expanded latent kernel's ring of key and value blocks, as a model run in random orders.

One warp copies the blocks of K_0 V_0 K_1 V_1 ..., another issues the products of two q tiles on
them, and the blocks' places are taken again when both q tiles are done with them.  The model asks
that every product reads the tile that it should and that the walk always ends.
"""
import random

import pytest

from tests.test_latent_phases import Bar

TILES = 4


class Model:
    def __init__(self, n, key_blocks, value_blocks, ring, rng, early=False):
        self.n, self.kb, self.vb, self.ring, self.rng = n, key_blocks, value_blocks, ring, rng
        self.last = 1 if n[1] > 0 else 0
        self.early = early      # hand a value tile on behind the first q tile's product
        self.per = key_blocks + value_blocks
        self.full = [Bar(key_blocks if v == 0 else value_blocks)
                     for _ in range(TILES) for v in range(2)]
        self.empty = [Bar(1) for _ in range(2 * TILES)]
        self.s_full, self.p_full = [Bar(1), Bar(1)], [Bar(1), Bar(1)]
        self.place, self.flying, self.queue = [None] * ring, [], []

    @staticmethod
    def bar(j, v):
        return 2 * (j % TILES) + v

    def there(self, j, v):
        return self.full[self.bar(j, v)].done((j // TILES) & 1)

    def copies(self):
        for c in range(max(self.n) * self.per):
            before, j, e = c - self.ring, c // self.per, c % self.per
            if before >= 0:
                bj, bv = before // self.per, before % self.per >= self.kb
                while not self.empty[self.bar(bj, bv)].done((bj // TILES) & 1):
                    yield
            self.full[self.bar(j, e >= self.kb)].arrive(1)
            self.flying.append((c % self.ring, c, self.bar(j, e >= self.kb)))
            yield

    def land(self):
        while True:
            if self.flying:
                place, c, bar = self.flying.pop(self.rng.randrange(len(self.flying)))
                self.place[place] = c
                self.full[bar].bytes(1)
            yield

    def issue(self):
        nt, out = max(self.n), self.queue
        for j in range(nt + 1):
            i = j - 1
            while i >= 0 and not self.there(i, 1):
                yield
            for qt in range(2):
                if 0 <= i < self.n[qt]:
                    while not self.p_full[qt].done(i & 1):
                        yield
                    out += [("read", i * self.per + self.kb + e) for e in range(self.vb)]
                if i >= 0 and qt == (0 if self.early else self.last):
                    out.append(("commit", self.empty[self.bar(i, 1)]))
                if j < self.n[qt]:
                    while not self.there(j, 0):
                        yield
                    out += [("read", j * self.per + e) for e in range(self.kb)]
                    out.append(("commit", self.s_full[qt]))
                yield

    def tensor(self):
        while True:
            if self.queue:
                x = self.queue.pop(0)
                if x[0] == "commit":
                    x[1].arrive()
                else:
                    assert self.place[x[1] % self.ring] == x[1], "another block's place"
            yield

    def softmax(self, qt):
        for t in range(self.n[qt]):
            while not self.s_full[qt].done(t & 1):
                yield
            if qt == self.last:     # both q tiles' products with the keys are done
                self.empty[self.bar(t, 0)].arrive()
            yield
            self.p_full[qt].arrive()
            yield

    def run(self):
        roles = [self.copies(), self.issue(), self.softmax(0), self.softmax(1)]
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
                    assert not any(x[0] == "read" and self.place[x[1] % self.ring] != x[1]
                                   for x in self.queue)
                    return
        raise AssertionError("the walk does not end")


# blocks of a key tile and of its values, and of the ring: as the kernel's head sizes give them
@pytest.mark.parametrize("key_blocks,value_blocks,ring", [(3, 2, 8), (3, 1, 8), (2, 2, 10), (2, 1, 10)])
def test_every_order_ends_and_reads_what_it_should(key_blocks, value_blocks, ring):
    for seed in range(60):
        rng = random.Random(seed)
        n1 = rng.randint(1, 14)
        n = rng.choice([(n1, 0), (rng.randint(0, n1), n1), (max(0, n1 - 1), n1)])
        Model(n, key_blocks, value_blocks, ring, rng).run()


def test_handing_on_a_block_that_is_still_read_is_noticed():
    with pytest.raises(AssertionError):
        for seed in range(60):
            Model((9, 9), 3, 2, 8, random.Random(seed), early=True).run()
