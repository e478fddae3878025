"""The absorbed latent kernel's softmax warps in full, as a model run in random orders: the barriers
by which they tell each other that a row's maximum moves (one a tile, and one that only such tiles
have), the buffers that go by a tile's parity, the rescaling of O, V's rows past the last key and the
end of a row tile.  And that both latent kernels' barriers are those that the models have.
"""
import os
import random
import re

import pytest

from tests import test_latent_phases as phases
from tests.test_latent_phases import Bar

WARPS = 8       # four lane quarters; warps w and w ^ 4 share rows, half of the columns each
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "varlen_gqa_attention_paged_gb300", "csrc")


class Model(phases.Model):
    """`moves[it][w]`: a row of warp w's half moves its maximum in tile it."""

    def __init__(self, segments, stages, rng, wrong=None):
        super().__init__(segments, stages, rng)
        self.wrong = wrong
        total = sum(segments)
        often = rng.choice([0.05, 0.3, 0.9])
        self.moves = [[rng.random() < often for _ in range(WARPS)] for _ in range(total)]
        at = 0
        for nt in segments:     # a row's first keys move it
            self.moves[at] = [rng.random() < 0.9 for _ in range(WARPS)]
            at += nt
        self.grown, self.scaled, self.meet = Bar(8), Bar(8), Bar(8)
        self.bare = [rng.choice([0, 0, 1, 2]) for _ in segments]
        none = [None] * WARPS
        self.s_grow, self.tops = [none[:], none[:]], [none[:], none[:]]     # by a tile's parity
        self.f = [none[:], none[:]]
        self.heard, self.used = [0] * WARPS, [0] * WARPS    # tiles whose buffers a warp is done with
        self.met = [0] * WARPS

    def together(self, warp):   # a named barrier of the softmax warps
        n = self.met[warp]
        self.met[warp] += 1
        self.meet.arrive()
        while not self.meet.done(n & 1):
            yield

    def softmax(self, warp, seen):
        it = moved = 0
        for sg, nt in enumerate(self.seg):
            for n in range(nt):
                par = it & 1
                while not self.s_full[it & 1].done((it >> 1) & 1):
                    yield
                assert self.s[it & 1] == it
                seen[warp] = it + 1
                self.read = min(seen)
                self.s_empty[it & 1].arrive()
                yield
                # the partner has read the maxima of two tiles before, all warps who moved
                assert self.heard[warp ^ 4] >= it - 1 and min(self.heard) >= it - 1, \
                    "overwritten before it was read"
                self.tops[par][warp] = it
                if self.moves[it][warp]:
                    self.s_grow[par][warp] = it + 1
                self.grown.arrive()
                yield
                while it > 0 and not self.pv_done.done((it - 1) & 1):
                    if self.wrong == "no wait for the product":
                        break
                    yield
                if self.wrong != "no wait for the others":
                    while not self.grown.done(it & 1):
                        yield
                said = [x == it + 1 for x in self.s_grow[par]]
                assert said == self.moves[it], "another tile's word"
                if any(said):
                    assert self.tops[par][warp ^ 4] == it, "another tile's maxima"
                self.heard[warp] = it + 1
                if any(said):
                    if warp < 4:
                        assert min(self.used) >= it - 1
                        self.f[par][warp] = it
                    yield
                    self.scaled.arrive()
                    phase = it if self.wrong == "a phase a tile" else moved
                    while self.wrong != "no wait for the factors" and \
                            not self.scaled.done(phase & 1):
                        yield
                    moved += 1
                    for _ in range(2):
                        assert self.f[par][:4] == [it] * 4, "another tile's factors"
                        yield
                    if n > 0:
                        assert self.o[:2] == ["sum", sg] and \
                            not any(x[0] == "pv" for x in self.queues[1]), "O still added to"
                self.used[warp] = it + 1
                yield
                assert not any(x[0] == "pv" for x in self.queues[1]), "weights still read"
                self.p = self.p or [None] * 8
                self.p[warp] = it
                if n == nt - 1:     # V's rows past the last key become zeros
                    assert all(self.tile[it % self.S][g] == it for g in range(1, phases.PARTS))
                self.p_full.arrive()
                it += 1
                yield
            while not self.pv_done.done((it - 1) & 1):
                yield
            yield from self.end(warp, it, sg, True)
            for e in range(self.bare[sg]):      # row tiles of which this share has no key
                yield from self.end(warp, it, (sg, e), False)

    def end(self, warp, it, tag, tiles):
        """The column halves' sums meet where the maxima were, then the factors of O's rows."""
        par = it & 1
        assert not tiles or self.o[1] == tag
        assert self.heard[warp ^ 4] >= it - 1
        self.tops[par][warp] = ("sum", tag)
        yield from self.together(warp)
        assert self.tops[par][warp ^ 4] == ("sum", tag)
        if warp < 4:
            assert min(self.used) >= it - 1
            self.f[par][warp] = ("end", tag)
        yield from self.together(warp)
        for _ in range(2):
            assert self.f[par][:4] == [("end", tag)] * 4, "factors overwritten before they were used"
            yield
        if tiles:
            self.o = ["out", tag, self.o[2] + 1 if self.o[0] == "out" else 1]
            self.o_empty.arrive()
        yield from self.together(warp)


def run(wrong=None, count=60, stages=2):
    for seed in range(count):
        rng = random.Random(seed)
        segments = [rng.randint(1, 7) for _ in range(rng.randint(1, 4))]
        Model(segments, stages, rng, wrong).run()


# (two parts and four stages: latents of 128; three and two: of 512)
@pytest.mark.parametrize("parts,stages", [(2, 4), (3, 4), (3, 2), (2, 2)])
def test_every_order_ends_and_reads_what_it_should(parts, stages, monkeypatch):
    monkeypatch.setattr(phases, "PARTS", parts)
    run(stages=stages)


@pytest.mark.parametrize("wrong", ["a phase a tile", "no wait for the product",
                                   "no wait for the others", "no wait for the factors"])
def test_what_the_model_would_notice(wrong):
    with pytest.raises(AssertionError):
        run(wrong)


# ------------------------------------------------------------------ the kernels' own barriers

def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"\s+", " ", re.sub(r"//.*", "", f.read()))


def waits(text):
    """(barrier, phase) of every bounded wait, in the order of the source."""
    found = re.findall(r"(?:pf_wait_warp|mbar_wait_bounded)\(", text)
    out = []
    for m in re.finditer(r"(?:pf_wait_warp|mbar_wait_bounded)\(", text):
        depth, arg, args = 1, "", []
        for ch in text[m.end():]:
            depth += ch in "([" and 1 or ch in ")]" and -1 or 0
            if depth == 0 or depth == 1 and ch == ",":
                args.append(arg.strip())
                arg = ""
                if depth == 0:
                    break
            else:
                arg += ch
        out.append(tuple(args[:2]))
    assert len(out) == len(found)
    return out


def test_the_absorbed_kernels_barriers_are_the_models():
    """Arrivals that end a phase, and the phase that each wait names: what the models above were
    written from.  A change here is a change to make there."""
    text = source("ua_latent.cuh")
    assert re.findall(r"mbar_init\((.*?), (\w+)\)", text) == [
        ("q_full", "1"), ("q_empty", "1"), ("&s_full[0]", "1"), ("&s_full[1]", "1"),
        ("p_full", "8"), ("pv_done", "1"), ("o_empty", "8"), ("fin", "2"), ("grown", "8"),
        ("scaled", "8"), ("&s_empty[0]", "8"), ("&s_empty[1]", "8"), ("&k_full[i]", "1"),
        ("&k_empty[i]", "1")]
    assert waits(text) == [
        # copies
        ("q_empty", "(sg - 1) & 1"), ("&k_empty[st * C::kParts + g]", "((it / S) - 1) & 1"),
        ("&k_full[i % S * C::kParts + g]", "(i / S) & 1"), ("q_full", "(sg - 1) & 1"),
        # Q K^T
        ("q_full", "sg & 1"), ("&s_empty[it & 1]", "((it >> 1) - 1) & 1"),
        ("&full[0]", "(it / S) & 1"), ("&full[1 + g]", "(it / S) & 1"), ("fin", "0"),
        # P.V
        ("p_full", "it & 1"), ("o_empty", "(sg - 1) & 1"), ("fin", "0"),
        # softmax
        ("&s_full[it & 1]", "(it >> 1) & 1"), ("pv_done", "(it - 1) & 1"), ("grown", "it & 1"),
        ("scaled", "moved & 1"), ("pv_done", "(it - 1) & 1")]
    assert len(re.findall(r"named_bar_sync\(1, 256\)", text)) == 3


def test_the_expanded_kernels_barriers_are_the_models():
    text = source("ua_latent_prefill.cuh")
    assert re.findall(r"mbar_init\((.*?), ([^,;]+)\);", text) == [
        ("&q_full[i]", "1"), ("&s_full[i]", "1"), ("&p_full[i]", "4"), ("&pv_done[i]", "1"),
        ("fin", "1"), ("&full[i]", "i % 2 == 0 ? C::kCB : C::kVB"), ("&empty[i]", "1")]
    assert waits(text) == [
        # copies
        ("&empty[bar_of(before / PER, before % PER >= C::kCB)]", "phase_of(before / PER)"),
        ("&full[bar_of(j, v)]", "phase_of(j)"), ("&q_full[qt]", "0"),
        # MMA issue
        ("&full[bar_of(i, 1)]", "phase_of(i)"), ("&p_full[qt]", "i & 1"), ("&q_full[qt]", "0"),
        ("&full[bar_of(j, 0)]", "phase_of(j)"), ("fin", "0"),
        # softmax
        ("&s_full[qt]", "n & 1"), ("&full[bar_of(n, 1)]", "phase_of(n)"), ("&pv_done[qt]", "0"),
        ("&pv_done[qt ^ 1]", "0")]
