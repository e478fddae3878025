"""Waits by parity on a barrier that completes one phase a tile, over every interleaving.

The one-tile prefill kernels wait for P.V of a tile on such a barrier: phase n completes some
time after the softmax has handed over the P of tile n (and after phase n - 1).  A wait names a
phase by its parity only, so it is right only while the barrier is at most one phase past the one
waited for: two past, it reads as not done, for good.  The model below runs a softmax warp's
operations against the tensor cores' progress in every order, and asks that no wait passes too
early and that the walk always ends.
"""
import pytest


def walk(n_tiles, rescaled, end):
    """The softmax's operations: ("read", n) S of tile n is there, ("wait", n) for phase n of P.V,
    ("give", n) hands over the P of tile n; then `end`."""
    ops = []
    for n in range(n_tiles):
        ops.append(("read", n))
        if n >= 1 and n in rescaled:
            ops.append(("wait", n - 1))
        ops.append(("give", n))
    return ops + end


def last_commit(n_tiles):
    """What the kernels wait for behind the walk: a barrier that completes once, after all P.V."""
    return [("last", n_tiles)]


def last_phases(n_tiles):
    """The last two phases instead."""
    return [("wait", n) for n in range(max(0, n_tiles - 2), n_tiles)]


def outcomes(ops):
    """What can happen: "done", "stuck" (a wait that never passes), "early" (one that passes
    before its phase is complete)."""
    seen, todo, out = set(), [(0, 0, 0)], set()
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        at, given, done = state      # the warp's next operation, tiles handed over, P.V complete
        moves = []
        if done < given:
            moves.append((at, given, done + 1))
        if at == len(ops):
            out.add("done")
        else:
            kind, n = ops[at]
            if kind == "give":
                moves.append((at + 1, n + 1, done))
            elif kind == "read":
                if done >= n - 1:                # S of tile n follows P.V n - 2
                    moves.append((at + 1, given, done))
            elif kind == "last":
                if done == n:
                    moves.append((at + 1, given, done))
            elif (done & 1) != (n & 1):          # the phase with this parity is complete
                if done <= n:
                    out.add("early")
                moves.append((at + 1, given, done))
        if not moves and at < len(ops):
            out.add("stuck")
        todo += moves
    return out


@pytest.mark.parametrize("n_tiles", range(1, 8))
def test_the_walk_always_ends_and_no_wait_passes_early(n_tiles):
    for mask in range(1 << n_tiles):
        rescaled = {n for n in range(n_tiles) if mask >> n & 1}
        assert outcomes(walk(n_tiles, rescaled, last_commit(n_tiles))) == {"done"}


def test_two_waits_behind_the_last_hand_over_can_miss_a_phase():
    assert "stuck" in outcomes(walk(2, set(), last_phases(2)))
    assert "stuck" in outcomes(walk(5, {1}, last_phases(5)))
    assert outcomes(walk(1, set(), last_phases(1))) == {"done"}
