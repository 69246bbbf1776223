"""How the expanded attention's softmax warps leave after a wait that gave up, on the CPU by random interleaving (on the GPU
no wait gives up unless a copy or a product never completes).

A CTA's processes: pairs of softmax warps, the copying warp that publishes pieces, the warp that issues products.  A wait on
an mbarrier ends when its condition holds or, at any time, by giving up; its process then is dead and goes on without
waiting until it leaves.  A named barrier has no such limit: it waits for all its members.  So whoever shares one has to
leave at the same place, or the others hang there."""
import random

import pytest

PAIRS, PIECES, STEPS = 3, 4, 2


class Hang(AssertionError):
    pass


class Barrier:
    """All members, or none: generation `round` is over when each has come."""

    def __init__(self, members):
        self.members, self.come, self.round, self.any, self.result = members, 0, 0, False, False

    def arrive(self, value):
        self.come, self.any, mine = self.come + 1, self.any or value, self.round
        if self.come == self.members:
            self.come, self.round, self.result, self.any = 0, self.round + 1, self.any, False
        return mine


def softmax(s, pair, cut, together):
    """One pair: pieces in turn, their steps, and for cut row tiles the join.  together: one vote of all pairs before each
    piece of a call that cuts row tiles."""
    dead = False
    for piece in range(PIECES + 1):
        if not dead:
            dead = not (yield lambda: s["published"] > piece, True)
        if cut and together:
            mine = s["all"].arrive(dead)
            yield lambda: s["all"].round > mine, False
            dead = s["all"].result
        if dead or piece == PIECES:
            break
        for step in range(STEPS):
            if not dead:
                dead = not (yield lambda: s["scores"][pair] > piece * STEPS + step, True)
            s["weights"][pair] += 1
        if cut:
            mine = s["all"].arrive(False)
            yield lambda: s["all"].round > mine, False
    s["left"] += 1


def copies(s):
    for _ in range(PIECES + 1):
        s["published"] += 1
        yield lambda: True, False


def products(s):
    for n in range(PIECES * STEPS):
        for pair in range(PAIRS):
            s["scores"][pair] += 1
            if not (yield lambda: s["weights"][pair] > n, True):
                return


def run(seed, cut, together, patience):
    """patience: one wait in so many that could go on gives up all the same."""
    rng = random.Random(seed)
    s = {"published": 0, "scores": [0] * PAIRS, "weights": [0] * PAIRS, "left": 0, "all": Barrier(PAIRS)}
    live = {g: next(g) for g in [softmax(s, p, cut, together) for p in range(PAIRS)] + [copies(s), products(s)]}
    while live:
        ready = [g for g, (holds, gives_up) in live.items() if gives_up or holds()]
        if not ready:
            raise Hang(f"seed {seed}: {s['left']} of {PAIRS} pairs have left, the others wait for them")
        g = rng.choice(ready)
        holds, gives_up = live[g]
        came = holds() and not (gives_up and rng.randrange(patience) == 0)
        if not came and holds() is False and rng.randrange(patience) and len(ready) > 1:
            continue                                         # not yet
        try:
            live[g] = g.send(came)
        except StopIteration:
            del live[g]
    assert s["left"] == PAIRS


@pytest.mark.parametrize("cut", [False, True])
def test_softmax_warps_leave_together(cut):
    for seed in range(3000):
        run(seed, cut, True, patience=2 + seed % 40)


def test_the_search_sees_a_pair_that_leaves_alone():
    with pytest.raises(Hang):
        for seed in range(3000):
            run(seed, True, False, patience=2 + seed % 40)
