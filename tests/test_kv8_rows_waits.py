"""The barriers between the softmax warps and the products of k_kv8_lists.cu, restated: a wait of parity P passes when the
phase before the one in progress has it. Every warp comes to its end, whatever runs late, and what was waited for is done."""
import random

import pytest


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passes(self, parity):
        return (self.phase - 1) % 2 == parity


class Tile:
    """One tile: products are done in their order, some time after they are issued; scores two steps ahead."""

    def __init__(self, rows, per_place):
        self.rows, self.per_place = rows, per_place  # steps of each row block
        self.scores = [Barrier(1), Barrier(1)]
        self.weights = [Barrier(4), Barrier(4)]
        self.values = [Barrier(1), Barrier(1)]
        self.queue, self.values_done = [], 0

    def done(self, c):
        """The barrier, and the parity, of the product with step c's values."""
        return (self.values[c & 1], c >> 1 & 1) if self.per_place else (self.values[0], c & 1)

    def products(self):
        first = 0
        for steps in self.rows:
            for c in range(first, first + min(steps, 2)):
                self.queue.append(("s", c))
            for c in range(first, first + steps):
                yield self.weights[c & 1], c >> 1 & 1
                self.queue.append(("v", c))
                if c + 2 < first + steps:
                    self.queue.append(("s", c + 2))
            first += steps

    def softmax(self, rng):
        first = 0
        for steps in self.rows:
            for c in range(first, first + steps):
                yield self.scores[c & 1], c >> 1 & 1
                if c > first and rng.random() < 0.3:  # its sum is scaled
                    yield self.done(c - 1)
                    assert self.values_done >= c
                self.weights[c & 1].arrive()
            first += steps
            if not self.per_place:
                yield self.done(first - 2)
            yield self.done(first - 1)
            assert self.values_done == first

    def unit(self):
        kind, c = self.queue.pop(0)
        if kind == "s":
            self.scores[c & 1].arrive()
        else:
            self.values_done += 1
            self.done(c)[0].arrive()


def ends(rows, seed, per_place):
    """Whether all warps come to their end with this order of events."""
    rng = random.Random(seed)
    t = Tile(rows, per_place)
    warps = [t.products()] + [t.softmax(rng) for _ in range(4)]
    waits = [next(w, None) for w in warps]
    slow = rng.choice([0.02, 0.2, 1.0])  # the slowest warp's or the products' share
    late = rng.randrange(6)
    while any(w is not None for w in waits):
        ready = [i for i, w in enumerate(waits) if w is not None and w[0].passes(w[1])] + ([5] if t.queue else [])
        if not ready:
            return False
        i = rng.choice(ready)
        if i == late and len(ready) > 1 and rng.random() > slow:
            continue
        if i == 5:
            t.unit()
        else:
            waits[i] = next(warps[i], None)
    return True


ROWS = [[1], [2], [3], [1, 1, 1], [2, 3, 1, 2], [53, 102, 5], [4, 1, 6, 2, 2]]


@pytest.mark.parametrize("rows", ROWS, ids=str)
def test_every_warp_comes_to_its_end(rows):
    assert all(ends(rows, seed, True) for seed in range(200))


def test_with_one_barrier_for_both_places_some_would_not():
    """The restatement sees what the second one is for."""
    assert not all(ends([4, 3], seed, False) for seed in range(200))
