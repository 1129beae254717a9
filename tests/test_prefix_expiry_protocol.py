"""Executable model of attn_prefix_kernel's waits running out (csrc/prefix.cuh; host only, no GPU): one signal is withheld, some
wait for it gives up, and every other wait then gives up at once.  Whatever the signal and the schedule: the block ends, every share of each softmax
warpgroup leaves a part, and a part that was not complete is marked as bad, so that the join never reads what the
workspace held before.  The mistake of leaving without marking is caught.
"""
import random

import pytest

from tests.test_prefix_protocol import GEOMETRIES, Prefix
from tests.test_sync_model import Violation

LIMIT = 300                                          # ticks after which a wait gives up (the model takes 400 idle ones for a deadlock)


class GaveUp(Exception):
    pass


class Expiring(Prefix):
    def __init__(self, shares, single, stages, rng, withheld, mistake=None):
        super().__init__(shares, single, stages, rng)
        self.leave, self.abort, self.parts = mistake == "leave", False, [[None] * len(shares) for _ in range(2)]
        bars = self.full + self.empty + self.s + self.p + self.o + [self.q, self.q_empty]
        bar, nth = bars[withheld[0] % len(bars)], withheld[1]
        arrive, seen = bar.arrive, [0]

        def some():
            seen[0] += 1
            if seen[0] != nth + 1:
                arrive()
        bar.arrive = some

    def wait(self, bar, phase):
        began = self.now
        while bar.done < phase + 1:
            if self.abort or self.now - began > LIMIT:
                self.abort = True
                raise GaveUp
            yield
        if bar.done > phase + 1:
            raise Violation("overrun on %s" % bar.name)

    def until(self, role):
        try:
            yield from role
        except GaveUp:
            return

    def loader(self, who):
        return self.until(super().loader(who))

    def mma(self):
        return self.until(super().mma())

    def softmax(self, t):
        count, ok = 0, True
        for n, steps in enumerate(self.shares):
            try:
                for jj in range(steps if ok else 0):
                    yield from self.wait(self.s[t], count)
                    if self.buf[t] != ("S", n, jj):
                        raise Violation("softmax %d read %s" % (jj, self.buf[t]))
                    yield
                    self.buf[t] = ("P", n, jj)
                    self.p[t].arrive()
                    count += 1
                if ok:
                    yield from self.wait(self.o[t], n)
            except GaveUp:
                ok = False
                if self.leave:
                    return
            if ok and self.acc[t] != (n, list(range(steps))):
                raise Violation("O read early")
            yield
            self.parts[t][n] = "whole" if ok else "bad"
            if ok:
                self.acc[t] = (None, [])

    def state(self):
        return super().state(), self.abort


def run(single, stages, rng, mistake=None):
    shares = rng.choice([[1], [9], [1, 1, 1], [3, 1, 4], [6, 6, 2], [2, 5, 2, 1]])
    x = Expiring(shares, single, stages, rng, (rng.randrange(64), rng.randrange(8)), mistake)
    x.run()
    return x


@pytest.mark.parametrize("single,stages", GEOMETRIES)
def test_every_share_leaves_a_part(single, stages):
    rng, expired = random.Random(stages), 0
    for _ in range(150):
        x = run(single, stages, rng)
        for parts in x.parts:
            assert None not in parts and parts == sorted(parts, key=lambda p: p == "bad")        # whole ones, then bad ones
            assert x.abort or "bad" not in parts
        expired += x.abort
    assert expired > 30


def test_leaving_without_marking_is_caught():
    rng, missing = random.Random(1), 0
    for _ in range(60):
        x = run(False, 4, rng, "leave")
        missing += any(None in parts for parts in x.parts)
    assert missing
