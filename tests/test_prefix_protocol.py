"""Executable model of attn_prefix_kernel's synchronisation (csrc/prefix.cuh; host only, no GPU): two loading warps, the
thread that issues the products and two softmax warpgroups, which meet only through mbarriers, under random schedules and
lengths of a range.  Checked: no deadlock, no wait two phases behind, every product reads the tiles (and the P) of its own
step, no tile is overwritten before its products have read it, and no load is signalled before it has landed.  Planted
mistakes are caught.  A change to the kernel's barriers or to the order of its loads must be made here too.
"""
import random

import pytest

from tests.test_sync_model import Barrier, Deadlock, Violation


class Prefix:
    def __init__(self, steps, single, stages, lag, rng, mistake=None):
        self.steps, self.single, self.stages, self.lag, self.rng, self.mistake = steps, single, stages, lag, rng, mistake
        self.full = [Barrier("full%d" % i, 2) for i in range(stages)]
        self.empty = [Barrier("empty%d" % i, 1) for i in range(stages)]
        self.q = Barrier("q", 2)
        self.s, self.p, self.o = ([Barrier("%s%d" % (n, i), 1) for i in range(2)] for n in "spo")
        self.slot = [[None, None] for _ in range(stages)]      # what each half of a slot holds
        self.buf = [None, None]                                 # ("S" or "P", step) in TMEM
        self.acc = [[], []]                                     # steps accumulated in O
        self.pending, self.now, self.seq, self.mma_free = [], 0, 0, 0

    def later(self, fn, in_order=False):
        t = self.now + self.rng.randint(1, 30)
        if in_order:
            t = self.mma_free = max(t, self.mma_free + 1)
        self.seq += 1
        self.pending.append((t, self.seq, fn))

    def wait(self, bar, phase):
        while True:
            if bar.done > phase + 1:
                raise Violation("overrun on %s" % bar.name)
            if bar.done == phase + 1:
                return
            yield

    # what load `pos` brings: ("K" or "V", step, which tile of it), as the loading warps count it
    def load_at(self, pos):
        if not self.single:
            return ("V" if pos & 1 else "K", pos >> 1, 0)
        if pos < 2:
            return ("K", 0, pos)
        g, r = (pos - 2) >> 2, (pos - 2) & 3
        if g < self.steps - 1:
            return ("V", g, r >> 1) if not r & 1 else ("K", g + 1, r >> 1)
        return ("V", g, r)

    def loader(self, half):
        total, landed = (4 if self.single else 2) * self.steps, []
        for pos in range(total):
            slot = pos % self.stages
            if pos >= self.stages and self.mistake != "no empty wait":
                yield from self.wait(self.empty[slot], pos // self.stages - 1)
            landed.append(False)
            self.slot[slot][half] = None

            def land(pos=pos, slot=slot):
                self.slot[slot][half] = self.load_at(pos)
                landed[pos] = True
            self.later(land)
            if pos >= self.lag:
                while self.mistake != "no landing wait" and not all(landed[:pos - self.lag + 1]):
                    yield
                self.full[(pos - self.lag) % self.stages].arrive()
            yield
        while not all(landed):
            yield
        for pos in range(max(total - self.lag, 0), total):
            self.full[pos % self.stages].arrive()

    def mma(self):
        yield from self.wait(self.q, 0)

        def landed(at):
            yield from self.wait(self.full[at % self.stages], at // self.stages)

        def read(slot, what):
            if self.slot[slot] != [what, what]:
                raise Violation("product of %s read %s" % (what, self.slot[slot]))

        def issue_s(t, at, step):
            what = ("K", step, t if self.single else 0)

            def run():
                read(at % self.stages, what)
                if step and self.acc[t] != list(range(step)):
                    raise Violation("S over a P that was not used")
                self.buf[t] = ("S", step)
            self.later(run, True)
            self.later(self.s[t].arrive, True)

        def issue_o(t, at, step):
            what = ("V", step, t if self.single else 0)

            def run():
                read(at % self.stages, what)
                if self.buf[t] != ("P", step):
                    raise Violation("PV of step %d read %s" % (step, self.buf[t]))
                self.acc[t].append(step)
            self.later(run, True)

        def release(at):
            self.later(self.empty[at % self.stages].arrive, True)
        single = self.single
        yield from landed(0)
        issue_s(0, 0, 0)
        if single:
            release(0)
            yield from landed(1)
        issue_s(1, 1 if single else 0, 0)
        release(1 if single else 0)
        pos = 2 if single else 1
        for jj in range(self.steps):
            more = jj + 1 < self.steps
            v = [pos, pos + (2 if more else 1) if single else pos]
            k = [pos + 1, pos + 3 if single else pos + 1]
            for t in range(2):
                yield from landed(v[t])
                if self.mistake != "no P wait":
                    yield from self.wait(self.p[t], jj)
                issue_o(t, v[t], jj)
                if not more:
                    self.later(self.o[t].arrive, True)
                if single or t == 1 or self.mistake == "early release":
                    release(v[t])
                if more:
                    yield from landed(k[t])
                    issue_s(t, k[t], jj + 1)
                    if single or t == 1:
                        release(k[t])
            pos += (2 if single else 1) * (2 if more else 1)

    def softmax(self, t):
        self.q.arrive()
        for jj in range(self.steps):
            yield from self.wait(self.s[t], jj)
            if self.buf[t] != ("S", jj):
                raise Violation("softmax %d read %s" % (jj, self.buf[t]))
            yield
            self.buf[t] = ("P", jj)
            self.p[t].arrive()
        yield from self.wait(self.o[t], 0)
        if self.acc[t] != list(range(self.steps)):
            raise Violation("O read early")

    def run(self):
        roles = [self.loader(0), self.loader(1), self.mma(), self.softmax(0), self.softmax(1)]
        idle = 0
        while roles or self.pending:
            self.now += 1
            before = self.seq, sum(b.done * 3 + b.pending for b in self.full + self.empty + self.s + self.p + self.o + [self.q])
            for x in sorted(x for x in self.pending if x[0] <= self.now):
                self.pending.remove(x)
                x[2]()
            role = self.rng.choice(roles) if roles else None
            if role is not None:
                try:
                    next(role)
                except StopIteration:
                    roles.remove(role)
            after = self.seq, sum(b.done * 3 + b.pending for b in self.full + self.empty + self.s + self.p + self.o + [self.q])
            idle = 0 if after != before or self.pending else idle + 1
            if idle > 400:
                raise Deadlock()


GEOMETRIES = [(False, 5, 2), (True, 6, 2), (False, 12, 5), (True, 13, 5)]     # single, stages, lag: d = 128, then 64


@pytest.mark.parametrize("single,stages,lag", GEOMETRIES)
def test_runs_to_the_end(single, stages, lag):
    rng = random.Random(stages)
    for steps in list(range(1, 12)) + [25, 40]:
        for _ in range(6):
            Prefix(steps, single, stages, lag, rng).run()


@pytest.mark.parametrize("mistake", ["no empty wait", "no landing wait", "no P wait", "early release"])
def test_mistakes_are_caught(mistake):
    rng, caught = random.Random(1), 0
    for _ in range(20):
        try:
            Prefix(30, False, 5, 2, rng, mistake).run()
        except (Violation, Deadlock):
            caught += 1
    assert caught
