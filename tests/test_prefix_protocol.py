"""Executable model of attn_prefix_kernel's synchronisation (csrc/prefix.cuh; host only, no GPU): three or six warps that copy keys and
values and the queries, whose barriers count them as they land, the thread that issues the products and two softmax warpgroups,
which meet only through mbarriers, under random schedules and shares of a range.  Checked: no deadlock, no wait two phases behind, every product
reads the tiles (and the queries and the P) of its own step, and nothing is overwritten before its products have read it.  Planted mistakes are caught.  A change to the kernel's barriers or to the order of
its loads must be made here too.
"""
import random

import pytest

from tests.test_sync_model import Barrier, Deadlock, Violation


class Prefix:
    """shares: the steps of each unit that the CTA meets."""

    def __init__(self, shares, single, stages, rng, mistake=None):
        self.shares, self.single, self.stages, self.rng, self.mistake = shares, single, stages, rng, mistake
        self.loaders = loaders = 6 if single else 3
        self.full = [Barrier("full%d" % i, loaders) for i in range(stages)]
        self.empty = [Barrier("empty%d" % i, 1) for i in range(stages)]
        self.q, self.q_empty = Barrier("q", loaders), Barrier("q_empty", 1)
        self.s, self.p, self.o = ([Barrier("%s%d" % (n, i), 1) for i in range(2)] for n in "spo")
        self.slot = [[None] * loaders for _ in range(stages)]        # what each warp has put into a slot
        self.queries = [None] * loaders                               # whose queries each warp has brought
        self.buf = [None, None]                                 # ("S" or "P", share, step) in TMEM
        self.acc = [(None, []), (None, [])]                     # share and steps accumulated in O
        self.pending, self.now, self.seq, self.mma_free = [], 0, 0, 0

    def later(self, fn, in_order=False):
        t = self.now + self.rng.randint(1, 30 if in_order else 120)
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

    def loads(self):
        """("K" or "V", share, step, which tile of it) in the order in which the loading warps count them."""
        for n, steps in enumerate(self.shares):
            for at in range((4 if self.single else 2) * steps):
                if not self.single:
                    yield ("V" if at & 1 else "K", n, at >> 1, 0)
                elif at < 2:
                    yield ("K", n, 0, at)
                else:
                    g, r = (at - 2) >> 2, (at - 2) & 3
                    if g < steps - 1:
                        yield ("V", n, g, r >> 1) if not r & 1 else ("K", n, g + 1, r >> 1)
                    else:
                        yield ("V", n, g, r)

    def loader(self, who):
        share = -1
        for pos, what in enumerate(self.loads()):
            if what[1] != share:
                share = what[1]
                if share and self.mistake != "no query wait":
                    yield from self.wait(self.q_empty, share - 1)
                self.queries[who] = None

                def bring(share=share):
                    self.queries[who] = share
                    self.q.arrive()
                self.later(bring)
                yield
            slot = pos % self.stages
            if pos >= self.stages and self.mistake != "no empty wait":
                yield from self.wait(self.empty[slot], pos // self.stages - 1)
            self.slot[slot][who] = None

            def land(slot=slot, what=what):
                self.slot[slot][who] = what
                self.full[slot].arrive()
            self.later(land)
            if self.mistake == "signalled at once":
                self.full[slot].arrive()
            yield

    def mma(self):
        def landed(at):
            yield from self.wait(self.full[at % self.stages], at // self.stages)

        def read(slot, what):
            if self.slot[slot] != [what] * self.loaders:
                raise Violation("product of %s read %s" % (what, self.slot[slot]))

        def issue_s(t, at, n, step):
            what = ("K", n, step, t if self.single else 0)

            def run():
                read(at % self.stages, what)
                if self.queries != [n] * self.loaders:
                    raise Violation("S of share %d read queries of %s" % (n, self.queries))
                if step and self.acc[t] != (n, list(range(step))):
                    raise Violation("S over a P that was not used")
                self.buf[t] = ("S", n, step)
            self.later(run, True)
            self.later(self.s[t].arrive, True)

        def issue_o(t, at, n, step):
            what = ("V", n, step, t if self.single else 0)

            def run():
                read(at % self.stages, what)
                if self.buf[t] != ("P", n, step):
                    raise Violation("PV of step %d read %s" % (step, self.buf[t]))
                if step == 0:
                    if self.acc[t][1] and self.acc[t][0] is not None:
                        raise Violation("O overwritten before it was read")
                    self.acc[t] = (n, [])
                self.acc[t][1].append(step)
            self.later(run, True)

        def release(at):
            self.later(self.empty[at % self.stages].arrive, True)
        single, pos, count = self.single, 0, 0
        for n, steps in enumerate(self.shares):
            yield from self.wait(self.q, n)
            yield from landed(pos)
            issue_s(0, pos, n, 0)
            if single:
                release(pos)
                pos += 1
                yield from landed(pos)
            issue_s(1, pos, n, 0)
            release(pos)
            pos += 1
            if steps == 1:
                self.later(self.q_empty.arrive, True)
            for jj in range(steps):
                more = jj + 1 < steps
                v = [pos, pos + (2 if more else 1) if single else pos]
                k = [pos + 1, pos + 3 if single else pos + 1]
                for t in range(2):
                    if single or t == 0:
                        yield from landed(v[t])
                    if self.mistake != "no P wait":
                        yield from self.wait(self.p[t], count + jj)
                    issue_o(t, v[t], n, jj)
                    if not more:
                        self.later(self.o[t].arrive, True)
                    if single or t == 1 or self.mistake == "early release":
                        release(v[t])
                    if more:
                        if single or t == 0:
                            yield from landed(k[t])
                        issue_s(t, k[t], n, jj + 1)
                        if single or t == 1:
                            release(k[t])
                        if t == 1 and jj + 2 == steps:
                            self.later(self.q_empty.arrive, True)
                pos += (2 if single else 1) * (2 if more else 1)
            count += steps

    def softmax(self, t):
        count = 0
        for n, steps in enumerate(self.shares):
            for jj in range(steps):
                yield from self.wait(self.s[t], count)
                if self.buf[t] != ("S", n, jj):
                    raise Violation("softmax %d read %s" % (jj, self.buf[t]))
                yield
                self.buf[t] = ("P", n, jj)
                self.p[t].arrive()
                count += 1
            if self.mistake != "no O wait":
                yield from self.wait(self.o[t], n)
            if self.acc[t] != (n, list(range(steps))):
                raise Violation("O read early")
            yield
            self.acc[t] = (None, [])

    def state(self):
        return self.seq, sum(b.done * 8 + b.pending for b in
                             self.full + self.empty + self.s + self.p + self.o + [self.q, self.q_empty])

    def run(self):
        roles = [self.loader(i) for i in range(self.loaders)] + [self.mma(), self.softmax(0), self.softmax(1)]
        idle = 0
        while roles or self.pending:
            self.now += 1
            before = self.state()
            for x in sorted(x for x in self.pending if x[0] <= self.now):
                self.pending.remove(x)
                x[2]()
            role = self.rng.choice(roles) if roles else None
            if role is not None:
                try:
                    next(role)
                except StopIteration:
                    roles.remove(role)
            idle = 0 if self.state() != before or self.pending else idle + 1
            if idle > 400:
                raise Deadlock()


GEOMETRIES = [(False, 4), (True, 5), (False, 10), (True, 11)]     # single, stages: d = 128, then 64


@pytest.mark.parametrize("single,stages", GEOMETRIES)
def test_runs_to_the_end(single, stages):
    rng = random.Random(stages)
    for shares in [[n] for n in list(range(1, 12)) + [25]] + [[1, 1], [1, 1, 1, 1], [3, 1], [1, 7], [2, 5, 2], [6, 6, 6, 2], [1, 2, 3, 4, 1]]:
        for _ in range(6):
            Prefix(shares, single, stages, rng).run()


@pytest.mark.parametrize("mistake", ["no empty wait", "signalled at once", "no P wait", "early release", "no O wait", "no query wait"])
def test_mistakes_are_caught(mistake):
    rng, caught = random.Random(1), 0
    for _ in range(20):
        try:
            Prefix([20, 3, 10], False, 4, rng, mistake).run()
        except (Violation, Deadlock):
            caught += 1
    assert caught
