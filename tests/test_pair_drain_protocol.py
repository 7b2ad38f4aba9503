"""A discrete-event model of the barriers of the product's pair kernel, checked on the CPU: the loads of two CTAs, the
products, the readers of the sums, and the end after a wait that ran out.

Two CTAs load halves of a step into S stages and count their bytes on the first one's barrier of the stage (one
arrival, by the first CTA, which expects the bytes of both); the first CTA gives steps to the tensor cores, which
signal both CTAs' barriers when a step is done, and at a tile's end the barriers of the sums; readers of both CTAs
give accumulators back.  A barrier is waited on by the parity of a phase, and the hardware compares parities alone.

In the model a CTA withholds its loads from some step on, or a reader stops, and every wait has a limit that may be
shorter than a load takes; a CTA's waits end with the first of them that runs out, its roles then, and the other CTA
learns of it before the barrier of the cluster that ends them.  Whatever was issued has to have landed when the CTAs leave, and the end must not lean on
its own limit.  An end that only sleeps for the waits' limit once more leaves loads in flight.
"""
from __future__ import annotations

import heapq
import random

import pytest

INF = float("inf")


class Bar:
    def __init__(self, count):
        self.count = self.pending = count
        self.tx = self.phase = 0

    def change(self, arrive=0, tx=0):
        self.pending -= arrive
        self.tx += tx
        assert self.pending >= 0
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def done(self, parity):
        return (self.phase & 1) != parity


class Model:
    """Roles are generators that yield ("sleep", t), or ("wait", barrier, parity), which answers whether it came in
    time, or ("drain", barrier, parity), a wait of the end."""

    def __init__(self, seed, stages, steps, tiles, stall=None, reader_stops=None, limit=5.0, sleep_only=False):
        self.rng = random.Random(seed)
        self.S, self.steps, self.tiles = stages, steps, tiles
        self.stall, self.reader_stops, self.limit, self.sleep_only = stall, reader_stops, limit, sleep_only
        self.now, self.events, self.seq = 0.0, [], 0
        self.full = [Bar(1) for _ in range(stages)]
        self.empty = [[Bar(1) for _ in range(stages)] for _ in range(2)]
        self.sums = [[Bar(1) for _ in range(2)] for _ in range(2)]
        self.freed = [Bar(2) for _ in range(2)]
        self.aborted = [False, False]
        self.flying = 0              # loads and signals that have not landed
        self.issued, self.stepped, self.tiled = [0, 0], 0, 0
        self.waiting = {}            # role -> (kind, barrier, parity, deadline)
        self.drain_ran_out = False
        self.left_flying = None

    def at(self, dt, f):
        self.seq += 1
        heapq.heappush(self.events, (self.now + dt, self.seq, f))

    def land(self, dt, f):
        self.flying += 1

        def landed():
            self.flying -= 1
            f()
        self.at(dt, landed)

    @property
    def abort(self):
        return any(self.aborted)

    # ---- the roles, as in the kernel

    def producer(self, r):
        n, ok = 0, True
        while ok and n < self.steps * self.tiles:
            st = n % self.S
            if n >= self.S:
                ok = yield "wait", self.empty[r][st], ((n // self.S) - 1) & 1
            if self.stall == (r, n):
                ok = False
            if not ok:
                break
            if r == 0:
                self.full[st].change(arrive=1, tx=2)
            self.land(self.rng.uniform(1, 40 if self.rng.random() < 0.2 else 4), lambda st=st: self.full[st].change(tx=-1))
            n += 1
            yield "sleep", self.rng.uniform(0, 1)
        self.issued[r] = n
        i = max(0, n - self.S)
        while ok and i < n:
            ok = yield "wait", self.empty[r][i % self.S], (i // self.S) & 1
            i += 1

    def products(self):
        n, k, ok = 0, 0, True
        while ok and k < self.tiles:
            if k >= 1:
                ok = yield "wait", self.freed[(k - 1) & 1], ((k - 1) >> 1) & 1
            i = 0
            while ok and i < self.steps:
                st = n % self.S
                ok = yield "wait", self.full[st], (n // self.S) & 1
                if not ok:
                    break
                for r in range(2):
                    self.land(self.rng.uniform(0.5, 6), lambda st=st, r=r: self.empty[r][st].change(arrive=1))
                n, i = n + 1, i + 1
                yield "sleep", self.rng.uniform(0, 1)
            if not ok:
                break
            for r in range(2):
                self.land(self.rng.uniform(0.5, 6), lambda k=k, r=r: self.sums[r][k & 1].change(arrive=1))
            k += 1
        self.stepped, self.tiled = n, k

    def reader(self, r):
        for k in range(self.tiles):
            if not (yield "wait", self.sums[r][k & 1], (k >> 1) & 1):
                return
            if self.reader_stops == (r, k):
                yield "sleep", 10 * self.limit + 50
                return
            yield "sleep", self.rng.uniform(0, 2)
            self.freed[k & 1].change(arrive=1)

    def end(self, r):
        """After the barrier of the cluster; CTA r's thread 0."""
        if not self.abort:           # (either CTA's: the flag was passed on before the barrier)
            return
        if self.sleep_only:
            yield "sleep", self.limit
            return
        for i in range(max(0, self.stepped - self.S), self.stepped):
            yield "drain", self.empty[r][i % self.S], (i // self.S) & 1
        for k in range(max(0, self.tiled - 2), self.tiled):
            yield "drain", self.sums[r][k & 1], (k >> 1) & 1
        if r == 0:
            loads = max(self.issued)
            for i in range(max(0, loads - self.S), loads):
                b = self.full[i % self.S]
                if i >= self.issued[0]:
                    b.change(arrive=1, tx=1)
                if i >= self.issued[1]:
                    b.change(tx=-1)
                yield "drain", b, (i // self.S) & 1

    # ---- the machine

    def run_roles(self, *roles):
        """roles: (CTA, generator)."""
        live = {(key, cta): g for key, (cta, g) in enumerate(roles)}

        def resume(key, value):
            try:
                got = live[key].send(value)
            except StopIteration:
                del live[key]
                return
            if got[0] == "sleep":
                self.at(got[1], lambda: resume(key, None))
            else:
                limit = self.limit if got[0] == "wait" else 1000.0
                self.waiting[key] = (*got, self.now + limit)
                self.at(limit + 1e-6, lambda: None)        # (so that the run-out is looked at)

        for key in list(live):
            resume(key, None)
        while live:
            for key, (kind, bar, parity, deadline) in list(self.waiting.items()):
                answer = True if bar.done(parity) else None
                if answer is None and kind == "wait" and (self.aborted[key[1]] or self.now > deadline):
                    self.aborted[key[1]], answer = True, False
                if answer is None and kind == "drain" and self.now > deadline:
                    self.drain_ran_out, answer = True, False
                if answer is not None:
                    del self.waiting[key]
                    resume(key, answer)
                    break
            else:
                if live:
                    self.now, _, f = heapq.heappop(self.events)
                    f()

    def run(self):
        self.run_roles((0, self.producer(0)), (1, self.producer(1)), (0, self.products()), (0, self.reader(0)), (1, self.reader(1)))
        self.run_roles((0, self.end(0)), (1, self.end(1)))
        self.left_flying = self.flying
        return self


def _cases():
    rng = random.Random(1)
    for seed in range(400):
        stages, steps, tiles = rng.randint(2, 6), rng.randint(1, 9), rng.randint(1, 5)
        total = steps * tiles
        what = seed % 3
        stall = (rng.randint(0, 1), rng.randrange(total)) if what != 2 else None
        stops = (rng.randint(0, 1), rng.randrange(tiles)) if what == 2 else None
        yield seed, dict(stages=stages, steps=steps, tiles=tiles, stall=stall, reader_stops=stops,
                         limit=rng.choice([0.5, 3.0, 30.0, 300.0]))


def test_nothing_is_in_flight_when_the_pair_leaves():
    ran_out = 0
    for seed, kw in _cases():
        m = Model(seed, **kw).run()
        ran_out += m.abort
        assert m.left_flying == 0 and not m.drain_ran_out, (seed, kw)
    assert ran_out > 250


def test_without_a_fault_every_step_and_tile_is_done():
    for seed in range(60):
        m = Model(seed, stages=2 + seed % 5, steps=1 + seed % 7, tiles=1 + seed % 4, limit=INF).run()
        assert not m.abort and m.left_flying == 0
        total = (1 + seed % 7) * (1 + seed % 4)
        assert m.issued == [total, total] and m.stepped == total and m.tiled == 1 + seed % 4


def test_sleeping_for_the_limit_once_more_leaves_loads_in_flight():
    """What the end is there for: the model sees the fault that it mends."""
    assert sum(Model(seed, sleep_only=True, **kw).run().left_flying > 0 for seed, kw in _cases()) > 50


@pytest.mark.parametrize("half", [0, 1])
def test_loads_that_only_one_cta_issued(half):
    """One CTA stops first and the other runs up to all stages ahead: both ways of closing a phase are met.  (The
    limit is past all delays of the ten loads together, so that the withheld one alone runs out.)"""
    m = Model(half, stages=4, steps=20, tiles=1, stall=(half, 6), limit=1000.0).run()
    assert m.abort and m.issued[half] == 6 and m.issued[1 - half] == 10 and m.left_flying == 0
