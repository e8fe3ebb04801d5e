"""The few-row paged kernel's ring of tiles, as a model (no GPU): one loader fills slots with copies
that may end out of order, warps take tiles in order, and both sides wait on mbarriers by
the parity of a phase, as the kernel does.  A wait by parity is right only for a waiter that is at
most one phase ahead; the model raises where a warp takes a slot that does not hold its tile, where
a slot is overwritten under a reader, and where a barrier gets an arrival too many."""
import heapq
import random

import pytest


class Bar:
    def __init__(self, count):
        self.count = self.pending = count
        self.tx = self.phase = 0

    def arrive(self, tx=0):
        if self.pending == 0:
            raise RuntimeError("an arrival too many")
        self.pending -= 1
        self.tx += tx
        self._flip()

    def complete(self, tx):
        self.tx -= tx
        self._flip()

    def _flip(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def done(self, parity):  # what try_wait.parity answers
        return (self.phase & 1) != parity


def run(slots, groups, warps, tiles, seed):
    r = random.Random(seed)
    full, empty = [Bar(1) for _ in range(slots)], [Bar(warps) for _ in range(slots)]
    holds = [None] * slots
    events, state = [], dict(t=0.0, n=0, taken=0)

    def after(dt, f):
        state["n"] += 1
        heapq.heappush(events, (state["t"] + dt, state["n"], f))

    def loader(it):
        if it >= 2 * tiles:
            return
        s = it % slots
        if not empty[s].done(((it // slots) & 1) ^ 1):
            return after(0.05, lambda: loader(it))
        full[s].arrive(1)
        holds[s] = None

        def landed():
            holds[s] = it
            full[s].complete(1)

        after(1 + r.random() * (8 if r.random() < 0.05 else 0.5), landed)  # now and then a late one
        after(0.02, lambda: loader(it + 1))

    def warp(tile, half, step):
        if tile >= tiles:
            return
        it = 2 * tile + half
        s = it % slots
        if not full[s].done((it // slots) & 1):
            return after(0.05, lambda: warp(tile, half, step))
        if holds[s] != it:
            raise RuntimeError("a slot that holds another tile")

        def release():
            if holds[s] != it:
                raise RuntimeError("overwritten under a reader")
            empty[s].arrive()
            state["taken"] += 1
            warp(*((tile, 1) if half == 0 else (tile + groups, 0)), step)

        after(r.random() * step, release)

    after(0, lambda: loader(0))
    for g in range(groups):
        for _ in range(warps):
            after(0, lambda g=g: warp(g, 0, 0.5 * groups))
    while events:
        state["t"], _, f = heapq.heappop(events)
        f()
    return state["taken"]


# (slots, computing warps) of a group: d = 128 and d = 64, bf16 and e4m3.  Groups share nothing.
@pytest.mark.parametrize("slots,warps", [(2, 4), (4, 4), (2, 2), (4, 2)])
def test_every_tile_is_taken_whole_and_once(slots, warps):
    for seed in range(25):
        for tiles in (1, 2, 3, 7, 150):
            assert run(slots, 1, warps, tiles, seed) == 2 * tiles * warps


def test_groups_that_share_slots_would_not_do():
    """Three groups that take the tiles of one ring of four slot pairs in turn meet one another's slots: why every
    group of the kernel has its own."""
    failed = 0
    for seed in range(25):
        try:
            run(8, 3, 4, 150, seed)
        except RuntimeError:
            failed += 1
    assert failed > 10
