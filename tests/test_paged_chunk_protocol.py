"""The chunk kernel's hand-offs between two MMA issuers, two softmax warpgroups and the tensor core, as
a model (no GPU).  The roles are coroutines in random order; products run behind their issuer, each
issuer's in order and the two in any order; waits go by the parity of a phase, as in the kernel.
The model raises where scores, P or sums are not those a role counts on, and where a named
barrier gets an arrival too many; a schedule in which nobody can go on fails too."""
import random

import pytest


class Bar:
    def __init__(self):
        self.phase = 0

    def arrive(self):
        self.phase += 1

    def done(self, parity):
        return (self.phase & 1) != (parity & 1)


class Model:
    """parts: (units, tiles) of a block's parts in order.  alone: the variant for calls whose items all
    have one unit, scores in both units' S columns in turn."""

    def __init__(self, parts, seed, alone, *, wait_rescale=True):
        self.parts, self.alone, self.wait_rescale = parts, alone, wait_rescale
        self.r = random.Random(seed)
        self.s_full, self.o_done, self.o_free = ([Bar(), Bar()] for _ in range(3))
        self.pv_done = Bar()
        self.turn = 0
        self.named = [0, 0]                 # P handed over and not taken
        self.queue = [[], []]               # the products of each issuer that have not run
        self.cols = [None, None]            # what the S columns hold: ("S" or "P", part, unit, tile)
        self.o = [None, None]               # (part, products summed)
        self.out = []

    def check(self, ok, what):
        if not ok:
            raise AssertionError(what)

    # products: run at some time after they are queued
    def s_mma(self, y, tag):
        def run():
            self.cols[y] = ("S",) + tag
        return run

    def pv_mma(self, y, x, part, j):
        def run():
            self.check(self.cols[y] == ("P", part, x, j), "P V found %s for %s" % (self.cols[y], (part, x, j)))
            self.check(j == 0 or self.o[x] == (part, j), "sums of another item")
            self.o[x] = (part, j + 1)
        return run

    def issuer(self, x):
        seq = qit = 0
        for k, (nx, n) in enumerate(self.parts):
            ahead = 2 if self.alone and n >= 2 else 1
            if x >= nx:
                seq += n + ahead
                continue
            q = self.queue[x]
            for i in range(ahead):
                yield lambda s=seq: self.turn == s + x
                q.append(self.s_mma(x + i, (k, x, i)))
                q.append(self.s_full[x + i].arrive)
                if i + 1 < ahead:
                    seq += 1
                self.turn = seq + x + (0 if i + 1 < ahead else 1)
            for j in range(n):
                y = j & 1 if ahead == 2 else x
                mine = seq + nx * (j + 1) + x
                yield lambda m=mine: self.turn == m
                if j == 0:
                    yield lambda t=qit: self.o_free[x].done((t & 1) ^ 1)
                yield lambda yy=y: self.named[yy] > 0
                self.named[y] -= 1
                q.append(self.pv_mma(y, x, k, j))
                if self.alone:
                    q.append(self.pv_done.arrive)
                if j + ahead < n:
                    q.append(self.s_mma(y, (k, x, j + ahead)))
                    q.append(self.s_full[y].arrive)
                if j + 1 == n:
                    q.append(self.o_done[x].arrive)
                self.turn = mine + 1
            seq += nx * (n + 1)
            qit += 1

    def softmax(self, x):
        sit, pvs, iit = [0, 0], 0, 0
        for k, (nx, n) in enumerate(self.parts):
            if x >= nx:
                continue
            two = self.alone and n >= 2
            for j in range(n):
                y = (j & 1 if two else 0) if self.alone else x
                use = 1 if self.alone and y else 0
                yield lambda b=self.s_full[y], ph=sit[use]: b.done(ph)
                sit[use] += 1
                self.check(self.cols[y] == ("S", k, x, j), "softmax found %s for %s" % (self.cols[y], (k, x, j)))
                if j > 0 and self.r.random() < 0.3:  # the sums are rescaled
                    if self.alone and self.wait_rescale:
                        yield lambda ph=pvs + j - 1: self.pv_done.done(ph)
                    self.check(self.o[x] == (k, j), "rescaled at the wrong time")
                yield lambda: True
                self.cols[y] = ("P", k, x, j)
                self.named[y] += 1
                self.check(self.named[y] == 1, "an arrival too many on a named barrier")
            pvs += n
            yield lambda ph=iit: self.o_done[x].done(ph)
            iit += 1
            self.check(self.o[x] == (k, n), "sums %s of item %s" % (self.o[x], (k, n)))
            self.out.append((k, x))
            self.o_free[x].arrive()

    def run(self):
        roles = [self.issuer(0), self.softmax(0)] + ([] if self.alone else [self.issuer(1), self.softmax(1)])
        waits = [next(g, None) for g in roles]
        while any(w is not None for w in waits) or any(self.queue):
            choices = [("role", i) for i, w in enumerate(waits) if w is not None and w()]
            choices += [("pipe", i) for i in (0, 1) if self.queue[i]]
            if not choices:
                raise AssertionError("nobody can go on")
            kind, i = self.r.choice(choices)
            if kind == "pipe":
                self.queue[i].pop(0)()
            else:
                waits[i] = next(roles[i], None)
        assert sorted(self.out) == [(k, x) for k, (nx, _) in enumerate(self.parts) for x in range(nx)]


def _parts(seed, alone):
    r = random.Random(seed)
    return [(1 if alone else r.choice([1, 2]), r.choice([1, 1, 2, 3, 4, 7])) for _ in range(r.randint(1, 9))]


@pytest.mark.parametrize("alone", [False, True])
@pytest.mark.parametrize("block", range(4))
def test_every_schedule_ends_with_the_right_sums(block, alone):
    for seed in range(400):
        Model(_parts(block * 1000 + seed, alone), seed, alone).run()


def test_a_unit_alone_has_to_wait_before_it_rescales():
    """Its S(j) is signalled before P V(j - 1) has run: the sums may not be touched yet."""
    failed = 0
    for seed in range(400):
        try:
            Model(_parts(seed, True), seed, True, wait_rescale=False).run()
        except AssertionError:
            failed += 1
    assert failed > 50
