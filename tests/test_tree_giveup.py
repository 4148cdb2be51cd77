"""Waits that give up in the tensor-core kernel of the rule over trees (csrc/gdr_tree_tc.cu), as a model on the CPU.

Every wait of the kernel has a limit, and may run out of it in one warp while the phase completes for another.  The
named barriers of a role have none: all of the role's warps have to come to each of them, or none.  The roles that have
several warps are modelled with their waits, votes and barriers in the kernel's order; a wait gives up at random, warp by
warp, and the model checks that every warp ends."""

import random

import pytest


class Stuck(Exception):
    pass


class Named:
    """A named barrier of `count` warps, with an OR of what they bring."""

    def __init__(self, count):
        self.count, self.here, self.any, self.result, self.round = count, 0, False, False, 0

    def vote(self, value):
        mine = self.round
        self.here, self.any = self.here + 1, self.any or value
        if self.here == self.count:
            self.result, self.here, self.any, self.round = self.any, 0, False, mine + 1
        while self.round == mine:
            yield
        return self.result


class Model:
    def __init__(self, seed, pairs, rate, alone=False):
        self.rng, self.pairs, self.rate = random.Random(seed), pairs, rate
        self.alone = alone  # a warp of the states whose last wait of a pair gives up leaves by itself
        self.heads = [self.rng.random() < 0.5 for _ in range(pairs)]  # a pair that the factors take with the next

    def wait(self):
        """A wait of one warp: whether it ended by its phase."""
        for _ in range(self.rng.randint(0, 3)):
            yield
        return self.rng.random() >= self.rate

    def states(self, bar, stages):
        ok = True
        for i in range(self.pairs):
            ok = (i == 0 or (yield from self.wait())) and ok  # kFirst
            for _ in range(stages):
                ok = ok and (yield from self.wait())  # kSFull
                if (yield from bar.vote(not ok)):
                    return
            if i > 0:
                if not (yield from self.wait()):  # kRParts
                    if self.alone:
                        return
                    ok = False

    def rows(self, bar):
        ok = True
        for i in range(self.pairs):
            for _ in range(3):  # kGateFull, kVFull, kFirst
                ok = (yield from self.wait()) and ok
            if (yield from bar.vote(not ok)):
                return
            odd = yield from bar.vote(self.rng.random() < 0.3)
            ok = (yield from self.wait()) and ok  # kSecond
            if odd:
                yield from bar.vote(False)

    def factors(self, bar):
        def voted():
            return (yield from bar.vote(not (yield from self.wait())))

        def sync(n):
            for _ in range(n):
                yield from bar.vote(False)

        i = 0
        while i < self.pairs:
            yield from sync(1)  # K and Q
            if (yield from voted()):  # kTables
                return
            two = i + 1 < self.pairs and self.heads[i]
            if two and (yield from voted()):
                return
            if (yield from voted()):  # kGram
                return
            yield from sync(9)
            for j in (i, i + 1) if two else (i,):
                if j > 0 and (yield from voted()):  # kBFree
                    return
                yield from sync(2)
            i += 2 if two else 1

    def run(self):
        warps = [self.rows(b) for b in [Named(16)] for _ in range(16)]
        warps += [self.states(b, 4) for b in (Named(4), Named(4)) for _ in range(4)]
        warps += [self.factors(b) for b in [Named(6)] for _ in range(6)]
        left, idle = list(range(len(warps))), 0
        while left:
            w, idle = self.rng.choice(left), idle + 1
            try:
                next(warps[w])
            except StopIteration:
                left.remove(w)
                idle = 0
            if idle > 20000:
                raise Stuck(left)


def models(count, **kw):
    for seed in range(count):
        r = random.Random(seed)
        yield Model(seed, r.randint(1, 5), r.choice([0.0, 0.003, 0.02, 0.2, 1.0]), **kw)


def test_every_warp_ends():
    for m in models(150):
        m.run()


def test_the_model_finds_a_warp_that_leaves_by_itself():
    with pytest.raises(Stuck):
        for m in models(150, alone=True):
            m.run()
