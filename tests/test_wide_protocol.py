"""The barrier protocol of the attention kernel for many rows (csrc/gdr_attn_wide.cu) as a model on the CPU.

Every role is a generator that waits, arrives and touches buffers as the kernel's role does, with the kernel's own
indices and phases, in random order; loads land in any order, MMAs and the arrivals committed behind them complete in
the order of their issue.  Every use of a buffer is checked to find what its user means.  B blocks of rows share a
worker's keys and values; a barrier that counts several warps of a role is one arrival of it."""

import random

import pytest

# head size, blocks of rows -> stages of the ring, places for Q
SHAPES = {(64, 1): (8, 2), (128, 1): (8, 2), (256, 1): (5, 1), (64, 2): (8, 2), (128, 2): (6, 2)}


class Wrong(Exception):
    """A buffer does not hold what its user means, or nothing can go on."""


def check(ok, *what):
    if not ok:
        raise Wrong(what)


class Bar:
    def __init__(self, count):
        self.count = self.pending = count
        self.phase = 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.phase, self.pending = self.phase + 1, self.count


class Model:
    def __init__(self, seed, triples, d, blocks, without=None):
        self.rng, self.triples, self.B, self.without = random.Random(seed), triples, blocks, without
        self.N, self.QS = SHAPES[d, blocks]
        sizes = dict(QFull=self.QS, QEmpty=self.QS, KvFull=self.N, KvEmpty=self.N, SFull=2 * blocks, PFull=2 * blocks,
                     PvDone=2 * blocks, ODone=1, OFree=1)
        self.bars = {name: [Bar(blocks if name == "OFree" else 1) for _ in range(m)] for name, m in sizes.items()}
        self.loads, self.mmas = [], []
        self.ring, self.q, self.s = [None] * self.N, [None] * self.QS, [None] * (2 * blocks)
        self.o = [None] * blocks
        self.done = [0] * blocks

    def wait(self, role, name, i, parity):
        if self.without == (role, name):
            return
        bar = self.bars[name][i]
        while (bar.phase & 1) == (parity & 1):
            yield

    def arrive(self, name, i=0):
        self.bars[name][i].arrive()

    def load(self, where, i, what, name):
        """A copy under way, whose landing arrives."""
        where[i] = ("on its way", what)

        def land():
            where[i] = what
            self.arrive(name, i)
        self.loads.append(land)

    def stages(self):
        """(stage's number, what it holds), K0, K1, V0, K2, V1, ...; the last value leaves one out."""
        tiles = sum(self.triples)
        key = [(0 if g == 0 else 2 * g - 1, ("k", g)) for g in range(tiles)]
        return sorted(key + [(2 * g + 2, ("v", g)) for g in range(tiles)])

    def loader(self, kind):
        for i, what in self.stages():
            if what[0] != kind:
                continue
            st, use = i % self.N, i // self.N
            if use > 0:
                yield from self.wait("loads", "KvEmpty", st, use - 1)
            self.load(self.ring, st, what, "KvFull")
            yield

    def queries(self):
        for it in range(len(self.triples)):
            z = it % self.QS
            if it >= self.QS:
                yield from self.wait("Q", "QEmpty", z, it // self.QS - 1)
            self.load(self.q, z, it, "QFull")
            yield

    def mma(self, run):
        self.mmas.append(run)

    def products(self):
        triples = self.triples
        tile_of = [(it, tile) for it, m in enumerate(triples) for tile in range(m)]
        gs, kt = 0, -1

        def keys():
            nonlocal kt
            it, tile = tile_of[gs]
            if tile == 0:
                kt = it
                yield from self.wait("MMAs", "QFull", it % self.QS, it // self.QS)
            i = 0 if gs == 0 else 2 * gs - 1
            yield from self.wait("MMAs", "KvFull", i % self.N, i // self.N)

        def score(b):
            it, tile = tile_of[gs]
            g, i = gs, 0 if gs == 0 else 2 * gs - 1

            def run():
                check(self.q[it % self.QS] == it and self.ring[i % self.N] == ("k", g), "S's operands", g)
                check(self.s[2 * b + (g & 1)] in (None, ("used", g - 2)), "S's tile", b, g, self.s)
                self.s[2 * b + (g & 1)] = ("s", g)
            self.mma(run)
            self.mma(lambda: self.arrive("SFull", 2 * b + (g & 1)))
            if b == self.B - 1:
                self.mma(lambda: self.arrive("KvEmpty", i % self.N))
                if tile == triples[it] - 1:
                    self.mma(lambda: self.arrive("QEmpty", it % self.QS))

        total = len(tile_of)
        for _ in range(2):
            if gs == total:
                break
            yield from keys()
            for b in range(self.B):
                score(b)
            gs += 1
        g = 0
        for it, m in enumerate(triples):
            for tile in range(m):
                ahead = g > 0 and gs < total
                if ahead:
                    yield from keys()
                i = 2 * g + 2
                for b in range(self.B):
                    if ahead:
                        score(b)
                    if b == 0:
                        if tile == 0 and it > 0:
                            yield from self.wait("MMAs", "OFree", 0, it - 1)
                        yield from self.wait("MMAs", "KvFull", i % self.N, i // self.N)
                    yield from self.wait("MMAs", "PFull", 2 * b + (g & 1), g >> 1)

                    def run(g=g, b=b, it=it, tile=tile, i=i):
                        check(self.ring[i % self.N] == ("v", g), "V", g, self.ring)
                        check(self.s[2 * b + (g & 1)] == ("p", g), "P", b, g, self.s)
                        check(self.o[b] in ((None, ("read", it - 1)) if tile == 0 else (("o", it, tile - 1),)), "O", self.o)
                        self.s[2 * b + (g & 1)] = ("used", g)
                        self.o[b] = ("o", it, tile)
                    self.mma(run)
                    self.mma(lambda b=b, g=g: self.arrive("PvDone", 2 * b + (g & 1)))
                    if b == self.B - 1:
                        self.mma(lambda i=i: self.arrive("KvEmpty", i % self.N))
                        if tile == m - 1:
                            self.mma(lambda: self.arrive("ODone"))
                    yield
                if ahead:
                    gs += 1
                g += 1

    def rows(self, b):
        g = 0
        for it, m in enumerate(self.triples):
            for tile in range(m):
                st = 2 * b + (g & 1)
                yield from self.wait("rows", "SFull", st, g >> 1)
                check(self.s[st] == ("s", g), "S", b, g, self.s)
                if tile > 0 and self.rng.random() < 0.4:  # O is scaled
                    yield from self.wait("rows", "PvDone", 2 * b + (g - 1 & 1), (g - 1) >> 1)
                    check(self.o[b] == ("o", it, tile - 1), "O to scale", b, self.o)
                    yield
                    check(self.o[b] == ("o", it, tile - 1), "O while scaled", b, self.o)
                self.s[st] = ("p", g)
                self.arrive("PFull", st)
                yield
                g += 1
            yield from self.wait("rows", "ODone", 0, it)
            for _ in range(self.rng.randint(1, 4)):
                check(self.o[b] == ("o", it, m - 1), "O to store", b, self.o)
                yield
            self.o[b] = ("read", it)
            self.arrive("OFree")
            self.done[b] += 1

    def run(self):
        roles = [self.loader("k"), self.loader("v"), self.queries(), self.products()] + [self.rows(b) for b in range(self.B)]
        pace = [self.rng.uniform(0.05, 1) for _ in roles] + [self.rng.uniform(0.1, 1) for _ in range(2)]
        alive, idle = set(range(len(roles))), 0
        while alive:
            x = self.rng.choices(range(len(pace)), pace)[0]
            before = len(self.loads), len(self.mmas), len(alive), [b.phase for bs in self.bars.values() for b in bs]
            if x == len(roles):
                if self.loads:
                    self.loads.pop(self.rng.randrange(len(self.loads)))()
            elif x == len(roles) + 1:
                if self.mmas:
                    self.mmas.pop(0)()
            elif x in alive:
                try:
                    next(roles[x])
                except StopIteration:
                    alive.discard(x)
            after = len(self.loads), len(self.mmas), len(alive), [b.phase for bs in self.bars.values() for b in bs]
            idle = 0 if before != after else idle + 1
            check(idle < 3000, "nothing goes on", alive)
        check(self.done == [len(self.triples)] * self.B, "all triples")


def models(count, d, blocks, without=None):
    for seed in range(count):
        r = random.Random(seed)
        yield Model(seed, [r.choice([1, 1, 2, 3, 7]) for _ in range(r.randint(1, 6))], d, blocks, without)


@pytest.mark.parametrize("d,blocks", sorted(SHAPES))
def test_every_order_goes_through(d, blocks):
    for m in models(150, d, blocks):
        m.run()


@pytest.mark.parametrize("d,blocks", [(256, 1), (128, 2)])
@pytest.mark.parametrize("without", [("loads", "KvEmpty"), ("Q", "QEmpty"), ("MMAs", "QFull"), ("MMAs", "KvFull"),
                                     ("MMAs", "PFull"), ("rows", "SFull"), ("rows", "PvDone"), ("rows", "ODone")])
def test_every_wait_is_needed(without, d, blocks):
    """The model finds what goes wrong without it.  (The MMAs' wait for O's reader is implied by that for P: the rows
    read O before they make the next triple's P.)"""
    with pytest.raises(Wrong):
        for m in models(300, d, blocks, without):
            m.run()
