"""The barrier protocol of the two-SM attention kernel (csrc/gdr_attn_prefill.cu) as a model on the CPU.

Every role of the kernel is a generator that waits, arrives and touches buffers as the kernel's role does, with the
kernel's own indices and phases; the model runs them in random order, lets loads land in any order and MMAs complete
in the order of their issue, and checks at every use that a buffer holds what its user means: stages of the ring, Q,
S and P tiles, O, the entries of the blocks, the references and sums handed between the warpgroups.  A pair of CTAs
is one here: both run the same steps, and a barrier that counts several warps is one arrival of their role.

The kernel's names: block `it` of a pair has n tiles, of which those from j_clean on are looked through; g counts
tiles through all blocks, i counts ring stages."""

import random

import pytest

# head size -> tiles by which S runs ahead of P V, ring stages, S tiles, Q tiles
SHAPES = {64: (2, 8, 3, 2), 128: (2, 8, 3, 2), 256: (1, 5, 2, 1)}


class Wrong(Exception):
    """A buffer does not hold what its user means, or a wait meant another phase than the barrier's."""


def check(ok, *what):
    if not ok:
        raise Wrong(what)


class Bar:
    def __init__(self, count):
        self.count = self.pending = count
        self.phase = 0  # completed ones

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.phase, self.pending = self.phase + 1, self.count


class Model:
    def __init__(self, blocks, d, seed, without=None):
        self.blocks, self.rng, self.without = blocks, random.Random(seed), without
        self.A, self.N, self.S, self.QT = SHAPES[d]
        sizes = dict(QFull=2, QEmpty=2, KvFull=self.N, KvEmpty=self.N, VLocal=self.N, SFull=self.S, PFull=self.S,
                     PvDone=2, ODone=1, OFree=1, MReady=1, Patch=4, Block=4, Read=4, LOther=2, Inv=2)
        # entry, flags and 1 / l of a block are read by the two P warpgroups and the O warpgroup
        self.bars = {name: [Bar(3 if name == "Read" else 1) for _ in range(m)] for name, m in sizes.items()}
        self.loads, self.mmas = [], []  # under way: loads end in any order, MMAs in this one
        self.ring, self.q, self.s = [None] * self.N, [None] * self.QT, [None] * self.S
        self.entries, self.inv, self.sums = [None] * 4, [None] * 2, [None] * 2
        self.o, self.m, self.done = (None, []), None, []

    def wait(self, role, name, i, phase):
        """The kernel's parity wait, where only completed phase number `phase` or the one before can be met."""
        bar = self.bars[name][i]
        if self.without == (role, name):
            return
        while (bar.phase & 1) == (phase & 1):
            check(bar.phase <= phase, "overtaken", role, name, i, phase, bar.phase)
            yield
        check(bar.phase == phase + 1, "another phase", role, name, i, phase, bar.phase)

    def ready(self, name, i, phase):
        return (self.bars[name][i].phase & 1) != (phase & 1)

    def arrive(self, name, i):
        self.bars[name][i].arrive()

    def fetch(self, role, it):
        """Block `it`: tiles and the first to be looked through; 0 tiles: there is none."""
        yield from self.wait(role, "Block", it & 3, it >> 2)
        entry = self.entries[it & 3]
        check(entry is not None and entry[0] == it, "entry", role, it, entry)
        return entry[1:]

    # --- roles ----------------------------------------------------------------------------------------------

    def load(self):
        role, i, k_it, kj, kn, more, q_waits = "load", 0, -1, 0, 0, True, False

        def land(where, slot, what, name, index):
            def end():
                where[slot] = what
                self.arrive(name, index)
            self.loads.append(end)

        def load_q(block):
            nonlocal q_waits
            if not q_waits:
                return
            slot, use = k_it % self.QT, k_it // self.QT
            if use > 0:
                if block:
                    yield from self.wait(role, "QEmpty", slot, use - 1)
                elif not self.ready("QEmpty", slot, use - 1):
                    return
            land(self.q, slot, k_it, "QFull", slot)
            q_waits = False

        def free_stage():
            st, use = i % self.N, i // self.N
            if use > 0:
                while q_waits and not self.ready("KvEmpty", st, use - 1):
                    yield from load_q(False)
                    yield
                yield from self.wait(role, "KvEmpty", st, use - 1)
            return st

        def load_k():
            nonlocal i, k_it, kj, kn, more, q_waits
            if kj == kn:
                yield from load_q(True)
                k_it, kj = k_it + 1, 0
                more = k_it < len(self.blocks)
                kn, j_clean = self.blocks[k_it] if more else (0, 0)
                if k_it >= 4:
                    yield from self.wait(role, "Read", k_it & 3, (k_it >> 2) - 1)
                self.entries[k_it & 3] = (k_it, kn, j_clean)
                self.arrive("Block", k_it & 3)
                if not more:
                    return
                q_waits = True
                yield from load_q(False)
            st = yield from free_stage()
            land(self.ring, st, ("K", k_it, kj), "KvFull", st)
            kj, i = kj + 1, i + 1

        ahead = 0
        while ahead <= self.A and more:
            yield from load_k()
            ahead += 1
        v_it, vj, start = 0, 0, True
        n, j_clean = yield from self.fetch(role, 0)
        while n > 0:
            if not start and more:
                yield from load_k()
            start = False
            st = yield from free_stage()
            land(self.ring, st, ("V", v_it, vj), "VLocal" if vj >= j_clean else "KvFull", st)
            i, vj = i + 1, vj + 1
            if vj == n:
                v_it, vj = v_it + 1, 0
                n, j_clean = yield from self.fetch(role, v_it)
            yield from load_q(False)
        yield from load_q(True)

    def mma(self):
        role, i, gs, g, k_it, kj, kn, more = "mma", 0, 0, 0, -1, 0, 0, True

        def score():
            nonlocal i, gs, k_it, kj, kn, more
            if kj == kn:
                k_it, kj = k_it + 1, 0
                kn, _ = yield from self.fetch(role, k_it)
                more = kn > 0
                if not more:
                    return
                yield from self.wait(role, "QFull", k_it % self.QT, k_it // self.QT)
            st, t = i % self.N, gs % self.S
            yield from self.wait(role, "KvFull", st, i // self.N)

            def end(st=st, t=t, it=k_it, j=kj, gs=gs, last=kj == kn - 1):
                check(self.ring[st] == ("K", it, j), "K stage", self.ring[st], it, j)
                check(self.q[it % self.QT] == it, "Q", self.q, it)
                check(self.s[t] is None, "S over", self.s[t], gs)
                self.s[t] = ("S", gs)
                self.arrive("KvEmpty", st)
                self.arrive("SFull", t)
                if last:
                    self.arrive("QEmpty", it % self.QT)
            self.mmas.append(end)
            kj, gs, i = kj + 1, gs + 1, i + 1

        ahead = 0
        while ahead <= self.A and more:
            yield from score()
            ahead += 1
        v_it = vj = 0
        n, _ = yield from self.fetch(role, 0)
        while n > 0:
            if g > 0 and more:
                yield from score()
            st, t = i % self.N, g % self.S
            if vj == 0 and v_it > 0:
                yield from self.wait(role, "OFree", 0, v_it - 1)
            yield from self.wait(role, "KvFull", st, i // self.N)
            yield from self.wait(role, "PFull", t, g // self.S)

            def end(st=st, t=t, it=v_it, j=vj, g=g, last=vj == n - 1):
                check(self.ring[st] == ("V", it, j), "V stage", self.ring[st], it, j)
                check(self.s[t] == ("P", g), "P", self.s[t], g)
                self.s[t] = None
                if j == 0:
                    check(self.o[0] is None, "O over", self.o[0], it)
                    self.o = (it, [])
                check(self.o[0] == it, "O", self.o[0], it)
                self.o[1].append(g)
                self.arrive("KvEmpty", st)
                self.arrive("PvDone", g & 1)
                if last:
                    self.arrive("ODone", 0)
            self.mmas.append(end)
            i, g, vj = i + 1, g + 1, vj + 1
            if vj == n:
                v_it, vj = v_it + 1, 0
                n, _ = yield from self.fetch(role, v_it)

    def look(self):
        """Looks value tiles through and reports their stages."""
        role, g, k_count, k_it, it, more, turns = "look", 0, 0, 0, 0, True, [0] * self.N
        while True:
            n, j_clean = yield from self.fetch(role, it)
            if n == 0:
                return
            for j in range(n):
                if j >= j_clean:
                    while more and k_count < g + self.A + 1:
                        kn, _ = yield from self.fetch(role, k_it)
                        k_it, more, k_count = k_it + 1, kn > 0, k_count + kn
                    st = (g + min(g + self.A + 1, k_count)) % self.N
                    yield from self.wait(role, "VLocal", st, turns[st])
                    turns[st] += 1
                    check(self.ring[st] == ("V", it, j), "looked-through stage", self.ring[st], it, j)
                    self.arrive("KvFull", st)
                g += 1
            self.arrive("Patch", it & 3)
            it += 1

    def softmax(self, wg):
        role, g0, it, others = "softmax", 0, 0, [0, 0]
        while True:
            n, _ = yield from self.fetch(role, it)
            if n == 0:
                return
            self.arrive("Read", it & 3)
            for j in range((g0 ^ wg) & 1, n, 2):
                g = g0 + j
                t, slot = g % self.S, it & 1
                yield from self.wait(role, "SFull", t, g // self.S)
                check(self.s[t] == ("S", g), "S", self.s[t], g)
                if self.rng.random() < 0.5:
                    yield
                if g > 0:
                    yield from self.wait(role, "MReady", 0, g - 1)
                    check(self.m == g - 1, "reference", self.m, g)
                self.m = g
                self.arrive("MReady", 0)
                if j > 0 and self.rng.random() < 0.5:  # raises the reference and rescales O
                    yield from self.wait(role, "PvDone", (g - 1) & 1, (g - 1) >> 1)
                    check(self.o[0] == it and self.o[1][-1:] == [g - 1], "rescaled O", self.o, it, g)
                if self.rng.random() < 0.5:
                    yield
                check(self.s[t] == ("S", g), "P over", self.s[t], g)
                self.s[t] = ("P", g)
                self.arrive("PFull", t)
                if j == n - 2:
                    check(self.sums[slot] is None, "sum over", self.sums[slot], it)
                    self.sums[slot] = it
                    self.arrive("LOther", slot)
                elif j == n - 1:
                    if n > 1:
                        yield from self.wait(role, "LOther", slot, others[slot])
                        check(self.sums[slot] == it, "other sum", self.sums[slot], it)
                        self.sums[slot] = None
                    if it >= 2:
                        yield from self.wait(role, "Read", (it - 2) & 3, (it - 2) >> 2)
                    check(self.inv[slot] is None, "1 / l over", self.inv[slot], it)
                    self.inv[slot] = it
                    self.arrive("Inv", slot)
            g0 += n
            if n > 1:
                others[it & 1] += 1
            it += 1

    def output(self):
        role, it = "output", 0
        while True:
            n, _ = yield from self.fetch(role, it)
            if n == 0:
                return
            yield from self.wait(role, "Inv", it & 1, it >> 1)
            check(self.inv[it & 1] == it, "1 / l", self.inv[it & 1], it)
            yield from self.wait(role, "Patch", it & 3, it >> 2)
            yield from self.wait(role, "ODone", 0, it)
            yield
            check(self.o[0] == it and len(self.o[1]) == n, "O read", self.o, it)
            self.o, self.inv[it & 1] = (None, []), None
            self.done.append(it)
            self.arrive("OFree", 0)
            self.arrive("Read", it & 3)
            it += 1

    def run(self):
        roles = dict(load=self.load(), mma=self.mma(), look=self.look(), even=self.softmax(0), odd=self.softmax(1),
                     output=self.output())
        names = list(roles) + ["a load lands", "an MMA completes"]
        weights = [self.rng.choice([1, 1, 3, 10, 30]) for _ in names]  # some roles far slower than others
        for _ in range(400000):
            if not roles:
                break
            turn = self.rng.choices(names, weights)[0]
            if turn == "a load lands" and self.loads:
                self.loads.pop(self.rng.randrange(len(self.loads)))()
            elif turn == "an MMA completes" and self.mmas:
                self.mmas.pop(0)()
            elif turn in roles:
                try:
                    next(roles[turn])
                except StopIteration:
                    del roles[turn]
        check(not roles, "stuck", list(roles))
        check(self.done == list(range(len(self.blocks))), "blocks", self.done)


def blocks_of(seed):
    rng = random.Random(7 * seed + 1)
    most = rng.choice([1, 1, 2, 4, 9])
    sizes = [rng.randint(1, most) for _ in range(rng.randint(0, 14))]
    return [(n, max(0, n - rng.randint(1, 3))) for n in sizes]


@pytest.mark.parametrize("d", SHAPES)
def test_every_use_finds_what_it_means(d):
    for seed in range(150):
        Model(blocks_of(seed), d, seed).run()


@pytest.mark.parametrize("role,name", [
    ("load", "KvEmpty"), ("load", "QEmpty"), ("load", "Read"), ("mma", "QFull"), ("mma", "KvFull"), ("mma", "PFull"),
    ("mma", "OFree"), ("look", "VLocal"), ("softmax", "SFull"), ("softmax", "MReady"), ("softmax", "PvDone"),
    ("softmax", "LOther"), ("softmax", "Read"), ("output", "Inv"), ("output", "ODone"),
])
def test_the_model_finds_a_wait_left_out(role, name):
    """The model without one of its waits: some order of events shows it."""
    with pytest.raises(Wrong):
        for seed in range(300):
            for d in SHAPES:
                Model(blocks_of(seed), d, seed, without=(role, name)).run()
