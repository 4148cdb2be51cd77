"""The barrier protocol of the tensor-core kernel of the rule over trees (csrc/gdr_tree_tc.cu) as a model on the CPU.

Every role is a generator that waits, arrives and touches buffers as the kernel's role does, with the kernel's own
indices and phases; the model runs them in random order and checks at every use that a buffer holds what its user
means.  The states' warps are one role, the rows' warps two that vote (named barriers), as any two of theirs would; a
commit's arrival follows its MMAs."""

import random

import pytest


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
    def __init__(self, seed, items, share, per, without=None):
        """`items` pairs of a block: `per` V heads a tree, of which `share` have a QK head in common."""
        self.rng, self.without, self.items = random.Random(seed), without, []
        tree = head = None
        for i in range(items):
            t, h = i // per, (i // per, i % per // share)
            self.items.append((i, t != tree, h != head))
            tree, head = t, h
        sizes = dict(Tables=2, KqFull=2, GateFull=4, TabFree=2, BFull=1, BFree=1, First=1, Second=1, RParts=1, Parts=1,
                     XFree=1)
        # both of the rows' groups let X go
        self.bars = {name: [Bar(2 if name == "XFree" else 1) for _ in range(m)] for name, m in sizes.items()}
        self.tables, self.tree, self.kq, self.gate = [None] * 2, [None] * 4, [None] * 2, [None] * 4
        self.a = self.b = self.x = self.odd = None
        self.votes, self.round, self.result = [], 0, False

    def wait(self, role, name, i, parity):
        if self.without == (role, name):
            return
        bar = self.bars[name][i]
        while (bar.phase & 1) == (parity & 1):
            yield "waits"

    def arrive(self, name, i=0):
        self.bars[name][i].arrive()

    def gates(self):
        tree = -1
        for i, new_tree, _ in self.items:
            yield
            if i >= 2:
                yield from self.wait("gates", "TabFree", i & 1, (i - 2) >> 1)
            if new_tree:
                tree += 1
                self.tree[tree & 3] = tree
                yield
            self.tables[i & 1] = i
            yield
            self.arrive("Tables", i & 1)

    def factors(self):
        kq, tree, k = 0, -1, 0
        items = self.items
        while k < len(items):
            i, new_tree, new_kq = items[k]
            two = k + 1 < len(items) and not items[k + 1][2]  # another V head of this QK head with it
            tree += new_tree
            if new_kq:
                self.kq[kq] = i
                self.arrive("KqFull", kq)
                yield
            yield from self.wait("factors", "Tables", i & 1, i >> 1)
            if two:
                yield from self.wait("factors", "Tables", (i + 1) & 1, (i + 1) >> 1)
            both = (i, i + 1) if two else (i,)
            for j in both:
                check(self.tree[tree & 3] == tree and self.tables[j & 1] == j, "tables", j)
            yield
            for j in both:
                self.gate[j & 3] = j
            yield
            for j in both:
                check(self.tables[j & 1] == j, "tables", j)
                self.arrive("GateFull", j & 3)
                self.arrive("TabFree", j & 1)
            yield
            check(self.tree[tree & 3] == tree, "tree", i)
            for j in both:
                if j > 0:
                    yield from self.wait("factors", "BFree", 0, j - 1)
                after = i + len(both)
                if j == i and after < len(items) and items[after][2]:
                    self.kq[kq ^ 1] = ("on its way", after)
                yield
                check(self.tree[tree & 3] == tree and self.gate[j & 3] == j, "tree and gates", j)
                self.b = ("half", j)
                yield
                self.b = j
                yield
                self.arrive("BFull")
                yield
            k = i + len(both)
            if k < len(items) and items[k][2]:
                kq ^= 1

    def mmas(self):
        loads, held = -1, None
        for i, _, new_kq in self.items:
            if new_kq:
                loads += 1
                held = i
                yield from self.wait("MMAs", "KqFull", loads & 1, loads >> 1)
            yield from self.wait("MMAs", "Parts", 0, i)
            if i > 0:
                yield from self.wait("MMAs", "XFree", 0, i - 1)
            self.x = ("half", i)
            for _ in range(self.rng.randint(1, 4)):
                check(self.kq[loads & 1] == held and self.a == i, "first", i, self.kq, self.a)
                yield
            self.x = ("x", i)
            self.arrive("First")
            yield
            yield from self.wait("MMAs", "BFull", 0, i)
            yield from self.wait("MMAs", "RParts", 0, i)
            odd = self.odd
            for _ in range(self.rng.randint(1, 4)):
                check(self.b == i, "second", i, self.b)
                yield
            self.x = ("u", i)
            if not odd:
                self.arrive("BFree")
            yield
            self.arrive("Second")
            yield

    def vote(self, value):
        mine = self.round
        self.votes.append(value)
        if len(self.votes) == 2:
            self.result, self.votes, self.round = any(self.votes), [], mine + 1
        while self.round == mine:
            yield "waits"
        return self.result

    def rows(self, me):
        tree = -1
        for i, new_tree, _ in self.items:
            tree += new_tree
            yield
            yield from self.wait("rows", "GateFull", i & 3, i >> 2)
            yield from self.wait("rows", "First", 0, i)
            yield from self.vote(False)
            check(self.x == ("x", i) and self.gate[i & 3] == i and self.tree[tree & 3] == tree, "R", i)
            yield
            check(self.gate[i & 3] == i and self.tree[tree & 3] == tree, "gates", i)
            odd = yield from self.vote(self.rng.random() < 0.2)
            if me == 0:
                self.odd = odd
                self.arrive("RParts")
            yield
            yield from self.wait("rows", "Second", 0, i)
            check(self.x == ("u", i), "U and O", i)
            if odd:
                for _ in range(self.rng.randint(1, 5)):
                    check(self.b == i and self.tree[tree & 3] == tree, "odd values", i)
                    yield
                yield from self.vote(False)
                if me == 0:
                    self.arrive("BFree")
            for _ in range(self.rng.randint(1, 5)):
                check(self.x == ("u", i), "U and O", i)
                yield
            self.arrive("XFree")
            yield

    def states(self):
        for i, _, _ in self.items:
            if i > 0:  # the product that reads the parts before these is done
                yield from self.wait("states", "First", 0, i - 1)
            self.a = ("half", i)
            yield
            self.a = i
            self.arrive("Parts")
            yield

    def run(self):
        roles = [self.gates(), self.factors(), self.mmas(), self.rows(0), self.rows(1), self.states()]
        pace = [self.rng.uniform(0.05, 1) for _ in roles]
        left, idle = set(range(len(roles))), 0
        while left:
            order = sorted(left)
            r = self.rng.choices(order, [pace[x] for x in order])[0]
            try:
                idle = idle + 1 if next(roles[r]) == "waits" else 0
            except StopIteration:
                left.discard(r)
                idle = 0
            check(idle < 4000, "nothing goes on", sorted(left))


def models(count, without=None):
    for seed in range(count):
        r = random.Random(seed)
        share = r.choice([1, 2, 3, 4])
        yield Model(seed, r.randint(1, 14), share, r.choice([1, 2, 4]) * share, without)


def test_every_order_goes_through():
    for m in models(800):
        m.run()


@pytest.mark.parametrize("without", [
    ("gates", "TabFree"), ("factors", "Tables"), ("factors", "BFree"), ("MMAs", "KqFull"), ("MMAs", "Parts"),
    ("MMAs", "XFree"), ("MMAs", "BFull"), ("MMAs", "RParts"), ("rows", "GateFull"), ("rows", "First"), ("rows", "Second"),
    ("states", "First"),
])
def test_every_wait_is_needed(without):
    """The model finds what goes wrong without it."""
    with pytest.raises(Wrong):
        for m in models(400, without):
            m.run()
