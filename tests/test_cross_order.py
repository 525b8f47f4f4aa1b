"""The waits of cross attention's issuers, producer and softmax warpgroups on the CPU: barriers that
tell a phase by its parity alone, as the hardware's do, loads that land when they like, products
that run in order but late.  Whatever the order, no one may pass a wait for a load that has
not landed, no product may read a buffer that holds something else, and everyone ends."""
import random

import pytest


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phases = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phases = self.count, self.phases + 1

    def passes(self, parity):
        return self.phases & 1 != parity


class Wrong(Exception):
    pass


class Model:
    """items: (key tiles, two query tiles?).  come: an issuer waits for the producer to have come to
    a tile's place before it waits for the tile, as the kernel does."""

    def __init__(self, items, stages, r, come=True):
        self.items, self.st, self.r, self.come = items, stages, r, come
        self.full, self.empty = [Barrier(1) for _ in range(stages)], [Barrier(2) for _ in range(stages)]
        self.q_full, self.q_empty = [Barrier(1) for _ in range(2)], [Barrier(2) for _ in range(2)]
        for name in ("turn", "s_ready", "p_half", "p_ready", "o_done", "o_free"):
            setattr(self, name, [Barrier(1), Barrier(1)])
        self.other_ready = Barrier(1)
        self.ring, self.q, self.issued = [None] * stages, [None, None], 0
        self.loads, self.mmas = [], ([], [])           # on their way; of each issuer, in order

    # what a thread waits for is a function; the scheduler goes on with it once that is true
    def producer(self):
        pos = nq = 0
        for tiles, two in self.items:
            for _ in range(1 + two):
                b, fill = nq & 1, nq >> 1
                if nq >= 2:
                    yield lambda: self.q_empty[b].passes((fill - 1) & 1)
                self.loads.append((self.q, b, nq, self.q_full[b]))
                nq += 1
            for _ in range(2 * tiles):
                s = pos % self.st
                if pos >= self.st:
                    yield lambda: self.empty[s].passes((pos // self.st - 1) & 1)
                self.loads.append((self.ring, s, pos, self.full[s]))
                pos += 1
                self.issued = pos

    def issuer(self, y):
        base = np = nit = nq = turns = 0
        others = False
        mma = self.mmas[y].append

        def landed(memory, at, what):
            if memory[at] != what:
                raise Wrong(f"issuer {y} took {memory[at]} for {what}")

        def q_wait(n):
            yield lambda: self.q_full[n & 1].passes((n >> 1) & 1)
            landed(self.q, n & 1, n)

        def tile(place):
            at = base + place
            if self.come:
                yield lambda: self.issued > at
            yield lambda: self.full[at % self.st].passes((at // self.st) & 1)
            landed(self.ring, at % self.st, at)
            return at

        for tiles, two in self.items:
            k_place = lambda i: 0 if i == 0 else 2 * i - 1                       # noqa: E731
            v_place = lambda i: 2 * tiles - 1 if i == tiles - 1 else 2 * i + 2   # noqa: E731
            step, first, mine = (1, 0, nq + y) if two else (2, y, nq)
            yield from q_wait(mine)

            def release(at):
                for _ in range(1 if two else 2):
                    mma(("arrive", self.empty[at % self.st]))

            def release_q():
                for n in range(1 + two):
                    mma(("arrive", self.q_empty[(nq + n) & 1]))

            def scores(i):
                at = yield from tile(k_place(i))
                mma(("reads", self.q, mine & 1, mine))
                mma(("reads", self.ring, at % self.st, at))
                mma(("arrive", self.s_ready[y]))
                return at

            if first < tiles:
                release((yield from scores(first)))
            if first + step >= tiles:
                release_q()
            for i in range(first, tiles, step):
                yield lambda: self.p_half[y].passes(np & 1)
                if i == first and nit >= 1:
                    yield lambda: self.o_free[y].passes((nit - 1) & 1)
                v = yield from tile(v_place(i))
                if two and (y == 1 or others):
                    yield lambda: self.turn[y].passes(turns & 1)
                    turns += 1
                others |= two
                mma(("reads", self.ring, v % self.st, v))
                yield lambda: self.p_ready[y].passes(np & 1)
                np += 1
                if i + step < tiles:
                    k = yield from scores(i + step)
                    if two:
                        self.turn[y ^ 1].arrive()
                    release(v)
                    release(k)
                    if i + 2 * step >= tiles:
                        release_q()
                else:
                    if two:
                        self.turn[y ^ 1].arrive()
                    mma(("arrive", self.o_done[y]))
                    release(v)
            nit += first < tiles
            nq += 2 if two else 1
            base += 2 * tiles

    def softmax(self, y):
        ns = nit = nother = 0
        for tiles, two in self.items:
            steps = tiles if two else len(range(y, tiles, 2))
            for _ in range(steps):
                yield lambda: self.s_ready[y].passes(ns & 1)
                ns += 1
                self.p_half[y].arrive()
                yield lambda: True
                self.p_ready[y].arrive()
            if steps == 0:
                continue
            yield lambda: self.o_done[y].passes(nit & 1)
            nit += 1
            join = not two and tiles > 1
            if join and y != (tiles - 1) & 1:
                self.other_ready.arrive()
                nother += 1
                continue
            if join:
                yield lambda: self.other_ready.passes(nother & 1)
                nother += 1
            self.o_free[y].arrive()
            if join:
                self.o_free[y ^ 1].arrive()

    def run(self):
        """In an order of r's: some loads land, and some threads go on, when nobody else can."""
        r, late = self.r, self.r.choice([0.05, 0.3, 0.6])
        threads = [self.producer(), self.issuer(0), self.issuer(1), self.softmax(0), self.softmax(1)]
        waits = [lambda: True] * len(threads)
        lazy = [r.random() < 0.15 for _ in threads]
        slow = [r.random() < 0.3 for _ in range(97)]     # loads, by what they load
        while threads or self.loads or any(self.mmas):
            able = [i for i, w in enumerate(waits) if w()]
            ready = [i for i in able if not lazy[i]]
            events = [("load", i) for i, x in enumerate(self.loads) if not slow[(x[2] + 31 * (x[0] is self.q)) % 97]]
            events += [("mma", y) for y in range(2) if self.mmas[y]]
            if not ready and not events:
                ready, events = able, [("load", i) for i in range(len(self.loads))]
            if ready and (not events or r.random() > late):
                i = r.choice(ready)
                try:
                    waits[i] = next(threads[i])
                except StopIteration:
                    del threads[i], waits[i], lazy[i]
            elif events:
                kind, i = r.choice(events)
                if kind == "load":
                    memory, at, what, bar = self.loads.pop(i)
                    memory[at] = what
                    bar.arrive()
                else:
                    op = self.mmas[i].pop(0)
                    if op[0] == "arrive":
                        op[1].arrive()
                    elif op[1][op[2]] != op[3]:
                        raise Wrong(f"a product read {op[1][op[2]]} for {op[3]}")
            else:
                raise Wrong("nobody can go on")


def _items(r):
    few = r.random() < 0.5
    return [(r.choice([1, 1, 1, 2] if few else [1, 2, 3, 4, 9]), r.random() < 0.5) for _ in range(r.randint(1, 12))]


@pytest.mark.parametrize("stages", [4, 5, 8])
def test_waits_take_their_own_phase(stages):
    """(An issuer never waits for the other's query tile of a pair.  The next tile in that buffer is
    for it behind one that the producer loads when both have given back the pair, each after
    its own tile had landed.)"""
    for seed in range(400):
        r = random.Random(1000 * stages + seed)
        Model(_items(r), stages, r).run()


@pytest.mark.parametrize("stages", [5, 8])
def test_the_model_finds_a_tile_taken_too_early(stages):
    """Units of one query tile whose key tiles only one of the issuers looks at, waited for as soon
    as the issuer has come to them: the phase before the last passes for the last one."""
    wrong = 0
    for seed in range(300):
        r = random.Random(seed)
        try:
            Model([(r.choice([1, 3, 9]), False) for _ in range(12)], stages, r, come=False).run()
        except Wrong:
            wrong += 1
    assert wrong
