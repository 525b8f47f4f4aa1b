"""Requests that grow when blocks run short, and hold their partial last blocks together with
others at lengths of their own: nobody is granted a token in a block that others still hold.
Against a form that takes one sequence after the other and decides by what the counts and the
free blocks are at its turn, and by what every request reads of its own tokens afterwards."""
import numpy as np
import pytest
import torch

import paged_kv_cache_98_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
NO_BLOCKS = 0x10


@pytest.fixture(scope="module", autouse=True)
def _library():
    from paged_kv_cache_98_gb300 import _build
    _build.build()
    pkv.load()
    torch.cuda.init()


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, torch.int32)


def blocks(n):
    return -(-n // 16)


def counts_of(tables, lens, pool):
    counts = np.zeros(pool, np.int64)
    for t, n in zip(tables, lens):
        np.add.at(counts, t[:blocks(n)], 1)
    return counts


def by_turns(tables, counts, rows, cached, new, num_new):
    """Blocks behind the new lengths go back; then each sequence in batch order takes what it
    needs of the free ones: a copy of a partial last block whose count is above 1 now, and what
    it opens.  After the first that does not get all of it nobody gets any."""
    tables, counts = tables.astype(np.int64), counts.astype(np.int64)
    for i, r in enumerate(rows):
        if r >= 0:
            for b in range(blocks(new[i]), blocks(cached[i])):
                counts[tables[r, b]] -= 1
                tables[r, b] = -1
    free, at, short = np.flatnonzero(counts == 0), 0, False
    granted, opened, pairs = np.zeros(len(rows), np.int64), [], np.full((len(rows), 2), -1)
    for i, r in enumerate(rows):
        if r < 0:
            continue
        granted[i] = new[i]
        if new[i] <= cached[i]:
            continue
        last = cached[i] // 16
        copy = cached[i] % 16 != 0 and counts[tables[r, last]] > 1
        want = copy + blocks(new[i]) - blocks(cached[i])
        if want and (short or at + want > len(free)):
            granted[i], short = cached[i], True
            continue
        if copy:
            pairs[i] = tables[r, last], free[at]
            counts[tables[r, last]] -= 1
        for b, e in zip(range(blocks(cached[i]) - copy, blocks(new[i])), free[at:at + want]):
            tables[r, b], counts[e] = e, 1
            if b >= blocks(cached[i]):
                opened.append(e)
        at += want
    return tables, counts, granted, np.array((opened + [-1] * num_new)[:num_new]), pairs, NO_BLOCKS * short


def resize(tables, counts, rows, cached, new, num_new):
    S, err = len(rows), torch.zeros(1, dtype=torch.int32, device=DEV)
    t = [ints(tables), ints(counts), ints(rows), ints(cached), ints(new), ints(np.full(S, -5)),
         ints(np.full(num_new, -5)), ints(np.full((S, 2), -5))]
    pkv.resize_requests(*t, device_errors=err)
    return [t[i].cpu().numpy() for i in (0, 1, 5, 6, 7)] + [pkv.check_errors(err)]


class Pool:
    """Requests with tokens of their own: what a program that writes granted tokens has left."""

    def __init__(self, tables, lens, pool, seed=0):
        self.r = np.random.RandomState(seed)
        self.tables, self.lens = tables.astype(np.int64), lens.astype(np.int64)
        self.counts = counts_of(tables, lens, pool)
        self.cache = self.r.randint(1 << 30, size=(pool, 16))
        self.want = [self.read(i) for i in range(len(lens))]

    def read(self, i):
        return self.cache[self.tables[i, :blocks(self.lens[i])]].reshape(-1)[:self.lens[i]].copy()

    def step(self, rows, new, num_new=4096):
        """A call, its copies, and the new tokens written; everything checked."""
        rows, new = np.asarray(rows), np.asarray(new)
        cached = np.where(rows >= 0, self.lens[rows], 0)
        got = resize(self.tables, self.counts, rows, cached, new, num_new)
        for g, w in zip(got, by_turns(self.tables, self.counts, rows, cached, new, num_new)):
            np.testing.assert_array_equal(g, w)
        self.tables, self.counts, granted, _, pairs, flags = got
        for src, dst in pairs:
            if src >= 0:
                self.cache[dst] = self.cache[src]
        live = rows >= 0
        self.lens[rows[live]] = granted[live]
        for i, r in enumerate(rows):
            if r < 0:
                continue
            fresh = self.r.randint(1 << 30, size=max(0, granted[i] - cached[i]))
            for j, x in enumerate(fresh):
                b = self.tables[r, (cached[i] + j) // 16]
                assert self.counts[b] == 1, (i, b)        # nobody else's
                self.cache[b, (cached[i] + j) % 16] = x
            self.want[r] = np.concatenate([self.want[r][:granted[i]], fresh])
        for i, w in enumerate(self.want):
            np.testing.assert_array_equal(self.read(i), w)
        np.testing.assert_array_equal(self.counts, counts_of(self.tables, self.lens, len(self.counts)))
        return granted, flags


@pytest.mark.parametrize("lens,new", [((5, 3), (6, 4)), ((12, 9), (14, 11)), ((3, 5), (4, 6)), ((15, 1), (16, 16)),
                                      ((4, 4), (5, 5)), ((28, 21), (29, 22)), ((9, 9, 2), (10, 10, 3))])
def test_holders_of_one_block_and_no_free_one(lens, new):
    """All of them would grow, the last one without a block: none does."""
    n = blocks(lens[0])
    p = Pool(np.tile(np.r_[np.arange(n), -1], (len(lens), 1)), np.array(lens), n)
    granted, flags = p.step(np.arange(len(lens)), new)
    assert granted.tolist() == list(lens) and flags == NO_BLOCKS
    # nor with the batch the other way round, one call after the other
    granted, flags = p.step(np.arange(len(lens))[::-1], new[::-1])
    assert granted.tolist() == list(lens[::-1]) and flags == NO_BLOCKS


def test_equal_holders_in_two_orders():
    """(A, B), then (B, A), with one free block in between: one of them moves, then the other has
    the block for itself."""
    p = Pool(np.zeros((2, 1), int), np.array([12, 12]), 1)
    assert p.step([0, 1], [13, 13])[0].tolist() == [12, 12]
    p.cache, p.counts = np.concatenate([p.cache, [[0] * 16]]), np.append(p.counts, 0)
    assert p.step([1, 0], [14, 14])[0].tolist() == [14, 14]
    assert p.step([0, 1], [16, 16])[0].tolist() == [16, 16]


@pytest.mark.parametrize("free", [0, 1, 2, 3])
def test_keepers_before_and_behind_the_shortage(free):
    """Three blocks with two holders each, of which the second ones need no block: they grow as long
    as the first ones got their copies.  Then one alone in its block, which grows in any case,
    one that shrinks and one that opens a block."""
    tables = np.array([[0, -1], [0, -1], [1, -1], [1, -1], [2, -1], [2, -1], [3, -1], [4, -1], [5, -1]])
    p = Pool(tables, np.array([5, 3, 7, 7, 2, 9, 4, 11, 16]), 6 + free)
    granted, flags = p.step(np.arange(9), [6, 4, 8, 8, 3, 10, 5, 1, 17])
    want = [[5, 3, 7, 7, 2, 9], [6, 4, 7, 7, 2, 9], [6, 4, 8, 8, 2, 9], [6, 4, 8, 8, 3, 10]][free]
    assert granted.tolist() == want + [5, 1, 16] and flags == NO_BLOCKS


@pytest.mark.parametrize("S,pool,spread", [(12, 90, 1.0), (60, 400, 1.0), (500, 3000, 1.0), (60, 40000, 0.0),
                                           (700, 9000, 1.0), (3000, 30000, 1.0)])
@pytest.mark.parametrize("seed", range(3))
def test_groups_at_lengths_of_their_own(S, pool, spread, seed):
    """Groups of one to five requests with the same blocks and last blocks cut to other lengths, in any
    batch order, some idle or shrinking, and free blocks for a part of what they need: by one CTA
    and by a cluster.  Three calls, then more blocks."""
    r = np.random.RandomState(100 * S + seed)
    width, R = 5, S + 5
    group = np.repeat(np.arange(R), r.randint(1, 6, R))[:R]
    full = r.randint(0, 4, R)[group]                   # blocks before the last one
    lens = 16 * full + r.randint(1, 16, R)
    lens[r.rand(R) < 0.05] = 0
    # entries in use spread over the whole pool, or at its front
    ids, tables, used = r.permutation(pool) if spread else np.arange(pool), np.full((R, width), -1), 0
    for g in np.unique(group):
        n = int(full[group == g].max()) + 1
        tables[group == g, :n] = ids[used:used + n]
        used += n
    tables = np.where(np.arange(width) < blocks(lens)[:, None], tables, -1)
    p = Pool(tables, lens, pool, seed)
    # free blocks for about a third of the needs: others hold the rest
    idle = np.flatnonzero(p.counts == 0)
    held = r.permutation(idle)[S // 3:]
    extra = np.full((len(held), width), -1)
    extra[:, 0] = held
    p = Pool(np.concatenate([p.tables, extra]), np.concatenate([lens, np.ones(len(held), int)]), pool, seed)
    short = 0
    for it in range(3):
        rows = r.permutation(R)[:S]
        now = p.lens[rows]
        new = np.minimum(now + r.choice([0, 1, 1, 2, 9, 20], S), 16 * width)
        new = np.where(r.rand(S) < 0.1, (now * r.rand(S)).astype(int), new)
        rows = np.where(r.rand(S) < 0.05, -1, rows)
        if it == 2:                                    # some of the others leave
            gone = R + np.arange(len(held))[::2]
            p.step(gone[:16384], np.zeros(len(gone[:16384]), int))
        short += p.step(rows, new)[1] == NO_BLOCKS
    assert short >= 1
