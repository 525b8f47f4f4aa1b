"""Requests whose block lists live on the GPU (fork, resize) and moves in the caches of all
layers (copies, compaction), against plain implementations that take one sequence, block
and token after the other.  Everything here is whole numbers and bytes: equal."""
import numpy as np
import pytest
import torch

import paged_kv_cache_98_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
BLOCK_ID, CONTEXT, NO_BLOCKS, SHARED = 0x1, 0x2, 0x10, 0x20


@pytest.fixture(scope="module", autouse=True)
def _library():
    from paged_kv_cache_98_gb300 import _build
    _build.build()
    pkv.load()
    torch.cuda.init()


def word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def ints(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dtype)


def blocks(n):
    return -(-n // 16)


# ---- fork ------------------------------------------------------------------------------------

def plain_fork(out, tables, lens, counts, parents):
    out, counts, cap = out.copy(), counts.copy(), tables.shape[1] * 16
    lens_out, nb = np.zeros(len(parents), np.int64), len(counts)
    lens = np.clip(lens, 0, cap)
    for i, p in enumerate(parents):
        if 0 <= p < len(lens):
            n = blocks(lens[p])
            lens_out[i], out[i, :n] = lens[p], tables[p, :n]
            for b in tables[p, :n]:
                if 0 <= b < nb:
                    counts[b] += 1
    for p, n in enumerate(lens):
        for b in tables[p, :blocks(n)]:
            if 0 <= b < nb:
                counts[b] -= 1
    return out, lens_out, counts


def counts_of(tables, lens, pool):
    counts = np.zeros(pool, np.int64)
    for t, n in zip(tables, lens):
        np.add.at(counts, t[:blocks(n)], 1)
    return counts


def run_fork(out, tables, lens, counts, parents, err=None, **kw):
    t = [ints(x) for x in (out, np.zeros(len(parents)), tables, lens, counts, parents)]
    pkv.fork_requests(*t, device_errors=err, **kw)
    return [t[i].cpu().numpy() for i in (0, 1, 4)]


@pytest.mark.parametrize("n_in,n_out,width,most", [
    (1, 1, 1, 16), (3, 5, 7, 100), (64, 64, 129, 2064), (5, 9, 2500, 40000), (40, 0, 9, 100),
    (0, 4, 9, 1), (1300, 1500, 5, 80), (5000, 3, 3, 48), (3, 4100, 33, 500), (6, 6, 4097, 65552),
])
def test_fork(n_in, n_out, width, most):
    r = np.random.RandomState(n_in + n_out)
    lens = r.randint(0, most + 1, n_in)
    pool = max(1, int(blocks(lens).sum()) // 2 + 3)
    tables = r.randint(0, pool, (n_in, width))
    counts = counts_of(tables, lens, pool)
    out = np.full((n_out, width), -7)
    parents = r.randint(-1, max(n_in, 1), n_out) if n_in else np.full(n_out, -1)
    err = word()
    got = run_fork(out, tables, lens, counts, parents, err)
    want = plain_fork(out, tables, lens, counts, parents)
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g, w)
    np.testing.assert_array_equal(got[2], counts_of(want[0], want[1], pool))  # what they are said to be
    assert pkv.check_errors(err) == 0


def test_fork_of_everything_into_one_and_of_one_into_everything():
    r = np.random.RandomState(3)
    lens, tables = np.array([31, 0, 2500, 16]), r.permutation(4 * 160).reshape(4, 160)
    counts = counts_of(tables, lens, 640)
    for parents in (np.zeros(3000, int) + 2, np.array([1]), np.array([-1]), np.array([3, -1, -1, 0])):
        out = np.full((len(parents), 160), -1)
        for g, w in zip(run_fork(out, tables, lens, counts, parents), plain_fork(out, tables, lens, counts, parents)):
            np.testing.assert_array_equal(g, w)


def test_fork_flags():
    r = np.random.RandomState(4)
    tables = r.randint(0, 30, (4, 6))
    out = np.full((3, 6), -1)
    for what, bits in (("parent", CONTEXT), ("long", CONTEXT), ("negative", CONTEXT), ("entry", BLOCK_ID),
                       ("dropped entry", BLOCK_ID)):
        t, lens, parents = tables.copy(), np.array([90, 5, 40, 96]), np.array([2, 0, 2])
        if what == "parent":
            parents[1] = 4
        if what == "long":
            lens[0] = 97
        if what == "negative":
            lens[2] = -3
        if what == "entry":
            t[0, 5], t[2, 0] = 30, -1
        if what == "dropped entry":
            t[1, 0] = 1 << 30
        counts, err = np.full(30, 50), word()
        for g, w in zip(run_fork(out, t, lens, counts, parents, err), plain_fork(out, t, lens, counts, parents)):
            np.testing.assert_array_equal(g, w)
        assert pkv.check_errors(err) == bits


# ---- resize ----------------------------------------------------------------------------------

def plain_resize(tables, counts, rows, cached, new, num_new):
    """The definition, sequence by sequence; the copies by what is left at each one's turn."""
    tables, counts = tables.copy().astype(np.int64), counts.copy().astype(np.int64)
    S, cap, nb, flags = len(rows), tables.shape[1] * 16, len(counts), 0
    ok = [0 <= rows[i] < len(tables) and 0 <= cached[i] <= cap and 0 <= new[i] <= cap for i in range(S)]
    if any(not o and rows[i] >= 0 for i, o in enumerate(ok)):
        flags |= CONTEXT
    for i in range(S):
        if ok[i]:
            for b in range(blocks(new[i]), blocks(cached[i])):
                e, tables[rows[i], b] = tables[rows[i], b], -1
                if 0 <= e < nb:
                    counts[e] -= 1
                else:
                    flags |= BLOCK_ID
    free = np.flatnonzero(counts == 0)
    # holders that grow, in batch order; the last of a block whose holders all do keeps it
    holders = {}
    for i in range(S):
        if ok[i] and new[i] > cached[i] and cached[i] % 16:
            e = int(tables[rows[i], cached[i] // 16])
            if 0 <= e < nb:
                holders.setdefault(e, []).append(i)
            else:
                flags |= BLOCK_ID
    copies = {i: e for e, h in holders.items() if counts[e] > 1
              for i in (h[:-1] if len(h) == counts[e] else h)}
    granted, opened, pairs, at = np.zeros(S, np.int64), [], np.full((S, 2), -1, np.int64), 0
    for i in range(S):
        if not ok[i]:
            continue
        granted[i] = new[i]
        want = max(0, blocks(new[i]) - blocks(cached[i])) + (i in copies)
        if want and at + want > len(free):
            granted[i], at, flags = cached[i], 1 << 60, flags | NO_BLOCKS
            continue
        if i in copies:
            pairs[i] = copies[i], free[at]
            counts[copies[i]] -= 1
            counts[free[at]] = 1
            tables[rows[i], cached[i] // 16] = free[at]
            at += 1
        for b in range(blocks(cached[i]), blocks(new[i])):
            tables[rows[i], b] = free[at]
            counts[free[at]] = 1
            opened.append(free[at])
            at += 1
    if len(opened) > num_new:
        flags |= BLOCK_ID
    opened = np.array((opened + [-1] * num_new)[:num_new], np.int64)
    return tables, counts, granted, opened, pairs, flags


def run_resize(tables, counts, rows, cached, new, num_new, offset=0):
    S, err = len(rows), word()
    c = ints(np.concatenate([np.zeros(offset), counts]))[offset:]
    t = [ints(tables), c, ints(rows), ints(cached), ints(new), ints(np.full(S, -5)),
         ints(np.full(num_new, -5)), ints(np.full((S, 2), -5))]
    pkv.resize_requests(*t, device_errors=err)
    return [t[i].cpu().numpy() for i in (0, 1, 5, 6, 7)] + [pkv.check_errors(err)]


def same(got, want):
    for g, w in zip(got[:-1], want[:-1]):
        np.testing.assert_array_equal(g, w)
    assert got[-1] == want[-1]


def requests(r, S, width, pool, group=3, spare=3):
    """Requests in groups that share the front of their block lists, and the counts."""
    R = S + spare
    cached = np.repeat(r.randint(0, width * 16 + 1, -(-R // group)), group)[:R]
    tables, ids, at = np.full((R, width), -1), r.permutation(pool), 0
    for g0 in range(0, R, group):
        n = blocks(cached[g0])
        alike = r.randint(0, n + 1) if r.rand() < 0.5 else n
        for row in range(g0, min(R, g0 + group)):
            if row == g0:
                tables[row, :n] = ids[at:at + n]
                at += n
            else:
                tables[row, :alike] = tables[g0, :alike]
                tables[row, alike:n] = ids[at:at + n - alike]
                at += n - alike
    assert at <= pool
    rows = r.permutation(R)[:S]
    return tables, counts_of(tables, cached, pool), rows, cached[rows]


@pytest.mark.parametrize("S,width,pool,grow,shrink", [
    (1, 1, 5, 3, 0.0), (5, 4, 60, 20, 0.3), (64, 20, 2500, 1, 0.0), (64, 20, 2500, 64, 0.9),
    (100, 33, 7001, 200, 0.4), (1000, 9, 20000, 30, 0.3), (3000, 40, 200000, 17, 0.5),
])
@pytest.mark.parametrize("offset", [0, 1])
def test_resize(S, width, pool, grow, shrink, offset):
    r = np.random.RandomState(S + grow)
    tables, counts, rows, cached = requests(r, S, width, pool)
    new = np.minimum(cached + r.randint(0, grow + 1, S), width * 16)
    new = np.where(r.rand(S) < shrink, (cached * r.rand(S)).astype(int), new)
    rows = np.where(r.rand(S) < 0.1, -1, rows)
    n = int(np.maximum(blocks(new) - blocks(cached), 0).sum()) + 5
    want = plain_resize(tables, counts, rows, cached, new, n)
    same(run_resize(tables, counts, rows, cached, new, n, offset), want)
    assert want[-1] == 0 and (S < 60 or grow != 1 or (want[4][:, 0] >= 0).any())


@pytest.mark.parametrize("S,group", [(16384, 1), (16384, 5), (9000, 9000), (8193, 2)])
def test_resize_of_very_many(S, group):
    """One request a place, two in some threads; shared last blocks all over, or one shared by all."""
    r = np.random.RandomState(S)
    pool, width = 3 * S + 10, 4
    ids, owner = r.permutation(pool), np.arange(S) // group
    tables = np.full((S, width), -1)
    tables[:, 0] = ids[owner]
    cached = np.full(S, 7)
    counts = counts_of(tables, cached, pool)
    new = cached + r.choice([1, 9, 10, 25], S)
    if group == 9000:
        new[17] = 7                       # one holder that does not grow: everybody copies
    rows = r.permutation(S)
    n = int((blocks(new) - 1).sum())
    same(run_resize(tables, counts, rows, cached, new, n), plain_resize(tables, counts, rows, cached, new, n))


def test_resize_when_blocks_run_out():
    """Those that still fit are served in order; the first that does not, and all behind it that
    need blocks, stay as they are; those that need none still grow."""
    r = np.random.RandomState(9)
    for pool_free in (0, 1, 2, 5, 9, 40):
        S, width = 12, 6
        tables = np.arange(S * width).reshape(S, width)
        cached = np.array([16, 10, 32, 5, 48, 17, 1, 16, 33, 10, 80, 0])
        new = np.array([17, 12, 90, 5, 30, 18, 40, 33, 34, 96, 96, 16])
        tables[1, 0] = tables[9, 0]       # a shared partial block
        pool = S * width + pool_free
        counts = np.ones(pool, int)
        counts[S * width:] = 0
        counts[tables[9, 0]] = 2
        perm = r.permutation(pool)
        want = plain_resize(perm[tables], counts[np.argsort(perm)], np.arange(S), cached, new, 9)
        same(run_resize(perm[tables], counts[np.argsort(perm)], np.arange(S), cached, new, 9), want)
        assert bool(want[-1] & NO_BLOCKS) == (pool_free < 20)


def test_resize_flags():
    r = np.random.RandomState(10)
    tables, counts, rows, cached = requests(r, 8, 6, 90)
    base = np.where(cached > 40, cached - 20, np.minimum(cached + 20, 96))
    for what in ("row", "cached", "new", "negative", "gone", "tail", "list"):
        t, c, rw, ca, nw, n = tables.copy(), counts.copy(), rows.copy(), cached.copy(), base.copy(), 40
        if what == "row":
            rw[2] = len(tables)
        if what == "cached":
            ca[1] = 97
        if what == "new":
            nw[0] = 97
        if what == "negative":
            nw[0] = -1
        if what == "gone":
            ca[3], nw[3] = 60, 20
            t[rw[3], 2] = 90
        if what == "tail":
            ca[4], nw[4] = 20, 30
            t[rw[4], 1] = -3
        if what == "list":
            n = 1
        want = plain_resize(t, c, rw, ca, nw, n)
        same(run_resize(t, c, rw, ca, nw, n), want)
        assert want[-1] != 0, what


def test_resize_no_new_list_and_no_sequences():
    z = torch.zeros(0, dtype=torch.int32, device=DEV)
    new_blocks = ints(np.full(5, 3))
    pkv.resize_requests(ints(np.zeros((2, 3))), ints(np.zeros(9)), z, z, z, z, new_blocks, z.view(0, 2))
    assert (new_blocks == -1).all()
    tables, counts = ints(np.array([[4, -1, -1]])), ints(np.arange(9) == 4)
    granted, pairs = ints([0]), ints([[0, 0]])
    pkv.resize_requests(tables, counts, ints([0]), ints([16]), ints([0]), granted, z, pairs)
    assert tables.tolist() == [[-1, -1, -1]] and counts.tolist() == [0] * 9 and granted.item() == 0


# ---- copies and compaction -------------------------------------------------------------------

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def caches(layers, nb, heads, d, kind, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n = layers * 2 * nb * heads * 16 * d * (1 if kind == "e4m3" else 2)
    return torch.randint(0, 256, (n,), generator=g, device=DEV, dtype=torch.uint8).view(DT[kind]).view(
        layers, 2, nb, heads, 16, d)


def raw(x):
    return x.view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("layers,heads,d,kind,listed", [
    (1, 1, 64, "e4m3", False), (3, 8, 128, "bf16", True), (2, 5, 64, "f16", False), (130, 1, 64, "f16", True),
    (2, 40, 128, "bf16", False),
])
def test_copy_layers(layers, heads, d, kind, listed):
    x = caches(layers, 23, heads, d, kind)
    r = np.random.RandomState(layers)
    ids = r.permutation(23)
    pairs = np.stack([ids[r.randint(0, 10, 9)], ids[10:19]], 1)
    pairs[[1, 5]] = -1
    pairs[7] = -1, 4                      # a negative source: nothing, whatever the destination
    want, err = raw(x), word()
    for s, t in pairs:
        if s >= 0:
            want[:, :, t] = want[:, :, s]
    k, v = ([y[0] for y in x], [y[1] for y in x]) if listed else (x[:, 0], x[:, 1])
    pkv.copy_blocks_layers(k, v, ints(pairs), device_errors=err)
    np.testing.assert_array_equal(raw(x), want)
    assert pkv.check_errors(err) == 0
    pkv.copy_blocks_layers(k, v, ints([[3, 23], [23, 2], [1, -1]]), device_errors=err)
    np.testing.assert_array_equal(raw(x), want)
    assert pkv.check_errors(err) == BLOCK_ID


def plain_compact(x, tables, ctx, base, starts, keep, counts):
    """Token by token, in ascending order; x: [layers, 2, nb, heads, 16, row bytes]."""
    nb, cap, flags = x.shape[2], tables.shape[1] * 16, 0
    new = np.zeros(len(ctx), np.int64)
    for s in range(len(ctx)):
        k0, k1 = starts[s], starts[s + 1]
        new[s] = np.clip(ctx[s], 0, cap)
        if not (0 <= ctx[s] <= cap and 0 <= base[s] <= ctx[s] and 0 <= k0 <= k1 <= len(keep)):
            flags |= CONTEXT
            continue
        mine = keep[k0:k1]
        if np.any(np.diff(np.concatenate([[base[s] - 1], mine])) <= 0) or np.any(mine >= ctx[s]):
            flags |= CONTEXT
            continue
        to = {int(base[s] + j) // 16 for j, p in enumerate(mine) if p != base[s] + j}
        if counts is not None and any(0 <= tables[s, b] < nb and counts[tables[s, b]] > 1 for b in to):
            flags |= SHARED
            continue
        new[s] = base[s] + len(mine)
        for j, p in enumerate(mine):
            t = base[s] + j
            if t == p:
                continue
            a, b = tables[s, p // 16], tables[s, t // 16]
            if not (0 <= a < nb and 0 <= b < nb):
                flags |= BLOCK_ID
                continue
            x[:, :, b, :, t % 16] = x[:, :, a, :, p % 16]
    return x, new, flags


def run_compact(x, tables, ctx, base, starts, keep, counts):
    err, new = word(), ints(np.full(len(ctx), -5))
    pkv.compact_tokens(x[:, 0], x[:, 1], ints(tables), ints(ctx), ints(base), ints(starts), ints(keep), new,
                       ref_counts=None if counts is None else ints(counts), device_errors=err)
    return raw(x), new.cpu().numpy(), pkv.check_errors(err)


def lists(r, S, most, tail, share):
    ctx = r.randint(0, most + 1, S)
    base = np.maximum(ctx - tail, 0) if tail else r.randint(0, ctx + 1)
    keep = [b + np.flatnonzero(r.rand(c - b) < share) for b, c in zip(base, ctx)]
    width = max(1, blocks(most))
    tables = r.permutation(S * width + 5)[:S * width].reshape(S, width)
    return tables, ctx, base, np.concatenate([[0], np.cumsum([len(k) for k in keep])]), np.concatenate(keep)


@pytest.mark.parametrize("layers,heads,d,kind", [(1, 1, 64, "e4m3"), (2, 3, 64, "f16"), (2, 2, 128, "bf16"),
                                                 (1, 2, 128, "e4m3"), (129, 1, 64, "e4m3")])
@pytest.mark.parametrize("S,most,tail,share", [(1, 1, 0, 0.5), (7, 64, 64, 0.1), (5, 333, 64, 0.5),
                                               (3, 700, 0, 0.97), (2, 1500, 2000, 0.5), (4, 100, 0, 0.0)])
def test_compact(layers, heads, d, kind, S, most, tail, share):
    if layers > 2 and most > 400:
        pytest.skip("many layers with short contexts only")
    r = np.random.RandomState(S + most)
    tables, ctx, base, starts, keep = lists(r, S, most, tail, share)
    x = caches(layers, tables.size + 5, heads, d, kind, seed=S)
    want = plain_compact(raw(x), tables, ctx, base, starts, keep, None)
    got = run_compact(x, tables, ctx, base, starts, keep, np.ones(tables.size + 5))
    np.testing.assert_array_equal(got[0], want[0])
    np.testing.assert_array_equal(got[1], want[1])
    assert got[2] == want[2] == 0


def test_blocks_past_32_bits():
    """Copies and moves between the first and the last blocks of caches of more than 2^32 elements."""
    nb, heads, d = (1 << 32) // (8 * 16 * 128) + 600, 8, 128
    x = torch.empty(1, 2, nb, heads, 16, d, dtype=torch.float16, device=DEV)
    small = caches(1, 12, heads, d, "f16", seed=3)
    ids = np.array([0, 1, 2, 3, 4, 5] + [nb - i for i in range(6, 0, -1)])
    at = ints(ids).long()
    x[:, :, at] = small
    pairs = np.array([[0, 11], [10, 1], [3, 6]])
    pkv.copy_blocks_layers(x[:, 0], x[:, 1], ints(ids[pairs]))
    tables = np.array([[2, 9, 8, 4], [5, 7, 10, 0]])
    ctx, base, starts = np.array([64, 60]), np.array([3, 0]), np.array([0, 20, 50])
    keep = np.concatenate([np.arange(20) * 3 + 4, np.arange(30) * 2])
    new = ints([0, 0])
    pkv.compact_tokens(x[:, 0], x[:, 1], ints(ids[tables]), ints(ctx), ints(base), ints(starts), ints(keep), new)
    want = raw(small)
    for a, b in pairs:
        want[:, :, b] = want[:, :, a]
    want = plain_compact(want, tables, ctx, base, starts, keep, None)
    np.testing.assert_array_equal(raw(x[:, :, at].contiguous()), want[0])
    np.testing.assert_array_equal(new.cpu().numpy(), want[1])


@pytest.mark.parametrize("d,kind", [(64, "e4m3"), (64, "f16"), (128, "e4m3"), (128, "bf16")])
@pytest.mark.parametrize("S,layers,heads,most", [
    (20, 8, 5, 150),     # lists of tens of tokens and many units: a warp moves one
    (12, 8, 5, 400),     # longer lists: a CTA moves one, of whole rows
    (9, 2, 3, 90),       # few units, short lists: a CTA moves 64 bytes of each row
    (1, 1, 1, 30),       # one unit
])
def test_compact_units(S, layers, heads, most, d, kind):
    """Short and long lists in many and few units, several turns each, every row size."""
    r = np.random.RandomState(S + d)
    tables, ctx, base, starts, keep = lists(r, S, most, 0, 0.6)
    ctx[0], base[0] = most, 1
    keep0 = 1 + np.flatnonzero(r.rand(most - 1) < 0.6)
    keep, starts = np.concatenate([keep0, keep[starts[1]:]]), starts + len(keep0) - starts[1]
    starts[0] = 0
    x = caches(layers, tables.size + 5, heads, d, kind, seed=S)
    want = plain_compact(raw(x), tables, ctx, base, starts, keep, None)
    got = run_compact(x, tables, ctx, base, starts, keep, np.ones(tables.size + 5))
    np.testing.assert_array_equal(got[0], want[0])
    np.testing.assert_array_equal(got[1], want[1])
    assert got[2] == want[2] == 0


@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("what", ["twice", "falls", "early", "late", "context", "base", "starts", "shared",
                                  "shared but in place", "source block", "place's block"])
def test_compact_flags(what, long):
    """A sequence that is not as it should be stays as it was, the others move."""
    r = np.random.RandomState(8)
    S, most = 5, 900 if long else 90
    tables, ctx, base, starts, keep = lists(r, S, most, 0, 0.5)
    ctx[:], base[:] = most - 3, 10
    mine = [10 + np.sort(r.permutation(most - 13)[:(most - 13) // 2 + i]) for i in range(S)]
    mine[2][:12] = 10 + np.arange(12)     # (the first ones are in place)
    mine[2] = np.unique(mine[2])
    keep, starts = np.concatenate(mine), np.concatenate([[0], np.cumsum([len(k) for k in mine])])
    counts, at = np.ones(tables.size + 5, int), starts[2]
    n2 = starts[3] - at
    if what == "twice":
        keep[at + 20] = keep[at + 19]
    if what == "falls":
        keep[at + 20] = keep[at + 18]
    if what == "early":
        keep[at] = 9
    if what == "late":
        keep[starts[3] - 1] = ctx[2]
    if what == "context":
        ctx[2] = tables.shape[1] * 16 + 1
    if what == "base":
        base[2] = ctx[2] + 1
    if what == "starts":
        starts[2], starts[3] = starts[3], starts[2]    # (its list and its neighbours' are no lists)
    if what == "shared":
        counts[tables[2, (10 + n2 - 1) // 16]] = 2
    if what == "shared but in place":
        counts[tables[2, 0]] = 2
    if what == "source block":
        tables[2, (most - 5) // 16] = -1
    if what == "place's block":
        tables[2, 2] = 1 << 29
    x = caches(2, tables.size + 5 if what != "place's block" else S * blocks(most) + 5, 2, 64, "f16")
    want = plain_compact(raw(x), tables, ctx, base, starts, keep, counts)
    got = run_compact(x, tables, ctx, base, starts, keep, counts)
    np.testing.assert_array_equal(got[0], want[0])
    np.testing.assert_array_equal(got[1], want[1])
    assert got[2] == want[2]
    assert (got[2] != 0) == (what != "shared but in place")


# ---- streams, graphs, a run of them ------------------------------------------------------------

def test_calls_on_another_stream():
    r = np.random.RandomState(12)
    tables, counts, rows, cached = requests(r, 40, 8, 700)
    new = np.minimum(cached + 9, 128)
    want = plain_resize(tables, counts, rows, cached, new, 60)
    side = torch.cuda.Stream()
    t = [ints(x) for x in (tables, counts, rows, cached, new, np.zeros(40), np.zeros(60), np.zeros((40, 2)))]
    x = caches(2, 700, 2, 64, "f16")
    bytes_ = raw(x)
    side.wait_stream(torch.cuda.current_stream())
    pkv.resize_requests(*t, stream=side)
    pkv.copy_blocks_layers(x[:, 0], x[:, 1], t[7], stream=side)
    side.synchronize()
    same([t[i].cpu().numpy() for i in (0, 1, 5, 6, 7)] + [0], want)
    for s, d in want[4]:
        if s >= 0:
            bytes_[:, :, d] = bytes_[:, :, s]
    np.testing.assert_array_equal(raw(x), bytes_)


def test_beam_steps_in_a_graph():
    """Beam search of three requests: fork by the parents, one token more, shared last blocks
    copied, the token's K and V written by the step's maps; captured once, replayed with other
    parents.  Every beam's tokens, read through its table, are those it should have; the
    counts are what the tables say."""
    r = np.random.RandomState(13)
    B, W, MB, NB, steps, start = 3, 4, 8, 90, 40, 21
    n, d = B * W, 64
    i32 = dict(dtype=torch.int32, device=DEV)
    tables = [torch.full((n, MB), -1, **i32) for _ in range(2)]
    lens = [torch.zeros(n, **i32) for _ in range(2)]
    counts, err = torch.zeros(NB, **i32), word()
    rows, parents, grown, granted = torch.arange(n, **i32), torch.zeros(n, **i32), torch.zeros(n, **i32), torch.zeros(n, **i32)
    opened, pairs = torch.zeros(n, **i32), torch.zeros((n, 2), **i32)
    kc, vc = (torch.zeros((2, NB, 1, 16, d), dtype=torch.float16, device=DEV) for _ in range(2))
    bt, ctx, qsl = torch.zeros((n, MB), **i32), torch.zeros(n, **i32), torch.zeros(n + 1, **i32)
    slots, pos, one = torch.zeros(n, dtype=torch.int64, device=DEV), torch.zeros(n, **i32), torch.ones(n, **i32)
    tokens = torch.zeros((n, 1, d), dtype=torch.float16, device=DEV)

    # the prompts: one row of each request takes its blocks, the beams are forked from it
    many = torch.zeros(n * MB, **i32)
    first = torch.tensor([start if i % W == 0 else 0 for i in range(n)], **i32)
    pkv.resize_requests(tables[0], counts, rows, lens[0], first, lens[1], many, pairs, device_errors=err)
    lens[0].copy_(lens[1])
    history = [[] for _ in range(n)]
    for i in range(0, n, W):
        history[i] = [float(100 + i)] * start
        for t in range(start):
            b = int(tables[0][i, t // 16])
            kc[:, b, :, t % 16] = 100 + i
            vc[:, b, :, t % 16] = -100 - i
    parents.copy_(torch.arange(n, **i32) // W * W)

    def step(a, b):
        pkv.fork_requests(tables[b], lens[b], tables[a], lens[a], counts, parents, device_errors=err)
        torch.add(lens[b], 1, out=grown)
        pkv.resize_requests(tables[b], counts, rows, lens[b], grown, granted, opened, pairs, device_errors=err)
        pkv.copy_blocks_layers(kc, vc, pairs, device_errors=err)
        pkv.build_step_maps(bt, ctx, qsl, slots, pos, tables[b], rows, lens[b], one, opened, NB, device_errors=err)
        for l in range(2):
            pkv.reshape_and_cache(tokens, -tokens, kc[l], vc[l], slots, device_errors=err)
        lens[b].copy_(granted)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    saved = [t.clone() for t in (tables[0], tables[1], lens[0], lens[1], counts, kc, vc)]
    step(0, 1)                            # (sets up what a first call sets up)
    for t, s in zip((tables[0], tables[1], lens[0], lens[1], counts, kc, vc), saved):
        t.copy_(s)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(0, 1)
        step(1, 0)                        # (with the same parents: the second goes on from the first)
    for it in range(steps // 2):
        p = parents.cpu().tolist()
        tok = torch.arange(n, dtype=torch.float16) + 200 + 16 * it
        tokens.copy_(tok.view(n, 1, 1).expand(n, 1, d))
        graph.replay()
        for _ in range(2):
            history = [history[p[i]] + [float(tok[i])] for i in range(n)]
        parents.copy_(torch.tensor([int(i // W * W + r.randint(W)) for i in range(n)], **i32))
    torch.cuda.synchronize()
    assert pkv.check_errors(err) == 0
    t, l = tables[0].cpu().numpy(), lens[0].cpu().numpy()
    assert (l == start + 2 * (steps // 2)).all()
    np.testing.assert_array_equal(counts.cpu().numpy(), counts_of(t, l, NB))
    for i in range(n):
        for x, sign in ((kc, 1), (vc, -1)):
            for layer in range(2):
                got = x[layer, t[i, :blocks(l[i])], 0, :, 5].reshape(-1)[:l[i]].cpu().numpy()
                np.testing.assert_array_equal(got, sign * np.array(history[i], np.float16))
    # freed by a fork that names nobody
    pkv.fork_requests(tables[1], lens[1], tables[0], lens[0], counts, torch.full((n,), -1, **i32))
    assert (counts == 0).all() and (lens[1] == 0).all()
