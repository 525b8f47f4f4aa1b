"""Step maps and rotary positions with the cache write on the GPU, against plain
64-bit implementations.

Tolerances.  Maps are whole numbers: equal.  A rotated element is u = a c - b s
with c, s in fp32 (an error of at most 2^-22 each: the fraction of a turn is
rounded to 2^-25 turns, 2^-22.3 radians, and sincospif adds 2 ulp) and two fp32
roundings, so it is off by at most (|a| + |b|) f 2^-21 before the one rounding of
the output, half a step: 2^-8 |u| in bf16, 2^-11 |u| in fp16 (2^-25 below its
normal range); an E4M3 code stands for a value within 2^-4 |x / scale| or half
its smallest step, 2^-10.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_98_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


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


# ---- step maps -------------------------------------------------------------------------------

def plain_maps(bt, tables, rows, cached, q, new, num_tokens, num_blocks):
    """The definition, one sequence and one token at a time."""
    S, bt, tables = len(rows), bt.copy(), tables.copy()
    ctx, qsl = np.zeros(S, np.int64), np.zeros(S + 1, np.int64)
    slots, pos = np.full(num_tokens, -1, np.int64), np.full(num_tokens, -1, np.int64)
    at = 0
    for s in range(S):
        c, n = (int(cached[s]), int(q[s])) if rows[s] >= 0 else (0, 0)
        ctx[s], qsl[s + 1] = c + n, min(qsl[s] + n, num_tokens)
        have, need = -(-c // 16), -(-(c + n) // 16)
        for b in range(have, need):
            tables[rows[s], b] = new[at] if at < len(new) else -1
            at += 1
        if need:
            bt[s, :need] = tables[rows[s], :need]
        for i in range(n):
            t, p = qsl[s] + i, c + i
            if t < num_tokens:
                b = tables[rows[s], p // 16]
                slots[t] = b * 16 + p % 16 if 0 <= b < num_blocks else -1
                pos[t] = p
    return bt, ctx, qsl, slots, pos, tables


def batch(r, S, table, max_q, zero_q=0.2):
    q = np.where(r.rand(S) < zero_q, 0, r.randint(1, max_q + 1, S))
    cached = np.minimum(r.randint(0, table * 16, S), table * 16 - q)
    have, need = -(-cached // 16), -(-(cached + q) // 16)
    nb = int(need.sum()) + 7
    ids, rows = r.permutation(nb), r.permutation(S + 3)[:S]
    tables = np.full((S + 3, table), -9, np.int64)
    new, at = [], 0
    for s in range(S):
        tables[rows[s], :have[s]] = ids[at:at + have[s]]
        new += list(ids[at + have[s]:at + need[s]])
        at += need[s]
    return tables, rows, cached, q, np.array(new, np.int64), nb


def run_maps(tables, rows, cached, q, new, nb, num_tokens, err=None, stream=None):
    S, table = len(rows), tables.shape[1]
    out = [torch.full((S, table), -5, dtype=torch.int32, device=DEV),
           torch.full((S,), -5, dtype=torch.int32, device=DEV),
           torch.full((S + 1,), -5, dtype=torch.int32, device=DEV),
           torch.full((num_tokens,), -5, dtype=torch.int64, device=DEV),
           torch.full((num_tokens,), -5, dtype=torch.int32, device=DEV), ints(tables)]
    args = [ints(x) for x in (rows, cached, q, new)]
    torch.cuda.synchronize()
    pkv.build_step_maps(*out, *args, nb, device_errors=err, stream=stream)
    return out, args


def check_maps(out, tables, rows, cached, q, new, nb, num_tokens):
    bt = np.full((len(rows), tables.shape[1]), -5, np.int64)
    for got, want in zip(out, plain_maps(bt, tables, rows, cached, q, new, num_tokens, nb)):
        np.testing.assert_array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("S,table,max_q,room", [
    (1, 1, 1, 0), (1, 1, 16, 3), (3, 5, 40, 0), (8, 64, 1, 9), (33, 17, 100, 1), (256, 9, 30, 0),
    (257, 300, 20, 5), (1000, 40, 64, 100), (7001, 3, 5, 0), (16384, 2, 2, 1), (2, 8192, 5000, 7)])
def test_maps(S, table, max_q, room):
    r = np.random.RandomState(S + table)
    b = batch(r, S, table, max_q)
    T = int(b[3].sum()) + room
    err = word()
    out, _ = run_maps(*b, T, err)
    check_maps(out, *b, T)
    assert pkv.check_errors(err) == 0


def test_maps_without_sequences_or_tokens():
    b = batch(np.random.RandomState(0), 4, 3, 5)
    out, _ = run_maps(b[0], b[1][:0], b[2][:0], b[3][:0], b[4], b[5], 6)
    check_maps(out, b[0], b[1][:0], b[2][:0], b[3][:0], b[4], b[5], 6)
    q0 = 0 * b[3]
    out, _ = run_maps(b[0], b[1], b[2], q0, b[4][:0], b[5], 0)
    check_maps(out, b[0], b[1], b[2], q0, b[4][:0], b[5], 0)


def test_maps_padding_rows_and_bad_inputs():
    r = np.random.RandomState(5)
    tables, rows, cached, q, new, nb = batch(r, 40, 8, 30, zero_q=0.0)
    keep = r.rand(40) < 0.6
    # padding sequences anywhere: their lengths, whatever they are, count for nothing
    have, need = -(-cached // 16), -(-(cached + q) // 16)
    owner = np.repeat(np.arange(40), need - have)
    pad_rows, pad_new = np.where(keep, rows, -1), new[keep[owner]]
    T, err = int(q[keep].sum()) + 4, word()
    out, _ = run_maps(tables, pad_rows, cached, q, pad_new, nb, T, err)
    check_maps(out, tables, pad_rows, cached, q, pad_new, nb, T)
    assert pkv.check_errors(err) == 0
    # a row past the tables, negative lengths, a context past the table: padding, and flagged
    for change in (dict(rows=len(tables)), dict(cached=-1), dict(q=-3), dict(q=2 ** 31 - 1),
                   dict(cached=2 ** 31 - 1), dict(cached=8 * 16)):
        v = dict(rows=rows.copy(), cached=cached.copy(), q=q.copy())
        (name, value), = change.items()
        v[name][7] = value
        good = np.arange(40) != 7
        want_rows, want_new = np.where(good, rows, -1), new[good[owner]]
        T = int(q[good].sum())
        out, _ = run_maps(tables, v["rows"], v["cached"], v["q"], want_new, nb, T, err)
        check_maps(out, tables, want_rows, cached, q, want_new, nb, T)
        assert pkv.check_errors(err) == 2
    # every length at its largest: the sums pass 32 bits, and nothing is written out of place
    big = np.full(40, 8 * 16)
    out, _ = run_maps(tables, rows, 0 * cached, big, new, nb, 50, err)
    check_maps(out, tables, rows, 0 * cached, big, new, nb, 50)
    assert pkv.check_errors(err) & 2
    # the list of new blocks runs out; an id outside the pool
    T = int(q.sum())
    out, _ = run_maps(tables, rows, cached, q, new[:-3], nb, T, err)
    check_maps(out, tables, rows, cached, q, new[:-3], nb, T)
    assert pkv.check_errors(err) == 1
    wrong = new.copy()
    wrong[len(wrong) // 2] = nb
    out, _ = run_maps(tables, rows, cached, q, wrong, nb, T, err)
    check_maps(out, tables, rows, cached, q, wrong, nb, T)
    assert pkv.check_errors(err) == 1
    # queries cut off at num_tokens
    out, _ = run_maps(tables, rows, cached, q, new, nb, T - 5, err)
    check_maps(out, tables, rows, cached, q, new, nb, T - 5)
    assert pkv.check_errors(err) == 2


def test_maps_twice_on_a_side_stream_and_in_a_graph():
    r = np.random.RandomState(9)
    a, b = batch(r, 30, 12, 20), batch(r, 30, 12, 20)
    T = int(max(a[3].sum(), b[3].sum())) + 2
    s = torch.cuda.Stream()
    out, args = run_maps(*a, T, stream=s)
    s.synchronize()
    check_maps(out, *a, T)
    # captured, then replayed on another batch of the same size written in place
    nb, room = max(a[5], b[5]), max(len(a[4]), len(b[4]))
    new = torch.zeros(room, dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pkv.build_step_maps(*out, *args[:3], new, nb)
    out[5].copy_(ints(b[0]))
    for dst, src in zip(args[:3], b[1:4]):
        dst.copy_(ints(src))
    new[:len(b[4])] = ints(b[4])
    out[0].fill_(-5)
    g.replay()
    torch.cuda.synchronize()
    check_maps(out, *b[:4], b[4], nb, T)
    # the same step once more changes nothing
    g.replay()
    torch.cuda.synchronize()
    check_maps(out, *b[:4], b[4], nb, T)


def test_maps_feed_on_the_pool():
    """Blocks that the host pool hands out, step by step, through the device maps."""
    pool, table, R = pkv.BlockPool(400), 20, 6
    reqs, lens = [pool.request() for _ in range(R)], np.zeros(R, np.int64)
    tables = torch.full((R, table), -1, dtype=torch.int32, device=DEV)
    r = np.random.RandomState(2)
    for step in range(12):
        rows = r.permutation(R)[:r.randint(1, R + 1)]
        q = r.randint(0, 25, len(rows))
        slots, new = [], []
        for row, n in zip(rows, q):
            had = len(reqs[row].block_table())
            sl, cow = reqs[row].append(list(r.randint(0, 1000, n))) if n else ([], None)
            assert cow is None
            slots += list(sl)
            new += list(reqs[row].block_table()[had:])
        S, T = len(rows), len(slots)
        out = [torch.zeros((S, table), dtype=torch.int32, device=DEV),
               torch.empty(S, dtype=torch.int32, device=DEV),
               torch.empty(S + 1, dtype=torch.int32, device=DEV),
               torch.empty(T, dtype=torch.int64, device=DEV),
               torch.empty(T, dtype=torch.int32, device=DEV)]
        pkv.build_step_maps(*out, tables, ints(rows), ints(lens[rows]), ints(q),
                            ints(np.array(new, np.int64)), 400)
        lens[rows] += q
        bt, cl = pool.block_tables([reqs[i] for i in rows], table)
        np.testing.assert_array_equal(out[0].cpu().numpy(), bt)
        np.testing.assert_array_equal(out[1].cpu().numpy(), cl)
        np.testing.assert_array_equal(out[3].cpu().numpy(), slots)
        lens_now = [x.num_tokens for x in reqs]
        np.testing.assert_array_equal(lens, lens_now)
    pool.close()


# ---- rotary ----------------------------------------------------------------------------------

TD = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF_STEP = {torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float16: (2.0 ** -11, 2.0 ** -25),
             torch.float8_e4m3fn: (2.0 ** -4, 2.0 ** -10)}


def plain_rotary(x, pos, inv, layout, factor):
    """(rotated [T, H, D] float64, bound of the fp32 error) of x."""
    x = x.double().cpu()
    half = len(inv)
    ang = pos.cpu().double()[:, None] * torch.from_numpy(inv)
    c, s = factor * torch.cos(ang)[:, None], factor * torch.sin(ang)[:, None]
    i = torch.arange(half)
    ia, ib = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
    a, b = x[..., ia], x[..., ib]
    out, off = x.clone(), torch.zeros_like(x)
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    off[..., ia] = off[..., ib] = (a.abs() + b.abs()) * abs(factor) * 2.0 ** -21
    return out, off


def near(got, want, off, what):
    rel, low = HALF_STEP[got.dtype]
    got = got.double().cpu()
    bound = off * (1 + rel) + rel * want.abs() + low
    bad = (got - want).abs() > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, first {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("dtype,kv,layout,T,H,hkv,D,rot,fused,far,factor", [
    ("bf16", "same", "half", 1, 8, 2, 128, 128, False, 0, 1.0),
    ("bf16", "same", "half", 7, 4, 4, 64, 64, True, 131072, 1.0),
    ("fp16", "same", "interleaved", 33, 8, 2, 128, 64, True, 1000000, 1.25),
    ("fp16", "same", "half", 65, 14, 2, 128, 96, True, 2000, 1.0),
    ("bf16", "same", "half", 19, 3, 1, 128, 6, False, 5000, 1.0),
    ("fp16", "same", "half", 5, 3, 1, 64, 62, True, 5000, -0.5),
    ("bf16", "same", "interleaved", 16, 5, 5, 64, 2, False, 5000, 1.0),
    ("fp16", "same", "interleaved", 40, 2, 1, 128, 126, True, 2 ** 30, 1.0),
    ("bf16", "e4m3", "half", 50, 8, 2, 128, 128, True, 131072, 1.1),
    ("fp16", "e4m3", "half", 21, 6, 3, 64, 20, False, 9000, 1.0),
    ("fp16", "e4m3", "interleaved", 64, 16, 1, 128, 32, True, 9000, 1.0),
    ("bf16", "same", "half", 1301, 64, 8, 128, 128, True, 131072, 1.0),
    ("bf16", "e4m3", "interleaved", 1217, 8, 8, 128, 128, True, 131072, 1.0),
])
def test_rotary(dtype, kv, layout, T, H, hkv, D, rot, fused, far, factor):
    g = torch.Generator(device=DEV).manual_seed(T * H + rot)
    r = np.random.RandomState(T + rot)
    td = TD[dtype]
    row = (H + 2 * hkv) * D + 8 * (T % 3)  # the projection's rows may be padded
    qkv = torch.randn((T, row), generator=g, device=DEV).to(td)
    q, k, v = (qkv[:, a:a + n * D].unflatten(1, (n, D))
               for a, n in ((0, H), (H * D, hkv), ((H + hkv) * D, hkv)))
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    nb = -(-T // 16) + 3
    slots = r.permutation(nb * 16)[:T].astype(np.int64)
    pos = np.maximum(far - 1 - r.permutation(T), 0)
    slots[T // 2] = -1 if T > 4 else slots[T // 2]        # rotated, not cached
    if T > 10:
        pos[T // 3], slots[T // 5] = -1, nb * 16          # padding; a slot past the pool
    inv = np.array([500000.0 ** (-2 * i / rot) for i in range(rot // 2)])
    ct = td if kv == "same" else torch.float8_e4m3fn
    ks, vs = (0.013, 0.011) if kv == "e4m3" else (1.0, 1.0)
    bits = torch.uint8 if kv == "e4m3" else torch.int16
    kc, vc = (torch.full((nb, hkv, 16, D), 77, dtype=bits, device=DEV).view(ct) for _ in range(2))
    out, err = torch.full((T, H, D), 3.0, dtype=td, device=DEV), word()
    pkv.rotary_and_cache(out, q, k, v, kc, vc, ints(slots, torch.int64), ints(pos), inv, layout, factor,
                         ks, vs, device_errors=err)
    assert pkv.check_errors(err) == (4 if T > 10 else 0)
    p = torch.from_numpy(pos)
    live = p >= 0
    want, off = plain_rotary(q, p.clamp(min=0), inv, layout, factor)
    near(out[live.to(DEV)], want[live], off[live], "q")
    assert torch.equal(out[~live.to(DEV)], torch.full_like(out[~live.to(DEV)], 3.0))
    wk, ok = plain_rotary(k, p.clamp(min=0), inv, layout, factor)
    at = live & torch.from_numpy((slots >= 0) & (slots < nb * 16))
    sl = torch.from_numpy(slots)[at]
    for cache, w, o, scale, what in ((kc, wk, ok, ks, "k"), (vc, v.double().cpu(), 0 * ok, vs, "v")):
        flat = cache.view(bits).transpose(1, 2).reshape(nb * 16, hkv, D)
        got = flat[sl.to(DEV)].view(ct)
        near(got, (w[at] / scale).clamp(-448, 448) if kv == "e4m3" else w[at], o[at] / scale, what)
        # nothing else is touched
        rest = torch.ones(nb * 16, dtype=torch.bool)
        rest[sl] = False
        assert bool((flat[rest.to(DEV)] == 77).all()), what
    # bits that only pass are copied
    if kv == "same":
        flat = vc.view(bits).transpose(1, 2).reshape(nb * 16, hkv, D)
        assert torch.equal(flat[sl.to(DEV)], v[at.to(DEV)].contiguous().view(bits))
    assert torch.equal(out[live.to(DEV)][..., rot:], q[live.to(DEV)][..., rot:])


def test_rotary_in_place_on_a_stream_and_in_a_graph():
    T, H, hkv, D = 37, 8, 2, 128
    g = torch.Generator(device=DEV).manual_seed(4)
    q, k, v = (torch.randn((T, n, D), generator=g, device=DEV).to(torch.bfloat16) for n in (H, hkv, hkv))
    inv, attn = pkv.rotary_frequencies(D, 10000.0, "yarn", 4.0, 1.0, 32.0, 4096)
    kc, vc = (torch.zeros((3, hkv, 16, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    slots, pos = torch.arange(T, device=DEV), torch.arange(100, 100 + T, dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    pkv.rotary_and_cache(out, q, k, v, kc, vc, slots, pos, inv, "half", attn)
    same, kc2, vc2 = q.clone(), torch.zeros_like(kc), torch.zeros_like(vc)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    pkv.rotary_and_cache(same, same, k, v, kc2, vc2, slots, pos, inv, "half", attn, stream=s)
    s.synchronize()
    assert torch.equal(same, out) and torch.equal(kc2, kc) and torch.equal(vc2, vc)
    graph = torch.cuda.CUDAGraph()
    out2 = torch.zeros_like(q)
    with torch.cuda.graph(graph):
        pkv.rotary_and_cache(out2, q, k, v, kc2, vc2, slots, pos, inv, "half", attn)
    inv[:] = 0.0  # read during the call
    pos += 7
    graph.replay()
    torch.cuda.synchronize()
    inv, _ = pkv.rotary_frequencies(D, 10000.0, "yarn", 4.0, 1.0, 32.0, 4096)
    pkv.rotary_and_cache(out, q, k, v, kc, vc, slots, pos, inv, "half", attn)
    assert torch.equal(out2, out) and torch.equal(kc2, kc) and torch.equal(vc2, vc)


def test_rotary_keeps_infinities_and_nan_in_their_pairs():
    q = torch.ones((1, 1, 64), dtype=torch.float16, device=DEV)
    q[0, 0, 3], q[0, 0, 40] = float("nan"), float("inf")
    k = torch.full((1, 1, 64), 1.0, dtype=torch.float16, device=DEV)
    kc, vc = (torch.zeros((1, 1, 16, 64), dtype=torch.float16, device=DEV) for _ in range(2))
    out = torch.empty_like(q)
    pkv.rotary_and_cache(out, q, k, k, kc, vc, torch.zeros(1, dtype=torch.int64, device=DEV),
                         torch.ones(1, dtype=torch.int32, device=DEV), np.full(32, 0.5))
    odd = ~torch.isfinite(out[0, 0]).cpu()
    assert odd.nonzero().flatten().tolist() == [3, 8, 35, 40]
