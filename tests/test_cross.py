"""Host side of cross attention: refusals before anything is launched, the workspace, what the
binding bounds and holds, and the walk of the line of work that the kernel cuts a call into."""
import contextlib

import pytest
import torch

import paged_kv_cache_98_gb300 as pkv
from paged_kv_cache_98_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.load()


def _cross(lib, **over):
    a = dict(out=1 << 20, q=1 << 22, k=1 << 24, v=1 << 25, tables=4096, lens=8192, starts=8448, num_seqs=2,
             total_q=6, max_q=4, heads=8, kv_heads=2, head_dim=128, block_size=16, width=8, num_blocks=64,
             max_enc=100, scale=0.1, q_dtype=1, kv_dtype=1, k_scale=1.0, v_scale=1.0, ws=None, ws_bytes=0,
             errors=None, stream=None)
    a.update(over)
    return lib.pkv_paged_attention_cross(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(out=None), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(tables=None), -1),
    (dict(lens=None), -1), (dict(starts=None), -1), (dict(num_seqs=-1), -1), (dict(total_q=-1), -1),
    (dict(max_q=-1), -1), (dict(max_enc=-1), -1), (dict(heads=0), -1), (dict(kv_heads=0), -1),
    (dict(heads=9), -1), (dict(width=0), -1), (dict(num_blocks=0), -1), (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1), (dict(out=(1 << 20) + 8), -1), (dict(q=(1 << 22) + 2), -1),
    (dict(tables=4098), -1), (dict(lens=8193), -1), (dict(starts=8450), -1), (dict(errors=1), -1),
    # over q, into the caches
    (dict(out=1 << 22), -1), (dict(out=(1 << 22) + 6 * 8 * 256 - 16), -1), (dict(out=(1 << 24) + 16), -1),
    (dict(k=(1 << 20) + 16), -1),
    (dict(head_dim=96), -2), (dict(block_size=32), -2), (dict(heads=34), -2), (dict(q_dtype=2), -2),
    (dict(kv_dtype=0), -2), (dict(width=1 << 27), -2), (dict(num_blocks=1 << 27), -2),
    (dict(num_blocks=(1 << 31) - 1, kv_heads=8), -2), (dict(total_q=1 << 28), -2),
    (dict(kv_dtype=2, k_scale=0.0), -1), (dict(kv_dtype=2, v_scale=float("inf")), -1),
    # inputs that may be cut need the workspace
    (dict(max_enc=129), -3), (dict(max_enc=129, ws=1 << 26, ws_bytes=4096), -3),
    (dict(max_enc=129, ws=(1 << 26) + 16, ws_bytes=1 << 30), -1),
])
def test_refusals(lib, over, status):
    assert _cross(lib, **over) == status


def test_nothing_to_do(lib):
    none = dict(out=None, q=None, tables=None, lens=None, starts=None)
    assert _cross(lib, num_seqs=0, **none) == 0
    assert _cross(lib, total_q=0, max_enc=1000, **none) == 0
    assert _cross(lib, max_q=0) == 0
    assert _cross(lib, num_seqs=0, head_dim=96, **none) == -2  # other arguments are still looked at


def test_workspace_size():
    size = lambda **k: pkv.cross_workspace_size(**{**dict(  # noqa: E731
        num_seqs=4, total_q=40, num_heads=8, num_kv_heads=2, head_dim=128, max_encoder_len=1000, max_q_len=10), **k})
    rows = 2 * 152 * 10 * 4               # two partials a processor, of the rows of ten tokens
    assert size() == 2 * 152 * 16 + rows * 4 + rows * 128 * 4
    assert size(max_encoder_len=128) == 0  # one key tile: nothing is cut
    rows = 2 * 152 * 32 * 4
    assert size(max_q_len=32) == 2 * 152 * 16 + rows * 4 + rows * 128 * 4
    rows = 2 * 152 * 256
    assert size(max_q_len=33) == size(max_q_len=40) == 2 * 152 * 16 + rows * 4 + rows * 128 * 4
    assert size(max_q_len=4000) == size(max_q_len=40)  # no sequence has more than all rows
    for k in (dict(num_seqs=0), dict(total_q=0), dict(max_q_len=0), dict(num_heads=9), dict(num_heads=40),
              dict(num_kv_heads=0), dict(head_dim=0), dict(max_encoder_len=0)):
        assert size(**k) == 0
    assert size(total_q=(1 << 31) - 1, max_q_len=(1 << 31) - 1, max_encoder_len=(1 << 31) - 1) == size(max_q_len=40)


def _args():
    t = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    return dict(out=t(6, 8, 128), q=t(6, 8, 128), k_cache=t(9, 2, 16, 128), v_cache=t(9, 2, 16, 128),
                block_tables=torch.zeros(2, 5, dtype=torch.int32), encoder_lens=torch.zeros(2, dtype=torch.int32),
                query_start_loc=torch.tensor([0, 4, 6], dtype=torch.int32), scale=0.1)


def test_left_out_bounds_read_nothing_back(monkeypatch):
    seen = {}

    class Lib:
        @staticmethod
        def pkv_cross_workspace_size(*a):
            return 0

        @staticmethod
        def pkv_paged_attention_cross(*a):
            seen.update(seqs=a[7], rows=a[8], max_q=a[9], max_enc=a[16])
            return 0

    def read(*a, **k):
        raise AssertionError("a device value was read")
    monkeypatch.setattr(pkv, "_stream_on", lambda device, stream, tensors: (7, contextlib.nullcontext()))
    monkeypatch.setattr(pkv, "_lib", Lib())
    monkeypatch.setattr(torch.Tensor, "item", read)
    pkv.paged_attention_cross(**_args())
    assert seen == dict(seqs=2, rows=6, max_q=6, max_enc=80)
    pkv.paged_attention_cross(**_args(), max_q_len=4, max_encoder_len=70)
    assert seen == dict(seqs=2, rows=6, max_q=4, max_enc=70)


def test_empty_through_the_binding(monkeypatch):
    _build.build()
    monkeypatch.setattr(pkv, "_stream_on", lambda device, stream, tensors: (7, contextlib.nullcontext()))
    a = _args()
    a.update(out=a["out"][:0], q=a["q"][:0], query_start_loc=torch.zeros(3, dtype=torch.int32))
    assert pkv.paged_attention_cross(**a, max_encoder_len=0).shape[0] == 0
    a.update(block_tables=a["block_tables"][:0], encoder_lens=a["encoder_lens"][:0],
             query_start_loc=a["query_start_loc"][:1])
    assert pkv.paged_attention_cross(**a, max_encoder_len=0).shape[0] == 0


# ---- the line of work -------------------------------------------------------------------------
# The cuts in integers, as the kernel takes them: every key tile of every unit in exactly one
# part, the parts of a cut unit one after the other, each with a tile, and the last of them
# the one that the first one names.

COST1, COST2, UNIT, LEAST, CTAS = 4, 6, 14, 8, 152


def _walk(seqs, hkv, rpt):
    """{part: [(unit, first tile, last tile + 1, names the unit's last part)]}, and the units."""
    work = lambda q, n: hkv * n * ((-(-q // rpt) >> 1) * COST2 + (-(-q // rpt) & 1) * COST1)  # noqa: E731
    count = lambda q: hkv * ((-(-q // rpt) + 1) >> 1)  # noqa: E731
    tiles = [(q, -(-e // 128)) for q, e in seqs]
    once = max(min(sum(work(*t) for t in tiles) // (2 * CTAS), UNIT), 1)
    start = [0]
    for q, n in tiles:
        start.append(start[-1] + work(q, n) + once * count(q))
    T = start[-1]
    parts = max(min(CTAS, T // LEAST), 1)
    got, units = {}, {}
    for s, (q, n) in enumerate(tiles):
        t = -(-q // rpt)
        for k in range(count(q)):
            units[s, k] = n
    for part in range(CTAS):
        w, w1 = (T * part // parts, T * (part + 1) // parts) if part < parts else (0, 0)
        s = max((i for i in range(len(seqs)) if start[i] <= w), default=0)
        while w < w1:
            q, n = tiles[s]
            t = -(-q // rpt)
            u2, u1, twos, off = n * COST2 + once, n * COST1 + once, hkv * (t >> 1), w - start[s]
            two = off < twos * u2
            k = off // u2 if two else twos + (off - twos * u2) // u1
            u0 = start[s] + (k * u2 if two else twos * u2 + (k - twos) * u1)
            u, cost = (u2, COST2) if two else (u1, COST1)
            at = lambda x: 0 if x - u0 - once <= 0 else min(-(-(x - u0 - once) // cost), n)  # noqa: E731
            a, b, begins = 0 if w <= u0 else at(w), n if w1 >= u0 + u else at(w1), w <= u0
            w, unit = u0 + u, (s, k)
            while s + 1 < len(seqs) and start[s + 1] <= w:
                s += 1
            if a >= b and not (n == 0 and begins):
                continue
            last = None
            if a == 0 and b < n:
                p = u0 + once + (n - 1) * cost
                last = -(-((p + 1) * parts) // T) - 1
            got.setdefault(part, []).append((unit, a, b, last))
    return got, units


@pytest.mark.parametrize("seed", range(60))
def test_line_of_work(seed):
    import random
    r = random.Random(seed)
    hkv, rpt = r.choice([1, 2, 8, 16]), r.choice([8, 9, 32, 128])
    S = r.choice([1, 2, 5, 30])
    most = r.choice([1, 100, 3000, 100000])
    seqs = [(r.choice([0, 1, rpt, rpt + 1, r.randint(0, 7 * rpt)]), r.choice([0, 1, 128, 129, r.randint(0, most)]))
            for _ in range(S)]
    got, units = _walk(seqs, hkv, rpt)
    seen, where = {}, {}
    for part, items in got.items():
        cut = 0
        for i, (unit, a, b, last) in enumerate(items):
            assert a < b or (a == b == 0 == units[unit])
            seen.setdefault(unit, []).append((a, b))
            where.setdefault(unit, []).append((part, last))
            if (a, b) != (0, units[unit]):
                # at most a first partial (a > 0) and a second one (a == 0) for each part
                assert (i == 0) if a > 0 else (i == len(items) - 1)
                cut += 1
        assert cut <= 2
    assert set(seen) == set(units)
    for unit, runs in seen.items():
        assert sorted(runs) == runs and runs[0][0] == 0 and runs[-1][1] == units[unit]
        assert all(x[1] == y[0] for x, y in zip(runs, runs[1:]))
        parts = [p for p, _ in where[unit]]
        assert parts == list(range(parts[0], parts[0] + len(parts)))
        if len(parts) > 1:
            assert where[unit][0][1] == parts[-1]
