"""Infinities and NaN in the K and V that some rows of a biased attention call see and
others do not, against a plain 64-bit softmax.

An output element sum_j w_j v_j whose row sees a v_j that is not finite is the infinity
of their sign, or NaN (the weights are positive): compared as such.  All others are
within the bounds of test_gpu_biased.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_98_gb300 as pkv
from test_gpu_biased import DEV, Batch, Decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    from paged_kv_cache_98_gb300 import _build
    _build.build()
    pkv.load()
    torch.cuda.init()


def plant(b, what):
    """Sets V (which "v") or K ("k") of tokens: what is a list of (which, sequence, token,
    dimensions, value); in an E4M3 cache every such value is its NaN."""
    for name, cache, host in (("v", b.vc, b.v), ("k", b.kc, b.k)):
        mine = [w for w in what if w[0] == name]
        if not mine:
            continue
        flat = cache.cpu().clone()
        for _, s, tok, dims, value in mine:
            if b.kv == "e4m3":
                flat.view(torch.uint8)[int(b.tables[s, tok // 16]), :, tok % 16, dims] = 0x7F
                host[s][tok, :, dims] = math.nan
            else:
                flat[int(b.tables[s, tok // 16]), :, tok % 16, dims] = value
                host[s][tok, :, dims] = value
        cache.copy_(flat)


def check(b, got):
    want, bound = b.plain()
    got = got.double().cpu()
    finite = torch.isfinite(want)
    assert not finite.all() and finite.any()
    off = (got - want).abs()
    bad = ~(off <= bound) & finite
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} elements, first {bad.nonzero()[0].tolist()}"
    odd = ~finite
    same = (torch.isnan(got) & torch.isnan(want)) | (got == want)
    assert same[odd].all(), (odd & ~same).nonzero()[0].tolist()


def twice(b):
    """Called two times: the same bits."""
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got, again = b.call(errors=err), b.call(errors=err)
    assert pkv.check_errors(err) == 0
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))
    return got


KINDS = [math.inf, -math.inf, math.nan]


@pytest.mark.parametrize("kw", [
    dict(H=8, hkv=2), dict(H=8, hkv=2, window=50), dict(H=8, hkv=8, D=64, alibi=True, dtype="fp16"),
    dict(H=14, hkv=2, softcap=9.0), dict(H=8, hkv=2, kv="e4m3", dtype="fp16", window=70),
    dict(H=4, hkv=2, D=64, kv="e4m3"), dict(H=16, hkv=1, softcap=9.0, alibi=True, window=33),
    dict(H=8, hkv=2, prefix=[100, 130])],
    ids=lambda k: "-".join(f"{a}{b if isinstance(b, (int, str, float)) else ''}" for a, b in k.items()))
def test_hidden_and_visible(kw):
    """Tokens whose V is not finite in some dimensions, in documents of their own and in
    others' sight: before, inside and behind the rows of an item."""
    starts = None if "window" in kw or "prefix" in kw else lambda s, p: max([0] + [c for c in (70, 140, 290) if c <= p])
    b = Batch(101, [(200, 200), (20, 300), (150, 400)][:2 if "prefix" in kw else 3], starts=starts, **kw)
    D = b.D
    what = [("v", 0, 3, slice(0, 5), math.inf), ("v", 0, 69, slice(4, D), -math.inf), ("v", 0, 71, [7, D - 1], math.nan),
            ("v", 0, 150, slice(2, 3), math.inf), ("v", 0, 150, slice(9, 10), -math.inf),
            ("v", 1, 289, slice(0, D, 3), math.inf), ("v", 1, 299, slice(1, 2), math.nan)]
    if "prefix" not in kw:
        what += [("v", 2, 255, slice(0, D), math.nan), ("v", 2, 333, slice(D // 2, D), math.inf)]
    lo = np.concatenate(b.lo)
    what = [w for w in what if not (w[1] == 1 and w[2] < lo[200])]  # (blocks that are in no table)
    plant(b, what)
    check(b, twice(b))


@pytest.mark.parametrize("kw", [dict(H=8, hkv=8), dict(H=8, hkv=8, D=64, alibi=True, dtype="fp16"),
                                dict(H=8, hkv=8, kv="e4m3", softcap=9.0)],
                         ids=lambda k: "-".join(k))
def test_more_odd_items_than_a_processor_lists(kw):
    """Six thousand items, every one with rows that a hidden V would reach and rows that see
    it: a processor lists as many as it can and leaves the others of the grid alone."""
    r = np.random.RandomState(5)
    lens = [int(x) for x in r.randint(12, 24, 800)]
    b = Batch(103, [(n, n) for n in lens], starts=lambda s, p: 9 if p >= 9 else 0, **kw)
    plant(b, [("v", s, 4, slice(s % 7, b.D, 7), KINDS[s % 3]) for s in range(800)] +
             [("v", s, 10, slice(s % 5, b.D, 11), KINDS[s % 2]) for s in range(0, 800, 4)])
    check(b, twice(b))


# ---- which form of the cap --------------------------------------------------------------------

def bits(t):
    return t.view(torch.int16).cpu()


@pytest.mark.parametrize("kw", [dict(H=8, hkv=2), dict(H=14, hkv=2, dtype="fp16"), dict(H=8, hkv=2, kv="e4m3"),
                                dict(H=4, hkv=4, D=64, alibi=True)],
                         ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()))
def test_large_scores_beside_small_ones_under_a_large_cap(kw):
    """One row whose scores pass half a cap of a million; its neighbours' scores are near one
    and keep their own precision."""
    b = Batch(107, [(60, 90), (30, 200)], softcap=1e6, **kw)
    b.q[17] *= 2.0 ** 13 if b.dtype == "fp16" else 2.0 ** 20
    if b.dtype == "fp16":
        b.scale *= 2.0 ** 8
        b.q[:17] *= 2.0 ** -8
        b.q[18:] *= 2.0 ** -8
    got = b.call()
    b.check(got, skip=[17])  # (its own scores are a step of their type apart, which is thousands)
    assert torch.isfinite(got[17].float()).all()


@pytest.mark.parametrize("kw", [dict(H=14, hkv=2, dtype="fp16"), dict(H=8, hkv=2), dict(H=5, hkv=1, D=64, dtype="fp16")],
                         ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()))
def test_neighbours_in_the_batch_choose_nothing(kw):
    """A chunk's bits, with small and with large queries of the sequence after it, and
    after a call that leaves large queries in the processors' memory."""
    b = Batch(113, [(90, 90)] * 8 + [(10, 90), (10, 90)], softcap=30.0, **kw)
    n = int(b.qsl[-2])
    big = Batch(115, [(128, 128)] * 64, H=8, hkv=8, D=b.D, dtype=b.dtype, spread=1e4)
    plain = [bits(b.call())[:n]]
    big.call()
    plain.append(bits(b.call())[:n])
    q = b.q.clone()
    q[n:] *= 1e3
    plain.append(bits(b.call(q=q.to(DEV)))[:n])
    assert torch.equal(plain[0], plain[1]) and torch.equal(plain[0], plain[2])


@pytest.mark.parametrize("cls,kw", [
    (Batch, dict(H=8, hkv=2)), (Batch, dict(H=8, hkv=2, window=50)), (Batch, dict(H=8, hkv=8, D=64, alibi=True)),
    (Batch, dict(H=8, hkv=2, window=70, dtype="fp16")),
    (Decode, dict(H=8, hkv=2, dtype="fp16")), (Decode, dict(H=8, hkv=2, window=50, dtype="fp16")),
    (Decode, dict(H=16, hkv=1, window=50, dtype="fp16")), (Decode, dict(H=4, hkv=4, window=50))],
    ids=lambda k: k.__name__ if isinstance(k, type) else "-".join(f"{a}{b}" for a, b in k.items()))
@pytest.mark.parametrize("value", [math.inf, -1e4])
def test_hidden_scores_choose_nothing(cls, kw, value):
    """K that no row sees, behind the contexts and before the windows, at zero and then not:
    the same bits.  In a chunk also K that only later rows see: the earlier ones' bits."""
    seqs = [(60, 90), (41, 203), (1, 333)] if cls is Batch else [90, 203, 333, 29, *range(101, 700, 13)]
    b = cls(109, seqs, softcap=30.0, **kw)
    later = 40 if cls is Batch else 0  # in the first sequence: seen by its rows from 10 on

    def call(x):
        kc = b.kc.cpu().clone()
        for s, c in enumerate(b.ctx):
            first = int(b.lo[s].min())
            for tok in list(range(first // 16 * 16, first)) + list(range(c, -(-c // 16) * 16)):
                kc[int(b.tables[s, tok // 16]), :, tok % 16] = x
        if later:
            kc[int(b.tables[0, later // 16]), :, later % 16] = x
        b.kc.copy_(kc)
        return bits(b.call())

    zero, odd = call(0.0), call(value)
    rows = [r for r in range(b.rows) if not later or r < 10 or r >= int(b.qsl[1])]
    assert torch.equal(zero[rows], odd[rows])


@pytest.mark.parametrize("kw", [dict(H=6, hkv=2, dtype="fp16"), dict(H=5, hkv=1, dtype="fp16", window=100),
                                dict(H=12, hkv=1, dtype="fp16"), dict(H=5, hkv=1, kv="e4m3", dtype="fp16")],
                         ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()))
def test_heads_past_the_group_choose_nothing(kw):
    """Every other sequence's bits, with small and with large queries of those between: the
    rows of Q that a group leaves free hold the next heads."""
    b = Decode(117, list(range(60, 700, 9)), softcap=30.0, **kw)
    q = b.q.clone()
    q[1::2] *= 1e3
    assert torch.equal(bits(b.call())[::2], bits(b.call(q=q.to(DEV)))[::2])


# ---- scores of minus infinity -------------------------------------------------------------------

def sink(b, s, toks):
    """K of the tokens such that every head's score is -inf: a weight of zero."""
    b.q[:, :, 0] = b.q[:, :, 0].abs() + 0.5
    kc = b.kc.cpu().clone()
    for t in toks:
        kc[int(b.tables[s, t // 16]), :, t % 16, 0] = -math.inf
    b.kc.copy_(kc)


LOW = [dict(H=8, hkv=2), dict(H=8, hkv=2, dtype="fp16", alibi=True), dict(H=16, hkv=1), dict(H=3, hkv=3),
       dict(H=4, hkv=2, D=64, dtype="fp16"), dict(H=14, hkv=2)]


@pytest.mark.parametrize("kw", LOW, ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()))
def test_decode_first_score_is_minus_infinity(kw):
    """As many keys as are recomputed key by key, and more: the others share the weight."""
    b = Decode(121, [2, 20, 32, 33, 34, 513, 1025], **kw)
    for s in range(len(b.ctx)):
        sink(b, s, [0])
        b.lo[s] = b.lo[s] + 1
    b.check(b.call())


@pytest.mark.parametrize("kw", LOW, ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()))
def test_decode_scores_of_a_whole_partition_are_minus_infinity(kw):
    """The last partition's, the first one's: the row is the others'.  All: NaN."""
    b = Decode(123, [513, 1030, 1100, 600], **kw)
    for s, lo, hi in ((0, 0, 512), (1, 0, 1024), (2, 600, 1100)):
        sink(b, s, [t for t in range(b.ctx[s]) if not lo <= t < hi])
        b.lo[s], b.hi[s] = b.lo[s] * 0 + lo, b.hi[s] * 0 + hi
    sink(b, 3, range(600))
    got = b.call()
    b.check(got, skip=[3])
    assert torch.isnan(got[3].float()).all()


@pytest.mark.parametrize("kw", [dict(H=8, hkv=2), dict(H=4, hkv=4, D=64, dtype="fp16", alibi=True)],
                         ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()))
def test_prefill_first_score_is_minus_infinity_in_rows_recomputed(kw):
    b = Batch(125, [(64, 64), (30, 100)], **kw)
    plant(b, [("v", 0, 40, slice(0, b.D, 2), math.inf)])  # hidden from the rows before it
    sink(b, 0, [0])
    b.lo[0] = np.maximum(b.lo[0], 1)
    got = b.call()
    assert torch.isnan(got[0].float()).all()  # it sees that key alone
    got[0] = 0
    check(b, got)
