"""Decode and prefill attention under score modifiers (capped scores, distance
bias, window, first keys, two-way prefixes) against a plain 64-bit softmax.

Tolerance of an output element o = sum_j w_j v_j, derived from what the kernels
round:
  - the output, half a step u: 2^-8 |o| in bf16, 2^-11 |o| in fp16;
  - the softmax weights, to the matrix instruction's input, half a step each:
    2^-8 (bf16 or two E4M3 terms) or 2^-11 (fp16) of A = sum_j w_j |v_j|; a weight
    far below the row's largest can vanish: 2^-17 of B = sum_j |v_j| / l, l the
    sum of the weights over the largest one;
  - the scores, by at most d, which moves a weight by 2 d relative, so 2 d A:
    fp32 products and sums (D + 8) 2^-24 S, S the row's largest |scale| sum |q||k|
    plus its bias; the cap 2^-19 of the score; exponentials 2^-21; an E4M3 cache's
    fp16 query, split in two E4M3 terms, 2^-8 S (a bf16 one is split exactly, but for
    elements that fall below the codes of a row scaled to at least 224: 2^-17 of the
    row's largest |q| times |scale| sum |k|).
The sums of all three are taken with 1 % for their products.

On the whole the roundings are independent: the output's and the weights' are each
at most u / sqrt(3) of the norm, so the norm of all errors stays below 1.5 u of the
outputs' norm (u of the coarser of the two), where scores are exact to that.  That
catches a weight that lost its low term, which no single element's bound does.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_98_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
TD = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _library():
    from paged_kv_cache_98_gb300 import _build
    _build.build()
    pkv.load()
    torch.cuda.init()


class Batch:
    """Queries and paged caches of sequences (q_len, context), and what they see.

    Every byte of the caches that no row sees is NaN; table entries that no row
    needs are outside the pool."""

    def __init__(self, seed, seqs, H, hkv, D=128, dtype="bf16", kv="same", softcap=0.0, alibi=False,
                 window=0, starts=None, prefix=None, spread=2.0, slack=2):
        g = torch.Generator().manual_seed(seed)
        r = np.random.RandomState(seed)
        self.H, self.hkv, self.D, self.dtype, self.kv = H, hkv, D, dtype, kv
        self.softcap, self.window = softcap, window
        self.q_len = np.array([a for a, _ in seqs])
        self.ctx = np.array([c for _, c in seqs])
        self.qsl = np.concatenate([[0], np.cumsum(self.q_len)])
        self.rows = int(self.qsl[-1])
        self.prefix = None if prefix is None else np.array(prefix)
        self.start = None
        lo, hi = [], []
        for s, (n, c) in enumerate(seqs):
            pos = np.arange(c - n, c)
            a = np.zeros(n, np.int64)
            if starts is not None:
                a = np.array([starts(s, p) for p in pos], np.int64).reshape(n)
            self.start = a if self.start is None else np.concatenate([self.start, a])
            b = pos + 1 if prefix is None else np.maximum(pos + 1, min(prefix[s], c))
            if window:
                a = np.maximum(a, pos - window + 1)
            a = np.maximum(a, 0)
            lo.append(np.minimum(a, b))
            hi.append(b)
        if starts is None:
            self.start = None
        self.lo, self.hi = lo, hi
        need = -(-self.ctx // 16)
        self.nb = int(need.sum()) + 3
        ids = r.permutation(self.nb)
        self.tables = np.full((len(seqs), max(1, int(need.max())) + slack), -7, np.int64)
        kind = torch.float8_e4m3fn if kv == "e4m3" else TD[dtype]
        bits, nan = (torch.uint8, 0x7F) if kv == "e4m3" else (torch.int16, 0x7FFF)
        self.ks, self.vs = (0.011, 0.013) if kv == "e4m3" else (1.0, 1.0)
        cache = [torch.full((self.nb, 16, hkv, D), nan, dtype=bits) for _ in range(2)]
        self.k, self.v, at = [], [], 0
        for s, c in enumerate(self.ctx):
            mine = ids[at:at + need[s]]
            at += need[s]
            kv_s = [torch.randn((c, hkv, D), generator=g) / x for x in (self.ks, self.vs)]
            kv_s = [x.clamp(-448, 448).to(kind) if kv == "e4m3" else x.to(kind) for x in kv_s]
            seen = np.zeros(c, bool)
            for a, b in zip(lo[s], hi[s]):
                seen[a:b] = True
            j = np.nonzero(seen)[0]
            for dst, x in zip(cache, kv_s):
                dst[mine[j // 16], j % 16] = x.view(bits)[j]
            for b in set(j // 16):
                self.tables[s, b] = mine[b]
            self.k.append(kv_s[0].double() * self.ks)
            self.v.append(kv_s[1].double() * self.vs)
        self.kc, self.vc = (x.transpose(1, 2).contiguous().view(kind).to(DEV) for x in cache)
        self.q = (torch.randn((self.rows, H, D), generator=g) * spread).to(TD[dtype])
        self.scale = D ** -0.5
        self.slopes = 2.0 ** (-8.0 * torch.arange(1, H + 1, dtype=torch.float32) / H) if alibi else None

    def call(self, out=None, stream=None, workspace=None, errors=None, q=None):
        i = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV, torch.int32)  # noqa: E731
        self.dev = [i(self.tables), i(self.ctx), i(self.qsl), i(self.start), i(self.prefix),
                    None if self.slopes is None else self.slopes.to(DEV)]
        bt, cl, qsl, start, prefix, slopes = self.dev
        q = self.q.to(DEV) if q is None else q
        out = torch.full_like(q, 5.0) if out is None else out
        kw = dict(softcap=self.softcap, alibi_slopes=slopes, window=self.window, key_start=start,
                  max_context_len=int(self.ctx.max()) if len(self.ctx) else 0, k_scale=self.ks, v_scale=self.vs,
                  device_errors=errors, stream=stream)
        torch.cuda.synchronize()
        if self.is_decode:
            return pkv.paged_attention_decode_biased(out, q, self.kc, self.vc, bt, cl, self.scale,
                                                     workspace=workspace, **kw)
        return pkv.paged_attention_prefill_biased(out, q, self.kc, self.vc, bt, cl, qsl, self.scale,
                                                  prefix_lens=prefix, max_q_len=int(self.q_len.max()), **kw)

    is_decode = False

    def plain(self):
        """(output, bound) of every row, in 64 bits."""
        out = torch.zeros((self.rows, self.H, self.D), dtype=torch.float64)
        bound = torch.zeros_like(out)
        g, u = self.H // self.hkv, U[self.dtype]
        for s in range(len(self.ctx)):
            pos = np.arange(self.ctx[s] - self.q_len[s], self.ctx[s])
            for i, (a, b) in enumerate(zip(self.lo[s], self.hi[s])):
                if a >= b:
                    continue
                row = int(self.qsl[s]) + i
                q = self.q[row].double().view(self.hkv, g, self.D)
                k, v = self.k[s][a:b].transpose(0, 1), self.v[s][a:b].transpose(0, 1)  # [hkv, n, D]
                x = self.scale * torch.einsum("hgd,hnd->hgn", q, k)
                # S is a magnitude: |scale| (a negative scale would make d negative, and the
                # bound smaller than the rounding of the weights alone)
                size = abs(self.scale) * torch.einsum("hgd,hnd->hgn", q.abs(), k.abs())
                cap = 0.0
                if self.softcap:
                    x = self.softcap * torch.tanh(x / self.softcap)
                    cap = 2.0 ** -19 * x.abs()
                if self.slopes is not None:
                    bias = self.slopes.double().view(self.hkv, g, 1) * torch.from_numpy(
                        np.abs(pos[i] - np.arange(a, b))).double()
                    x, size = x - bias, size + bias
                d = (self.D + 8) * 2.0 ** -24 * size
                if self.kv == "e4m3" and self.dtype == "fp16":
                    d = d + 2.0 ** -8 * size
                elif self.kv == "e4m3":
                    d = d + 2.0 ** -17 * abs(self.scale) * q.abs().amax(-1)[..., None] * k.abs().sum(-1)[:, None]
                d = (d + cap).amax(-1, keepdim=True) + 2.0 ** -21
                w = torch.softmax(x, -1)
                top = w.amax(-1, keepdim=True)
                o = torch.einsum("hgn,hnd->hgd", w, v)
                A = torch.einsum("hgn,hnd->hgd", w, v.abs())
                B = v.abs().sum(1)[:, None] * top
                up = 2.0 ** -8 if self.kv == "e4m3" else u
                e = u * o.abs() + (up + 2 * d) * A + 2.0 ** -17 * B
                out[row], bound[row] = o.reshape(self.H, self.D), 1.01 * e.reshape(self.H, self.D)
        return out, bound + 2.0 ** -24

    def check(self, got, skip=()):
        want, bound = self.plain()
        got = got.double().cpu()
        keep = torch.ones(self.rows, dtype=torch.bool)
        keep[list(skip)] = False
        off = (got - want).abs()
        bad = ~(off <= bound)
        bad[~keep] = False
        assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} elements, first {bad.nonzero()[0].tolist()}: "
                               f"got {got[bad][0]:.6g} want {want[bad][0]:.6g} bound {bound[bad][0]:.3g}")


class Decode(Batch):
    is_decode = True

    def __init__(self, seed, ctx, *a, **k):
        super().__init__(seed, [(1, c) for c in ctx], *a, **k)


def run(b, flags=0, whole=True):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = b.call(errors=err)
    assert pkv.check_errors(err) == flags
    b.check(got)
    want = b.plain()[0]
    if whole and float(want.norm()):
        u = 2.0 ** -8 if b.kv == "e4m3" else U[b.dtype]
        assert float((got.double().cpu() - want).norm() / want.norm()) < 1.5 * u


EDGES = [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300, 511, 512, 513, 700, 1024, 1025]

DECODE = [
    dict(H=8, hkv=2), dict(H=8, hkv=2, softcap=30.0), dict(H=8, hkv=2, alibi=True),
    dict(H=8, hkv=2, window=1), dict(H=8, hkv=2, window=16, dtype="fp16"),
    dict(H=8, hkv=2, window=17, softcap=5.0, alibi=True), dict(H=8, hkv=2, window=200, dtype="fp16"),
    dict(H=8, hkv=2, window=500), dict(H=8, hkv=2, window=513, alibi=True, dtype="fp16"),
    dict(H=16, hkv=2, softcap=50.0, window=300), dict(H=14, hkv=2, softcap=50.0, dtype="fp16"),
    dict(H=12, hkv=2, alibi=True), dict(H=16, hkv=1, window=100, softcap=20.0),
    dict(H=16, hkv=1, alibi=True, dtype="fp16"), dict(H=3, hkv=3, softcap=10.0, window=77),
    dict(H=4, hkv=4, alibi=True, dtype="fp16"), dict(H=8, hkv=2, D=64, softcap=30.0, window=130),
    dict(H=5, hkv=1, D=64, alibi=True, dtype="fp16"), dict(H=2, hkv=2, D=64, window=33),
    dict(H=8, hkv=2, kv="e4m3", softcap=30.0), dict(H=8, hkv=2, kv="e4m3", window=200, dtype="fp16"),
    dict(H=16, hkv=2, kv="e4m3", alibi=True), dict(H=16, hkv=1, kv="e4m3", window=17, softcap=8.0),
    dict(H=14, hkv=2, kv="e4m3", dtype="fp16"), dict(H=4, hkv=4, kv="e4m3", alibi=True, softcap=9.0),
    dict(H=4, hkv=2, D=64, kv="e4m3", window=40),
]


@pytest.mark.parametrize("kw", DECODE, ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()))
def test_decode(kw):
    run(Decode(sum(map(ord, str(kw))), EDGES, **kw))


@pytest.mark.parametrize("kw", [dict(H=8, hkv=2), dict(H=8, hkv=2, kv="e4m3", dtype="fp16"),
                                dict(H=3, hkv=3), dict(H=4, hkv=2, D=64, softcap=7.0),
                                dict(H=16, hkv=1, window=90, alibi=True)])
def test_decode_first_keys(kw):
    """Contexts of no token, and first keys before, at, inside and behind the context."""
    ctx = [0, 1, 40, 40, 40, 40, 600, 600, 600, 1100, 0, 1100]
    first = [0, 0, -5, 39, 40, 99, 16, 513, 85, 511, 3, 1099]
    b = Decode(7, ctx, starts=lambda s, p: first[s], **kw)
    run(b)
    got = b.call().cpu()
    for s in (0, 4, 5, 10):
        assert not got[s].any()  # a row that sees nothing


def test_decode_one_partition_leaves_empty_rows_zero():
    run(Decode(3, [0, 5, 0, 300], H=8, hkv=2, softcap=3.0))
    run(Decode(3, [0, 0], H=8, hkv=2))
    run(Decode(3, [0], H=2, hkv=2))


def test_decode_modifiers_off_equal_plain_decode():
    for kw in (dict(H=8, hkv=2), dict(H=2, hkv=2), dict(H=8, hkv=2, D=64)):
        b = Decode(11, [1, 33, 400, 512, 900], **kw)
        got = b.call()
        bt, cl = b.dev[:2]
        want = torch.empty_like(got)
        pkv.paged_attention_decode(want, b.q.to(DEV), b.kc, b.vc, bt, cl, b.scale, max_context_len=900)
        b.check(got)
        b.check(want)


def test_decode_scales_caps_and_large_scores():
    b = Decode(5, [100, 700], H=8, hkv=2, softcap=50.0, spread=40.0)
    run(b, whole=False)  # (scores of 300 are not exact to a bf16 step)
    b.scale = -b.scale
    run(b, whole=False)
    b.scale = 0.0
    run(b)
    b = Decode(5, [100, 700], H=8, hkv=2, softcap=1e6, spread=3.0)
    run(b)
    run(Decode(6, [100, 700], H=8, hkv=2, softcap=1e-3, spread=3.0))
    run(Decode(6, [100, 700], H=2, hkv=2, softcap=1e6, spread=3.0))


def test_decode_many_sequences():
    ctx = [(37 * s) % 90 for s in range(1500)]
    run(Decode(13, ctx, H=2, hkv=1, window=30, softcap=20.0))


def test_decode_a_window_deep_in_a_long_context():
    """Contexts whose partitions without the window would need more than the workspace holds."""
    b = Decode(17, [5000, 4999, 20, 4096], H=8, hkv=2, window=600, alibi=True)
    n = pkv.decode_biased_workspace_size(4, 8, 128, 5000, 600)
    assert n == pkv.decode_biased_workspace_size(4, 8, 128, 700)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    b.check(b.call(workspace=ws))
    with pytest.raises(pkv.PagedKVError):
        b.call(workspace=ws[:-256])


def test_decode_flags():
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for kw in (dict(H=8, hkv=2), dict(H=2, hkv=2)):
        b = Decode(19, [100, 200, 300], window=50, **kw)
        b.tables[1, 199 // 16] = b.nb  # a block id past the pool, in sight
        b.call(errors=err)
        assert pkv.check_errors(err) == 1
        b = Decode(19, [100, 200, 300], **kw)
        got = b.call(errors=err)
        assert pkv.check_errors(err) == 0
        b.ctx[2] = -4  # refused on the device, read as no context
        out = b.call(errors=err)
        assert pkv.check_errors(err) == 2 and not out[2].any()
        assert torch.equal(out[:2], got[:2])


def test_decode_two_streams_and_a_graph():
    a, b = (Decode(s, [900, 13, 1400], H=8, hkv=2, softcap=20.0, window=700) for s in (1, 2))
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(3):
        outs = [a.call(stream=sa), b.call(stream=sb)]
    torch.cuda.synchronize()
    a.check(outs[0])
    b.check(outs[1])
    # one graph of two calls that share a workspace in stream order, replayed on other queries
    n = pkv.decode_biased_workspace_size(3, 8, 128, 1400, 700)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    qa, qb = a.q.to(DEV), b.q.to(DEV)
    oa, ob = torch.empty_like(qa), torch.empty_like(qb)
    kw = dict(softcap=20.0, window=700, max_context_len=1400, workspace=ws)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pkv.paged_attention_decode_biased(oa, qa, a.kc, a.vc, a.dev[0], a.dev[1], a.scale, **kw)
        pkv.paged_attention_decode_biased(ob, qb, b.kc, b.vc, b.dev[0], b.dev[1], b.scale, **kw)
    for x, q in ((a, qa), (b, qb)):
        x.q = (-x.q).roll(1, 0)
        q.copy_(x.q)
    g.replay()
    torch.cuda.synchronize()
    a.check(oa)
    b.check(ob)


# ---- prefill ---------------------------------------------------------------------------------

def docs(cuts):
    return lambda s, p: max([0] + [c for c in cuts if c <= p])


MIXED = [(1, 1), (3, 3), (1, 40), (17, 40), (0, 9), (100, 100), (40, 300), (2, 513)]
PREFILL = [
    dict(H=8, hkv=2), dict(H=8, hkv=2, softcap=30.0), dict(H=8, hkv=2, alibi=True, dtype="fp16"),
    dict(H=8, hkv=2, window=1), dict(H=8, hkv=2, window=33, softcap=9.0),
    dict(H=8, hkv=2, window=150, alibi=True), dict(H=8, hkv=8, window=64, dtype="fp16"),
    dict(H=16, hkv=1, softcap=20.0), dict(H=14, hkv=2, softcap=50.0, window=50),
    dict(H=6, hkv=2, alibi=True), dict(H=5, hkv=1, dtype="fp16", window=130),
    dict(H=8, hkv=2, starts=docs([2, 50, 51, 130, 200, 290])),
    dict(H=8, hkv=2, starts=docs([30, 60]), alibi=True, window=25, dtype="fp16"),
    dict(H=8, hkv=2, prefix=[1, 2, 40, 20, 9, 64, 290, 600]),
    dict(H=8, hkv=2, prefix=[0, 9, 30, 40, 0, 100, 100, 512], softcap=12.0, alibi=True),
    dict(H=8, hkv=2, prefix=[1, 2, 40, 35, 9, 64, 290, 600], window=60, dtype="fp16"),
    dict(H=4, hkv=4, D=64, softcap=30.0, window=90), dict(H=5, hkv=1, D=64, alibi=True),
    dict(H=8, hkv=2, D=64, dtype="fp16"), dict(H=16, hkv=1, D=64, alibi=True, softcap=6.0),
    dict(H=8, hkv=2, D=64, kv="e4m3", prefix=[1, 2, 40, 35, 9, 64, 290, 600]),
    dict(H=7, hkv=1, D=64, kv="e4m3", dtype="fp16", alibi=True, starts=docs([2, 50, 51, 130, 200, 290])),
    dict(H=8, hkv=2, kv="e4m3", softcap=30.0), dict(H=8, hkv=2, kv="e4m3", alibi=True, dtype="fp16"),
    dict(H=16, hkv=2, kv="e4m3", prefix=[1, 2, 40, 35, 9, 64, 290, 600]),
    dict(H=14, hkv=2, kv="e4m3", window=70, dtype="fp16"),
    dict(H=4, hkv=4, D=64, kv="e4m3", window=45, softcap=9.0),
]


@pytest.mark.parametrize("kw", PREFILL, ids=lambda k: "-".join(
    f"{a}{b if isinstance(b, (int, str, float)) else ''}" for a, b in k.items()))
def test_prefill(kw):
    run(Batch(sum(map(ord, str(sorted(k for k in kw if k not in ("starts", "prefix"))))), MIXED, **kw))


@pytest.mark.parametrize("kw", [
    dict(H=8, hkv=2, window=200, softcap=40.0), dict(H=8, hkv=1, starts=docs([100, 131, 300, 301, 555])),
    dict(H=4, hkv=1, prefix=[400], dtype="fp16"), dict(H=4, hkv=1, kv="e4m3", window=300),
    dict(H=3, hkv=1, alibi=True), dict(H=4, hkv=1, D=64, softcap=40.0),
    dict(H=4, hkv=1, D=64, kv="e4m3", window=300, alibi=True)])
def test_prefill_long_chunk(kw):
    run(Batch(23, [(650, 650)], **kw))
    if "prefix" not in kw:
        run(Batch(24, [(129, 1153)], **kw))


def test_prefill_modifiers_off_equal_plain_prefill():
    b = Batch(31, [(40, 100), (130, 130), (1, 600)], H=8, hkv=2)
    got = b.call()
    bt, cl, qsl = b.dev[:3]
    want = torch.empty_like(got)
    pkv.paged_attention_prefill_chunk(want, b.q.to(DEV), b.kc, b.vc, bt, cl, qsl, b.scale, max_q_len=130,
                                      max_context_len=600)
    b.check(got)
    b.check(want)


@pytest.mark.parametrize("kw", [dict(H=8, hkv=2), dict(H=8, hkv=2, kv="e4m3", dtype="fp16"),
                                dict(H=4, hkv=4, D=64), dict(H=8, hkv=2, softcap=9.0, alibi=True)])
def test_prefill_hidden_infinities(kw):
    """A document whose V is infinite and whose K is NaN: the next documents do not see it."""
    b = Batch(37, [(200, 200), (20, 300)], starts=docs([70, 140, 290]), **kw)
    kind = b.kc.dtype
    for s, tok in ((0, 69), (0, 3), (1, 289)):
        blk = int(b.tables[s, tok // 16])
        kc, vc = b.kc.view(torch.uint8), b.vc.view(torch.uint8)
        if b.kv == "e4m3":
            kc[blk, :, tok % 16], vc[blk, :, tok % 16] = 0x7F, 0xFF
        else:
            b.kc[blk, :, tok % 16], b.vc[blk, :, tok % 16] = float("nan"), float("-inf")
    assert b.kc.dtype == kind
    got = b.call()
    # rows of the documents that hold those tokens see them
    b.check(got, skip=list(range(70)) + list(range(200, 210)))
    assert torch.isfinite(got[70:200].float()).all() and torch.isfinite(got[210:].float()).all()
    assert not torch.isfinite(got[69].float()).any()
    if b.softcap == 0:  # rows before the token do not see it either
        assert torch.isfinite(got[:3].float()).all()


@pytest.mark.parametrize("kw", [dict(H=8, hkv=2), dict(H=8, hkv=2, kv="e4m3", dtype="fp16"),
                                dict(H=4, hkv=4, D=64), dict(H=8, hkv=2, softcap=9.0, alibi=True)])
@pytest.mark.parametrize("odd", [float("nan"), float("inf")])
def test_queries_that_are_not_finite_stay_in_their_rows(kw, odd):
    """One element of a row and head: its output is not a number throughout where the
    element is none (an infinite one makes scores of both signs, and the largest of
    them inf - inf), all the others are what they were."""
    for b, row in ((Batch(39, [(150, 400), (3, 60)], **kw), 131), (Decode(40, [33, 700, 200], **kw), 1)):
        if math.isinf(odd) and b.softcap:
            continue  # (capped, an infinite score is a finite one)
        q = b.q.clone()
        q[row, 2, 7] = odd
        got = b.call(q=q.to(DEV))
        assert torch.isnan(got[row, 2].float()).all()
        mine = got.clone()
        mine[row, 2] = b.plain()[0][row, 2].to(mine.dtype).to(DEV)
        b.check(mine)


def test_prefill_rows_behind_the_last_sequence_stay():
    for kw in (dict(H=8, hkv=2), dict(H=8, hkv=2, D=64), dict(H=8, hkv=2, kv="e4m3")):
        b = Batch(41, [(5, 20), (30, 600), (0, 0)], window=40, **kw)
        q = torch.cat([b.q, torch.zeros((7, 8, b.D), dtype=b.q.dtype)]).to(DEV)
        out = torch.full_like(q, 5.0)
        b.call(out=out, q=q)
        torch.cuda.synchronize()
        b.check(out[:35])
        assert bool((out[35:] == 5.0).all())


def test_prefill_empty_rows_are_zero():
    for kw in (dict(H=8, hkv=2), dict(H=4, hkv=4, D=64), dict(H=8, hkv=2, kv="e4m3")):
        b = Batch(43, [(60, 90), (140, 140), (3, 600)], starts=lambda s, p: p + 1 if s != 1 or p > 99 else 0, **kw)
        run(b)
        got = b.call().cpu()
        assert not got[:60].any() and not got[160:].any()


def test_prefill_more_queries_than_context_is_flagged():
    for kw in (dict(H=8, hkv=2), dict(H=4, hkv=4, D=64)):
        b = Batch(47, [(40, 60), (10, 50)], **kw)
        good = b.call()
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        b.ctx[0] = 30
        out = b.call(errors=err)
        assert pkv.check_errors(err) & 2
        assert torch.equal(out[40:], good[40:])


def test_prefill_streams_and_a_graph():
    a = Batch(51, [(70, 200), (1, 33), (130, 513)], H=8, hkv=2, softcap=20.0, window=90)
    b = Batch(52, [(70, 200), (1, 33), (130, 513)], H=8, hkv=2, kv="e4m3", alibi=True)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(3):
        outs = [a.call(stream=sa), b.call(stream=sb)]
    torch.cuda.synchronize()
    a.check(outs[0])
    b.check(outs[1])
    q = a.q.to(DEV)
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pkv.paged_attention_prefill_biased(out, q, a.kc, a.vc, *a.dev[:3], a.scale, softcap=20.0, window=90,
                                           max_q_len=130, max_context_len=513)
    a.q = (-a.q).roll(3, 0)
    q.copy_(a.q)
    g.replay()
    torch.cuda.synchronize()
    a.check(out)


# ---- a serving step --------------------------------------------------------------------------

@pytest.mark.parametrize("kv", ["same", "e4m3"])
def test_steps_of_a_small_server(kv):
    """Maps, rotary with the cache write and both attentions, run as a server runs them:
    prompts in chunks, then tokens, against one pass over the whole sequences."""
    H, hkv, D, W, cap = 8, 2, 128, 100, 25.0
    g = torch.Generator().manual_seed(3)
    total, R, table = [150, 37, 260], 3, 20
    x = [torch.randn((n, H + 2 * hkv, D), generator=g).to(torch.bfloat16) for n in total]
    inv, attn = pkv.rotary_frequencies(D, 10000.0, "bands", 4.0, 1.0, 4.0, 64)
    pool = pkv.BlockPool(64)
    reqs = [pool.request() for _ in range(R)]
    kind = torch.bfloat16 if kv == "same" else torch.float8_e4m3fn
    ks, vs = (1.0, 1.0) if kv == "same" else (0.012, 0.01)
    bits, nan = (torch.int16, 0x7FFF) if kv == "same" else (torch.uint8, 0x7F)
    kc, vc = (torch.full((64, hkv, 16, D), nan, dtype=bits, device=DEV).view(kind) for _ in range(2))
    tables = torch.full((R, table), -1, dtype=torch.int32, device=DEV)
    done, outs = [0] * R, [[] for _ in range(R)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    while any(d < n for d, n in zip(done, total)):
        # chunks of 64 while a prompt lasts, the last five tokens one at a time
        todo = [(r, min(64, total[r] - 5 - done[r]) if done[r] < total[r] - 5 else 1)
                for r in range(R) if done[r] < total[r]]
        todo.sort(key=lambda t: t[1] > 1)  # decode rows first
        rows, q_lens = [r for r, _ in todo], [n for _, n in todo]
        new = []
        for r, n in todo:
            had = len(reqs[r].block_table())
            reqs[r].append(list(range(n)))
            new += list(reqs[r].block_table()[had:])
        S, T = len(todo), sum(q_lens) + 3
        bt, cl, qsl = (torch.full((S, table), -1, dtype=torch.int32, device=DEV),
                       torch.empty(S, dtype=torch.int32, device=DEV),
                       torch.empty(S + 1, dtype=torch.int32, device=DEV))
        slots, pos = (torch.empty(T, dtype=t, device=DEV) for t in (torch.int64, torch.int32))
        pkv.build_step_maps(bt, cl, qsl, slots, pos, tables, i32(rows), i32([done[r] for r in rows]),
                            i32(q_lens), i32([int(b) for b in new]), 64, device_errors=err)
        qkv = torch.zeros((T, (H + 2 * hkv) * D), dtype=torch.bfloat16)
        at = 0
        for r, n in todo:
            qkv[at:at + n] = x[r][done[r]:done[r] + n].flatten(1)
            at += n
        q, k, v = (y.unflatten(1, (-1, D)) for y in qkv.to(DEV).split([H * D, hkv * D, hkv * D], 1))
        qr = torch.empty((T, H, D), dtype=torch.bfloat16, device=DEV)
        pkv.rotary_and_cache(qr, q, k, v, kc, vc, slots, pos, inv, "half", attn, ks, vs, device_errors=err)
        out = torch.full_like(qr, 9.0)
        nd = sum(n == 1 for n in q_lens)
        kw = dict(softcap=cap, window=W, k_scale=ks, v_scale=vs, max_context_len=table * 16, device_errors=err)
        if nd:
            pkv.paged_attention_decode_biased(out[:nd], qr[:nd], kc, vc, bt[:nd], cl[:nd], D ** -0.5, **kw)
        if nd < S:
            sub = qsl[nd:] - qsl[nd]
            pkv.paged_attention_prefill_biased(out[nd:], qr[nd:], kc, vc, bt[nd:], cl[nd:], sub, D ** -0.5,
                                               max_q_len=64, **kw)
        at = 0
        for r, n in todo:
            outs[r].append(out[at:at + n].double().cpu())
            done[r] += n
            at += n
        assert bool((out[at:] == 9.0).all())
    assert pkv.check_errors(err) == 0
    pool.close()
    for r in range(R):
        n = total[r]
        y = x[r].double()
        ang = torch.arange(n).double()[:, None] * torch.from_numpy(inv)
        c, s = attn * torch.cos(ang)[:, None], attn * torch.sin(ang)[:, None]

        def turn(z):
            a, b = z[..., :D // 2], z[..., D // 2:]
            return torch.cat([a * c - b * s, b * c + a * s], -1)

        q, k, v = turn(y[:, :H]), turn(y[:, H:H + hkv]), y[:, H + hkv:]
        i = torch.arange(n)
        hidden = (i[None] > i[:, None]) | (i[None] <= i[:, None] - W)
        k, v = k.repeat_interleave(H // hkv, 1), v.repeat_interleave(H // hkv, 1)
        sc = cap * torch.tanh(torch.einsum("ihd,jhd->hij", q, k) * D ** -0.5 / cap)
        w = torch.softmax(sc.masked_fill(hidden, -math.inf), -1)
        want, size = torch.einsum("hij,jhd->ihd", w, v), torch.einsum("hij,jhd->ihd", w, v.abs())
        # q and K rounded to bf16 (K and V to E4M3): scores off by at most u (|q||k|), u = 2^-8 + 2^-8
        # (2^-8 + 2^-4), and the values of E4M3 by 2^-4 of themselves
        S = (torch.einsum("ihd,jhd->hij", q.abs(), k.abs()) * D ** -0.5).masked_fill(hidden, 0).amax(-1)
        uk, uv = (2.0 ** -8, 0.0) if kv == "same" else (2.0 ** -4, 2.0 ** -4)
        d = (2.0 ** -8 + uk + 2.0 ** -8) * S.transpose(0, 1)[..., None]
        bound = 2.0 ** -8 * want.abs() + (2.0 ** -8 + uv + torch.expm1(2 * d)) * size * 1.05
        got = torch.cat(outs[r])
        assert bool(((got - want).abs() <= bound).all())
        # the worst case above is loose: on the whole the outputs are far nearer
        far = float((got - want).norm() / want.norm())
        assert far < (2.0 ** -6 if kv == "same" else 2.0 ** -3)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 128), ("bf16", 64), ("fp16", 64)])
def test_prefill_every_e4m3_code(dtype, D):
    """A window of one key returns that key's V: every code of an E4M3 cache, subnormal and
    NaN ones among them, in every position of a tile."""
    b = Batch(61, [(200, 200)], H=4, hkv=1, D=D, dtype=dtype, kv="e4m3", window=1)
    codes = torch.arange(200 * D, dtype=torch.int64).view(200, D)
    codes = ((codes * 37 + codes // 256) % 256).to(torch.uint8)
    for s in range(200):
        b.vc.view(torch.uint8)[int(b.tables[0, s // 16]), 0, s % 16] = codes[s].to(DEV)
    b.vs = 0.5
    got = b.call().double().cpu()
    want = codes.view(torch.float8_e4m3fn).double().mul(0.5)[:, None].expand(200, 4, D)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))


@pytest.mark.parametrize("kw", [dict(), dict(kv="e4m3"), dict(alibi=True), dict(kv="e4m3", alibi=True, softcap=9.0),
                                dict(D=64), dict(D=64, kv="e4m3")])
@pytest.mark.parametrize("skip", [1, 2, 5])
def test_prefill_wait_runs_out(kw, skip):
    """A tile copy that never comes: the call reports it, and the next one is whole."""
    b = Batch(67, [(300, 700), (40, 40)], H=8, hkv=2, **kw)
    good = b.call()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.debug_arm_wait_timeout(skip, 20000)
    b.call(errors=err)
    assert pkv.check_errors(err) & 8
    assert torch.equal(b.call(errors=err), good)
    assert pkv.check_errors(err) == 0


@pytest.mark.parametrize("kw", [dict(window=200), dict(kv="e4m3", softcap=9.0)])
def test_decode_wait_runs_out(kw):
    b = Decode(71, [900, 40, 1300], H=8, hkv=2, **kw)
    good = b.call()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.debug_arm_wait_timeout(2, 20000)
    b.call(errors=err)
    assert pkv.check_errors(err) & 8
    assert torch.equal(b.call(errors=err), good)
    assert pkv.check_errors(err) == 0


@pytest.mark.parametrize("kw", [dict(), dict(dtype="fp16", D=64), dict(window=300), dict(alibi=True), dict(softcap=60.0),
                                dict(kv="e4m3"), dict(starts=lambda s, p: p - p % 200)])
def test_prefill_large_scores(kw):
    """Scores of hundreds, whose running maximum moves at many steps."""
    run(Batch(83, [(150, 900), (70, 330)], H=8, hkv=2, spread=12.0, **kw), whole=False)


@pytest.mark.parametrize("kw", [
    dict(), dict(alibi=True, dtype="fp16"), dict(window=90), dict(D=64, alibi=True), dict(softcap=20.0),
    dict(softcap=20.0, alibi=True, D=64), dict(starts=lambda s, p: p - p % 50), dict(kv="e4m3"),
    dict(prefix=[(7 * s) % 90 for s in range(60)])],
    ids=lambda k: "-".join(k) or "keys")
def test_prefill_more_items_than_processors(kw):
    """Several hundred items of mixed lengths (empty ones, one key, query tiles that end apart):
    each processor takes many, one after another."""
    r = np.random.RandomState(7)
    seqs = []
    for s in range(60):
        n = int(r.randint(0, 40)) if s % 3 else int(r.randint(40, 300 if s % 9 == 0 else 70))
        seqs.append((n, n + (0 if s % 4 == 0 else int(r.randint(0, 400)))))
    run(Batch(79, seqs, H=8, hkv=8, **kw))


def test_prefill_many_sequences():
    """More sequences than one launch's tables hold."""
    seqs = [(1 + s % 3, 1 + s % 3 + (s * 7) % 50) for s in range(1100)]
    run(Batch(73, seqs, H=2, hkv=1, window=20, softcap=15.0))
    run(Batch(74, seqs[:1030], H=2, hkv=2, kv="e4m3", prefix=[s % 60 for s in range(1030)]))


@pytest.mark.parametrize("kv", ["same", "e4m3"])
def test_blocks_past_four_gigabytes(kv):
    """Caches whose byte offsets do not fit 32 bits: the sequences live in the last blocks."""
    dec = Decode(79, [40, 700], H=8, hkv=8, window=600, kv=kv)
    dec4 = Decode(79, [40, 700], H=16, hkv=8, softcap=9.0, kv=kv)
    pre = Batch(80, [(70, 200)], H=8, hkv=8, alibi=True, kv=kv)
    for b in (dec, dec4, pre):
        blocks = 5 * 2 ** 30 // (8 * 16 * 128 * (1 if kv == "e4m3" else 2))
        shift = blocks - b.nb
        for name in ("kc", "vc"):
            small = getattr(b, name)
            big = torch.empty((blocks, 8, 16, 128), dtype=small.dtype, device=DEV)
            big[shift:].view(torch.uint8).copy_(small.view(torch.uint8))
            setattr(b, name, big)
        b.tables = np.where(b.tables >= 0, b.tables + shift, b.tables)
        b.check(b.call())
