"""Cross attention over paged encoder states on the GPU, against softmax attention in 64 bits.

Tolerance of an element, with u half a step of the type (2^-8 bf16, 2^-11 fp16), p the exact
softmax weights, A = sum_j p_j |v_j| and N states:
  - the output's rounding: u |o|;
  - the weights' rounding, to the type or on an E4M3 cache to fp16 (half a step w): each is
    off by d_j <= w relative, and so is what the sum they are divided by is of, so the output is
    off by |sum_j p_j d_j (v_j - o)| / sum_j p_j (1 + d_j) <= 1.01 w (A + |o|).  fp16 weights
    below its normal range are off by 2^-25 absolutely, where the largest weight is 2^4 at
    least: 2^-29 (sum_j |v_j| + N |o|);
  - scores: a sum of D exact products in fp32 is off by at most D 2^-23 of the sum of their
    magnitudes (a step each), which moves a weight by as much relatively, and the sum of
    all by no more: 2 A E with E = D 2^-23 |scale| max_j sum_d |q_d k_jd|;
  - exponentials (2^-22, and their argument's rounding, 2^-24 of its magnitude, below 2^-20
    for arguments that leave a weight of 2^-16), sums of N terms in fp32 in runs of at most
    N, partial results joined: 2 A (2^-19 + N 2^-23).
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_98_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
TD = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
BLOCK_ID, CONTEXT, TIMEOUT = 0x1, 0x2, 0x8


@pytest.fixture(scope="module", autouse=True)
def _library():
    from paged_kv_cache_98_gb300 import _build
    _build.build()
    pkv.load()
    torch.cuda.init()


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, torch.int32)


class Case:
    """Sequences of `q` query rows over `enc` states each.  What no sequence has (rows of
    partial blocks behind the states, other blocks, entries behind the last) is NaN or
    outside the pool; `before` and `behind` rows belong to no sequence."""

    def __init__(self, seed, q, enc, H=4, hkv=2, D=128, dtype="bf16", kv="same", scale=None, before=0,
                 behind=0, q_size=2.0, k=None, v=None):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)
        r = np.random.RandomState(seed)
        self.q_lens, self.enc, self.H, self.hkv, self.D = np.asarray(q), np.asarray(enc), H, hkv, D
        self.dtype, self.kv, self.before = dtype, kv, before
        self.scale = D ** -0.5 if scale is None else scale
        S, dt = len(self.q_lens), TD[dtype]
        need = -(-self.enc // 16)
        self.nb, width = int(need.sum()) + 3, max(1, int(need.max(initial=0))) + 1
        ids, at = r.permutation(self.nb), 0
        self.tables = np.full((S, width), self.nb + 7)
        self.rows = before + int(self.q_lens.sum()) + behind
        self.qsl = before + np.concatenate([[0], np.cumsum(self.q_lens)])
        self.q = (self.rand(self.rows, H, D) * q_size).to(dt)
        self.ks, self.vs = (0.031, 0.027) if kv == "e4m3" else (1.0, 1.0)
        kt = torch.float8_e4m3fn if kv == "e4m3" else dt
        nan = 0x7f if kv == "e4m3" else 0x7fff
        bits = torch.uint8 if kv == "e4m3" else torch.int16
        self.kc = torch.full((self.nb, hkv, 16, D), nan, dtype=bits, device=DEV).view(kt)
        self.vc = self.kc.clone()
        self.k, self.v = [], []
        for s in range(S):
            n = int(self.enc[s])
            self.tables[s, :need[s]] = ids[at:at + need[s]]
            at += need[s]
            pair = []
            for cache, size, make in ((self.kc, self.ks, k), (self.vc, self.vs, v)):
                x = self.rand(n, hkv, D) if make is None else make(s, self.rand(n, hkv, D))
                x = (x / size).clamp(-448, 448).to(kt) if kv == "e4m3" else x.to(dt)
                blocks = torch.full((need[s] * 16, hkv, D), nan, dtype=bits, device=DEV)
                blocks[:n] = x.view(bits)
                blocks = blocks.view(need[s], 16, hkv, D).transpose(1, 2)
                cache.view(bits)[torch.from_numpy(self.tables[s, :need[s]]).to(DEV)] = blocks
                pair.append(x.double() * size)
            self.k.append(pair[0])
            self.v.append(pair[1])

    def rand(self, *shape):
        return torch.randn(shape, generator=self.g, device=DEV)

    def call(self, out=None, **kw):
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        if out is None:
            out = torch.full((self.rows, self.H, self.D), 77.0, dtype=TD[self.dtype], device=DEV)
        kw = {**dict(max_q_len=int(self.q_lens.max(initial=0)), max_encoder_len=int(self.enc.max(initial=0)),
                     k_scale=self.ks, v_scale=self.vs, device_errors=self.err), **kw}
        return pkv.paged_attention_cross(out, self.q, self.kc, self.vc, ints(self.tables), ints(self.enc),
                                         ints(self.qsl), self.scale, **kw)

    def check(self, out, seqs=None):
        G, u = self.H // self.hkv, U[self.dtype]
        w = U["fp16"] if self.kv == "e4m3" else u
        for s in range(len(self.q_lens)) if seqs is None else seqs:
            a, b = int(self.qsl[s]), int(self.qsl[s + 1])
            got, n = out[a:b].double(), int(self.enc[s])
            if a == b:
                continue
            if n == 0:
                assert not got.any(), s
                continue
            for h in range(self.H):
                q, k, v = self.q[a:b, h].double(), self.k[s][:, h // G], self.v[s][:, h // G]
                sc = q @ k.T * self.scale
                p = torch.softmax(sc, 1)
                o = p @ v
                A = p @ v.abs()
                E = self.D * 2.0 ** -23 * abs(self.scale) * (q.abs() @ k.abs().T).amax(1, keepdim=True)
                tol = u * o.abs() + 1.01 * w * (A + o.abs()) + A * (2 * E + 2 * (2.0 ** -19 + n * 2.0 ** -23))
                if w == U["fp16"]:
                    tol = tol + 2.0 ** -29 * (v.abs().sum(0) + n * o.abs())
                if self.dtype == "fp16":
                    tol = tol + 2.0 ** -25    # (the output's own steps below its normal range)
                far = (got[:, h] - o).abs() - tol
                assert torch.isfinite(got[:, h]).all(), (s, h)
                assert far.max() <= 0, (s, h, float(far.max()), float((got[:, h] - o).abs().max()))
        t = out[:self.before], out[int(self.qsl[-1]):]
        assert all((x == 77.0).all() for x in t)     # rows of no sequence


def run(case, **kw):
    out = case.call(**kw)
    case.check(out)
    assert pkv.check_errors(case.err) == 0
    assert torch.equal(out.view(torch.int16), case.call(**kw).view(torch.int16))
    return out


FORMS = [
    dict(H=4, hkv=4), dict(H=8, hkv=2), dict(H=8, hkv=2, dtype="fp16"), dict(H=3, hkv=1, D=64),
    dict(H=6, hkv=2, dtype="fp16"), dict(H=14, hkv=2), dict(H=16, hkv=1), dict(H=16, hkv=1, D=64, dtype="fp16"),
    dict(H=5, hkv=5, D=64), dict(H=12, hkv=1, D=64), dict(H=8, hkv=2, kv="e4m3"),
    dict(H=4, hkv=4, kv="e4m3", dtype="fp16"), dict(H=4, hkv=4, D=64, kv="e4m3"),
    dict(H=14, hkv=2, D=64, kv="e4m3", dtype="fp16"), dict(H=16, hkv=1, kv="e4m3"),
]
IDS = dict(ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()))
EDGES = [0, 1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 384, 385, 600, 1023, 2049]


@pytest.mark.parametrize("kw", FORMS, **IDS)
def test_one_token(kw):
    run(Case(1, [1] * len(EDGES), EDGES, **kw))


@pytest.mark.parametrize("kw", FORMS, **IDS)
def test_ragged(kw):
    """Odd numbers of query tiles and key tiles, sequences without queries, rows of no sequence."""
    rpt = 128 // (kw["H"] // kw["hkv"])
    q = [0, 1, rpt - 1, rpt, rpt + 1, 2 * rpt, 2 * rpt + 1, 3 * rpt, 0, 4 * rpt - 1, 5, 5 * rpt + 2]
    enc = [300, 129, 128, 17, 1, 385, 256, 700, 0, 0, 2000, 90]
    run(Case(2, q, enc, before=3, behind=5, **kw))


@pytest.mark.parametrize("kw", [FORMS[1], FORMS[4], FORMS[8], FORMS[10]], **IDS)
@pytest.mark.parametrize("q,enc", [([1], [1]), ([1], [128]), ([1], [129]), ([2], [40000]), ([700], [77]), ([300], [5000]),
                                   ([40, 1, 3], [20000, 3, 9000]), ([1] * 3, [0, 0, 0]), ([0, 0], [9, 200])])
def test_few_sequences(kw, q, enc):
    """One unit cut into as many parts as there are processors, and units that fill none."""
    run(Case(3, q, enc, **kw))


@pytest.mark.parametrize("S", [1024, 1025, 2100])
def test_many_sequences(S):
    """More sequences than a launch takes."""
    r = np.random.RandomState(S)
    run(Case(4, r.randint(0, 3, S), r.randint(0, 200, S), H=2, hkv=1, D=64, dtype="fp16"))


@pytest.mark.parametrize("scale", [-0.1, 0.0, 3.0])
def test_scales(scale):
    """Negative and zero ones, and scores so large that a state or two take all the weight."""
    run(Case(5, [1, 70, 140], [700, 333, 1030], H=8, hkv=2, scale=scale))
    run(Case(5, [1, 70, 140], [700, 333, 1030], H=4, hkv=4, D=64, dtype="fp16", scale=scale))


@pytest.mark.parametrize("kw", [FORMS[1], FORMS[7]], **IDS)
def test_rising_scores(kw):
    """Maxima that move at nearly every key tile: O is rescaled."""
    def rise(s, x):
        return x * 0.1 + torch.linspace(0, 6, len(x), device=DEV).view(-1, 1, 1)
    c = Case(6, [1, 200, 64], [3000, 1500, 900], k=rise, **kw)
    c.q.abs_()
    run(c)


@pytest.mark.parametrize("kw", [dict(H=8, hkv=2), dict(H=2, hkv=2, D=64, dtype="fp16")], **IDS)
@pytest.mark.parametrize("q", [1, 90])
def test_scores_of_minus_infinity(kw, q):
    """K whose scores are -inf: no weight, also where whole parts of a unit have no other; a row
    that has no other at all is NaN, as in the formula."""
    def k(s, x):
        x = x.clone()
        if s < 3:
            x[..., 0] = 0
            x[[slice(0, 1300), slice(500, None), slice(0, None, 2)][s], :, 0] = -torch.inf
        else:
            x[..., 0] = -torch.inf
        return x
    c = Case(7, [q] * 4, [1800, 1800, 700, 300], k=k, **kw)
    c.q.abs_()
    out = c.call()
    # (in the products inf meets finite numbers only; the plain form needs finite keys)
    for s in range(3):
        c.k[s][..., 0] = torch.where(c.k[s][..., 0] < 0, -1e30, c.k[s][..., 0])
    for s in range(3):
        a, b = int(c.qsl[s]), int(c.qsl[s + 1])
        for h in range(c.H):
            g = c.H // c.hkv
            qq, kk, vv = c.q[a:b, h].double(), c.k[s][:, h // g], c.v[s][:, h // g]
            p = torch.softmax(qq @ kk.T * c.scale, 1)
            want, A = p @ vv, p @ vv.abs()
            u = U[c.dtype]
            assert ((out[a:b, h].double() - want).abs() <= u * want.abs() + A * (u + 2.0 ** -10) + 2.0 ** -12).all()
    assert out[int(c.qsl[3]):].isnan().all()


def test_states_that_are_not_finite():
    """A visible infinity or NaN leaves its rows and dimensions not finite, and no others."""
    def v(s, x):
        x = x.clone()
        if s == 1:
            x[5, 0, 3], x[200, 1, 100] = torch.inf, torch.nan
        return x
    c = Case(8, [3, 130, 2], [300, 301, 299], H=8, hkv=2, v=v)
    out = c.call()
    bad = ~torch.isfinite(out)
    a, b = int(c.qsl[1]), int(c.qsl[2])
    want = torch.zeros_like(bad)
    want[a:b, :4, 3] = True
    want[a:b, 4:, 100] = True
    assert torch.equal(bad, want)
    c.check(out, [0, 2])
    c = Case(8, [3, 130, 2], [300, 301, 299], H=8, hkv=2, k=v)
    out = c.call()
    assert out[a:b, 4:].isnan().all() and torch.isfinite(out[:a]).all() and torch.isfinite(out[b:]).all()
    c.check(out, [0, 2])


def test_left_out_bounds_and_given_workspace():
    c = Case(9, [5, 100, 1], [900, 50, 2000], H=8, hkv=2)
    want = run(c)
    assert torch.equal(want, c.call(max_q_len=None, max_encoder_len=None))
    n = pkv.cross_workspace_size(3, c.rows, 8, 2, 128, 2000, 100)
    for fill in (0, 255):      # its contents do not matter
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        assert torch.equal(want, c.call(workspace=ws))
    with pytest.raises(pkv.PagedKVError):
        c.call(workspace=torch.empty(n - 1, dtype=torch.uint8, device=DEV))


def test_flags():
    def flagged(change, bits, rows=None, **kw):
        c = Case(10, [4, 200, 3], [333, 700, 90], H=8, hkv=2, behind=2)
        change(c)
        out = c.call(**kw)
        assert pkv.check_errors(c.err) == bits
        return c, out

    def entry(c):
        c.tables[1, 2] = c.nb
        c.tables[2, 5] = -1
    c, out = flagged(entry, BLOCK_ID)
    c.check(out, [0])
    c, out = flagged(lambda c: None, CONTEXT, max_encoder_len=400)       # states past the bound are cut
    c.check(out, [0, 2])
    c.k[1], c.v[1], c.enc[1] = c.k[1][:400], c.v[1][:400], 400
    c.check(out)
    c, out = flagged(lambda c: None, CONTEXT, max_q_len=150)             # and queries past it left alone
    c.check(out[:154], [0])
    assert (out[154:204] == 77).all() and (out[-2:] == 77).all()
    c.check(out, [2])

    def offsets(c):
        c.qsl = np.array([0, 4, 2, 209])
    c, out = flagged(offsets, CONTEXT, max_q_len=300)
    assert (out[-2:] != 77).any()    # (sequence 2 owns 2 .. 208 now)

    def beyond(c):
        c.qsl = np.array([0, 4, 204, 300])
    c, out = flagged(beyond, CONTEXT, max_q_len=300)
    assert (out[204:] == 77).all()
    c.qsl = np.array([0, 4, 204, 204])
    c.check(out, [0, 1])

    def negative(c):
        c.enc = np.array([333, -5, 90])
    c, out = flagged(negative, CONTEXT)
    assert not out[4:204].any()


def test_beams_are_queries():
    """Beams of a request, one after the other, read its states once; the order of the rows
    does not matter to any of them."""
    c = Case(11, [5, 4, 5], [700, 1500, 64], H=8, hkv=2)
    out = run(c)
    perm = torch.tensor([4, 2, 0, 1, 3, 5, 8, 7, 6, 13, 12, 11, 10, 9], device=DEV)
    c.q = c.q[perm].contiguous()
    assert torch.equal(c.call(), out[perm])


def test_on_another_stream_and_two_at_once():
    c, d = Case(12, [1, 300], [3000, 800], H=8, hkv=2), Case(13, [40] * 4, [900] * 4, H=4, hkv=4, D=64, dtype="fp16")
    a, b = run(c), run(d)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        outs.append((c.call(stream=s), d.call(stream=t)))
    torch.cuda.synchronize()
    assert all(torch.equal(x, a) and torch.equal(y, b) for x, y in outs)


def test_in_a_graph():
    """Captured with bounds, replayed with other queries and lengths."""
    c, d = Case(14, [4, 30, 1], [900, 200, 2000], H=8, hkv=2), Case(15, [4, 30, 1], [100, 1999, 7], H=8, hkv=2)
    n = max(c.nb, d.nb)
    kc, vc = (torch.zeros((n, 2, 16, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q, width = c.q.clone(), max(c.tables.shape[1], d.tables.shape[1])
    tables, enc, qsl = ints(np.zeros((3, width))), ints(c.enc), ints(c.qsl)
    out = torch.zeros_like(q)
    ws = torch.empty(pkv.cross_workspace_size(3, 35, 8, 2, 128, 2000, 30), dtype=torch.uint8, device=DEV)

    def fill(x):
        kc[:x.nb], vc[:x.nb] = x.kc, x.vc
        tables[:, :x.tables.shape[1]] = ints(x.tables)
        enc.copy_(ints(x.enc))
        q.copy_(x.q)

    def call():
        pkv.paged_attention_cross(out, q, kc, vc, tables, enc, qsl, c.scale, max_q_len=30,
                                  max_encoder_len=2000, workspace=ws)
    fill(c)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for x in (d, c, d):
        fill(x)
        out.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        x.check(out)


@pytest.mark.parametrize("kw", [dict(H=8, hkv=2), dict(H=4, hkv=4, D=64, dtype="fp16"), dict(H=8, hkv=2, kv="e4m3")], **IDS)
@pytest.mark.parametrize("q,skip", [(1, 1), (1, 3), (300, 1), (300, 2), (300, 7)])
def test_a_wait_runs_out(kw, q, skip):
    """A tile copy that is never issued: the call gives up, reports it, and the next one is fine."""
    # (the first processor's part of the work has to hold that copy)
    c = Case(16, [q] * 3, [30000 if skip > 3 else 3000, 900, 2000], **kw)
    pkv.debug_arm_wait_timeout(skip, 20000)
    c.call()
    assert pkv.check_errors(c.err) & TIMEOUT
    run(c)


def test_refusals():
    c = Case(17, [2], [40], H=8, hkv=2)
    out = torch.empty_like(c.q)
    args = [out, c.q, c.kc, c.vc, ints(c.tables), ints(c.enc), ints(c.qsl), 0.1]

    def refused(error, i, x, **kw):
        a = list(args)
        a[i] = x
        with pytest.raises(error):
            pkv.paged_attention_cross(*a, **kw)
    refused(TypeError, 1, c.q.float())
    refused(TypeError, 0, out.to(torch.float16))
    refused(TypeError, 5, args[5].long())
    refused(ValueError, 0, out[:1])
    refused(ValueError, 6, args[6][:1])
    refused(ValueError, 3, c.vc[:2])
    refused(ValueError, 1, c.q.cpu())
    refused(ValueError, 4, args[4].cpu())
    refused(pkv.PagedKVError, 0, c.q)                        # in place
    refused(pkv.PagedKVError, 7, float("nan"))
    refused(ValueError, 0, torch.empty(2, 8, 256, dtype=c.q.dtype, device=DEV)[..., ::2])


@pytest.mark.parametrize("kv", ["same", "e4m3"])
def test_blocks_past_32_bits(kv):
    """States in blocks whose elements lie more than 2^32 into caches of 10 or 20 GB."""
    c = Case(18, [1, 3, 150], [333, 2000, 140], H=16, hkv=8, kv=kv)
    want, nb = run(c), (1 << 32) // (8 * 16 * 128) + c.nb + 1000
    for name in ("kc", "vc"):
        small = getattr(c, name)
        big = torch.empty(nb, *small.shape[1:], dtype=small.dtype, device=DEV)
        big.view(torch.uint8)[-c.nb:] = small.view(torch.uint8)
        setattr(c, name, big)
    c.tables += nb - c.nb         # (entries behind a sequence's last stay outside the pool)
    assert torch.equal(want, c.call())
    assert pkv.check_errors(c.err) == 0
