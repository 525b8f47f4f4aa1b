"""The calls on requests, layers and encoder states together, as a program uses them: beam
search of an encoder-decoder model in a captured step, and drafted trees verified, cut to the
accepted path and given back, with the sequences that come of them against plain ones."""
import numpy as np
import pytest
import torch

import paged_kv_cache_98_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = dict(dtype=torch.int32, device=DEV)


@pytest.fixture(scope="module", autouse=True)
def _library():
    from paged_kv_cache_98_gb300 import _build
    _build.build()
    pkv.load()
    torch.cuda.init()


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, torch.int32)


def attend(q, k, v, scale):
    """q [H, D], k and v [T, hkv, D] in 64 bits: [H, D]."""
    g = q.shape[0] // k.shape[1]
    k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    return torch.einsum("ht,thd->hd", torch.softmax(torch.einsum("hd,thd->ht", q, k) * scale, 1), v)


def test_encoder_decoder_beams_in_a_graph():
    """Three requests of four beams over encoder inputs of 1, 333 and 90 states: each step forks
    the beams by their parents, takes a token's place in every beam (copying shared last
    blocks), writes its K and V, attends to the beams' own tokens and to the encoder.
    Tolerance: half a step of bf16 for the output and for the weights, 2^-8 each, of the
    values' magnitudes, and fp32 terms far below (2^-14 stands for them)."""
    r = np.random.RandomState(3)
    B, W, H, hkv, D, mb, nb, L, steps = 3, 4, 8, 2, 128, 6, 100, 2, 40
    n, scale = B * W, D ** -0.5
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    enc = [1, 333, 90]
    eb = [-(-e // 16) for e in enc]
    ids = r.permutation(sum(eb))
    etab = np.full((B, max(eb)), -1)
    at = 0
    for i, k in enumerate(eb):
        etab[i, :k], at = ids[at:at + k], at + k
    ek, ev = rand(L, sum(eb), hkv, 16, D), rand(L, sum(eb), hkv, 16, D)
    kc, vc = rand(L, nb, hkv, 16, D), rand(L, nb, hkv, 16, D)
    tables = [torch.full((n, mb), -1, **I32) for _ in range(2)]
    lens = [torch.zeros(n, **I32) for _ in range(2)]
    counts, err = torch.zeros(nb, **I32), torch.zeros(1, **I32)
    rows, one, parents = torch.arange(n, **I32), torch.ones(n, **I32), torch.arange(n, **I32)
    grown, granted, opened, pairs = (torch.zeros(s, **I32) for s in (n, n, n, (n, 2)))
    bt, ctx, qsl, pos = (torch.zeros(s, **I32) for s in ((n, mb), n, n + 1, n))
    slots = torch.zeros(n, dtype=torch.int64, device=DEV)
    q, k, v = (torch.zeros((L, n, h, D), dtype=torch.bfloat16, device=DEV) for h in (H, hkv, hkv))
    own, cross = torch.zeros_like(q), torch.zeros_like(q)
    etables, elens, eqsl = ints(etab), ints(enc), ints(np.arange(B + 1) * W)
    ws = torch.empty(pkv.cross_workspace_size(B, n, H, hkv, D, 333, W), dtype=torch.uint8, device=DEV)
    dws = torch.empty(max(1, pkv.decode_workspace_size(n, H, D, mb * 16)), dtype=torch.uint8, device=DEV)

    def step(a, b):
        pkv.fork_requests(tables[b], lens[b], tables[a], lens[a], counts, parents, device_errors=err)
        torch.add(lens[b], 1, out=grown)
        pkv.resize_requests(tables[b], counts, rows, lens[b], grown, granted, opened, pairs, device_errors=err)
        pkv.copy_blocks_layers(kc, vc, pairs, device_errors=err)
        pkv.build_step_maps(bt, ctx, qsl, slots, pos, tables[b], rows, lens[b], one, opened, nb, device_errors=err)
        for i in range(L):
            pkv.reshape_and_cache(k[i], v[i], kc[i], vc[i], slots, device_errors=err)
            pkv.paged_attention_decode(own[i], q[i], kc[i], vc[i], bt, ctx, scale, max_context_len=mb * 16,
                                       workspace=dws, device_errors=err)
            pkv.paged_attention_cross(cross[i], q[i], ek[i], ev[i], etables, elens, eqsl, scale, max_q_len=W,
                                      max_encoder_len=333, workspace=ws, device_errors=err)
        lens[b].copy_(granted)

    step(0, 1)                              # (what a first call sets up)
    torch.cuda.synchronize()
    graphs = []
    for a, b in ((0, 1), (1, 0)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step(a, b)
    for t in (*tables, *lens, counts, err):
        t.zero_()
    history = [[] for _ in range(n)]        # (K, V) of each beam's tokens
    encoded = [[x[i, ints(etab[b, :eb[b]]).long()].transpose(1, 2).reshape(-1, hkv, D)[:enc[b]].double()
                for x in (ek, ev)] for i in range(L) for b in range(B)]

    def close(got, want, v):
        size = v.abs().amax(0).repeat_interleave(H // hkv, 0)
        assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -14) * size).all()

    for it in range(steps):
        par = r.randint(0, W, n) + np.arange(n) // W * W if it else np.arange(n)
        parents.copy_(ints(par))
        for t, h in ((q, H), (k, hkv), (v, hkv)):
            t.copy_(rand(L, n, h, D))
        graphs[it & 1].replay()
        history = [history[p] + [(k[:, i].clone(), v[:, i].clone())] for i, p in enumerate(par)]
        if it in (0, 15, 16, 17, 32, steps - 1):
            torch.cuda.synchronize()
            for i in range(n):
                for l in range(L):
                    hk, hv = (torch.stack([x[j][l] for x in history[i]]).double() for j in range(2))
                    close(own[l, i], attend(q[l, i].double(), hk, hv, scale), hv)
                    xk, xv = encoded[l * B + i // W]
                    close(cross[l, i], attend(q[l, i].double(), xk, xv, scale), xv)
    assert pkv.check_errors(err) == 0
    t, m = tables[steps & 1].cpu().numpy(), lens[steps & 1].cpu().numpy()
    want = np.zeros(nb, int)
    for i in range(n):
        np.add.at(want, t[i, :-(-m[i] // 16)], 1)
    np.testing.assert_array_equal(counts.cpu().numpy(), want)


def test_drafted_trees_kept_and_given_back():
    """Each step drafts a tree of tokens behind every request, verifies it in one pass, keeps a
    path from its root and gives the blocks behind back.  What the caches hold afterwards are the
    accepted tokens, and the verification of the next step sees them (tolerance as above)."""
    r = np.random.RandomState(5)
    S, H, hkv, D, mb, nb, L, T = 4, 8, 2, 128, 20, 120, 3, 24
    scale = D ** -0.5
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    kc, vc = rand(L, nb, hkv, 16, D), rand(L, nb, hkv, 16, D)
    tables, counts, err = torch.full((S, mb), -1, **I32), torch.zeros(nb, **I32), torch.zeros(1, **I32)
    rows, lens = torch.arange(S, **I32), np.zeros(S, int)
    opened, pairs, granted, new = (torch.zeros(s, **I32) for s in (S * 3, (S, 2), S, S))
    history = [[] for _ in range(S)]
    for it in range(8):
        size = r.randint(1, T + 1, S)
        parent = [np.array([-1] + [r.randint(0, j) for j in range(1, n)]) for n in size]
        pkv.resize_requests(tables, counts, rows, ints(lens), ints(lens + size), granted, opened, pairs,
                            device_errors=err)
        N = int(size.sum())
        bt, ctx, qsl, pos = (torch.zeros(s, **I32) for s in ((S, mb), S, S + 1, N))
        slots = torch.zeros(N, dtype=torch.int64, device=DEV)
        pkv.build_step_maps(bt, ctx, qsl, slots, pos, tables, rows, ints(lens), ints(size), opened, nb,
                            device_errors=err)
        q, k, v = rand(N, H, D), rand(L, N, hkv, D), rand(L, N, hkv, D)
        for l in range(L):
            pkv.reshape_and_cache(k[l], v[l], kc[l], vc[l], slots, device_errors=err)
        mask, at = np.zeros(N, np.uint64), 0
        for p in parent:
            for j in range(len(p)):
                mask[at + j] = np.uint64(1 << j) | (mask[at + p[j]] if p[j] >= 0 else np.uint64(0))
            at += len(p)
        out = torch.empty_like(q)
        pkv.paged_attention_prefill_tree(out, q, kc[1], vc[1], bt, ctx, qsl,
                                         torch.from_numpy(mask.view(np.int64)).to(DEV), scale, max_q_len=T,
                                         max_context_len=mb * 16, device_errors=err)
        keep, starts, at = [], [0], 0
        for s in range(S):
            # a path from the root, as long as a random leaf's
            path, j = [], r.randint(size[s])
            while j >= 0:
                path.append(int(j))
                j = parent[s][j]
            path = path[::-1]
            for j in range(size[s]):        # the verification's rows
                seen = [i for i in range(size[s]) if int(mask[at + j]) >> i & 1]
                hk, hv = (torch.stack([x[c][1] for x in history[s]] + [y[1, at + i] for i in seen]).double()
                          for c, y in ((0, k), (1, v)))
                want = attend(q[at + j].double(), hk, hv, scale)
                top = hv.abs().amax(0).repeat_interleave(H // hkv, 0)
                assert ((out[at + j].double() - want).abs() <=
                        2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -14) * top).all()
            keep += [int(lens[s]) + j for j in path]
            starts.append(len(keep))
            history[s] += [(k[:, at + j].clone(), v[:, at + j].clone()) for j in path]
            at += size[s]
        pkv.compact_tokens(kc, vc, tables, granted, ints(lens), ints(starts), ints(keep), new, ref_counts=counts,
                           device_errors=err)
        lens = new.cpu().numpy().astype(int)
        assert lens.tolist() == [len(h) for h in history]
        pkv.resize_requests(tables, counts, rows, granted.clone(), new, torch.zeros(S, **I32), opened, pairs,
                            device_errors=err)
        assert pkv.check_errors(err) == 0
        t = tables.cpu().numpy()
        want = np.zeros(nb, int)
        for s in range(S):
            n = -(-lens[s] // 16)
            assert (t[s, n:] == -1).all()
            np.add.at(want, t[s, :n], 1)
            for x, c in ((kc, 0), (vc, 1)):
                got = x[:, ints(t[s, :n]).long()].transpose(2, 3).reshape(L, -1, hkv, D)[:, :lens[s]]
                assert torch.equal(got, torch.stack([h[c] for h in history[s]], 1))
        np.testing.assert_array_equal(counts.cpu().numpy(), want)
