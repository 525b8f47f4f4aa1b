"""Cases for the serving-step operators around the paged cache.

A serving step of a paged-cache model runs four operators in this order:

  maps     block tables, context lengths, query offsets, slots and positions of
           a batch, built on the GPU from the requests' lengths
           (``build_step_maps``)
  rotary   the rotary rotation of Q and K, with K and V written into the paged
           cache on the way (``rotary_and_cache``)
  decode   one query token per sequence over the paged context, with capped
           scores, a distance bias, a sliding window or a document start
           (``paged_attention_decode_biased``)
  prefill  the same for chunks of queries, with a document mask per query or a
           bidirectional prefix (``paged_attention_prefill_biased``)

``run`` computes them from elementary torch operations in 32 bits (angles in
64), or, where ``own`` is true, through this repository's entry points.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
TD = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---- cases -----------------------------------------------------------------------------------

def listed():
    att = dict(head_dim=128, kv="same", softcap=0.0, alibi=False, window=0, docs=0, prefix=False)
    return [
        # eight running requests, one new token each: the launch latency a step pays
        dict(name="maps.decode8", op="maps", seqs=8, chunks=0, chunk=1, max_ctx=1000, table=64, lens=11),
        # a loaded server: 936 running requests and 64 prompt chunks of 512 tokens
        dict(name="maps.mixed1000", op="maps", seqs=1000, chunks=64, chunk=512, max_ctx=12000,
             table=1024, lens=12),
        # decode step of a 32-head model, 64 sequences around 4096 tokens
        dict(name="rotary.decode64", op="rotary", tokens=64, heads=32, kv_heads=32, head_dim=128,
             rot=128, layout="half", dtype="bf16", kv="same", fused=False, max_pos=4096, base=1e4),
        # a prompt of 8192 tokens, grouped heads, Q/K/V slices of one fused projection, half of
        # each head rotated, neighbouring elements paired
        dict(name="rotary.prompt8192", op="rotary", tokens=8192, heads=64, kv_heads=8, head_dim=128,
             rot=64, layout="interleaved", dtype="fp16", kv="same", fused=True, max_pos=8192,
             base=1e4),
        # a mixed batch (32 decode rows, 4 chunks of 512) of a long-context model into an 8-bit cache
        dict(name="rotary.mixed_e4m3", op="rotary", tokens=2080, heads=32, kv_heads=8, head_dim=128,
             rot=128, layout="half", dtype="bf16", kv="e4m3", fused=True, max_pos=131072, base=5e5),
        # three short chats: latency
        dict(att, name="decode.short_cap", op="decode", seqs=3, min_ctx=1, max_ctx=700, lens=21,
             heads=8, kv_heads=2, dtype="fp16", softcap=30.0),
        # the mixed batch's 32 decode rows with capped scores and a 4096-token window whose blocks
        # behind it went back to the pool
        dict(att, name="decode.window_cap", op="decode", seqs=32, min_ctx=1024, max_ctx=8192, lens=22,
             heads=32, kv_heads=8, dtype="bf16", softcap=50.0, window=4096),
        # one query head per KV head with a linear distance bias
        dict(att, name="decode.alibi_mha", op="decode", seqs=16, min_ctx=2048, max_ctx=4099, lens=23,
             heads=32, kv_heads=32, dtype="fp16", alibi=True),
        # eight long documents in an 8-bit cache, some of them starting late in their sequence
        dict(att, name="decode.long_e4m3", op="decode", seqs=8, min_ctx=100000, max_ctx=131071,
             lens=24, heads=32, kv_heads=8, dtype="bf16", kv="e4m3", softcap=50.0, docs=30000),
        # four prompt chunks of 512 tokens over 2048 prior ones, capped scores, window of 1024
        dict(att, name="prefill.window_cap", op="prefill", seqs=4, min_q=512, max_q=512, min_prior=2048,
             max_prior=2048, lens=31, heads=32, kv_heads=8, dtype="bf16", softcap=50.0, window=1024),
        # documents packed into one sequence of odd length, with a distance bias
        dict(att, name="prefill.packed_docs", op="prefill", seqs=1, min_q=8191, max_q=8191, min_prior=0,
             max_prior=0, lens=32, heads=32, kv_heads=8, dtype="fp16", alibi=True, docs=900),
        # whole prompts whose first part is seen in both directions, 8-bit cache
        dict(att, name="prefill.prefix_e4m3", op="prefill", seqs=6, min_q=37, max_q=1500, min_prior=0,
             max_prior=0, lens=33, heads=64, kv_heads=8, dtype="bf16", kv="e4m3", prefix=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["maps", "rotary", "decode", "prefill"])
    lens = rng.randrange(1 << 20)
    if op == "maps":
        seqs = _log_int(rng, 1, 1000)
        chunks = rng.randint(0, min(64, seqs))
        return dict(op=op, seqs=seqs, chunks=chunks, chunk=_log_int(rng, 1, 512),
                    max_ctx=_log_int(rng, 17, 12000), table=rng.choice([800, 1000, 1024]), lens=lens)
    if op == "rotary":
        heads, kv_heads = rng.choice([(32, 32), (32, 8), (64, 8), (8, 2), (4, 4)])
        d = rng.choice([64, 128, 128])
        return dict(op=op, tokens=_log_int(rng, 1, 8192), heads=heads, kv_heads=kv_heads, head_dim=d,
                    rot=rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)]),
                    layout=rng.choice(["half", "interleaved"]), dtype=rng.choice(["bf16", "fp16"]),
                    kv=rng.choice(["same", "e4m3"]), fused=rng.random() < 0.5,
                    max_pos=_log_int(rng, 8192, 131072), base=rng.choice([1e4, 5e5]))
    case = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), kv=rng.choice(["same", "same", "e4m3"]),
                head_dim=128, softcap=rng.choice([0.0, 30.0, 50.0]), alibi=rng.random() < 0.4,
                window=rng.choice([0, 0, _log_int(rng, 20, 4096)]), docs=0, prefix=False, lens=lens)
    if rng.random() < 0.3:
        case["docs"] = _log_int(rng, 16, 2000)
    if op == "decode":
        heads, kv_heads = rng.choice([(32, 32), (32, 8), (64, 8), (8, 2), (14, 2), (16, 1)])
        hi = _log_int(rng, 16, 8192)
        case.update(seqs=_log_int(rng, 1, 48), min_ctx=max(1, hi // rng.choice([1, 4, 50])), max_ctx=hi,
                    heads=heads, kv_heads=kv_heads, head_dim=rng.choice([128, 128, 64]))
    else:
        heads, kv_heads = rng.choice([(32, 8), (64, 8), (8, 2), (8, 8), (14, 2), (16, 1)])
        hi = _log_int(rng, 1, 700)
        prior = rng.choice([0, _log_int(rng, 1, 2100)])
        case.update(seqs=_log_int(rng, 1, 6), min_q=max(1, hi // rng.choice([1, 3, 20])), max_q=hi,
                    min_prior=prior // 2, max_prior=prior, heads=heads, kv_heads=kv_heads)
        case["prefix"] = rng.random() < 0.3
    return case


# ---- inputs ----------------------------------------------------------------------------------

def _lengths(case):
    """(query lengths, context lengths) of a case's sequences: the case's own, whatever the seed."""
    r = np.random.RandomState(case["lens"])
    s = case["seqs"]
    if case["op"] == "decode":
        return np.ones(s, np.int64), r.randint(case["min_ctx"], case["max_ctx"] + 1, s).astype(np.int64)
    if case["op"] == "prefill":
        q = r.randint(case["min_q"], case["max_q"] + 1, s).astype(np.int64)
        return q, q + r.randint(case["min_prior"], case["max_prior"] + 1, s)
    q = np.ones(s, np.int64)
    q[s - case["chunks"]:] = case["chunk"]
    cached = r.randint(0, case["max_ctx"] - 1, s).astype(np.int64)
    return q, q + cached


def _starts(case, ctx):
    """First position of the document that holds each position, per sequence (zeros without documents)."""
    r = np.random.RandomState(case["lens"] + 1)
    out = []
    for c in ctx:
        cuts = [0]
        while case["docs"] and cuts[-1] < c:
            cuts.append(cuts[-1] + 1 + int(r.randint(2 * case["docs"])))
        cuts = np.array(cuts, np.int64)
        out.append(cuts[np.searchsorted(cuts, np.arange(c), side="right") - 1])
    return out


def _prefixes(case, ctx):
    return np.random.RandomState(case["lens"] + 2).randint(0, ctx + 1) if case["prefix"] else 0 * ctx


def _intervals(case):
    """Per sequence: (lo, hi) of the keys each query row sees."""
    qlen, ctx = _lengths(case)
    pre, starts, out = _prefixes(case, ctx), _starts(case, ctx), []
    for q, c, p, st in zip(qlen, ctx, pre, starts):
        pos = np.arange(c - q, c)
        lo = st[c - q:]
        if case["window"]:
            lo = np.maximum(lo, pos - case["window"] + 1)
        out.append((np.maximum(lo, 0), np.maximum(pos + 1, p)))
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 31))
    st = dict(case=dict(case))
    dev = "cuda"

    def ints(a, dtype=torch.int32):
        return torch.from_numpy(np.ascontiguousarray(a)).to(dev, dtype)

    if case["op"] == "maps":
        qlen, ctx = _lengths(case)
        have, need = -(-(ctx - qlen) // BLOCK), -(-ctx // BLOCK)
        total = int(need.sum())
        st["num_blocks"] = total + total // 4 + 1
        ids = r.permutation(st["num_blocks"])[:total]
        rows = r.permutation(2 * case["seqs"])[:case["seqs"]]
        tables = np.full((2 * case["seqs"], case["table"]), -1, np.int64)
        new, at = [], 0
        for row, h, n in zip(rows, have, need):
            tables[row, :h] = ids[at:at + h]
            new.append(ids[at + h:at + n])
            at += n
        # a captured step runs at a fixed number of tokens: some room behind the last one
        st["cap"] = int(qlen.sum()) + case["seqs"] // 8
        st.update(tables=ints(tables), rows=ints(rows), cached=ints(ctx - qlen), qlen=ints(qlen),
                  new=ints(np.concatenate(new)))
        s = case["seqs"]
        st.update(bt=torch.full((s, case["table"]), -1, dtype=torch.int32, device=dev),
                  ctx=torch.zeros(s, dtype=torch.int32, device=dev),
                  qsl=torch.zeros(s + 1, dtype=torch.int32, device=dev),
                  slots=torch.zeros(st["cap"], dtype=torch.int64, device=dev),
                  pos=torch.zeros(st["cap"], dtype=torch.int32, device=dev))
        return st

    dt = TD[case["dtype"]]
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]

    def randn(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device=dev) * scale

    if case["op"] == "rotary":
        t = case["tokens"]
        if case["fused"]:  # slices of one projection's output
            qkv = randn(t, (h + 2 * hk) * d).to(dt)
            q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([h * d, hk * d, hk * d], 1))
        else:
            q, k, v = (randn(t, n, d).to(dt) for n in (h, hk, hk))
        nb = -(-t // BLOCK) * 5 // 4 + 1
        slots = (r.permutation(nb)[:-(-t // BLOCK), None] * BLOCK + np.arange(BLOCK)).reshape(-1)[:t]
        # decode rows sit anywhere in their contexts, prompt tokens behind one another
        pos = r.randint(0, case["max_pos"], t) if t <= 64 else \
            (r.randint(0, case["max_pos"] - t + 1) if t < case["max_pos"] else 0) + np.arange(t)
        inv = case["base"] ** (-np.arange(0, case["rot"], 2, dtype=np.float64) / case["rot"])
        kind = dt if case["kv"] == "same" else torch.float8_e4m3fn
        kc, vc = (torch.zeros((nb, hk, BLOCK, d), dtype=kind, device=dev) for _ in range(2))
        st.update(q=q, k=k, v=v, slots=ints(slots, torch.int64), pos=ints(pos), inv=inv, kc=kc, vc=vc,
                  out=torch.empty((t, h, d), dtype=dt, device=dev), k_scale=6.0 / 448, v_scale=6.0 / 448)
        return st

    qlen, ctx = _lengths(case)
    need = -(-ctx // BLOCK)
    total, width = int(need.sum()), int(need.max())
    nb = total + total // 4 + 1
    ids, at = r.permutation(nb), 0
    tables = np.zeros((case["seqs"], width), np.int64)
    for i, ((lo, _), n) in enumerate(zip(_intervals(case), need)):
        tables[i, :n] = ids[at:at + n]
        if case["window"]:  # blocks behind the window went back to the pool
            tables[i, :int(lo.min()) // BLOCK] = -1
        at += n

    def cache():
        x = randn(nb, hk, BLOCK, d)
        if case["kv"] == "same":
            return x.to(dt), 1.0
        scale = float(x.abs().amax()) / 448
        return (x / scale).clamp_(-448, 448).to(torch.float8_e4m3fn), scale

    (kc, ks), (vc, vs) = cache(), cache()
    rows = int(qlen.sum())
    starts = _starts(case, ctx)
    st.update(q=randn(rows, h, d, scale=2.0).to(dt), kc=kc, vc=vc, k_scale=ks, v_scale=vs,
              tables=ints(tables), ctx=ints(ctx), scale=d ** -0.5, max_ctx=int(ctx.max()),
              max_q=int(qlen.max()), qsl=ints(np.concatenate([[0], np.cumsum(qlen)])),
              slopes=(2.0 ** (-8.0 * torch.arange(1, h + 1, device=dev, dtype=torch.float32) / h)
                      if case["alibi"] else None),
              start=ints(np.concatenate([x[c - q:] for x, c, q in zip(starts, ctx, qlen)]))
              if case["docs"] else None,
              prefix=ints(_prefixes(case, ctx)) if case["prefix"] else None,
              out=torch.empty((rows, h, d), dtype=dt, device=dev))
    return st


# ---- one pass --------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return {"maps": _maps, "rotary": _rotary}.get(op, _attention)(state)


def _own(op, st):
    import paged_kv_cache_98_gb300 as pkv
    c = st["case"]
    if op == "maps":
        pkv.build_step_maps(st["bt"], st["ctx"], st["qsl"], st["slots"], st["pos"], st["tables"],
                            st["rows"], st["cached"], st["qlen"], st["new"], st["num_blocks"])
        return st["bt"], st["ctx"], st["qsl"], st["slots"], st["pos"], st["tables"]
    if op == "rotary":
        pkv.rotary_and_cache(st["out"], st["q"], st["k"], st["v"], st["kc"], st["vc"], st["slots"],
                             st["pos"], st["inv"], layout=c["layout"], k_scale=st["k_scale"],
                             v_scale=st["v_scale"])
        return st["out"], st["kc"], st["vc"]
    mods = dict(softcap=c["softcap"], alibi_slopes=st["slopes"], window=c["window"],
                key_start=st["start"], max_context_len=st["max_ctx"], k_scale=st["k_scale"],
                v_scale=st["v_scale"])
    if op == "decode":
        return pkv.paged_attention_decode_biased(st["out"], st["q"], st["kc"], st["vc"], st["tables"],
                                                 st["ctx"], st["scale"], **mods)
    return pkv.paged_attention_prefill_biased(st["out"], st["q"], st["kc"], st["vc"], st["tables"],
                                              st["ctx"], st["qsl"], st["scale"],
                                              prefix_lens=st["prefix"], max_q_len=st["max_q"], **mods)


def _maps(st):
    cached, qlen, tables, cap = st["cached"].long(), st["qlen"].long(), st["tables"], st["cap"]
    rows, new, width = st["rows"].long(), st["new"], tables.shape[1]
    ctx = cached + qlen
    have, need = (cached + BLOCK - 1) // BLOCK, (ctx + BLOCK - 1) // BLOCK
    grow = need - have
    col = torch.arange(width, device=tables.device)
    # the blocks this step opens follow those a request has, taken from the list in batch order
    src = (grow.cumsum(0) - grow - have)[:, None] + col
    fresh = (col >= have[:, None]) & (col < need[:, None])
    mine = torch.where(fresh, new[src.clamp(0, max(new.numel() - 1, 0))] if new.numel() else -1,
                       tables[rows])
    tables[rows] = mine
    bt = torch.where(col < need[:, None], mine, st["bt"])
    qsl = torch.cat([qlen.new_zeros(1), qlen.cumsum(0)])
    t = torch.arange(cap, device=tables.device)
    seq = (torch.searchsorted(qsl, t, right=True) - 1).clamp(max=rows.numel() - 1)
    live = t < qsl[-1]
    pos = cached[seq] + t - qsl[seq]
    blk = mine[seq, (pos // BLOCK).clamp(max=width - 1)].long()
    slots = torch.where(live, blk * BLOCK + pos % BLOCK, -1)
    return bt, ctx.int(), qsl.int(), slots, torch.where(live, pos, -1).int(), tables


def _rotary(st):
    c = st["case"]
    rot, d = c["rot"], c["head_dim"]
    ang = st["pos"].double()[:, None] * torch.from_numpy(st["inv"]).to(st["pos"].device)
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]

    def turn(x):
        x = x.float()
        y = x[..., :rot]
        a, b = (y[..., :rot // 2], y[..., rot // 2:]) if c["layout"] == "half" else \
            (y[..., 0::2], y[..., 1::2])
        u, w = a * cos - b * sin, b * cos + a * sin
        y = torch.cat([u, w], -1) if c["layout"] == "half" else torch.stack([u, w], -1).flatten(-2)
        return torch.cat([y, x[..., rot:]], -1)

    def put(cache, x, scale):
        if c["kv"] == "e4m3":
            x = (x / scale).clamp(-448, 448)
        blk, off = st["slots"] // BLOCK, st["slots"] % BLOCK
        bits = torch.uint8 if c["kv"] == "e4m3" else torch.int16
        cache.view(bits)[blk, :, off] = x.to(cache.dtype).view(bits)
        return cache

    return (turn(st["q"]).to(st["q"].dtype), put(st["kc"], turn(st["k"]), st["k_scale"]),
            put(st["vc"], st["v"].float(), st["v_scale"]))


def _attention(st):
    """Softmax attention of every query row over the keys of its interval, on padded batches."""
    c, q, qsl, ctx = st["case"], st["q"], st["qsl"].long(), st["ctx"].long()
    s, h, hk, d, lq = c["seqs"], c["heads"], c["kv_heads"], c["head_dim"], st["max_q"]
    dev, g = q.device, h // hk
    idx = st["tables"].long().clamp(min=0)
    keys = idx.shape[1] * BLOCK
    j = torch.arange(keys, device=dev)

    def gathered(cache, scale):
        x = cache.view(torch.uint8)[idx].view(cache.dtype) if c["kv"] == "e4m3" else cache[idx]
        x = x.transpose(1, 2).reshape(s, hk, keys, d).float()
        return x.mul_(scale) if c["kv"] == "e4m3" else x

    qlen = qsl[1:] - qsl[:-1]
    i = torch.arange(lq, device=dev)
    row = (qsl[:-1, None] + i).clamp(max=q.shape[0] - 1)                     # [s, lq]
    pos = (ctx - qlen)[:, None] + i
    lo = torch.zeros_like(pos) if st["start"] is None else st["start"].long()[row]
    if c["window"]:
        lo = torch.maximum(lo, pos - c["window"] + 1)
    hi = pos + 1 if st["prefix"] is None else torch.maximum(pos + 1, st["prefix"].long()[:, None])
    seen = (j >= lo[..., None]) & (j < hi[..., None])                        # [s, lq, keys]
    x = q.float()[row].view(s, lq, hk, g, d).permute(0, 2, 3, 1, 4).reshape(s, hk, g * lq, d)
    score = (x @ gathered(st["kc"], st["k_scale"]).transpose(-1, -2)).mul_(st["scale"])
    if c["softcap"]:
        score = score.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    score = score.view(s, hk, g, lq, keys)
    if st["slopes"] is not None:
        dist = (pos[..., None] - j).abs().float()
        score = score.sub_(st["slopes"].view(1, hk, g, 1, 1) * dist[:, None, None])
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    w = score.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = w.sum(-1, keepdim=True)
    v = gathered(st["vc"], st["v_scale"]).masked_fill_((j >= ctx[:, None])[:, None, :, None], 0.0)
    o = (w.view(s, hk, g * lq, keys) @ v).view(s, hk, g, lq, d) / total.masked_fill(total == 0, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(s, lq, h, d)
    t = torch.arange(q.shape[0], device=dev)
    seq = torch.searchsorted(qsl, t, right=True) - 1
    return o[seq, t - qsl[seq]].to(q.dtype)


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    if case["op"] == "maps":
        qlen, ctx = _lengths(case)
        need, have = -(-ctx // BLOCK), -(-(ctx - qlen) // BLOCK)
        s, grow = case["seqs"], int((need - have).sum())
        # block lists read and written, the list of new blocks, the lengths, per token slot and position
        return {"bytes": 8 * int(need.sum()) + 4 * grow + 4 * (3 * s) + 4 * (2 * s + 1)
                + 12 * (int(qlen.sum()) + s // 8), "flops": 4 * int(qlen.sum()) + 8 * s}
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    kvb = 2 if case["kv"] == "same" else 1
    if case["op"] == "rotary":
        t = case["tokens"]
        return {"bytes": t * (4 * h * d + 2 * hk * d * (2 + kvb) + 12),
                "flops": t * (3 * (h + hk) * case["rot"] + 20 * case["rot"])}
    keys = pairs = 0
    for lo, hi in _intervals(case):
        pairs += int((hi - lo).clip(0).sum())
        edge = np.zeros(int(hi.max()) + 1, np.int64)
        np.add.at(edge, lo, 1)
        np.add.at(edge, hi, -1)
        keys += int((edge.cumsum() > 0).sum())
    rows = int(_lengths(case)[0].sum())
    return {"bytes": 2 * keys * hk * d * kvb + 4 * rows * h * d + 4 * keys // BLOCK,
            "flops": 4 * pairs * h * d}


# ---- the definition in 64 bits -----------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "maps":
        rows, cached, qlen, new = (st[n].cpu().numpy().astype(np.int64)
                                   for n in ("rows", "cached", "qlen", "new"))
        tables, bt = st["tables"].cpu().numpy(), st["bt"].cpu().numpy()
        slots, pos = np.full(st["cap"], -1, np.int64), np.full(st["cap"], -1, np.int32)
        at = t = 0
        for i in range(case["seqs"]):
            mine = tables[rows[i]]
            for b in range(-(-cached[i] // BLOCK), -(-(cached[i] + qlen[i]) // BLOCK)):
                mine[b], at = new[at], at + 1
            n = -(-(cached[i] + qlen[i]) // BLOCK)
            bt[i, :n] = mine[:n]
            for p in range(cached[i], cached[i] + qlen[i]):
                slots[t], pos[t], t = int(mine[p // BLOCK]) * BLOCK + p % BLOCK, p, t + 1
        qsl = np.concatenate([[0], np.cumsum(qlen)])
        return (bt, (cached + qlen).astype(np.int32), qsl.astype(np.int32), slots, pos, tables)
    if case["op"] == "rotary":
        rot, d, half = case["rot"], case["head_dim"], case["rot"] // 2
        first = np.arange(half) if case["layout"] == "half" else np.arange(half) * 2
        second = first + (half if case["layout"] == "half" else 1)
        first, second = torch.from_numpy(first).cuda(), torch.from_numpy(second).cuda()
        z = torch.polar(torch.ones(case["tokens"], half, dtype=torch.float64, device="cuda"),
                        torch.outer(st["pos"].double(), torch.from_numpy(st["inv"]).cuda()))[:, None]

        def turned(x):
            y = x.double().clone()
            w = torch.complex(y[..., first], y[..., second]) * z
            y[..., first], y[..., second] = w.real, w.imag
            return y

        def cached(cache, x, scale):
            full = cache.double().permute(0, 2, 1, 3).reshape(-1, case["kv_heads"], d)
            full[st["slots"]] = x if case["kv"] == "same" else (x / scale).clamp(-448, 448)
            return full.view(-1, BLOCK, case["kv_heads"], d).permute(0, 2, 1, 3).contiguous()

        return (turned(st["q"]), cached(st["kc"], turned(st["k"]), st["k_scale"]),
                cached(st["vc"], st["v"].double(), st["v_scale"]))
    # attention, sequence by sequence and KV head by KV head
    qlen, ctx = _lengths(case)
    hk, d = case["kv_heads"], case["head_dim"]
    grp = case["heads"] // hk
    if float(qlen.max()) * float(ctx.max()) * hk * case["seqs"] > 3e9:
        return None
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    ks, vs = (st["k_scale"], st["v_scale"]) if case["kv"] == "e4m3" else (1.0, 1.0)
    r0 = 0
    for i, (lo, hi) in enumerate(_intervals(case)):
        n, c = int(qlen[i]), int(ctx[i])
        first = int(lo.min()) // BLOCK                       # no row looks at a block before
        ids = st["tables"][i, first:-(-c // BLOCK)].long()
        at = torch.arange(first * BLOCK, c, device="cuda")
        low, high = (torch.from_numpy(np.ascontiguousarray(x)).cuda()[:, None] for x in (lo, hi))
        hidden = (at < low) | (at >= high)
        here = torch.arange(c - n, c, device="cuda")[:, None]
        for kv in range(hk):
            key = st["kc"][:, kv].view(torch.uint8)[ids].view(st["kc"].dtype).double().reshape(-1, d)
            val = st["vc"][:, kv].view(torch.uint8)[ids].view(st["vc"].dtype).double().reshape(-1, d)
            key, val = key[:len(at)] * ks, val[:len(at)] * vs
            for head in range(kv * grp, (kv + 1) * grp):
                a = st["scale"] * torch.einsum("nd,kd->nk", st["q"][r0:r0 + n, head].double(), key)
                if case["softcap"]:
                    a = case["softcap"] * torch.tanh(a / case["softcap"])
                if case["alibi"]:
                    a = a - st["slopes"][head].double() * (here - at).abs()
                a[hidden] = -math.inf
                out[r0:r0 + n, head] = torch.softmax(a, 1).nan_to_num(0.0) @ val
        r0 += n
    return out
