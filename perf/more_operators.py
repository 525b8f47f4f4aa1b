"""Cases for encoder-decoder attention and for a block pool that lives on the GPU.

Five operators around the paged cache, for beam search, parallel samples and drafted
tokens without the host in the loop:

  cross    attention of ragged queries (a prompt, one token, a request's beams) to an
           encoder's states of another length in a paged cache
           (``paged_attention_cross``)
  fork     the block tables of a step's rows from those of their parents, with the
           blocks' reference counts (``fork_requests``)
  resize   blocks taken and given back as requests grow and shrink, with private copies
           of shared last blocks (``resize_requests``)
  copy     whole-block copies in the caches of all layers (``copy_blocks_layers``)
  compact  kept tokens of each sequence moved together in the caches of all layers
           (``compact_tokens``)

``run`` computes them from elementary torch operations in 32 bits, or, where ``own`` is
true, through this repository's entry points.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
TD = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # eight requests, one token each, encoder lengths from nothing to some 1500 states, one
        # head a group: the latency of a step
        dict(name="cross.greedy8", op="cross", seqs=8, min_q=1, max_q=1, min_enc=0, max_enc=1500, lens=41,
             heads=16, kv_heads=16, head_dim=64, dtype="fp16", kv="same"),
        # 32 requests of four to five beams over documents in an 8-bit cache
        dict(name="cross.beams_e4m3", op="cross", seqs=32, min_q=4, max_q=5, min_enc=512, max_enc=8192,
             lens=42, heads=32, kv_heads=8, head_dim=128, dtype="bf16", kv="e4m3"),
        # one token each over very long encoded inputs: every state is read for it
        dict(name="cross.long_decode", op="cross", seqs=4, min_q=1, max_q=1, min_enc=60000,
             max_enc=131071, lens=43, heads=64, kv_heads=8, head_dim=128, dtype="bf16", kv="same"),
        # target prompts (or a teacher-forced pass) over encoded documents, both ragged
        dict(name="cross.prompts", op="cross", seqs=6, min_q=300, max_q=1500, min_enc=700, max_enc=6000,
             lens=44, heads=32, kv_heads=8, head_dim=128, dtype="bf16", kv="same"),
        # beam search, 16 requests of 4 beams around 1000 tokens: the latency of a step
        dict(name="fork.beams64", op="fork", rows=64, group=4, table=128, max_ctx=1500, drop=0.0, lens=51),
        # 512 samples of long prompts, some of them finished
        dict(name="fork.long512", op="fork", rows=512, group=8, table=8192, max_ctx=131072, drop=0.05,
             lens=52),
        # a decode step of 64 beams: one token each, shared last blocks copied
        dict(name="resize.step64", op="resize", seqs=64, group=4, table=128, max_ctx=1500, grow=1,
             shrink=0.0, pool=16384, lens=53),
        # a loaded server: 8000 requests with drafts accepted and rejected, prompts admitted, some ended
        dict(name="resize.churn8000", op="resize", seqs=8000, group=2, table=256, max_ctx=1800, grow=64,
             shrink=0.3, pool=1000000, lens=54),
        # the copies of a step of a few beams
        dict(name="copy.beams8", op="copy", pairs=8, layers=4, kv_heads=8, head_dim=128, pool=64,
             dtype="fp16", skip=0.3, lens=61),
        # the copies of a step of 64 beams in all layers
        dict(name="copy.layers32", op="copy", pairs=64, layers=32, kv_heads=8, head_dim=128, pool=200,
             dtype="bf16", skip=0.3, lens=62),
        # drafted trees of 64 tokens verified, a path of each kept
        dict(name="compact.accept32", op="compact", seqs=32, layers=8, kv_heads=8, head_dim=128,
             dtype="bf16", max_ctx=1000, tail=64, share=0.07, lens=63),
        # long contexts of which half the tokens stay
        dict(name="compact.evict4", op="compact", seqs=4, layers=2, kv_heads=8, head_dim=128,
             dtype="fp16", max_ctx=16384, tail=16384, share=0.5, lens=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cross", "cross", "cross", "fork", "resize", "copy", "compact"])
    lens = rng.randrange(1 << 20)
    if op == "cross":
        heads, kv_heads = rng.choice([(32, 32), (32, 8), (64, 8), (16, 16), (14, 2), (16, 1), (12, 4)])
        most = _log_int(rng, 1, 1500)
        d = rng.choice([64, 128, 128])
        far = _log_int(rng, 16, 131071 if most < 4 else 20000 if most < 64 else 6000)
        far = min(far, 1500000000 // (4 * kv_heads * d))
        # at most the largest listed cases' bytes and products
        seqs = min(_log_int(rng, 1, 48), 1500000000 // (4 * kv_heads * d * far),
                   240000000000 // (4 * heads * d * most * far))
        return dict(op=op, seqs=max(1, seqs), min_q=max(1, most // rng.choice([1, 2, 30])), max_q=most,
                    min_enc=far // rng.choice([1, 2, 10 ** 6]), max_enc=far, lens=lens, heads=heads,
                    kv_heads=kv_heads, head_dim=d, dtype=rng.choice(["bf16", "fp16"]),
                    kv=rng.choice(["same", "same", "e4m3"]))
    if op == "fork":
        table = _log_int(rng, 4, 8192)
        return dict(op=op, rows=_log_int(rng, 1, 512), group=rng.choice([1, 2, 4, 5, 8]), table=table,
                    max_ctx=rng.randint(1, table * BLOCK), drop=rng.choice([0.0, 0.05, 0.5]), lens=lens)
    if op == "resize":
        seqs, table = _log_int(rng, 1, 8000), rng.choice([64, 100, 256])
        return dict(op=op, seqs=seqs, group=rng.choice([1, 2, 4, 5]), table=table,
                    max_ctx=rng.randint(20, table * BLOCK - 600), grow=_log_int(rng, 1, 512),
                    shrink=rng.choice([0.0, 0.3, 0.9]), lens=lens,
                    pool=min(1000000, seqs * table + _log_int(rng, 1, 10000)))
    layers, dtype = _log_int(rng, 1, 16), rng.choice(["bf16", "fp16"])
    kv_heads, d = rng.choice([1, 2, 8, 32]), rng.choice([64, 128])
    if op == "copy":
        pairs = _log_int(rng, 1, 64)
        return dict(op=op, pairs=pairs, layers=layers, kv_heads=kv_heads, head_dim=d,
                    pool=2 * pairs + rng.randint(1, 100), dtype=dtype, skip=rng.choice([0.0, 0.3]), lens=lens)
    seqs = _log_int(rng, 1, 32)
    most = max(20, (1 << 29) // (seqs * layers * kv_heads * d * 4))  # half a gigabyte of caches
    ctx = min(most, _log_int(rng, 20, 16384))
    return dict(op=op, seqs=seqs, layers=layers, kv_heads=kv_heads, head_dim=d, dtype=dtype, max_ctx=ctx,
                tail=rng.choice([ctx, min(ctx, 64)]), share=rng.choice([0.07, 0.5, 0.95]), lens=lens)


# ---- inputs ----------------------------------------------------------------------------------

def _cross_lengths(case):
    """(queries, encoder states) of a case's sequences: the case's own, whatever the seed."""
    r = np.random.RandomState(case["lens"])
    return (r.randint(case["min_q"], case["max_q"] + 1, case["seqs"]).astype(np.int64),
            r.randint(case["min_enc"], case["max_enc"] + 1, case["seqs"]).astype(np.int64))


def _groups(rows, group, max_ctx, r):
    """Context lengths of rows that came in groups of one prompt: equal in a group."""
    return np.repeat(r.randint(1, max_ctx + 1, -(-rows // group)), group)[:rows].astype(np.int64)


def _tables(ctx, group, table, pool, r):
    """Block tables of rows in groups that share their blocks up to the group's own first
    part, the reference counts, and the number of blocks of the pool in use."""
    rows = len(ctx)
    tables, counts, at = np.full((rows, table), -1, np.int64), np.zeros(pool, np.int64), 0
    ids = r.permutation(pool)
    for g0 in range(0, rows, group):
        n = -(-int(ctx[g0]) // BLOCK)
        alike = n if r.rand() < 0.5 else int(r.randint(0, n + 1))   # shared blocks of this group
        first = ids[at:at + n]
        at += n
        for row in range(g0, min(g0 + group, rows)):
            tables[row, :n] = first
            if row > g0 and alike < n:
                tables[row, alike:n] = ids[at:at + n - alike]
                at += n - alike
            counts[tables[row, :n]] += 1
    return tables, counts, at


def _parents(case, r):
    """Beams go on from beams of their own group; a row that is dropped has no parent."""
    rows, group = case["rows"], case["group"]
    first = np.arange(rows) // group * group
    par = first + r.randint(0, 1 << 30, rows) % np.minimum(group, rows - first)
    return np.where(r.rand(rows) < case["drop"], -1, par)


def _resize_lengths(case):
    r = np.random.RandomState(case["lens"])
    s = case["seqs"]
    cached = _groups(s, case["group"], case["max_ctx"], r)
    new = cached + r.randint(1, case["grow"] + 1, s)
    new = np.where(r.rand(s) < case["shrink"], (cached * r.rand(s)).astype(np.int64), new)
    rows = r.permutation(2 * s)[:s]
    rows[r.rand(s) < 0.02] = -1              # places of a captured step that nothing fills
    return rows, cached, new


def _kept(case):
    """(context lengths, first moved place, offsets of the kept lists, kept positions)."""
    r = np.random.RandomState(case["lens"])
    ctx = r.randint(max(1, case["max_ctx"] // 2), case["max_ctx"] + 1, case["seqs"]).astype(np.int64)
    base = np.maximum(ctx - case["tail"], 0)
    keep = [b + np.flatnonzero(r.rand(int(c - b)) < case["share"]) for b, c in zip(base, ctx)]
    return ctx, base, np.concatenate([[0], np.cumsum([len(k) for k in keep])]), np.concatenate(keep)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 31))
    dev, st = "cuda", dict(case=dict(case))

    def ints(a, dtype=torch.int32):
        return torch.from_numpy(np.ascontiguousarray(a)).to(dev, dtype)

    def randn(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device=dev) * scale

    if case["op"] == "cross":
        qlen, enc = _cross_lengths(case)
        dt, h, hk, d = TD[case["dtype"]], case["heads"], case["kv_heads"], case["head_dim"]
        need = -(-enc // BLOCK)
        width = max(1, int(need.max()))
        nb = int(need.sum()) * 5 // 4 + 1
        ids, at = r.permutation(nb), 0
        tables = np.full((case["seqs"], width), -1, np.int64)
        for i, n in enumerate(need):
            tables[i, :n] = ids[at:at + n]
            at += n

        def cache():
            if case["kv"] == "same":
                return torch.randn((nb, hk, BLOCK, d), generator=g, device=dev, dtype=dt), 1.0
            x = randn(nb, hk, BLOCK, d)
            scale = float(x.abs().amax()) / 448
            return (x / scale).clamp_(-448, 448).to(torch.float8_e4m3fn), scale

        (kc, ks), (vc, vs) = cache(), cache()
        rows = int(qlen.sum())
        st.update(q=randn(rows, h, d, scale=2.0).to(dt), kc=kc, vc=vc, k_scale=ks, v_scale=vs,
                  tables=ints(tables), enc=ints(enc), qsl=ints(np.concatenate([[0], np.cumsum(qlen)])),
                  scale=d ** -0.5, max_q=case["max_q"], max_enc=case["max_enc"],
                  out=torch.empty((rows, h, d), dtype=dt, device=dev))
        return st

    if case["op"] == "fork":
        rl = np.random.RandomState(case["lens"])
        ctx = _groups(case["rows"], case["group"], case["max_ctx"], rl)
        pool = int((-(-ctx // BLOCK)).sum()) + 16
        tables, counts, _ = _tables(ctx, case["group"], case["table"], pool, r)
        st.update(tables=ints(tables), lens=ints(ctx), counts=ints(counts), parents=ints(_parents(case, r)),
                  tables_out=torch.full((case["rows"], case["table"]), -1, dtype=torch.int32, device=dev),
                  lens_out=torch.zeros(case["rows"], dtype=torch.int32, device=dev),
                  work=torch.empty(pool, dtype=torch.int32, device=dev))
        return st

    if case["op"] == "resize":
        rows, cached, new = _resize_lengths(case)
        s = case["seqs"]
        tables, counts, _ = _tables(cached, case["group"], case["table"], case["pool"], r)
        held = np.full((2 * s, case["table"]), -1, np.int64)
        idle = rows < 0
        held[rows[~idle]] = tables[~idle]
        for row, n in zip(tables[idle], -(-cached[idle] // BLOCK)):   # nobody holds these
            counts[row[:n]] -= 1
        opens = int(np.maximum(-(-new // BLOCK) - -(-cached // BLOCK), 0).sum())
        st.update(tables=ints(held), counts=ints(counts), rows=ints(rows), cached=ints(cached),
                  new=ints(new), cap=opens + s // 8 + 1,
                  granted=torch.empty(s, dtype=torch.int32, device=dev),
                  opened=torch.empty(opens + s // 8 + 1, dtype=torch.int32, device=dev),
                  pairs=torch.empty((s, 2), dtype=torch.int32, device=dev))
        return st

    dt, hk, d = TD[case["dtype"]], case["kv_heads"], case["head_dim"]
    if case["op"] == "copy":
        ids = 1 + r.permutation(case["pool"] - 1)
        n = case["pairs"]
        pairs = np.stack([ids[r.randint(0, max(1, len(ids) - n), n)], ids[len(ids) - n:]], 1)
        pairs[r.rand(n) < case["skip"]] = -1        # a sequence that had nothing to copy
        nb = case["pool"]
        st.update(pairs=ints(pairs))
    else:
        ctx, base, ksl, keep = _kept(case)
        need = -(-ctx // BLOCK)
        nb = int(need.sum()) + 7
        ids, at = r.permutation(nb), 0
        tables = np.full((case["seqs"], int(need.max())), -1, np.int64)
        for i, n in enumerate(need):
            tables[i, :n] = ids[at:at + n]
            at += n
        st.update(tables=ints(tables), ctx=ints(ctx), base=ints(base), ksl=ints(ksl), keep=ints(keep),
                  counts=ints(np.isin(np.arange(nb), ids[:at])),
                  new=torch.empty(case["seqs"], dtype=torch.int32, device=dev))
    caches = torch.randn((case["layers"], 2, nb, hk, BLOCK, d), generator=g, device=dev, dtype=dt)
    st.update(caches=caches, k_caches=caches[:, 0], v_caches=caches[:, 1])
    return st


# ---- one pass --------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return {"cross": _cross, "fork": _fork, "resize": _resize, "copy": _copy, "compact": _compact}[op](state)


def _own(op, st):
    import paged_kv_cache_98_gb300 as pkv
    if op == "cross":
        return pkv.paged_attention_cross(st["out"], st["q"], st["kc"], st["vc"], st["tables"], st["enc"],
                                         st["qsl"], st["scale"], max_q_len=st["max_q"],
                                         max_encoder_len=st["max_enc"], k_scale=st["k_scale"],
                                         v_scale=st["v_scale"])
    if op == "fork":
        counts = st["work"].copy_(st["counts"])    # (the call updates them in place)
        pkv.fork_requests(st["tables_out"], st["lens_out"], st["tables"], st["lens"], counts, st["parents"])
        return st["tables_out"], st["lens_out"], counts
    if op == "resize":
        tables, counts = st["tables"].clone(), st["counts"].clone()
        pkv.resize_requests(tables, counts, st["rows"], st["cached"], st["new"], st["granted"],
                            st["opened"], st["pairs"])
        return tables, counts, st["granted"], st["opened"], st["pairs"]
    if op == "copy":
        pkv.copy_blocks_layers(st["k_caches"], st["v_caches"], st["pairs"])
        return st["caches"]
    pkv.compact_tokens(st["k_caches"], st["v_caches"], st["tables"], st["ctx"], st["base"], st["ksl"],
                       st["keep"], st["new"], ref_counts=st["counts"])
    return st["caches"], st["new"]


def _cross(st):
    """Softmax attention of every query row over its sequence's encoder states, on padded batches."""
    c, q, qsl, enc = st["case"], st["q"], st["qsl"].long(), st["enc"].long()
    s, h, hk, d, lq = c["seqs"], c["heads"], c["kv_heads"], c["head_dim"], st["max_q"]
    dev, g = q.device, h // hk
    idx = st["tables"].long().clamp(min=0)
    keys = idx.shape[1] * BLOCK

    def gathered(cache, scale):
        x = cache.view(torch.uint8)[idx].view(cache.dtype) if c["kv"] == "e4m3" else cache[idx]
        x = x.transpose(1, 2).reshape(s, hk, keys, d).float()
        return x.mul_(scale) if c["kv"] == "e4m3" else x

    row = (qsl[:-1, None] + torch.arange(lq, device=dev)).clamp(max=q.shape[0] - 1)      # [s, lq]
    past = torch.arange(keys, device=dev) >= enc[:, None]                                # [s, keys]
    x = q.float()[row].view(s, lq, hk, g, d).permute(0, 2, 3, 1, 4).reshape(s, hk, g * lq, d)
    score = (x @ gathered(st["kc"], st["k_scale"]).transpose(-1, -2)).mul_(st["scale"])
    score = score.masked_fill_(past[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    w = score.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = w.sum(-1, keepdim=True)
    v = gathered(st["vc"], st["v_scale"]).masked_fill_(past[:, None, :, None], 0.0)
    o = (w @ v).view(s, hk, g, lq, d) / total.masked_fill(total == 0, 1.0).view(s, hk, g, lq, 1)
    o = o.permute(0, 3, 1, 2, 4).reshape(s, lq, h, d)
    t = torch.arange(q.shape[0], device=dev)
    seq = torch.searchsorted(qsl, t, right=True) - 1
    return o[seq, t - qsl[seq]].to(q.dtype)


def _fork(st):
    tables, lens, par = st["tables"], st["lens"].long(), st["parents"].long()
    counts = st["work"].copy_(st["counts"])
    from_, has = par.clamp(min=0), par >= 0
    col = torch.arange(tables.shape[1], device=tables.device)
    lens_out = torch.where(has, lens[from_], 0)
    mine = col < ((lens_out + BLOCK - 1) // BLOCK)[:, None]
    tables_out = torch.where(mine, tables[from_], st["tables_out"])
    # a row's blocks gain a holder for each child and lose the row itself
    change = torch.zeros_like(lens).index_add_(0, from_, has.long()) - 1
    held = col < ((lens + BLOCK - 1) // BLOCK)[:, None]
    counts.index_add_(0, tables.clamp(min=0).view(-1).long(), (held * change[:, None]).view(-1).int())
    return tables_out, lens_out.int(), counts


def _resize(st):
    dev = st["tables"].device
    tables, counts = st["tables"].clone(), st["counts"].long()
    rows, pool = st["rows"].long(), st["counts"].numel()
    live = rows >= 0
    rows = rows.clamp(min=0)
    cached, new = torch.where(live, st["cached"].long(), 0), torch.where(live, st["new"].long(), 0)
    s, width = rows.numel(), tables.shape[1]
    col, order = torch.arange(width, device=dev), torch.arange(s, device=dev)
    mine = tables[rows].long()
    have, need = (cached + BLOCK - 1) // BLOCK, (new + BLOCK - 1) // BLOCK
    # blocks behind the new lengths go back
    gone = (col >= need[:, None]) & (col < have[:, None])
    counts.index_add_(0, mine.clamp(min=0).view(-1), -gone.view(-1).long())
    mine = torch.where(gone, -1, mine)
    # a partial last block that others hold too is copied, but by the last of its holders
    # where all of them grow
    last = (cached // BLOCK).clamp(max=width - 1)[:, None]
    part = (new > cached) & (cached % BLOCK != 0)
    tail = torch.where(part, mine.gather(1, last)[:, 0], pool)
    holders = torch.zeros(pool + 1, dtype=torch.long, device=dev).index_add_(0, tail, torch.ones_like(tail))
    latest = torch.full((pool + 1,), -1, device=dev).scatter_reduce_(0, tail, order, "amax")
    held = torch.cat([counts, counts.new_zeros(1)])[tail]
    copies = part & (held > 1) & ~((holders[tail] == held) & (latest[tail] == order))
    opens = (need - have).clamp(min=0)
    # free blocks in the order of their ids, to the sequences in batch order
    want = opens + copies
    end = want.cumsum(0)
    free = counts == 0
    granted = (want == 0) | (end <= free.sum())
    rank = torch.where(free, free.cumsum(0) - 1, pool)
    ids = torch.full((pool + 1,), -1, device=dev).scatter_(0, rank, torch.arange(pool, device=dev))
    begin = end - want
    copies, opens = copies & granted, torch.where(granted, opens, 0)
    copy = ids[begin.clamp(max=pool)]
    mine.scatter_(1, last, torch.where(copies, copy, mine.gather(1, last)[:, 0])[:, None])
    at = begin[:, None] + copies[:, None].long() + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < (have + opens)[:, None])
    mine = torch.where(fresh, ids[at.clamp(0, pool)], mine)
    counts.index_add_(0, torch.where(copies, tail, 0), -copies.long())
    counts = torch.where(free & (rank < torch.where(granted, want, 0).sum()), 1, counts)
    tables = torch.cat([tables, tables[:1]]).index_copy_(
        0, torch.where(live, rows, tables.shape[0]), mine.int())[:-1]
    off = opens.cumsum(0) - opens
    n = torch.arange(st["cap"], device=dev)
    seq = torch.searchsorted(opens.cumsum(0), n, right=True).clamp(max=s - 1)
    opened = mine[seq, (have[seq] + n - off[seq]).clamp(max=width - 1)]
    opened = torch.where(n < opens.sum(), opened, -1)
    pairs = torch.where(copies[:, None], torch.stack([tail, copy], 1), -1)
    return (tables, counts.int(), torch.where(live, torch.where(granted, new, cached), 0).int(),
            opened.int(), pairs.int())


def _copy(st):
    src, dst = st["pairs"].long().unbind(1)
    dst = torch.where(src < 0, 0, dst)               # (block 0, which no pair names, onto itself)
    st["caches"][:, :, dst] = st["caches"][:, :, src.clamp(min=0)]
    return st["caches"]


def _compact(st):
    ksl, base, tables, keep = st["ksl"].long(), st["base"].long(), st["tables"].long(), st["keep"].long()
    t = torch.arange(keep.numel(), device=keep.device)
    seq = torch.searchsorted(ksl, t, right=True) - 1
    to = base[seq] + t - ksl[seq]
    rows = st["caches"][:, :, tables[seq, keep // BLOCK], :, keep % BLOCK]
    st["caches"][:, :, tables[seq, to // BLOCK], :, to % BLOCK] = rows
    return st["caches"], (base + ksl[1:] - ksl[:-1]).int()


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    if case["op"] == "cross":
        qlen, enc = _cross_lengths(case)
        h, hk, d, rows = case["heads"], case["kv_heads"], case["head_dim"], int(qlen.sum())
        keys = int(enc[qlen > 0].sum())
        return {"bytes": 2 * keys * hk * d * (2 if case["kv"] == "same" else 1) + 4 * rows * h * d
                + 4 * keys // BLOCK, "flops": 4 * int((qlen * enc).sum()) * h * d}
    if case["op"] == "fork":
        ctx = _groups(case["rows"], case["group"], case["max_ctx"], np.random.RandomState(case["lens"]))
        held = int((-(-ctx // BLOCK)).sum())
        # the tables read and written, and the counts of their blocks read and written
        return {"bytes": 16 * held + 12 * case["rows"], "flops": held}
    if case["op"] == "resize":
        rows, cached, new = _resize_lengths(case)
        moved = int(np.abs(-(-new // BLOCK) - -(-cached // BLOCK))[rows >= 0].sum())
        # the lengths, pairs and tables' ends, the entries and counts that change, and the
        # counts up to the last block that is handed out (the pool is the least that is known)
        return {"bytes": 28 * case["seqs"] + 16 * moved + 4 * case["pool"], "flops": case["pool"]}
    row = case["kv_heads"] * case["head_dim"] * 4 * case["layers"]   # of K and V, all layers
    if case["op"] == "copy":
        n = case["pairs"] * (1 - case["skip"])
        return {"bytes": 2 * n * BLOCK * row, "flops": 0}
    ctx, base, ksl, keep = _kept(case)
    to = np.concatenate([b + np.arange(n) for b, n in zip(base, np.diff(ksl))])
    moved = int((to != keep).sum())
    return {"bytes": 2 * moved * row + 8 * len(keep), "flops": 0}


# ---- the definition, in 64 bits and one after the other ------------------------------------------

def exact(case, seed):
    if case["op"] in ("copy", "compact"):
        return None
    st = prepare(case, seed)
    if case["op"] == "cross":
        qlen, enc = _cross_lengths(case)
        if float((qlen * enc).sum()) * case["heads"] > 3e9:
            return None
        hk, d = case["kv_heads"], case["head_dim"]
        grp = case["heads"] // hk
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        ks, vs = (st["k_scale"], st["v_scale"]) if case["kv"] == "e4m3" else (1.0, 1.0)
        r0 = 0
        for i in range(case["seqs"]):
            n, c = int(qlen[i]), int(enc[i])
            ids = st["tables"][i, :-(-c // BLOCK)].long()
            for kv in range(hk if c else 0):
                key, val = (x[:, kv].view(torch.uint8)[ids].view(x.dtype).double().reshape(-1, d)[:c]
                            for x in (st["kc"], st["vc"]))
                for head in range(kv * grp, (kv + 1) * grp):
                    a = torch.einsum("nd,kd->nk", st["q"][r0:r0 + n, head].double(), key)
                    a = torch.softmax(a * (st["scale"] * ks), 1)
                    out[r0:r0 + n, head] = torch.einsum("nk,kd->nd", a, val) * vs
            r0 += n
        return out
    if case["op"] == "fork":
        tables, lens, counts, par = (st[n].cpu().numpy() for n in ("tables", "lens", "counts", "parents"))
        tables_out, lens_out = st["tables_out"].cpu().numpy(), st["lens_out"].cpu().numpy()
        for i, p in enumerate(par):
            lens_out[i] = lens[p] if p >= 0 else 0
            n = -(-lens_out[i] // BLOCK)
            tables_out[i, :n] = tables[p, :n]
            np.add.at(counts, tables_out[i, :n], 1)
        for i, c in enumerate(lens):
            np.add.at(counts, tables[i, :-(-c // BLOCK)], -1)
        return tables_out, lens_out, counts
    tables, counts, rows, cached, new = (st[n].cpu().numpy().astype(np.int64)
                                         for n in ("tables", "counts", "rows", "cached", "new"))
    s = case["seqs"]
    for i in range(s):
        if rows[i] >= 0:
            for b in range(-(-new[i] // BLOCK), -(-cached[i] // BLOCK)):
                counts[tables[rows[i], b]] -= 1
                tables[rows[i], b] = -1
    free = iter(np.flatnonzero(counts == 0).tolist())
    left = int((counts == 0).sum())
    granted, opened, pairs = np.zeros(s, np.int64), [], np.full((s, 2), -1, np.int64)
    for i in range(s):
        if rows[i] < 0:
            continue
        mine, have, need = tables[rows[i]], -(-cached[i] // BLOCK), -(-new[i] // BLOCK)
        granted[i] = new[i]
        if new[i] <= cached[i]:
            continue
        old = mine[have - 1] if cached[i] % BLOCK else -1
        copy = old >= 0 and counts[old] > 1
        want = need - have + copy
        assert want <= left, "the cases' pools are large enough"
        left -= want
        if copy:
            mine[have - 1] = next(free)
            counts[mine[have - 1]] = 1
            counts[old] -= 1
            pairs[i] = old, mine[have - 1]
        for b in range(have, need):
            mine[b] = next(free)
            counts[mine[b]] = 1
            opened.append(mine[b])
    opened = np.array(opened + [-1] * (st["cap"] - len(opened)))
    return tuple(x.astype(np.int32) for x in (tables, counts, granted, opened, pairs))
