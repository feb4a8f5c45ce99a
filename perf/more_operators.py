"""Cases for the pages of the cache, sparse attention over them and the selection of beams.

Five operators of a serving loop over the paged KV cache:

* ``beam``     beam search's selection: log-softmax of each beam's logits, added to the beam's score,
               the best continuations over beams and vocabulary, ties to the lowest index;
* ``pages``    what follows it on the cache's block tables: the children take their parents' blocks,
               blocks of the next tokens are reserved with copies where a partly filled block is
               shared, the pages are copied in every layer's pool, finished sequences are freed;
* ``compact``  the pool's live blocks moved into its low end, tables and counts with them;
* ``index``    the bounds of each block's keys that the sparse selection reads, after an append;
* ``sparse``   for each query token and KV head the blocks with the largest bound of q.k are selected
               (with the first and the last ones), and attention runs over those alone.

Layouts are the library's: q ``[n, Hq, D]``, pool ``[num_blocks, 2, Hkv, 16, D]``, block tables
``[rows, max_blocks]``, reference counts ``[num_blocks]`` (0: the block is free).
"""

import math

import numpy as np
import torch

own = False

BLOCK = 16
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one request of a small model, 4 beams: the latency of the call
        dict(name="beam 4 beams", op="beam", batch=1, beams=4, vocab=32000, num=4, dtype="bf16",
             done=0.0, pad=0),
        # an odd vocabulary whose rows start unaligned, 10 candidates for 5 beams, some finished
        dict(name="beam odd vocabulary", op="beam", batch=37, beams=5, vocab=50257, num=10,
             dtype="fp16", done=0.2, pad=0),
        # a busy server: 64 requests of 8 beams, logits kept in 32 bits by a padded projection
        dict(name="beam 512 beams", op="beam", batch=64, beams=8, vocab=128000, num=16,
             dtype="fp32", done=0.05, pad=256),
        # one request's 4 beams: the latency of the calls
        dict(name="pages 4 beams", op="pages", rows=4, group=4, hkv=8, d=64, layers=2, fp8=False,
             ctx_lo=300, ctx_hi=700, q_hi=1, done=0.0, lens=1),
        # 64 requests of 4 beams, contexts to 8192, four layers of the 8-bit pool
        dict(name="pages 256 beams", op="pages", rows=256, group=4, hkv=8, d=128, layers=4,
             fp8=True, ctx_lo=64, ctx_hi=8192, q_hi=3, done=0.1, lens=2),
        # a small pool after its long sequences ended
        dict(name="compact small pool", op="compact", blocks=1201, live=0.5, rows=9, hkv=2, d=64,
             layers=1, fp8=False, lens=3),
        # a large 8-bit pool, scattered: a third of it lives
        dict(name="compact large pool", op="compact", blocks=40000, live=0.35, rows=300, hkv=8,
             d=128, layers=2, fp8=True, lens=4),
        # after the append of one decode step of 256 sequences
        dict(name="index 256 decodes", op="index", hkv=8, d=128, seqs=256, q_lo=1, q_hi=1, chunk=0,
             lens=5),
        # after the append of long prompts: 30000 + 5000 tokens
        dict(name="index 35000 tokens", op="index", hkv=8, d=128, seqs=1, q_lo=5000, q_hi=5000,
             chunk=30000, lens=6),
        # one decode at 4096: the latency of the calls
        dict(name="sparse 1 decode", op="sparse", hq=16, hkv=8, d=128, seqs=1, q_lo=1, q_hi=1,
             ctx_lo=4096, ctx_hi=4096, num=32, sink=1, recent=2, lens=7),
        # verify windows on a small head, every length from the shortest contexts on
        dict(name="sparse verify windows", op="sparse", hq=8, hkv=2, d=64, seqs=61, q_lo=1, q_hi=6,
             ctx_lo=9, ctx_hi=16001, num=48, sink=2, recent=3, lens=8),
        # 24 decodes of very long contexts
        dict(name="sparse 24 decodes long", op="sparse", hq=40, hkv=8, d=128, seqs=24, q_lo=1,
             q_hi=1, ctx_lo=30000, ctx_hi=131072, num=128, sink=4, recent=8, lens=9),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["beam", "beam", "pages", "compact", "index", "sparse", "sparse"])
    hkv, group, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128])
    c = dict(op=op, lens=rng.randrange(1 << 30))
    if op == "beam":
        c["vocab"], c["beams"] = _log_int(rng, 100, 128000), rng.randint(1, 12)
        c["batch"] = _log_int(rng, 1, max(1, min(100, 30_000_000 // (c["vocab"] * c["beams"]))))
        c["num"] = rng.randint(1, 3 * c["beams"])
        c.update(dtype=rng.choice(list(DTYPES)), done=rng.choice([0.0, 0.3]), pad=rng.choice([0, 3, 128]))
    elif op == "pages":
        c["group"] = rng.choice([1, 2, 3, 4, 8])
        c["rows"] = c["group"] * _log_int(rng, 1, 256 // c["group"])
        c.update(hkv=hkv, d=d, layers=rng.randint(1, 4), fp8=rng.random() < 0.5, ctx_lo=1,
                 ctx_hi=_log_int(rng, 20, 8000), q_hi=rng.choice([1, 1, 5, 40]),
                 done=rng.choice([0.0, 0.3]))
    elif op == "compact":
        c["blocks"] = _log_int(rng, 10, 20000)
        c.update(live=rng.uniform(0.05, 0.95), rows=_log_int(rng, 1, 300), hkv=hkv, d=d,
                 layers=rng.randint(1, 2), fp8=rng.random() < 0.5)
    elif op == "index":
        c.update(hkv=hkv, d=d, seqs=_log_int(rng, 1, 400), q_lo=1, q_hi=rng.choice([1, 4, 60]))
        c["chunk"] = rng.choice([0, _log_int(rng, 17, 20000)])
    else:
        c.update(hq=hkv * group, hkv=hkv, d=d, seqs=_log_int(rng, 1, 64), q_lo=1,
                 q_hi=rng.choice([1, 1, 4, 9]), sink=rng.randint(0, 4), recent=rng.randint(1, 8))
        c["ctx_lo"], c["ctx_hi"] = 9, _log_int(rng, 40, min(100000, 1200000 // c["seqs"]))
        c["num"] = c["sink"] + c["recent"] + _log_int(rng, 1, 100)
    return c


# ----------------------------------------------------------------------------------- inputs

def _normal(g, shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _on(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _pools(g, case, blocks):
    """Every layer's pool, and the 8-bit pools' scales: the rows of all of them go with a block."""
    shape = (blocks, 2, case["hkv"], BLOCK, case["d"])
    pools = []
    for _ in range(case["layers"]):
        x = torch.empty(shape, dtype=torch.float8_e4m3fn if case["fp8"] else torch.bfloat16, device=DEV)
        step = max(1, (1 << 28) // (2 * case["hkv"] * BLOCK * case["d"]))
        for b in range(0, blocks, step):
            x[b:b + step] = _normal(g, (min(step, blocks - b), *shape[1:])).to(x.dtype)
        pools.append(x)
        if case["fp8"]:
            pools.append(torch.exp2(torch.randint(-9, 2, (blocks, case["hkv"], 2), generator=g,
                                                  device=DEV).float()))
    return pools


def _beam_tables(case):
    """Tables of beams that share a prompt, and each its own blocks after it; reference counts."""
    r = np.random.default_rng(case["lens"])
    rows, group = case["rows"], case["group"]
    lo, hi = case["ctx_lo"], max(case["ctx_lo"], case["ctx_hi"])
    prompt = np.exp(r.uniform(math.log(lo), math.log(hi + 1), size=rows // group)).astype(np.int64)
    prompt = np.clip(prompt, lo, hi)
    gone = r.integers(0, 70, size=rows // group)              # tokens generated since the prompt
    ctx = np.repeat(prompt + gone, group)
    kept = np.repeat(prompt // BLOCK, group)
    q = r.integers(1, case["q_hi"], size=rows, endpoint=True)
    need = -(-ctx // BLOCK)
    width = int((-(-(ctx + q) // BLOCK)).max()) + 1
    total = int((prompt // BLOCK).sum() + (need - kept).sum())
    blocks = total + total // 8 + rows * (2 + case["q_hi"] // BLOCK) + 3
    perm = r.permutation(blocks)
    table, refs, at = np.full((rows, width), -1, dtype=np.int64), np.zeros(blocks, dtype=np.int64), 0
    for s in range(rows):
        if s % group == 0:
            shared = perm[at:at + kept[s]]
            at += kept[s]
        table[s, :kept[s]] = shared
        table[s, kept[s]:need[s]] = perm[at:at + need[s] - kept[s]]
        at += need[s] - kept[s]
        refs[table[s, :need[s]]] += 1
    # the beams that go on: some parents twice, some not at all
    parents = np.arange(rows) // group * group + r.integers(0, group, size=rows)
    done = np.where(r.random(rows) < case["done"], np.arange(rows), -1)
    return ctx, q, table, refs, parents, done


def _scattered(case):
    """A pool some of whose blocks live, referred to by the tables of ragged sequences."""
    r = np.random.default_rng(case["lens"])
    blocks, rows = case["blocks"], case["rows"]
    live = max(1, int(blocks * case["live"]))
    ids = r.permutation(blocks)[:live]
    cut = np.sort(r.integers(0, live + 1, size=rows - 1)) if rows > 1 else np.zeros(0, dtype=np.int64)
    begin, end = np.concatenate([[0], cut]), np.concatenate([cut, [live]])
    width = int((end - begin).max()) + 2
    table, refs = np.full((rows, width), -1, dtype=np.int64), np.zeros(blocks, dtype=np.int64)
    ctx = np.zeros(rows, dtype=np.int64)
    for s, (a, b) in enumerate(zip(begin, end)):
        n = b - a
        table[s, :n] = ids[a:b]
        if s and s % 3 == 0:                  # a third of them go on from another's first blocks
            m = min(n, end[s - 1] - begin[s - 1]) // 2
            table[s, :m] = ids[begin[s - 1]:begin[s - 1] + m]
        ctx[s] = n * BLOCK - (r.integers(0, BLOCK) if n else 0)
        refs[table[s, :n]] += 1
    return ctx, table, refs


def _windows(case):
    """q_lens, context_lens and block tables of sequences with ragged contexts."""
    r = np.random.default_rng(case["lens"])
    q = r.integers(case["q_lo"], case["q_hi"], size=case["seqs"], endpoint=True)
    lo, hi = case["ctx_lo"], max(case["ctx_lo"], case["ctx_hi"])
    ctx = np.exp(r.uniform(math.log(lo), math.log(hi + 1), size=case["seqs"])).astype(np.int64)
    ctx = np.maximum(np.clip(ctx, lo, hi), q)
    need = -(-ctx // BLOCK)
    blocks = int(need.sum()) * 11 // 10 + 2
    perm = r.permutation(blocks)
    table, at = np.full((len(q), int(need.max())), -1, dtype=np.int64), 0
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n]
        at += n
    return q, ctx, table, blocks


def _written(case):
    """Slots of a step's new tokens, the pool's blocks: only blocks that the step writes."""
    r = np.random.default_rng(case["lens"])
    q = r.integers(case["q_lo"], case["q_hi"], size=case["seqs"], endpoint=True)
    first = r.integers(0, 200, size=case["seqs"])
    if case["chunk"]:
        q, first = np.concatenate([[case["chunk"]], q]), np.concatenate([[0], first])
    pos = np.concatenate([np.arange(f, f + n) for f, n in zip(first, q)])
    key = np.repeat(np.arange(len(q)), q) * (1 << 24) + pos // BLOCK
    uniq, inv = np.unique(key, return_inverse=True)
    blocks = len(uniq) + len(uniq) // 10 + 2
    return r.permutation(blocks)[inv] * BLOCK + pos % BLOCK, blocks


def _keyed_pool(g, blocks, hkv, d):
    """A bf16 pool whose keys lie about a centre of their block, as text's keys do."""
    pool = torch.empty((blocks, 2, hkv, BLOCK, d), dtype=torch.bfloat16, device=DEV)
    step = max(1, (1 << 27) // (2 * hkv * BLOCK * d))
    for b in range(0, blocks, step):
        n = min(step, blocks - b)
        x = _normal(g, (n, 2, hkv, BLOCK, d))
        x[:, 0] = 0.6 * x[:, 0] + 0.8 * _normal(g, (n, hkv, 1, d))
        pool[b:b + step] = x.to(torch.bfloat16)
    return pool


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, s = case["op"], dict(op=case["op"])
    i32 = dict(dtype=torch.int32, device=DEV)
    if op == "beam":
        b, k, v, m = case["batch"], case["beams"], case["vocab"], case["num"]
        rows = _normal(g, (b, k, v + case["pad"])).mul_(2.5).to(DTYPES[case["dtype"]])
        s.update(logits=rows[:, :, :v], num=m, pad_token=2 % v,
                 cum=(-20.0 * torch.rand((b, k), generator=g, device=DEV)).sort(1, descending=True)[0],
                 finished=torch.rand((b, k), generator=g, device=DEV) < case["done"],
                 scores=torch.empty((b, m), dtype=torch.float32, device=DEV),
                 tokens=torch.empty((b, m), **i32), parents=torch.empty((b, m), **i32))
    elif op == "pages":
        ctx, q, table, refs, parents, done = _beam_tables(case)
        s.update(ctx=_on(ctx), cu=_on(np.concatenate([[0], np.cumsum(q)])), table=_on(table),
                 refs0=_on(refs), refs=_on(refs), parents=_on(parents), done=_on(done),
                 new_table=torch.full(table.shape, -1, **i32), new_ctx=torch.zeros(len(ctx), **i32),
                 slots=torch.empty(int(q.sum()), **i32), src=torch.empty(len(ctx), **i32),
                 dst=torch.empty(len(ctx), **i32), pools=_pools(g, case, len(refs)))
    elif op == "compact":
        ctx, table, refs = _scattered(case)
        half = len(refs) // 2
        s.update(ctx=_on(ctx), table=_on(table), refs=_on(refs), new_table=torch.full(table.shape, -1, **i32),
                 new_refs=torch.empty(len(refs), **i32), src=torch.empty(half, **i32),
                 dst=torch.empty(half, **i32), count=torch.empty(1, **i32),
                 pools=_pools(g, case, len(refs)))
    elif op == "index":
        slots, blocks = _written(case)
        hkv, d = case["hkv"], case["d"]
        s.update(slots=_on(slots), pool=_keyed_pool(g, blocks, hkv, d),
                 index=torch.zeros((blocks, hkv, 2, d), dtype=torch.int8, device=DEV),
                 scales=torch.ones((blocks, hkv), dtype=torch.float32, device=DEV))
    else:
        q_lens, ctx, table, blocks = _windows(case)
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        n = int(q_lens.sum())
        pool = _keyed_pool(g, blocks, hkv, d)
        index, scales = _bounds(pool[:, 0].float(), None)
        token = np.repeat(np.arange(len(q_lens)), q_lens)
        nth = np.arange(n) - np.repeat(np.cumsum(q_lens) - q_lens, q_lens)
        s.update(q=_normal(g, (n, hq, d)).to(torch.bfloat16), pool=pool, index=index, scales=scales,
                 cu=_on(np.concatenate([[0], np.cumsum(q_lens)])), ctx=_on(ctx), table=_on(table),
                 seq=_on(token), pos=_on(ctx[token] - q_lens[token] + nth), num=case["num"],
                 sink=case["sink"], recent=case["recent"], scale=1.0 / math.sqrt(d),
                 selected=torch.empty((n, hkv, case["num"]), **i32),
                 out=torch.empty((n, hq, d), dtype=torch.bfloat16, device=DEV))
    if own:   # a loop's calls over its fixed buffers, checked once
        s["calls"] = _bind(s)
    return s


# ----------------------------------------------------------------------------- the framework

def _bind(s):
    import paged_kv_attention_append_gb300 as pkv
    if s["op"] == "beam":
        return [pkv.BoundBeamSelect(s["logits"], s["cum"], s["num"], finished=s["finished"],
                                    pad_token=s["pad_token"], scores=s["scores"],
                                    tokens=s["tokens"], parents=s["parents"])]
    if s["op"] == "pages":
        return [pkv.BoundForkSequences(s["parents"], s["table"], s["ctx"], s["refs"],
                                       s["new_table"], s["new_ctx"]),
                pkv.BoundReserveBlocks(s["cu"], s["new_table"], s["new_ctx"], s["refs"],
                                       slot_mapping=s["slots"], copy_src=s["src"],
                                       copy_dst=s["dst"]),
                pkv.BoundCopyBlocks(s["pools"], s["src"], s["dst"]),
                pkv.BoundFreeSequences(s["done"], s["new_table"], s["new_ctx"], s["refs"])]
    if s["op"] == "compact":
        return [pkv.BoundCompactBlocks(s["table"], s["ctx"], s["refs"], new_tables=s["new_table"],
                                       new_ref_counts=s["new_refs"], copy_src=s["src"],
                                       copy_dst=s["dst"], num_pairs=s["count"]),
                pkv.BoundCopyBlocks(s["pools"], s["src"], s["dst"], num_pairs=s["count"])]
    if s["op"] == "index":
        return [pkv.BoundIndexUpdate(s["pool"], s["slots"], s["index"], s["scales"])]
    return [pkv.BoundSelectBlocks(s["q"], s["cu"], s["ctx"], s["table"], s["index"], s["scales"],
                                  s["num"], sink_blocks=s["sink"], recent_blocks=s["recent"],
                                  selected=s["selected"]),
            pkv.BoundSparseAttention(s["q"], s["cu"], s["ctx"], s["table"], s["selected"],
                                     s["pool"], s["scale"], s["out"])]


def _outputs(s):
    if s["op"] == "beam":
        return s["scores"], s["tokens"], s["parents"]
    if s["op"] == "pages":
        return (s["new_table"], s["new_ctx"], s["refs"], s["slots"], s["src"], s["dst"], *s["pools"])
    if s["op"] == "compact":
        return s["new_table"], s["new_refs"], s["src"], s["dst"], s["count"], *s["pools"]
    if s["op"] == "index":
        return s["index"], s["scales"]
    return s["selected"], s["out"]


def run(state):
    if state["op"] == "pages":     # a pass begins with the counts that the tables stand for
        state["refs"].copy_(state["refs0"])
    if own:
        for call in state["calls"]:
            call.run()
    else:
        PLAIN[state["op"]](state)
    return _outputs(state)


# -------------------------------------------------------------------------------- plain forms

def _plain_beam(s):
    x, m = s["logits"], s["num"]
    b, k, v = x.shape
    f = x.float()
    top = f.amax(dim=-1, keepdim=True)
    lse = top[..., 0].double() + (f - top).exp().sum(dim=-1, dtype=torch.float64).log()
    best, token = torch.sort(x, dim=-1, descending=True, stable=True)
    best, token = best[..., :m].double(), token[..., :m]
    score = s["cum"].double()[..., None] + (best - lse[..., None])
    if best.shape[-1] < m:
        fill = (0, m - best.shape[-1])
        score = torch.nn.functional.pad(score, fill, value=-math.inf)
        token = torch.nn.functional.pad(token, fill)
    only = torch.arange(m, device=DEV) == 0            # a finished beam goes on as itself
    ended = s["finished"][..., None]
    score = torch.where(ended, torch.where(only, s["cum"].double()[..., None], -math.inf), score)
    token = torch.where(ended, s["pad_token"], token)
    score = torch.where(score.isfinite(), score, -math.inf).view(b, k * m)
    score, at = torch.sort(score, dim=-1, descending=True, stable=True)
    score, at = score[:, :m], at[:, :m]
    there = score > -math.inf
    row = torch.arange(b, device=DEV)[:, None] * k + at // m
    s["scores"].copy_(score)
    s["tokens"].copy_(torch.where(there, token.view(b, k * m).gather(1, at), -1))
    s["parents"].copy_(torch.where(there, row, -1))


def _used(ctx):
    return (ctx + BLOCK - 1) // BLOCK


def _plain_pages(s):
    table, ctx, refs, parents = s["table"].long(), s["ctx"].long(), s["refs"], s["parents"].long()
    rows, width = table.shape
    col = torch.arange(width, device=DEV)
    # fork: the children's tables, and one reference more or less for each child and parent
    change = torch.zeros(rows, dtype=torch.int32, device=DEV).index_add_(
        0, parents, torch.ones_like(s["parents"])) - 1
    held = col < _used(ctx)[:, None]
    refs.index_add_(0, table.clamp(min=0).flatten(), (change[:, None] * held).int().flatten())
    ctx = ctx[parents]
    new = torch.where(col < _used(ctx)[:, None], table[parents], s["new_table"].long())
    # reserve: who writes into a shared block takes a copy; the last of all its holders keeps it
    cu = s["cu"].long()
    q = cu[1:] - cu[:-1]
    row = torch.arange(rows, device=DEV)
    part = new.gather(1, (ctx // BLOCK)[:, None])[:, 0].clamp(min=0)
    writes = (q > 0) & (ctx % BLOCK > 0)
    writers = torch.zeros(len(refs), dtype=torch.int64, device=DEV).index_add_(0, part, writes.long())
    last = torch.full((len(refs),), -1, device=DEV).scatter_reduce(
        0, part, torch.where(writes, row, -1), "amax")
    copied = writes & ((writers[part] < refs[part]) | (last[part] != row))
    first = torch.where(copied, ctx // BLOCK, _used(ctx))
    need = torch.where(q > 0, _used(ctx + q), _used(ctx)) - first
    base = need.cumsum(0) - need
    free = torch.sort((refs != 0).int(), stable=True)[1]      # free blocks first, in order
    taken = (col >= first[:, None]) & (col < (first + need)[:, None])
    at = (base[:, None] + col - first[:, None]).clamp(0, len(refs) - 1)
    s["src"].copy_(torch.where(copied, part, -1))
    new = torch.where(taken, free[at], new)
    s["dst"].copy_(torch.where(copied, new.gather(1, (ctx // BLOCK)[:, None])[:, 0], -1))
    refs.index_add_(0, part, -copied.int())
    refs.index_add_(0, free, (torch.arange(len(refs), device=DEV) < need.sum()).int())
    of = torch.searchsorted(cu, torch.arange(len(s["slots"]), device=DEV), right=True) - 1
    pos = ctx[of] + torch.arange(len(s["slots"]), device=DEV) - cu[of]
    s["slots"].copy_(new[of, pos // BLOCK] * BLOCK + pos % BLOCK)
    # the pages, in every pool
    pair = copied.nonzero()[:, 0]
    src, dst = s["src"].long()[pair], s["dst"].long()[pair]
    for p in s["pools"]:
        _copy_rows(p, src, dst)
    # free the finished ones
    ctx = ctx + q
    ended = torch.zeros(rows + 1, dtype=torch.bool, device=DEV)
    ended[torch.where(s["done"] < 0, rows, s["done"].long())] = True
    ended = ended[:rows]
    gone = ended[:, None] & (col < _used(ctx)[:, None])
    refs.index_add_(0, new.clamp(min=0).flatten(), -gone.int().flatten())
    s["new_ctx"].copy_(torch.where(ended, 0, ctx))
    s["new_table"].copy_(new)


def _copy_rows(pool, src, dst):
    bits = pool.view(torch.uint8) if pool.element_size() == 1 else pool
    bits[dst] = bits[src]


def _plain_compact(s):
    refs, n = s["refs"], len(s["refs"])
    ids = torch.arange(n, device=DEV)
    live = refs != 0
    total = live.sum()
    holes, movers = ~live & (ids < total), live & (ids >= total)
    src = torch.sort((~movers).int(), stable=True)[1][:n // 2]
    dst = torch.sort((~holes).int(), stable=True)[1][:n // 2]
    pair = torch.arange(n // 2, device=DEV) < movers.sum()
    s["src"].copy_(torch.where(pair, src, -1))
    s["dst"].copy_(torch.where(pair, dst, -1))
    s["count"].copy_(movers.sum())
    to = torch.arange(n + 1, device=DEV)
    to[torch.where(pair, src, n)] = torch.where(pair, dst, n)
    s["new_refs"].zero_().scatter_add_(0, to[:n], refs)
    held = torch.arange(s["table"].shape[1], device=DEV) < _used(s["ctx"])[:, None]
    s["new_table"].copy_(torch.where(held, to[s["table"].long().clamp(min=0)], s["new_table"].long()))
    src, dst = src[pair], dst[pair]
    for p in s["pools"]:
        _copy_rows(p, src, dst)


def _bounds(keys, rows):
    """Bounds of the keys [n, Hkv, 16, D] of each block (its first `rows` rows) in 8 bits, and the
    power of two that they count in: the smallest, at least 2^-64, with |key| <= 127 of it."""
    if rows is not None:
        there = (torch.arange(BLOCK, device=DEV) < rows[:, None])[:, None, :, None]
        low, high = keys.masked_fill(~there, math.inf).amin(2), keys.masked_fill(~there, -math.inf).amax(2)
    else:
        low, high = keys.amin(2), keys.amax(2)
    m, e = torch.frexp(torch.maximum(low.abs(), high.abs()).amax(-1) / 127)
    scale = torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e).clamp(min=-64))
    index = torch.stack([(low / scale[..., None]).floor(), (high / scale[..., None]).ceil()], dim=2)
    return index.to(torch.int8), scale


def _plain_index(s):
    blocks = s["pool"].shape[0]
    slots = s["slots"].long()
    rows = torch.zeros(blocks, dtype=torch.int64, device=DEV).scatter_reduce(
        0, slots // BLOCK, slots % BLOCK + 1, "amax")
    touched = (slots // BLOCK).unique()
    index, scale = _bounds(s["pool"][touched, 0].float(), rows[touched])
    s["index"][touched] = index
    s["scales"][touched] = scale


def _plain_sparse(s):
    q, pool, num = s["q"], s["pool"], s["num"]
    n, hq, d = q.shape
    hkv = pool.shape[2]
    table, pos = s["table"].long().clamp(min=0)[s["seq"].long()], s["pos"].long()  # [n, blocks]
    nb = table.shape[1]
    # q in 11 bits and a sign, its positive and negative parts summed over the heads of a KV head
    f = q.float().view(n, hkv, hq // hkv, d)
    m, e = torch.frexp(f.abs().amax(dim=(2, 3)) / 2047)
    unit = torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e))[..., None, None]
    whole = (f.double() / unit).round()
    parts = torch.stack([whole.clamp(max=0).sum(2), whole.clamp(min=0).sum(2)], dim=2)  # [n, Hkv, 2, D]
    held = s["index"][table].double().permute(0, 2, 1, 3, 4).reshape(n, hkv, nb, 2 * d)
    score = torch.matmul(held, parts.view(n, hkv, 2 * d, 1))[..., 0].float()
    del held
    score = (score * s["scales"][table].permute(0, 2, 1)).double()
    block = torch.arange(nb, device=DEV)
    own_block = (pos // BLOCK)[:, None]
    seen = block <= own_block
    forced = seen & ((block < s["sink"]) | (block > own_block - s["recent"]))
    score = score.masked_fill(forced[:, None], math.inf).masked_fill(~seen[:, None], -math.inf)
    score, at = torch.sort(score, dim=-1, descending=True, stable=True)
    at = torch.where(score > -math.inf, at, nb)[..., :num]
    at = torch.nn.functional.pad(at, (0, num - at.shape[-1]), value=nb).sort(dim=-1)[0]
    s["selected"].copy_(torch.where(at < nb, at, -1))
    # attention over the selected blocks, a few tokens at a time
    step = max(1, (1 << 28) // (hkv * num * BLOCK * d))
    head = torch.arange(hkv, device=DEV)[:, None]
    for i in range(0, n, step):
        a = at[i:i + step]
        phys = table[i:i + step].gather(1, a.clamp(max=nb - 1).flatten(1)).view(a.shape)
        k, v = (pool[phys, j, head].float().flatten(2, 3) for j in (0, 1))   # [t, Hkv, keys, D]
        key = (a[..., None] * BLOCK + torch.arange(BLOCK, device=DEV)).flatten(2)
        x = torch.matmul(f[i:i + step], k.transpose(2, 3)) * s["scale"]
        x = x.masked_fill((key > pos[i:i + step, None, None])[:, :, None], -math.inf)
        x = (x - x.amax(dim=-1, keepdim=True)).exp()
        o = torch.matmul(x, v) / x.sum(dim=-1, keepdim=True)
        s["out"][i:i + step] = o.reshape(-1, hq, d)


PLAIN = dict(beam=_plain_beam, pages=_plain_pages, compact=_plain_compact, index=_plain_index,
             sparse=_plain_sparse)


# ------------------------------------------------------------------------------------- work

def _row_bytes(case):
    return case["layers"] * (2.0 * case["hkv"] * BLOCK * case["d"] * (1 if case["fp8"] else 2) +
                             (8 * case["hkv"] if case["fp8"] else 0))


def work(case):
    op = case["op"]
    if op == "beam":
        n = float(case["batch"] * case["beams"])
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": n * case["vocab"] * size + 5 * n + 12.0 * case["batch"] * case["num"],
                "flops": 3 * n * case["vocab"]}
    if op == "pages":
        ctx, q, table, refs, parents, _ = _beam_tables(case)
        ctx = ctx[parents]
        part = table[np.arange(len(q))[parents], ctx // BLOCK]
        copied = sum(1 for s in range(len(q)) if ctx[s] % BLOCK and part[s] in part[s + 1:])
        entries = float(np.sum(-(-ctx // BLOCK)))
        return {"bytes": 2 * copied * _row_bytes(case) + 8 * entries + 8.0 * len(refs) + 4.0 * len(q),
                "flops": 2 * entries}
    if op == "compact":
        ctx, _, refs = _scattered(case)
        live = refs != 0
        moved = int(live[live.sum():].sum())
        return {"bytes": (2 * moved * _row_bytes(case) + 8.0 * float(np.sum(-(-ctx // BLOCK))) +
                          8.0 * len(refs) + 8.0 * moved),
                "flops": float(len(refs))}
    hkv, d = case["hkv"], case["d"]
    if op == "index":
        slots, _ = _written(case)
        rows = {}
        for x in slots.tolist():
            rows[x // BLOCK] = max(rows.get(x // BLOCK, 0), x % BLOCK + 1)
        return {"bytes": hkv * (2.0 * d * sum(rows.values()) + (2 * d + 4) * len(rows)) + 4.0 * len(slots),
                "flops": 2.0 * hkv * d * sum(rows.values())}
    q, ctx, _, _ = _windows(case)
    need = -(-ctx // BLOCK)
    keep = np.minimum(need, case["num"])
    n = float(q.sum())
    return {"bytes": float(hkv * np.sum(need * (2 * d + 4) + np.minimum(need, keep * q) * BLOCK * d * 4.0)) +
            n * (4.0 * case["hq"] * d + 4.0 * hkv * case["num"]),
            "flops": float(np.sum(q * (4.0 * d * hkv * need + 4.0 * d * case["hq"] * BLOCK * keep)))}


# ------------------------------------------------------------------------------------ exact

def _exact_beam(s):
    """Row by row in 64 bits; each request's candidates ordered by (-score, beam, token)."""
    b, k, v = s["logits"].shape
    m, out = s["num"], ([], [], [])
    cum, done = s["cum"].double().tolist(), s["finished"].tolist()
    for i in range(b):
        x = s["logits"][i].double()
        x = x - torch.logsumexp(x, dim=1, keepdim=True)
        found = []
        for j in range(k):
            if done[i][j]:
                found.append((-cum[i][j], j, s["pad_token"]))
                continue
            least = torch.topk(x[j], min(m, v))[0][-1]
            at = (x[j] >= least).nonzero()[:, 0]
            found += [(-(cum[i][j] + p), j, t) for p, t in zip(x[j][at].tolist(), at.tolist())]
        found = [c for c in sorted(found) if math.isfinite(c[0])][:m]
        found += [(math.inf, -1 - i * k, -1)] * (m - len(found))
        out[0].append([-c[0] for c in found])
        out[1].append([c[2] for c in found])
        out[2].append([i * k + c[1] for c in found])
    return (torch.tensor(out[0], dtype=torch.float64, device=DEV), _on(out[1]), _on(out[2]))


def _exact_copies(pools, src, dst):
    kept = [p.float().double() if p.numel() < 1 << 29 else None for p in pools]
    for p in kept:
        if p is not None:
            for a, b in zip(src, dst):
                if a >= 0:
                    p[b] = p[a]
    return kept


def _exact_pages(s):
    """One row after another, as a program on the host would."""
    table, ctx, refs = (s[n].cpu().numpy().astype(np.int64) for n in ("table", "ctx", "refs0"))
    parents, cu, done = (s[n].tolist() for n in ("parents", "cu", "done"))
    new, lens = np.full(table.shape, -1, dtype=np.int64), np.zeros(len(parents), dtype=np.int64)
    for i, p in enumerate(parents):
        used = -(-ctx[p] // BLOCK)
        new[i, :used], lens[i] = table[p, :used], ctx[p]
        refs[table[p, :used]] += 1
    for p in range(len(ctx)):
        refs[table[p, :-(-ctx[p] // BLOCK)]] -= 1
    free, slots = iter(np.flatnonzero(refs == 0).tolist()), []
    src, dst = [-1] * len(parents), [-1] * len(parents)
    for i in range(len(parents)):
        for t in range(lens[i], lens[i] + cu[i + 1] - cu[i]):
            j = t // BLOCK
            if t % BLOCK == 0:
                new[i, j] = next(free)
                refs[new[i, j]] += 1
            elif refs[new[i, j]] > 1:
                src[i] = int(new[i, j])
                refs[new[i, j]] -= 1
                new[i, j] = dst[i] = next(free)
                refs[new[i, j]] += 1
            slots.append(int(new[i, j]) * BLOCK + t % BLOCK)
        lens[i] += cu[i + 1] - cu[i]
    for i in set(x for x in done if x >= 0):
        refs[new[i, :-(-lens[i] // BLOCK)]] -= 1
        lens[i] = 0
    return (_on(new), _on(lens), _on(refs), _on(slots), _on(src), _on(dst),
            *_exact_copies(s["pools"], src, dst))


def _exact_compact(s):
    table, ctx, refs = (s[n].cpu().numpy().astype(np.int64) for n in ("table", "ctx", "refs"))
    total = np.count_nonzero(refs)
    dst = [x for x in range(total) if refs[x] == 0]
    src = [x for x in range(total, len(refs)) if refs[x] != 0]
    to = dict(zip(src, dst))
    new, counts = np.full(table.shape, -1, dtype=np.int64), np.zeros_like(refs)
    for r, c in enumerate(ctx):
        for j in range(-(-c // BLOCK)):
            new[r, j] = to.get(table[r, j], table[r, j])
            counts[new[r, j]] += 1
    none = [-1] * (len(refs) // 2 - len(src))
    return (_on(new), _on(counts), _on(src + none), _on(dst + none), _on([len(src)]),
            *_exact_copies(s["pools"], src, dst))


def _exact_bounds(keys):
    """Bounds of the keys [Hkv, rows, D] of one block."""
    top = np.abs(keys).max(axis=(1, 2))
    unit = np.exp2(np.maximum(np.ceil(np.log2(np.maximum(top, 1e-300) / 127)), -64))
    unit = np.where(unit / 2 * 127 >= top, np.maximum(unit / 2, 2.0 ** -64), unit)
    low, high = keys.min(axis=1), keys.max(axis=1)
    return np.stack([np.floor(low / unit[:, None]), np.ceil(high / unit[:, None])], axis=1), unit


def _exact_index(s):
    upto = {}
    for x in s["slots"].tolist():
        upto[x // BLOCK] = max(upto.get(x // BLOCK, 0), x % BLOCK + 1)
    keys = s["pool"][:, 0].float().cpu().numpy().astype(np.float64)
    index, scales = s["index"].cpu().numpy().copy(), s["scales"].cpu().double().numpy().copy()
    for b, n in upto.items():
        index[b], scales[b] = _exact_bounds(keys[b, :, :n])
    return torch.from_numpy(index).to(DEV), torch.from_numpy(scales).to(DEV)


def _exact_sparse(s):
    """Token by token: q.k's bound head by head with the larger of the two products."""
    q, pool, num = s["q"].double(), s["pool"], s["num"]
    n, hq, d = q.shape
    hkv = pool.shape[2]
    chosen, out = [], torch.empty((n, hq, d), dtype=torch.float64, device=DEV)
    seq, pos = s["seq"].tolist(), s["pos"].tolist()
    for t in range(n):
        ids = s["table"][seq[t], :pos[t] // BLOCK + 1].long()
        nb = len(ids)
        low, high = s["index"][ids].double().unbind(2)                    # [nb, Hkv, D]
        picked = []
        for h in range(hkv):
            x = q[t].view(hkv, -1, d)[h]
            top = float(x.abs().max())
            unit = 2.0 ** math.ceil(math.log2(max(top, 1e-300) / 2047))
            unit = unit / 2 if unit / 2 * 2047 >= top else unit
            x = (x / unit).round()
            bound = torch.maximum(x[:, None] * low[:, h], x[:, None] * high[:, h]).sum(dim=(0, 2))
            bound = (bound.float() * s["scales"][ids, h]).tolist()
            must = [b for b in range(nb) if b < s["sink"] or b >= nb - s["recent"]]
            rest = sorted((b for b in range(nb) if b not in must), key=lambda b: (-bound[b], b))
            sel = sorted((must + rest)[:num])
            picked.append(sel + [-1] * (num - len(sel)))
            at = ids[torch.tensor(sel, device=DEV)]
            k, v = (pool[at, j, h].double().reshape(-1, d) for j in (0, 1))
            key = (torch.tensor(sel, device=DEV)[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)).flatten()
            w = (q[t].view(hkv, -1, d)[h] @ k.T) * s["scale"]
            w = torch.softmax(w.masked_fill(key > pos[t], -math.inf), dim=1)
            out[t].view(hkv, -1, d)[h] = w @ torch.where((key > pos[t])[:, None], 0.0, v)
        chosen.append(picked)
    return _on(chosen), out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sparse" and case["seqs"] * (case["q_lo"] + case["q_hi"]) / 2 * case["hkv"] > 1500:
        return None
    return dict(beam=_exact_beam, pages=_exact_pages, compact=_exact_compact, index=_exact_index,
                sparse=_exact_sparse)[case["op"]](s)
