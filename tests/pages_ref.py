"""Plain host forms of the page calls, the beam selection and the sparse attention.

Rows and tokens one after another, in Python and numpy, 64 bits throughout; shared by the
tests of the kernels and checked against hand-made cases of their own.
"""

import numpy as np

BLOCK = 16


def used(ctx, width=1 << 30):
    return min(-(-max(int(ctx), 0) // BLOCK), width)


def fork(parents, tables, ctx, refs, new, new_ctx, keep):
    """In place on refs, new and new_ctx."""
    for i, p in enumerate(parents):
        n = used(ctx[p], tables.shape[1]) if 0 <= p < len(tables) else 0
        new_ctx[i] = max(ctx[p], 0) if 0 <= p < len(tables) else 0
        if n:
            new[i, :n] = tables[p, :n]
            for b in tables[p, :n]:
                if 0 <= b < len(refs):
                    refs[b] += 1
    if not keep:
        for r in range(len(tables)):
            for b in tables[r, :used(ctx[r], tables.shape[1])]:
                if 0 <= b < len(refs):
                    refs[b] -= 1


def free(rows, tables, ctx, refs):
    for r in rows:
        if 0 <= r < len(tables):
            for b in tables[r, :used(ctx[r], tables.shape[1])]:
                if 0 <= b < len(refs) and refs[b] > 0:
                    refs[b] -= 1
            ctx[r] = 0


def reserve(cu, tables, ctx, refs):
    """Token by token; returns slots, copy_src, copy_dst, or None when blocks or columns run
    out (the arrays are then to be thrown away)."""
    free_ids = iter(np.flatnonzero(refs == 0).tolist())
    rows, slots = len(tables), np.full(max(int(cu[-1]), 0), -1, dtype=np.int32)
    src, dst = np.full(rows, -1, dtype=np.int32), np.full(rows, -1, dtype=np.int32)
    for r in range(rows):
        for i in range(max(int(cu[r + 1]) - int(cu[r]), 0)):
            pos = max(int(ctx[r]), 0)
            j, off = divmod(pos, BLOCK)
            if j >= tables.shape[1]:
                return None
            if off == 0 or refs[tables[r, j]] > 1:
                b = next(free_ids, None)
                if b is None:
                    return None
                if off:
                    src[r], dst[r] = tables[r, j], b
                    refs[tables[r, j]] -= 1
                tables[r, j] = b
                refs[b] = 1
            slots[cu[r] + i] = tables[r, j] * BLOCK + off
            ctx[r] = pos + 1
    return slots, src, dst


def compact(tables, ctx, refs):
    """Returns new tables (used entries), new counts and the pairs."""
    live = int(np.count_nonzero(refs))
    dst = [x for x in range(live) if refs[x] == 0]
    src = [x for x in range(live, len(refs)) if refs[x] != 0]
    to = dict(zip(src, dst))
    new, counts = tables.copy(), np.zeros_like(refs)
    for x in np.flatnonzero(refs):
        counts[to.get(int(x), int(x))] = refs[x]
    for r in range(len(tables)):
        for j in range(used(ctx[r], tables.shape[1])):
            new[r, j] = to.get(int(tables[r, j]), tables[r, j])
    return new, counts, src, dst


def random_tables(rng, rows, width, blocks, share=0.5, longest=None):
    """Tables of ragged sequences, some of which go on from another's blocks; counts."""
    tables, ctx = np.full((rows, width), -1, dtype=np.int32), np.zeros(rows, dtype=np.int32)
    refs, ids = np.zeros(blocks, dtype=np.int32), iter(rng.permutation(blocks).tolist())
    longest = width * BLOCK if longest is None else longest
    for r in range(rows):
        ctx[r] = rng.choice([0, 1, 15, 16, 17, int(rng.integers(0, longest + 1))])
        ctx[r] = min(ctx[r], longest)
        n = used(ctx[r])
        shared = 0
        if r and rng.random() < share:
            o = int(rng.integers(0, r))
            shared = min(n, used(ctx[o]))
            if rng.random() < 0.5 and shared:      # a whole fork: the partly filled block too
                ctx[r] = min(ctx[r], ctx[o]) if rng.random() < 0.5 else ctx[o]
                n = shared = used(ctx[r])
            tables[r, :shared] = tables[o, :shared]
        for j in range(shared, n):
            tables[r, j] = next(ids)
        np.add.at(refs, tables[r, :n], 1)
    return tables, ctx, refs


def beam(logits, cum, num, finished=None, pad=0):
    """logits float64 [B, K, V].  Returns (scores, tokens, parents, score of every candidate)."""
    b, k, v = logits.shape
    with np.errstate(all="ignore"):
        top = logits.max(axis=2, keepdims=True)
        lse = np.log(np.exp(logits - top).sum(axis=2, keepdims=True))  # above top
        score = np.asarray(cum, dtype=np.float64)[..., None] + (logits - top - lse)
    if finished is not None:
        score[finished] = -np.inf
        score[finished, pad] = np.asarray(cum, dtype=np.float64)[finished]
    # (a finished beam's candidate is its pad token, so its order by token is its own)
    score[~np.isfinite(score)] = -np.inf
    out = np.full((b, num), -np.inf), np.full((b, num), -1), np.full((b, num), -1)
    for i in range(b):
        flat = score[i].reshape(-1)
        at = np.argsort(-flat, kind="stable")[:num]
        at = at[np.isfinite(flat[at])]
        n = len(at)
        out[0][i, :n], out[1][i, :n], out[2][i, :n] = flat[at], at % v, i * k + at // v
    return (*out, score)


def bounds(keys):
    """Bounds of the keys [Hkv, rows, D] (float64) of a block, and their unit."""
    keys = np.where(np.isfinite(keys), keys, 0.0)
    top = np.abs(keys).max(axis=(1, 2))
    unit = np.full(len(top), 2.0 ** -64)
    for h, t in enumerate(top):
        while t > 127 * unit[h]:
            unit[h] *= 2
    return (np.stack([np.floor(keys.min(axis=1) / unit[:, None]),
                      np.ceil(keys.max(axis=1) / unit[:, None])], axis=1), unit)


def scores(q, index, unit):
    """Scores of blocks, fp32: q float64 [G, D], index [nb, 2, D], unit [nb]."""
    q = np.where(np.isfinite(q), q, 0.0)
    top, u = np.abs(q).max(), 2.0 ** -160
    while top > 2047 * u:
        u *= 2
    w = np.rint(q / u) if top > 0 else q
    total = sum(np.where(x > 0, x * index[:, 1], x * index[:, 0]).sum(axis=1) for x in w)
    with np.errstate(over="ignore"):
        return total.astype(np.float32) * unit.astype(np.float32)


def select(q, pos, table, index, units, num, sink, recent):
    """One token's selection for each KV head: int32 [Hkv, num]."""
    nb, hkv = pos // BLOCK + 1, index.shape[1]
    out = np.full((hkv, num), -1, dtype=np.int32)
    q = q.reshape(hkv, -1, q.shape[-1])
    ids = table[:nb]
    for h in range(hkv):
        must = [b for b in range(nb) if b < sink or b >= nb - recent]
        if nb <= num:
            sel = list(range(nb))
        else:
            s = scores(q[h], index[ids, h].astype(np.float64), units[ids, h])
            rest = sorted(set(range(nb)) - set(must), key=lambda b: (-s[b], b))
            sel = sorted((must + rest)[:num])
        out[h, :len(sel)] = sel
    return out


def sparse_attention(q, pos, table, selected, pool, scale):
    """One token: q [Hq, D], selected [Hkv, n] (negative: none), pool [nb, 2, Hkv, 16, D], float64.
    Returns out [Hq, D] and, by element, the sum of |weight V| and the largest sum of |q K|."""
    hkv, d = pool.shape[2], pool.shape[4]
    g = q.shape[0] // hkv
    out, mag, dots = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[0])
    for h in range(hkv):
        sel = [int(b) for b in selected[h] if 0 <= b <= pos // BLOCK]
        if not sel:
            continue
        key = np.concatenate([np.arange(b * BLOCK, b * BLOCK + BLOCK) for b in sel])
        k, v = (pool[table[sel], j, h].reshape(-1, d)[key <= pos] for j in (0, 1))
        for i in range(h * g, h * g + g):
            s = (k @ q[i]) * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i], mag[i] = w @ v, w @ np.abs(v)
            dots[i] = (np.abs(k) @ np.abs(q[i])).max() * abs(scale)
    return out, mag, dots
