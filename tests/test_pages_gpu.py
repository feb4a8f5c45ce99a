"""GPU tests of the page calls (copy, fork, free, reserve, compact) and of the beam selection
against the plain host forms of pages_ref.py.

Tables, counts, slots, pairs and copied bytes have no tolerance.  A beam score is
cum + (x - lse) with lse = m + log(sum): the sum is taken in fp32.  A term is off by at most
2^-22 (ex2) plus the rounding of its exponent, 2^-24 |x - m| log2(e) ln 2 <= 2^-24 |x - m|, which
for the terms that count (|x - m| < 32; the others weigh below 2^-46) is 2^-19; a thread adds at
most 64 terms in a row, its warp, CTA and the splits 5 + 8 + 64 more, 2^-24 each.  So the sum is
off by less than 2^-19 + 2^-22 + 141 2^-24 < 2^-16 of itself, lse by as much, and the score by its
rounding, 2^-24 of itself, besides.
"""

import numpy as np
import pytest
import torch

import pages_ref as ref

pytestmark = pytest.mark.gpu

LSE_TOL = 2.0 ** -16


@pytest.fixture(scope="module")
def pkv(cuda_device):
    import paged_kv_attention_append_gb300 as m
    m.build()
    return m


def dev_i32(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)


def status_of(dev):
    return torch.zeros(1, dtype=torch.int32, device=dev)


def same(got, want):
    got = got.cpu().numpy() if isinstance(got, torch.Tensor) else got
    np.testing.assert_array_equal(got, np.asarray(want))


# ------------------------------------------------------------------------- copies

ROWS = [  # (dtype, row shape): widths of whole and partial units, 4-byte and 16-byte rows
    (torch.bfloat16, (2, 8, 16, 128)), (torch.bfloat16, (2, 1, 16, 64)), (torch.uint8, (2, 3, 16, 64)),
    (torch.float32, (1, 2)), (torch.float32, (3,)), (torch.int8, (4,)), (torch.int32, (1025,)),
    (torch.uint8, (4096 + 16,)),
]


@pytest.mark.parametrize("row", range(len(ROWS)))
@pytest.mark.parametrize("pairs", [1, 7, 400])
def test_copy_blocks(pkv, cuda_device, row, pairs):
    dtype, shape = ROWS[row]
    rng = np.random.default_rng(10 * row + pairs)
    blocks = 2 * pairs + 5
    raw = torch.from_numpy(rng.integers(0, 256, (blocks, int(np.prod(shape)) *
                                                 torch.empty(0, dtype=dtype).element_size()),
                                        dtype=np.uint8))
    pool = raw.to(cuda_device).view(dtype).view(blocks, *shape)
    ids = rng.permutation(blocks)
    src, dst = ids[:pairs].copy(), ids[pairs:2 * pairs].copy()
    src[rng.random(pairs) < 0.2] = -1
    dst[rng.random(pairs) < 0.1] = -5
    want = raw.numpy().copy()
    for s, d in zip(src, dst):
        if s >= 0 and d >= 0:
            want[d] = raw.numpy()[s]
    st = status_of(cuda_device)
    pkv.copy_blocks(pool, dev_i32(src, cuda_device), dev_i32(dst, cuda_device), dev_status=st)
    same(pool.view(blocks, -1).view(torch.uint8), want)
    assert int(st.item()) == 0


def test_copy_many_arrays_of_different_rows(pkv, cuda_device):
    """More arrays than one launch takes, wide and narrow ones, one of them not 16-byte aligned."""
    rng = np.random.default_rng(3)
    blocks = 9
    raw = [rng.integers(0, 256, (blocks, 4 * int(rng.choice([1, 3, 4, 8, 64, 2100]))), dtype=np.uint8)
           for _ in range(131)]
    pools = [torch.from_numpy(r).to(cuda_device) for r in raw]
    odd = torch.zeros(blocks * 64 + 4, dtype=torch.uint8, device=cuda_device)[4:].view(blocks, 64)
    odd.copy_(torch.from_numpy(rng.integers(0, 256, (blocks, 64), dtype=np.uint8)))
    raw.append(odd.cpu().numpy().copy())
    pkv.copy_blocks([*pools, odd], dev_i32([0, 3, 8], cuda_device), dev_i32([1, 5, 2], cuda_device))
    for r, p in zip(raw, [*pools, odd]):
        r[[1, 5, 2]] = r[[0, 3, 8]]
        same(p, r)


@pytest.mark.parametrize("count", [-3, 0, 2, 5, 100])
def test_copy_count_and_bad_ids(pkv, cuda_device, count):
    pool = torch.arange(12 * 64, dtype=torch.int32, device=cuda_device).view(12, 64)
    want = pool.cpu().numpy().copy()
    src, dst = [0, 1, 12, 2, 3], [5, 6, 7, 99, 8]
    for i in range(min(max(count, 0), 5)):
        if src[i] < 12 and dst[i] < 12:
            want[dst[i]] = want[src[i]]
    st = status_of(cuda_device)
    pkv.copy_blocks(pool, dev_i32(src, cuda_device), dev_i32(dst, cuda_device),
                    num_pairs=dev_i32([count], cuda_device), dev_status=st)
    same(pool, want)
    assert int(st.item()) == (2 if count > 2 else 0)


def test_copy_past_four_gigabytes(pkv, cuda_device):
    pool = torch.zeros((70000, 65536), dtype=torch.uint8, device=cuda_device)
    pool[69998] = torch.arange(65536, device=cuda_device).to(torch.uint8)
    pool[1] = 7
    pkv.copy_blocks(pool, dev_i32([69998, 1], cuda_device), dev_i32([3, 69999], cuda_device))
    assert torch.equal(pool[3], pool[69998]) and int(pool[69999].min()) == 7
    assert int(pool[4:69998].max()) == 0


# ------------------------------------------------------------------------- fork, free

@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("rows,n,width", [(1, 1, 1), (5, 9, 3), (9, 4, 37), (40, 40, 130), (300, 257, 9),
                                          (3, 5, 2500)])
def test_fork(pkv, cuda_device, keep, rows, n, width):
    rng = np.random.default_rng(rows * 1000 + n + keep)
    tables, ctx, refs = ref.random_tables(rng, rows, width, rows * width + 3)
    parents = rng.integers(-1, rows, n)
    new, new_ctx = np.full((n, width), -7), np.full(n, -7)
    want_refs = refs.copy()
    ref.fork(parents, tables, ctx, want_refs, new, new_ctx, keep)
    dev = cuda_device
    got, got_ctx = dev_i32(np.full((n, width), -7), dev), dev_i32(np.full(n, -7), dev)
    d_refs, st = dev_i32(refs, dev), status_of(dev)
    pkv.fork_sequences(dev_i32(parents, dev), dev_i32(tables, dev), dev_i32(ctx, dev), d_refs, got,
                       got_ctx, keep_parents=keep, dev_status=st)
    same(got, new)
    same(got_ctx, new_ctx)
    same(d_refs, want_refs)
    assert int(st.item()) == 0


def test_fork_bad_rows_blocks_and_counts(pkv, cuda_device):
    dev = cuda_device
    tables, ctx = np.array([[3, 9, 1], [2, -4, 0]]), np.array([40, 20])
    for parents, refs, code in (([0, 5], [0, 1, 1, 1], 6), ([0, 0], [0, 1, 1, 1], 2),
                                ([-1, -1], [0, 0, 1, 1], 8)):
        t = tables.copy()
        if code != 2:
            t[0, 1], t[1, 1] = 1, 3
        new, new_ctx = dev_i32(np.full((2, 3), -7), dev), dev_i32([-7, -7], dev)
        want, want_ctx, want_refs = np.full((2, 3), -7), np.full(2, -7), np.array(refs)
        ref.fork(parents, t, ctx, want_refs, want, want_ctx, False)
        d_refs, st = dev_i32(refs, dev), status_of(dev)
        pkv.fork_sequences(dev_i32(parents, dev), dev_i32(t, dev), dev_i32(ctx, dev), d_refs, new,
                           new_ctx, dev_status=st)
        same(new, want)
        same(new_ctx, want_ctx)
        same(d_refs, want_refs)
        assert int(st.item()) == code


@pytest.mark.parametrize("rows,width", [(1, 1), (7, 4), (120, 90), (2, 5000)])
def test_free(pkv, cuda_device, rows, width):
    rng = np.random.default_rng(rows + width)
    tables, ctx, refs = ref.random_tables(rng, rows, width, rows * width + 2)
    listed = rng.integers(-1, rows, rows + 3)       # with rows listed twice
    dev = cuda_device
    d_ctx, d_refs, st = dev_i32(ctx, dev), dev_i32(refs, dev), status_of(dev)
    pkv.free_sequences(dev_i32(listed, dev), dev_i32(tables, dev), d_ctx, d_refs, dev_status=st)
    ref.free(listed, tables, ctx, refs)
    same(d_ctx, ctx)
    same(d_refs, refs)
    assert int(st.item()) == 0


def test_free_reports(pkv, cuda_device):
    dev = cuda_device
    for listed, tables, refs, code in (([2], [[0], [1]], [1, 1], 6), ([0], [[4], [1]], [1, 1], 2),
                                       ([0, 1], [[0], [0]], [1, 1], 8)):
        ctx, st, d_refs = dev_i32([5, 5], dev), status_of(dev), dev_i32(refs, dev)
        pkv.free_sequences(dev_i32(listed, dev), dev_i32(tables, dev), ctx, d_refs, dev_status=st)
        assert int(st.item()) == code
        assert d_refs.cpu().tolist() == ([0, 1] if code == 8 else [1, 1])


# ------------------------------------------------------------------------- reserve

def run_reserve(pkv, dev, cu, tables, ctx, refs, **kw):
    d = [dev_i32(x, dev) for x in (cu, tables, ctx, refs)]
    st = status_of(dev)
    n = max(int(cu[-1]), 0)
    out = pkv.reserve_blocks(*d, num_tokens=n, dev_status=st, **kw)
    return d, out, int(st.item())


RESERVES = [  # rows, width, blocks, most new tokens, share
    (1, 1, 1, 3, 0.0), (1, 3, 5000, 40, 0.0), (4, 3, 30, 2, 1.0), (9, 12, 150, 17, 0.8),
    (64, 20, 4096, 1, 0.9), (65, 20, 4097, 5, 0.9), (300, 40, 20001, 3, 0.95),
    (1100, 6, 9000, 33, 0.7), (8192, 3, 30000, 4, 0.9), (3, 2000, 12300, 9000, 0.5),
]


@pytest.mark.parametrize("case", range(len(RESERVES)))
@pytest.mark.parametrize("seed", [0, 1])
def test_reserve(pkv, cuda_device, case, seed):
    rows, width, blocks, most, share = RESERVES[case]
    rng = np.random.default_rng(100 * case + seed)
    longest = max(width * 16 - most, 0)
    tables, ctx, refs = ref.random_tables(rng, rows, width, blocks, share, longest)
    n = rng.integers(0, most + 1, rows) if seed else np.full(rows, most)
    n = np.where(rng.random(rows) < 0.1 * seed, 0, n)
    cu = np.concatenate([[0], np.cumsum(n)])
    want = [tables.copy(), ctx.copy(), refs.copy()]
    pairs = ref.reserve(cu, *want)
    assert pairs is not None
    (_, t, c, r), (slots, src, dst), st = run_reserve(pkv, cuda_device, cu, tables, ctx, refs)
    assert st == 0
    for got, w in zip((t, c, r, slots, src, dst), (*want, *pairs)):
        same(got, w)


def test_reserve_leaves_everything_when_it_cannot(pkv, cuda_device):
    """Too few free blocks (by one), too few columns, a block outside the pool, counts below the
    writers: nothing changes, slots and pairs are -1."""
    tables = np.array([[4, 2, -1], [4, 2, -1], [-1, -1, -1]])
    ctx, refs, cu = np.array([20, 20, 0]), np.array([1, 3, 2, 0, 2]), [0, 1, 2, 5]
    cases = [(tables, ctx, refs, cu, 7),
             (tables, ctx, np.array([0, 0, 2, 0, 2]), [0, 1, 30, 30], 7),
             (np.where(tables == 2, 5, tables), ctx, np.zeros(5), cu, 2),
             (np.where(tables == 2, -1, tables), ctx, np.zeros(5), cu, 2),
             (tables, ctx, np.array([0, 0, 0, 0, 2]), cu, 8),
             (np.vstack([tables[:2], tables[:1]]), np.array([20, 20, 20]), np.array([0, 0, 2, 0, 2]),
              [0, 1, 2, 3], 8),
             (tables, ctx, np.array([0, 0, 2, 0, 2]), [0, 2 ** 31 - 40, 2 ** 31 - 39, 2 ** 31 - 38], 7)]
    for t, c, r, q, code in cases:
        d = [dev_i32(x, cuda_device) for x in (q, t, c, r)]
        st, slots = status_of(cuda_device), dev_i32(np.zeros(6), cuda_device)
        _, src, dst = pkv.reserve_blocks(*d, slot_mapping=slots, dev_status=st)
        assert int(st.item()) == code
        for got, w in zip(d[1:], (t, c, r)):
            same(got, w)
        for x in (slots, src, dst):
            assert set(x.cpu().tolist()) == {-1}


@pytest.mark.parametrize("rows", [1, 5, 1300])
@pytest.mark.parametrize("before,behind", [(0, 3), (4, 0), (2, 20000)])
def test_reserve_gives_padding_no_slot(pkv, cuda_device, rows, before, behind):
    """Slots before the first row's tokens and behind the last one's are -1, whatever they were;
    those past num_tokens are left."""
    rng = np.random.default_rng(rows)
    tables, ctx, refs = ref.random_tables(rng, rows, 4, 4 * rows + 20000, 0.5, 30)
    n = rng.integers(0, 20, rows)
    cu = before + np.concatenate([[0], np.cumsum(n)])
    want = [tables.copy(), ctx.copy(), refs.copy()]
    slots, _, _ = ref.reserve(cu, *want)
    d = [dev_i32(x, cuda_device) for x in (cu, tables, ctx, refs)]
    whole = dev_i32(np.full(len(slots) + behind + 5, 77), cuda_device)
    pkv.reserve_blocks(*d, slot_mapping=whole[:-5])
    same(whole, np.concatenate([slots, np.full(behind, -1), np.full(5, 77)]))
    for got, w in zip(d[1:], want):
        same(got, w)


def test_reserve_just_enough_and_unaligned_counts(pkv, cuda_device):
    """Every free block is taken, from counts that do not start on 16 bytes."""
    rng = np.random.default_rng(5)
    refs = (rng.random(9001) < 0.6).astype(np.int32)
    free = int((refs == 0).sum())
    tables, ctx = np.full((7, free), -1), np.zeros(7)
    n = rng.multinomial(free, [1 / 7] * 7) * 16
    cu = np.concatenate([[0], np.cumsum(n)])
    want = [tables.copy(), ctx.copy(), refs.copy()]
    slots, _, _ = ref.reserve(cu, *want)
    whole = dev_i32(np.concatenate([[9, 9, 9], refs]), cuda_device)
    t, c = dev_i32(tables, cuda_device), dev_i32(ctx, cuda_device)
    got, _, _ = pkv.reserve_blocks(dev_i32(cu, cuda_device), t, c, whole[3:], num_tokens=int(cu[-1]))
    same(got, slots)
    same(t, want[0])
    same(whole[3:], want[2])


# ------------------------------------------------------------------------- compact

@pytest.mark.parametrize("blocks", [1, 2, 17, 4095, 4096, 4097, 12289, 70001])
@pytest.mark.parametrize("live", [0.0, 0.3, 0.9, 1.0])
@pytest.mark.parametrize("place", [False, True])
def test_compact(pkv, cuda_device, blocks, live, place):
    rng = np.random.default_rng(blocks + int(10 * live))
    n = int(round(live * blocks))
    ids, rows = rng.permutation(blocks)[:n], 5
    width = n + 1
    tables, ctx, refs = np.full((rows, width), -1), np.zeros(rows, dtype=np.int64), np.zeros(blocks)
    cut = np.sort(rng.integers(0, n + 1, rows - 2))
    for r, (a, b) in enumerate(zip([0, *cut], [*cut, n])):
        tables[r, :b - a], ctx[r] = ids[a:b], (b - a) * 16 - (r if b > a else 0)
    tables[4], ctx[4] = tables[0], ctx[0]            # a fork
    for r in range(rows):
        np.add.at(refs, tables[r, :ref.used(ctx[r])], 1)
    refs[ids[:2]] += 3                               # held outside the tables, too
    new, counts, src, dst = ref.compact(tables, ctx, refs)
    dev = cuda_device
    t, r, st = dev_i32(tables, dev), dev_i32(refs, dev), status_of(dev)
    kw = {} if place else dict(new_tables=dev_i32(tables, dev), new_ref_counts=torch.empty_like(r))
    s, d, num = pkv.compact_blocks(t, dev_i32(ctx, dev), r, dev_status=st, **kw)
    same(kw.get("new_tables", t), new)
    same(kw.get("new_ref_counts", r), counts)
    fill = [-1] * (blocks // 2 - len(src))
    same(s, src + fill)
    same(d, dst + fill)
    assert int(num.item()) == len(src) and int(st.item()) == 0
    if not place:
        same(t, tables)
        same(r, refs)


def test_compact_reports_tables_that_do_not_fit(pkv, cuda_device):
    dev = cuda_device
    for table, code in (([[5, 3]], 8), ([[5, 9]], 2), ([[5, -2]], 2)):
        st, t = status_of(dev), dev_i32(table, dev)
        pkv.compact_blocks(t, dev_i32([32], dev), dev_i32([0, 0, 0, 0, 0, 1], dev), dev_status=st)
        assert int(st.item()) == code and t.cpu().tolist() == [[0, table[0][1]]]


# ------------------------------------------------------------------------- beams

def check_beams(got, want, all_scores, logits, finished):
    """The selection, up to candidates whose scores the tolerance does not tell apart (between
    beams; within a beam the order is that of the logits, then the token)."""
    s, t, p = (x.cpu().numpy() for x in got)
    ws, wt, wp = want
    b, k, v = logits.shape
    for i in range(b):
        n = int(np.isfinite(ws[i]).sum())
        assert np.isneginf(s[i, n:]).all() and (t[i, n:] == -1).all() and (p[i, n:] == -1).all()
        tol = LSE_TOL + 2.0 ** -24 * np.abs(ws[i, :n])
        assert (np.abs(s[i, :n] - ws[i, :n]) <= tol).all()
        pairs = list(zip(p[i, :n].tolist(), t[i, :n].tolist()))
        assert len(set(pairs)) == n and all(i * k <= x < i * k + k for x, _ in pairs)
        own = np.array([all_scores[i, x - i * k, y] for x, y in pairs])
        assert (np.abs(own - ws[i, :n]) <= 2 * tol).all()
        for x in range(k):
            mine = [y for q, y in pairs if q == i * k + x]
            if finished is not None and finished[i, x]:
                continue
            row = logits[i, x]
            assert mine == sorted(mine, key=lambda y: (-row[y], y))
            best = np.lexsort((np.arange(v), -row))[:len(mine)]
            assert mine == best.tolist()


def beam_case(rng, b, k, v, dtype, spread=3.0, pad=0, offset=0):
    whole = torch.from_numpy(rng.standard_normal(b * k * (v + pad) + offset) * spread).to(dtype)
    return whole[offset:].view(b, k, v + pad)[:, :, :v]


BEAMS = [(1, 1, 1, 1), (1, 4, 5, 9), (2, 3, 7, 4), (1, 4, 32000, 4), (3, 5, 50257, 10), (2, 8, 8193, 16),
         (5, 1, 2048, 33), (1, 64, 1000, 128), (7, 12, 333, 36), (40, 8, 20000, 8), (1, 1024, 40, 5),
         (2, 2, 128000, 128), (15, 2, 9047, 5), (41, 8, 295, 5), (43, 12, 586, 13), (1, 3, 200, 40),
         (80, 8, 4100, 9)]


@pytest.mark.parametrize("case", range(len(BEAMS)))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1)])
def test_beam_select(pkv, cuda_device, case, dtype, pad, offset):
    b, k, v, num = BEAMS[case]
    rng = np.random.default_rng(1000 + case)
    x = beam_case(rng, b, k, v, dtype, pad=pad, offset=offset)
    whole = torch.empty(b * k * (v + pad) + offset, dtype=dtype, device=cuda_device)
    on = whole[offset:].view(b, k, v + pad)[:, :, :v]
    on.copy_(x)
    cum = rng.uniform(-30, 0, (b, k)).astype(np.float32)
    finished = rng.random((b, k)) < 0.25 if case % 2 else None
    pad_token = 2 % v
    f64 = x.double().numpy()
    want = ref.beam(f64, cum, num, finished, pad_token)
    got = pkv.beam_select(on, torch.from_numpy(cum).to(cuda_device), num, pad_token=pad_token,
                          finished=None if finished is None else
                          torch.from_numpy(finished).to(cuda_device))
    check_beams(got, want[:3], want[3], f64, finished)


LOWEST = float(torch.finfo(torch.float32).min)
SHAPES = {  # rows that find the buffer's limits
    "equal": lambda rng, v: np.zeros(v),
    "rising": lambda rng, v: np.arange(v) / 64,
    "falling": lambda rng, v: -np.arange(v) / 64,
    "steps": lambda rng, v: np.floor(np.arange(v) / 1000),
    "two values": lambda rng, v: rng.integers(0, 2, v) * 1.0,
    "signed zeros": lambda rng, v: np.where(rng.random(v) < 0.5, -0.0, 0.0),
    "one": lambda rng, v: np.where(np.arange(v) == v - 1, 50.0, -50.0),
    "masked": lambda rng, v: np.where(rng.random(v) < 0.999, -np.inf, rng.standard_normal(v)),
    "large": lambda rng, v: rng.standard_normal(v) * 60000,
    "filled": lambda rng, v: np.where(rng.random(v) < 0.99, -1e4, rng.standard_normal(v)),
    "lowest": lambda rng, v: np.full(v, LOWEST),
    "lows": lambda rng, v: rng.choice([LOWEST, -3e38, -2.4e38, -np.inf], v, p=[.9, .05, .04, .01]),
    "lows apart": lambda rng, v: np.where(np.arange(v) < v // 2, LOWEST, -3e38),
    "few not lowest": lambda rng, v: np.where(rng.random(v) < 0.999, LOWEST, rng.standard_normal(v)),
}


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("v", [300, 8192, 70001])
@pytest.mark.parametrize("num", [3, 128])
@pytest.mark.parametrize("many", [False, True])
def test_beam_rows_of_all_shapes(pkv, cuda_device, shape, v, num, many):
    """Many rows take large tiles, few rows small ones; equal beams tie beam by beam."""
    rng = np.random.default_rng(v + num)
    b, k = (90, 4) if many and v > 300 else (1, 2)
    row = torch.from_numpy(SHAPES[shape](rng, v)).float()
    x = row.expand(1, k, v).contiguous()
    cum = np.zeros((1, k), dtype=np.float32)
    cum[0, 1] = -1e-3
    f64 = x.double().numpy()
    want = ref.beam(f64, cum, num)
    got = pkv.beam_select(x.to(cuda_device).expand(b, k, v).contiguous(),
                          torch.from_numpy(cum).to(cuda_device).expand(b, k).contiguous(), num)
    first = [g[:1] for g in got]
    check_beams(first, want[:3], want[3], f64, None)
    s, t, p = got
    assert torch.equal(s, s[:1].expand_as(s)) and torch.equal(t, t[:1].expand_as(t))
    at = torch.arange(b, device=cuda_device, dtype=torch.int32)[:, None] * k
    assert torch.equal(torch.where(p >= 0, p - at, -1), p[:1].expand_as(p))


@pytest.mark.parametrize("dtype,v,pad", [(torch.float16, 9001, 0), (torch.bfloat16, 20003, 5),
                                         (torch.float32, 5003, 0)])
def test_equal_beams_tie_to_the_lower_beam(pkv, cuda_device, dtype, v, pad):
    """The same logits in rows of different alignment give the same sums: every tie between
    the beams goes to the lower one."""
    rng = np.random.default_rng(v)
    k, num = 5, 20
    row = torch.from_numpy(rng.standard_normal(v) * 3).to(dtype)
    whole = torch.zeros((1, k, v + pad), dtype=dtype, device=cuda_device)
    x = whole[:, :, :v]
    x.copy_(row.expand(1, k, v))
    s, t, p = pkv.beam_select(x, torch.full((1, k), -2.0, device=cuda_device), num)
    value = np.tile(row.double().numpy(), k)       # by logit, then beam, then token
    want = np.lexsort((np.arange(k * v), -value))[:num]
    assert p[0].tolist() == (want // v).tolist() and t[0].tolist() == (want % v).tolist()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("v", [7, 3001, 200000])
def test_rows_masked_by_the_lowest_value(pkv, cuda_device, dtype, v):
    """All of a beam masked: every token alike, log v below the beam's score.  A NaN among them
    still takes the beam out, and a beam with one token left goes on with that."""
    low = torch.finfo(dtype).min
    x = torch.full((1, 4, v), low, dtype=dtype)
    x[0, 1, v // 2] = float("nan")
    x[0, 2, v - 1] = 1.0
    cum = np.array([[-1.0, 0.0, -20.0, -2.0]], dtype=np.float32)
    f64 = x.double().numpy()
    want = ref.beam(f64, cum, 9)
    got = pkv.beam_select(x.to(cuda_device), torch.from_numpy(cum).to(cuda_device), 9)
    check_beams(got, want[:3], want[3], f64, None)
    assert got[2][0, 0].item() == 0 and abs(got[0][0, 0].item() + 1 + np.log(v)) < 1e-4


def test_beams_that_are_not_there(pkv, cuda_device):
    """NaN, +inf and fully masked rows, beams of -inf, NaN and inf: no candidates of theirs."""
    rng = np.random.default_rng(8)
    v = 3000
    x = rng.standard_normal((1, 9, v)).astype(np.float32)
    x[0, 0, 1234] = np.nan
    x[0, 1, 7] = np.inf
    x[0, 2] = -np.inf
    x[0, 3, 5:] = -np.inf
    x[0, 7] = np.nan
    x[0, 8, 2999] = -np.nan
    cum = np.array([[0, 0, 0, -1, -np.inf, np.nan, np.inf, 0, 0]], dtype=np.float32)
    want = ref.beam(x.astype(np.float64), cum, 8)
    got = pkv.beam_select(torch.from_numpy(x).to(cuda_device), torch.from_numpy(cum).to(cuda_device), 8)
    check_beams(got, want[:3], want[3], x.astype(np.float64), None)
    assert got[2][0].tolist() == [3] * 5 + [-1] * 3
    none = pkv.beam_select(torch.full((2, 2, 50), -np.inf, device=cuda_device),
                           torch.zeros((2, 2), device=cuda_device), 3)
    assert none[1].tolist() == [[-1] * 3] * 2 and bool(torch.isneginf(none[0]).all())


def test_finished_beams_keep_their_score(pkv, cuda_device):
    x = torch.zeros((2, 3, 100), device=cuda_device)
    x[:, 1] = float("nan")                       # a finished beam's logits are not read
    cum = torch.tensor([[-9.0, -3.5, -1.0], [-2.0, -1.0, -float("inf")]], device=cuda_device)
    done = torch.tensor([[False, True, False], [False, True, True]], device=cuda_device)
    s, t, p = pkv.beam_select(x, cum, 3, finished=done, pad_token=77)
    assert t.tolist() == [[77, 0, 1], [77, 0, 1]] and p.tolist() == [[1, 2, 2], [4, 3, 3]]
    assert s[:, 0].tolist() == [-3.5, -1.0]
    assert torch.equal(s, pkv.beam_select(x, cum, 3, finished=done.to(torch.uint8), pad_token=77)[0])


# ------------------------------------------------------------------------- streams, graphs

def test_page_calls_captured_and_on_another_stream(pkv, cuda_device):
    """Fork, reserve, copy and free in one graph, replayed on the restored state twice; then the
    same on a side stream: the same arrays as one after another."""
    dev = cuda_device
    rng = np.random.default_rng(12)
    rows, width, blocks = 24, 12, 600
    tables, ctx, refs = ref.random_tables(rng, rows, width, blocks, 0.8, width * 16 - 20)
    parents, n = rng.integers(0, rows, rows), rng.integers(0, 20, rows)
    cu = np.concatenate([[0], np.cumsum(n)])
    done = np.array([3, 3, -1, 9])
    pool = torch.from_numpy(rng.integers(0, 256, (blocks, 512), dtype=np.uint8))
    new, new_ctx = np.full((rows, width), -1), np.zeros(rows, dtype=np.int64)
    want_refs = refs.copy()
    ref.fork(parents, tables, ctx, want_refs, new, new_ctx, False)
    slots, src, dst = ref.reserve(cu, new, new_ctx, want_refs)
    want_pool = pool.numpy().copy()
    for s, d in zip(src, dst):
        if s >= 0:
            want_pool[d] = want_pool[s]
    ref.free(done, new, new_ctx, want_refs)
    d = dict(tables=dev_i32(tables, dev), ctx=dev_i32(ctx, dev), refs=dev_i32(refs, dev),
             parents=dev_i32(parents, dev), cu=dev_i32(cu, dev), done=dev_i32(done, dev),
             new=dev_i32(np.full((rows, width), -1), dev), new_ctx=dev_i32(np.zeros(rows), dev),
             pool=pool.to(dev), st=status_of(dev))

    def bind(stream=None):
        kw = dict(dev_status=d["st"], stream=stream)
        fork = pkv.BoundForkSequences(d["parents"], d["tables"], d["ctx"], d["refs"], d["new"],
                                      d["new_ctx"], **kw)
        room = pkv.BoundReserveBlocks(d["cu"], d["new"], d["new_ctx"], d["refs"],
                                      num_tokens=int(cu[-1]), **kw)
        copy = pkv.BoundCopyBlocks([d["pool"]], room.copy_src, room.copy_dst, **kw)
        end = pkv.BoundFreeSequences(d["done"], d["new"], d["new_ctx"], d["refs"], **kw)
        return (fork, room, copy, end), room

    def restore():
        d["refs"].copy_(dev_i32(refs, dev))
        d["pool"].copy_(pool)
        d["new"].fill_(-1)

    def check(room):
        torch.cuda.synchronize(dev)
        for got, want in ((d["new"], new), (d["new_ctx"], new_ctx), (d["refs"], want_refs),
                          (room.slot_mapping, slots), (room.copy_src, src), (room.copy_dst, dst),
                          (d["pool"], want_pool)):
            same(got, want)
        assert int(d["st"].item()) == 0

    side = torch.cuda.Stream(dev)
    calls, room = bind(side)
    torch.cuda.synchronize(dev)
    for c in calls:
        c.run()
    check(room)
    restore()
    torch.cuda.synchronize(dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for c in calls:
            c.run()
    for _ in range(2):
        restore()
        graph.replay()
        check(room)


@pytest.mark.parametrize("seed", range(4))
def test_the_life_of_a_pool(pkv, cuda_device, seed):
    """Random forks (all rows reordered, or some added), reservations with their copies and
    writes, ends of sequences and compactions over one small pool: after each, tables, lengths and
    counts are those of the plain forms, and every row's blocks hold what the row has written."""
    dev, rng = cuda_device, np.random.default_rng(4000 + seed)
    rows, width, blocks = 12, 7, 70
    tables, ctx, refs = (np.full((rows, width), -1), np.zeros(rows, dtype=np.int64),
                         np.zeros(blocks, dtype=np.int64))
    pool = torch.zeros((blocks, 16), dtype=torch.int32, device=dev)   # a number a slot
    rowed = [[] for _ in range(rows)]
    d_tables, d_ctx, d_refs = (dev_i32(x, dev) for x in (tables, ctx, refs))
    st, stamp = status_of(dev), 0
    for step in range(80):
        kind = rng.choice(["fork", "reserve", "reserve", "free", "compact"])
        if kind == "fork":
            parents = np.where(rng.random(rows) < 0.6, np.arange(rows), rng.integers(-1, rows, rows))
            new, new_ctx = np.full((rows, width), -1), np.zeros(rows, dtype=np.int64)
            ref.fork(parents, tables, ctx, refs, new, new_ctx, False)
            d_new, d_new_ctx = dev_i32(np.full((rows, width), -1), dev), dev_i32(np.zeros(rows), dev)
            pkv.fork_sequences(dev_i32(parents, dev), d_tables, d_ctx, d_refs, d_new, d_new_ctx,
                               dev_status=st)
            tables, ctx, d_tables, d_ctx = new, new_ctx, d_new, d_new_ctx
            rowed = [list(rowed[p]) if p >= 0 else [] for p in parents]
        elif kind == "reserve":
            n = np.where(rng.random(rows) < 0.5, 0, rng.integers(0, 20, rows))
            cu = np.concatenate([[0], np.cumsum(n)])
            want = [tables.copy(), ctx.copy(), refs.copy()]
            got = ref.reserve(cu, *want)
            slots, src, dst = pkv.reserve_blocks(dev_i32(cu, dev), d_tables, d_ctx, d_refs,
                                                 num_tokens=int(cu[-1]), dev_status=st)
            if got is None:
                assert int(st.item()) == 7 and (slots.numel() == 0 or int(slots.max()) == -1)
                st.zero_()
            else:
                tables, ctx, refs = want
                for a, b in zip((slots, src, dst), got):
                    same(a, b)
                pkv.copy_blocks(pool, src, dst, dev_status=st)
                stamps = np.arange(stamp, stamp + int(cu[-1]))
                stamp += int(cu[-1])
                pool.view(-1)[slots.long()] = dev_i32(stamps, dev)
                for r in range(rows):
                    rowed[r] += stamps[cu[r]:cu[r + 1]].tolist()
        elif kind == "free":
            listed = rng.integers(-1, rows, 3)
            ref.free(listed, tables, ctx, refs)
            pkv.free_sequences(dev_i32(listed, dev), d_tables, d_ctx, d_refs, dev_status=st)
            for r in listed[listed >= 0]:
                rowed[r] = []
        else:
            tables, refs, src, dst = ref.compact(tables, ctx, refs)
            a, b, n = pkv.compact_blocks(d_tables, d_ctx, d_refs, dev_status=st)
            assert int(n.item()) == len(src) and a.tolist()[:len(src)] == src and b.tolist()[:len(src)] == dst
            pkv.copy_blocks([pool], a, b, num_pairs=n, dev_status=st)
        assert int(st.item()) == 0
        same(d_ctx, ctx)
        same(d_refs, refs)
        table, held = d_tables.cpu().numpy(), pool.cpu().numpy()
        for r in range(rows):
            n = ref.used(ctx[r])
            assert table[r, :n].tolist() == tables[r, :n].tolist()
            assert held[table[r, :n]].reshape(-1)[:ctx[r]].tolist() == rowed[r], (step, kind, r)


def test_python_refusals_on_device_tensors(pkv, cuda_device):
    dev = cuda_device
    t, c, r = dev_i32(np.zeros((4, 5)), dev), dev_i32(np.zeros(4), dev), dev_i32(np.zeros(9), dev)
    with pytest.raises(ValueError, match="overlap"):
        pkv.fork_sequences(c.clone(), t, c, r, t, c.clone())
    both = dev_i32(np.zeros((6, 5)), dev)
    with pytest.raises(ValueError, match="overlap"):
        pkv.fork_sequences(c.clone(), both[:4], c, r, both[2:], c.clone())
    with pytest.raises(ValueError, match="apart"):
        pkv.compact_blocks(both[:4], c, r, new_tables=both[2:])
    with pytest.raises(ValueError):
        pkv.fork_sequences(c, t, c, r, t[:, :4].contiguous(), c.clone())
    with pytest.raises(ValueError, match="num_tokens"):
        pkv.reserve_blocks(dev_i32(np.zeros(5), dev), t, c, r)
    with pytest.raises(ValueError):
        pkv.reserve_blocks(dev_i32(np.zeros(4), dev), t, c, r, num_tokens=1)
    with pytest.raises(TypeError):
        pkv.free_sequences(c.long(), t, c, r)
    with pytest.raises(ValueError, match="same number"):
        pkv.copy_blocks([t, r], c, c.clone())
    with pytest.raises(ValueError, match="multiple of 4"):
        pkv.copy_blocks(torch.zeros((4, 3), dtype=torch.uint8, device=dev), c, c.clone())
    x = torch.zeros((2, 3, 10), device=dev)
    cum = torch.zeros((2, 3), device=dev)
    for bad in (x.transpose(1, 2), x[:, :, ::2], torch.zeros((2, 4, 10), device=dev)[:, :3]):
        with pytest.raises(ValueError):
            pkv.beam_select(bad, cum if bad.shape[1] == 3 else torch.zeros(bad.shape[:2], device=dev), 2)
    with pytest.raises(ValueError, match="cum_scores"):
        pkv.beam_select(x, cum[:1], 2)
    with pytest.raises(TypeError):
        pkv.beam_select(x.double(), cum, 2)
    with pytest.raises(ValueError, match="overlap"):
        pkv.beam_select(x, cum, 3, scores=cum)
    with pytest.raises(pkv.PkvError):
        pkv.beam_select(x, cum, 129)


# ------------------------------------------------------------------------- beams: far scores, far logits

def live_rows(rng, x, live, mask):
    """All but `live` random tokens of each row masked by `mask`."""
    for row in x.view(-1, x.shape[-1]):
        row[torch.from_numpy(rng.permutation(len(row))[live:])] = mask
    return x


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("b,k,v,num", [(1, 1, 128000, 16), (1, 4, 32000, 16), (2, 2, 128000, 128),
                                       (1, 1, 50257, 128), (3, 40, 9001, 33)])
@pytest.mark.parametrize("far", [-1e6, -1e9, -1e12, -1e25, LOWEST])
def test_beams_far_below_are_ranked_by_their_logits(pkv, cuda_device, dtype, b, k, v, num, far):
    """Scores so low that the logits' differences vanish in them: the first beam has three tokens
    left, the others' candidates follow by their logits, over all ranges a row is cut into."""
    rng = np.random.default_rng(v + num)
    x = beam_case(rng, b, k, v, dtype)
    if k > 1:
        live_rows(rng, x[:, 0], 3, -np.inf)
    cum = np.full((b, k), far, dtype=np.float32)
    cum[:, 0] = -1.0 if k > 1 else far
    f64 = x.double().numpy()
    want = ref.beam(f64, cum, num)
    got = pkv.beam_select(x.to(cuda_device), torch.from_numpy(cum).to(cuda_device), num)
    check_beams(got, want[:3], want[3], f64, None)


@pytest.mark.parametrize("b,k,v,num", [(1, 1, 128000, 16), (1, 3, 32000, 128), (90, 4, 9001, 5)])
def test_logits_closer_than_a_score_can_tell(pkv, cuda_device, b, k, v, num):
    """Logits of 1e-30: every score of a beam is the same number, the order is the logits'."""
    rng = np.random.default_rng(v)
    x = (beam_case(rng, b, k, v, torch.float32) * 1e-30).float()
    cum = np.tile(-5.0 - np.arange(k, dtype=np.float32), (b, 1))
    f64 = x.double().numpy()
    s, t, p = (g.cpu().numpy() for g in
               pkv.beam_select(x.to(cuda_device), torch.from_numpy(cum).to(cuda_device), num))
    for i in range(b):
        best = np.lexsort((np.arange(v), -f64[i, 0]))[:num]
        assert t[i].tolist() == best.tolist() and (p[i] == i * k).all()
    assert (np.abs(s - (-5.0 - np.log(v))) <= LSE_TOL + 2.0 ** -24 * 20).all()


FAR = [-1e8, -7.4e8, -7.5e8, -1e9, -1e10, -1e12, -1e20, -1e30, -1e38, -2.3e38, -2.4e38, LOWEST]


@pytest.mark.parametrize("mask", FAR)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v,many", [(7, False), (300, False), (3001, False), (70001, False), (9001, True)])
def test_rows_masked_by_any_low_value(pkv, cuda_device, mask, dtype, v, many):
    """Most of a row, all of it, all but its last token, one end of it, or all but a second low
    value masked by a finite number: the live tokens' scores are those of the live tokens alone."""
    rng = np.random.default_rng(v)
    b, k = (60, 5) if many else (1, 5)
    x = beam_case(rng, 1, k, v, dtype)
    live_rows(rng, x[:, 0], max(v // 100, 1), mask)
    x[0, 1] = mask
    x[0, 2, :-1] = mask
    x[0, 3, v // 3:] = mask
    x[0, 4] = mask
    x[0, 4, [1, v // 2]] = max(2 * mask, LOWEST)
    cum = np.array([[-0.5, 0.0, -20.0, -2.0, -1.5]], dtype=np.float32)
    f64 = x.double().numpy()
    for num in (3, 40):
        want = ref.beam(f64, cum, num)
        got = pkv.beam_select(x.to(cuda_device).expand(b, k, v).contiguous(),
                              torch.from_numpy(cum).to(cuda_device).expand(b, k).contiguous(), num)
        check_beams([g[:1] for g in got], want[:3], want[3], f64, None)
        assert torch.equal(got[1], got[1][:1].expand_as(got[1]))


@pytest.mark.parametrize("top", [1e8, 7.4e8, 7.5e8, 1e10, 1e20, 2e38, 2.5e38, -LOWEST])
@pytest.mark.parametrize("v,many", [(7, False), (3001, False), (70001, False), (9001, True)])
def test_logits_of_any_finite_size(pkv, cuda_device, top, v, many):
    """Huge logits are numbers like others: one, several alike, beside ordinary and low ones."""
    rng = np.random.default_rng(v)
    b, k = (60, 4) if many else (1, 4)
    x = beam_case(rng, 1, k, v, torch.float32)
    x[0, 0, v // 2] = top
    x[0, 1, [0, v // 3, v - 1]] = top
    x[0, 2, v - 2], x[0, 2, v - 1] = top, top / 2
    x[0, 3] = torch.from_numpy(np.where(rng.random(v) < 0.5, top, -1e5)).float()
    cum = np.array([[-1.0, -2.0, -0.5, 0.0]], dtype=np.float32)
    f64 = x.double().numpy()
    for num in (4, 33):
        want = ref.beam(f64, cum, num)
        got = pkv.beam_select(x.to(cuda_device).expand(b, k, v).contiguous(),
                              torch.from_numpy(cum).to(cuda_device).expand(b, k).contiguous(), num)
        check_beams([g[:1] for g in got], want[:3], want[3], f64, None)
        assert torch.equal(got[1], got[1][:1].expand_as(got[1]))


def test_scores_past_fp32_are_not_candidates(pkv, cuda_device):
    x = torch.tensor([[[-LOWEST, LOWEST, -LOWEST], [LOWEST, LOWEST, LOWEST]]], device=cuda_device)
    s, t, p = pkv.beam_select(x, torch.tensor([[0.0, LOWEST]], device=cuda_device), 6)
    assert t[0].tolist() == [0, 2, 0, 1, 2, -1] and p[0].tolist() == [0, 0, 1, 1, 1, -1]
    assert s[0, 2:5].tolist() == [LOWEST] * 3 and bool(torch.isneginf(s[0, 5]))


# ------------------------------------------------------------------------- reserve without rows

@pytest.mark.parametrize("on_stream", [False, True])
def test_reserve_of_no_rows_gives_no_slot(pkv, cuda_device, on_stream):
    """A padded step none of whose rows is there: every slot is -1, whatever it was."""
    dev = cuda_device
    t, c, r = (torch.zeros(s, dtype=torch.int32, device=dev) for s in ((0, 4), (0,), (9,)))
    cu, whole = dev_i32([0], dev), dev_i32(np.full(12, 77), dev)
    stream = torch.cuda.Stream(dev) if on_stream else None
    torch.cuda.synchronize(dev)
    bound = pkv.BoundReserveBlocks(cu, t, c, r, slot_mapping=whole[:7], stream=stream)
    bound.run()
    torch.cuda.synchronize(dev)
    assert whole.cpu().tolist() == [-1] * 7 + [77] * 5
    slots, src, dst = pkv.reserve_blocks(cu, t, c, r, num_tokens=5)
    assert slots.cpu().tolist() == [-1] * 5 and src.numel() == 0 and dst.numel() == 0
    assert r.cpu().tolist() == [0] * 9
    pkv.reserve_blocks(cu, t, c, r, num_tokens=0)


@pytest.mark.parametrize("b,k,v,num", [(1, 4, 32000, 8), (1, 1, 128000, 16), (1, 2, 128000, 128), (3, 70, 9001, 20)])
def test_log_probabilities_of_confident_beams(pkv, cuda_device, b, k, v, num):
    """Logits that are log-probabilities: the best of a beam next to 0, or 0 itself, beside others
    far below; and some of them closer to each other than a score can tell."""
    rng = np.random.default_rng(num)
    x = beam_case(rng, b, k, v, torch.float32)
    x[:, ::2, v // 3] = 30.0
    x = torch.log_softmax(x, dim=-1)
    x[:, ::3, v // 2] = 0.0
    near = [v // 5, v // 4, v - 3]
    x[:, k - 1, near] = torch.tensor([-1e-9, -3e-9, -2e-9])
    cum = rng.uniform(-30, 0, (b, k)).astype(np.float32)
    f64 = x.double().numpy()
    want = ref.beam(f64, cum, num)
    got = pkv.beam_select(x.to(cuda_device), torch.from_numpy(cum).to(cuda_device), num)
    check_beams(got, want[:3], want[3], f64, None)


def test_scores_of_far_logits_are_rounded_once(pkv, cuda_device):
    """-1e10 beside -1e9: the difference is a tie between two fp32 numbers, the score is not."""
    x = torch.tensor([[[-1e9, -1e10, -1e10]]], device=cuda_device)
    s, t, _ = pkv.beam_select(x, torch.tensor([[-28.85]], device=cuda_device), 3)
    assert t[0].tolist() == [0, 1, 2] and s[0].tolist() == [np.float32(-28.85), -9000000512.0, -9000000512.0]
