"""GPU tests of the block index, the selection by it and the attention over selected blocks,
against the plain host forms of pages_ref.py.

Bounds, units and selected blocks are integers and powers of two: no tolerance.  Attention:
  - a score is an fp32 sum of D products of bf16 values: off by at most D 2^-24 S, S the sum of
    |q K| times |scale|; its scaling to log2 units and ex2 add 2^-22 and 2 |x| 2^-24 with |x| <= 2 S;
  - each weight is rounded to bf16 for the product with V, 2^-8 of itself (its sum L is not);
  - the sums over the keys (16 at a time by the tensor cores, the blocks one after another, the
    warps at the end) add less than 2^-14 for 2^9 blocks;
  - the result is rounded once to bf16, 2^-8 of itself.
With A = sum w |V|:  |got - want| <= 2^-8 |want| + A (2^-8 (1 + 2^-8) + 2 e), the score's
e = (D + 4) 2^-24 S + 2^-22 + 2^-14 counted for the weight and for L.
"""

import numpy as np
import pytest
import torch

import pages_ref as ref
import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv(cuda_device):
    import paged_kv_attention_append_gb300 as m
    m.build()
    return m


def dev_i32(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)


def status_of(dev):
    return torch.zeros(1, dtype=torch.int32, device=dev)


def bf16(x):
    return torch.from_numpy(np.asarray(x)).to(torch.bfloat16)


def make_pool(rng, blocks, hkv, d):
    x = rng.standard_normal((blocks, 2, hkv, 16, d), dtype=np.float32)
    x[:, 0] = 0.5 * x[:, 0] + rng.standard_normal((blocks, hkv, 1, d), dtype=np.float32)
    return bf16(x)


def whole_index(pool):
    """index and units of a pool's blocks, all rows of each."""
    k = pool[:, 0].double().numpy()
    both = [ref.bounds(b) for b in k]
    return (np.stack([b for b, _ in both]).astype(np.int8),
            np.stack([u for _, u in both]).astype(np.float32))


def check_out(got, want, mag, dots, d):
    got = got.double().cpu().numpy()
    e = (d + 4) * 2.0 ** -24 * dots[..., None] + 2.0 ** -22 + 2.0 ** -14
    tol = 2.0 ** -8 * np.abs(want) + mag * (2.0 ** -8 * (1 + 2.0 ** -8) + 2 * e)
    over = np.abs(got - want) - tol
    assert (over <= 0).all(), f"worst {over.max():.3e} over the bound at {np.unravel_index(over.argmax(), over.shape)}"


# ------------------------------------------------------------------------- the index

UPDATES = [  # (hkv, d, tokens of each sequence in the step, their contexts before it)
    (8, 128, [1, 1, 1, 1], [0, 15, 16, 30]), (2, 64, [5, 40, 1], [3, 14, 0]), (1, 128, [333], [0]),
    (3, 64, [1] * 40, list(range(40))), (5, 128, [17, 2], [15, 31]),
]


@pytest.mark.parametrize("case", range(len(UPDATES)))
def test_index_of_what_a_step_wrote(pkv, cuda_device, case):
    """Blocks written to get the bounds of their rows up to the last one written, others keep
    what they had; what lies past the rows does not count."""
    hkv, d, n, before = UPDATES[case]
    rng = np.random.default_rng(40 + case)
    need = [-(-(b + t) // 16) for b, t in zip(before, n)]
    perm = rng.permutation(sum(need) + 4)
    pool = make_pool(rng, len(perm), hkv, d)
    pool *= torch.from_numpy(np.exp2(rng.integers(-6, 7, (len(perm), 1, hkv, 1, 1)))).to(pool.dtype)
    slots, upto, at = [], {}, 0
    for b, t, m in zip(before, n, need):
        ids = perm[at:at + m]
        at += m
        for p in range(b, b + t):
            slots.append(ids[p // 16] * 16 + p % 16)
            upto[int(ids[p // 16])] = p % 16
    keys = pool[:, 0].double().numpy()
    for b, last in upto.items():
        pool[b, 0, :, last + 1:] = float("nan") if b % 2 else 1e30
    where = rng.permutation(len(slots)) if sum(n) <= 16 else np.arange(len(slots))
    slots = np.array(slots)[where].tolist() + [-1, -9]
    index, scales = (torch.from_numpy(rng.integers(-127, 128, (len(perm), hkv, 2, d), dtype=np.int8)),
                     torch.full((len(perm), hkv), 3.0))
    want, unit = index.numpy().copy(), scales.numpy().copy()
    for b, last in upto.items():
        want[b], unit[b] = ref.bounds(keys[b, :, :last + 1])
    dev = cuda_device
    index, scales, st = index.to(dev), scales.to(dev), status_of(dev)
    pkv.update_block_index(pool.to(dev), dev_i32(slots, dev), index, scales, dev_status=st)
    np.testing.assert_array_equal(scales.cpu().numpy(), unit)
    np.testing.assert_array_equal(index.cpu().numpy(), want)
    assert int(st.item()) == 0


def test_index_values_at_the_borders(pkv, cuda_device):
    """Largest keys next to 127 and 128 units, tiny, subnormal, zero, huge, not finite."""
    tops = [127.0, 127.5, 126.5, 128.0, 1.0, 1.984375, 1.9921875, 2.0 ** -70, 2.0 ** -64 * 127, 2.0 ** -130,
            0.0, 3.3895313892515355e38, 2.0 ** 100, 2.0 ** -57]
    rng = np.random.default_rng(7)
    x = rng.uniform(-1, 1, (len(tops), 2, 1, 16, 64)) * np.array(tops)[:, None, None, None, None]
    x[:, 0, 0, 3, 5], x[:, 0, 0, 9, 6] = tops, [-t for t in tops]
    x[:, 0, 0, 4, 7] = 2.0 ** -120
    x[:, 0, 0, :, 8] = -2.0 ** -133
    pool = bf16(x)
    pool[2, 0, 0, 1, 1], pool[2, 0, 0, 2, 2] = float("inf"), float("nan")
    pool[4, 0, 0, :, 3] = -float("inf")
    dev = cuda_device
    index, scales = pkv.block_index(len(tops), 1, 64, device=dev)
    pkv.update_block_index(pool.to(dev), dev_i32(np.arange(len(tops)) * 16 + 15, dev), index, scales)
    want, unit = whole_index(pool)
    np.testing.assert_array_equal(scales.cpu().numpy(), unit)
    np.testing.assert_array_equal(index.cpu().numpy(), want)


def test_index_after_rejected_tokens_and_bad_slots(pkv, cuda_device):
    dev = cuda_device
    pool = torch.zeros((3, 2, 1, 16, 64), dtype=torch.bfloat16, device=dev)
    pool[1, 0, 0, 4], pool[1, 0, 0, 5:8] = 1.0, 100.0
    index, scales = pkv.block_index(3, 1, 64, device=dev)
    pkv.update_block_index(pool, dev_i32([20, 21, 22, 23], dev), index, scales)
    assert int(index[1, 0, 1].max()) == 100 and float(scales[1]) == 1.0
    pool[1, 0, 0, 5] = 2.0                       # the three are rejected, one follows
    st = status_of(dev)
    pkv.update_block_index(pool, dev_i32([21, 48, -1, 2 ** 31 - 1], dev), index, scales, dev_status=st)
    assert float(scales[1]) == 2.0 ** -5 and int(index[1, 0, 1].max()) == 64 and int(st.item()) == 1
    assert int(index[0].abs().max()) == 0


# ------------------------------------------------------------------------- selection

SELECTS = [  # (hq, hkv, d, q_lens, contexts, num, sink, recent)
    (8, 2, 64, [1, 1, 1, 1], [1, 16, 17, 500], 4, 1, 1),
    (16, 8, 128, [1, 1], [4096, 3001], 32, 1, 2),
    (40, 8, 128, [1, 5, 0, 3], [9000, 700, 0, 33], 20, 2, 3),
    (5, 5, 64, [2, 1], [2000, 1], 9, 0, 9),
    (16, 1, 128, [1, 4], [30000, 100], 100, 4, 8),
    (6, 3, 128, [30], [1000], 7, 0, 1),
    (64, 16, 64, [1, 1, 1], [777, 20000, 40], 50, 3, 3),
    (2, 2, 64, [1], [170000], 300, 1, 1),
    (24, 12, 128, [9, 9, 1, 9, 9, 9, 0, 2], [9, 10, 400, 67, 150, 33, 5, 900], 6, 1, 2),  # many pairs
    (32, 16, 64, [4] * 8, [900, 4, 600, 513, 15, 1000, 530, 700], 32, 2, 3),
]


def select_case(case, seed=0, spoil=None):
    hq, hkv, d, n, ctx, num, sink, recent = SELECTS[case]
    rng = np.random.default_rng(200 + 10 * case + seed)
    meta = workloads.build_step("select", 1, n, ctx, hq, hkv, d, rng=rng)
    pool = make_pool(rng, meta.num_blocks, hkv, d)
    q = rng.standard_normal((meta.total_q, hq, d)) * np.exp2(rng.integers(-8, 9, (meta.total_q, hq, 1)))
    return meta, pool, bf16(q)


def expected(meta, q, index, unit, num, sink, recent):
    q = q.double().numpy()
    out = []
    for s, (n, c) in enumerate(zip(meta.q_lens, meta.context_lens)):
        for i in range(n):
            out.append(ref.select(q[len(out)], c - n + i, meta.block_tables[s], index, unit, num, sink,
                                  recent))
    return np.stack(out)


def run_select(pkv, dev, meta, q, index, unit, num, sink, recent, **kw):
    st = status_of(dev)
    got = pkv.select_blocks(q.to(dev), dev_i32(meta.cu_q_lens, dev), dev_i32(meta.context_lens, dev),
                            dev_i32(meta.block_tables, dev), torch.as_tensor(index).to(dev),
                            torch.as_tensor(unit).to(dev), num, sink_blocks=sink,
                            recent_blocks=recent, dev_status=st, **kw)
    return got, int(st.item())


@pytest.mark.parametrize("case", range(len(SELECTS)))
@pytest.mark.parametrize("seed", [0, 1])
def test_selection(pkv, cuda_device, case, seed):
    meta, pool, q = select_case(case, seed)
    index, unit = whole_index(pool)
    args = SELECTS[case][5:]
    got, st = run_select(pkv, cuda_device, meta, q, index, unit, *args)
    np.testing.assert_array_equal(got.cpu().numpy(), expected(meta, q, index, unit, *args))
    assert st == 0


@pytest.mark.parametrize("kind", ["equal", "few values", "units far apart", "zeros", "both signs"])
@pytest.mark.parametrize("ctx", [1500, 140000])
def test_selection_among_ties(pkv, cuda_device, kind, ctx):
    """Scores that coincide, by the hundred and at the border of the selection."""
    rng = np.random.default_rng(ctx)
    meta = workloads.build_step("ties", 1, [1], [ctx], 4, 2, 64, rng=rng)
    shape = (meta.num_blocks, 2, 2, 64)
    index = rng.integers(-127, 128, shape, dtype=np.int8)
    unit = np.ones(shape[:2], dtype=np.float32)
    if kind == "equal":
        index[:] = index[:1]
    elif kind == "few values":
        index[:] = index[rng.integers(0, 5, len(index))]
    elif kind == "units far apart":
        unit = np.exp2(rng.choice([-64, -3, 0, 90, 121], unit.shape)).astype(np.float32)
    elif kind == "zeros":
        index[rng.random(len(index)) < 0.9] = 0
    else:
        index = np.sign(index) * np.int8(1)
    q = bf16(rng.standard_normal((1, 4, 64)))
    if kind == "equal":
        q[:, 2:] = 0
    for num, sink, recent in ((40, 1, 2), (7, 0, 1), (63, 20, 10)):
        got, st = run_select(pkv, cuda_device, meta, q, index, unit, num, sink, recent)
        np.testing.assert_array_equal(got.cpu().numpy(),
                                      expected(meta, q, index, unit, num, sink, recent))
        assert st == 0


def test_selection_queries_of_all_sizes(pkv, cuda_device):
    """Zero, subnormal, huge, infinite and NaN queries; the unit goes by the group's largest."""
    meta, pool, _ = select_case(0)
    rng = np.random.default_rng(9)
    index, unit = whole_index(pool)
    index = rng.integers(-127, 128, index.shape, dtype=np.int8)
    for q in (0.0, 2.0 ** -133, 2.0 ** -126, 2.0 ** -20, 1.9921875, 2.0 ** 30, 3.3e38):
        x = bf16(rng.uniform(-1, 1, (meta.total_q, 8, 64)) * q)
        x[0, 0, 3], x[-1, 5, 9], x[-1, 1, 1] = float("inf"), float("nan"), -float("inf")
        got, st = run_select(pkv, cuda_device, meta, x, index, unit, 5, 1, 1)
        np.testing.assert_array_equal(got.cpu().numpy(), expected(meta, x, index, unit, 5, 1, 1))


def test_selection_in_several_passes(pkv, cuda_device):
    """A workspace of any size from one token's on gives the same selection."""
    meta, pool, q = select_case(2)
    index, unit = whole_index(pool)
    dev, args = cuda_device, SELECTS[2][5:]
    want, _ = run_select(pkv, dev, meta, q, index, unit, *args)
    lib, width = pkv._load(), meta.block_tables.shape[1]
    one = lib.pkv_select_workspace_size(1, 8, width)
    d = [x.to(dev) for x in (q, torch.as_tensor(index), torch.as_tensor(unit))]
    cu, ctx, table = (dev_i32(x, dev) for x in (meta.cu_q_lens, meta.context_lens, meta.block_tables))
    import ctypes
    for size in (one, 2 * one + 7, 100 * one):
        ws = torch.empty(size, dtype=torch.uint8, device=dev)
        out = torch.full_like(want, -7)
        st = lib.pkv_select_blocks(
            d[0].data_ptr(), cu.data_ptr(), ctx.data_ptr(), table.data_ptr(), width, len(ctx),
            q.shape[0], 40, d[1].data_ptr(), d[2].data_ptr(),
            ctypes.byref(pkv.PoolDesc(meta.num_blocks, 16, 8, 128)), *args, out.data_ptr(),
            ws.data_ptr(), size, None, torch.cuda.current_stream(dev).cuda_stream)
        assert st == 0 and torch.equal(out, want)


def test_selection_and_attention_of_tokens_without_a_place(pkv, cuda_device):
    """Rows behind the last sequence (a padded batch) and windows longer than their context."""
    dev = cuda_device
    meta, pool, q = select_case(0)
    index, unit = (torch.as_tensor(x).to(dev) for x in whole_index(pool))
    more = torch.cat([q, q[:3]]).to(dev)
    cu, ctx = dev_i32(meta.cu_q_lens, dev), meta.context_lens.copy()
    table, st = dev_i32(meta.block_tables, dev), status_of(dev)
    want, _ = run_select(pkv, dev, meta, q, index, unit, 4, 1, 1)
    sel = pkv.select_blocks(more, cu, dev_i32(ctx, dev), table, index, unit, 4, sink_blocks=1,
                            recent_blocks=1, dev_status=st)
    assert torch.equal(sel[:4], want) and int(sel[4:].max()) == -1 and int(st.item()) == 0
    out = torch.full_like(more, 7.0)
    pkv.paged_sparse_attention(more, cu, dev_i32(ctx, dev), table, sel, pool.to(dev), 0.1, out=out,
                               dev_status=st)
    assert bool((out[4:] == 7.0).all()) and int(st.item()) == 0 and not bool((out[:4] == 7.0).any())
    for bad in (0, 16 * meta.block_tables.shape[1] + 1):
        ctx[1] = bad
        st.zero_()
        sel = pkv.select_blocks(q.to(dev), cu, dev_i32(ctx, dev), table, index, unit, 4, sink_blocks=1,
                                recent_blocks=1, dev_status=st)
        assert int(sel[1].max()) == -1 and int(st.item()) == 4 and torch.equal(sel[2:], want[2:])
        st.zero_()
        out = torch.full_like(more[:4], 7.0)
        pkv.paged_sparse_attention(q.to(dev), cu, dev_i32(ctx, dev), table, want, pool.to(dev), 0.1,
                                   out=out, dev_status=st)
        assert bool((out[1] == 7.0).all()) and int(st.item()) == 4
        assert not bool((out[[0, 2, 3]] == 7.0).any())


def test_bad_blocks(pkv, cuda_device):
    """A block id outside the pool is never read: it scores -inf, and attention leaves it out."""
    dev = cuda_device
    meta, pool, q = select_case(1)
    index, unit = whole_index(pool)
    table = meta.block_tables.copy()
    table[0, [5, 100]], table[1, 7] = [-3, meta.num_blocks], 2 ** 31 - 1
    good = dict(zip(("index", "unit"), (index, unit)))
    meta.block_tables = table
    got, st = run_select(pkv, dev, meta, q, good["index"], good["unit"], 32, 1, 2)
    sel = got.cpu().numpy()
    assert st == 2 and not np.isin(sel[0], [5, 100]).any() and not np.isin(sel[1], [7]).any()
    assert (np.diff(sel, axis=2) > 0).all()
    mine = np.sort(np.concatenate([sel[:, :, :-1], np.full((2, 8, 1), 5)], axis=2), axis=2)
    mine[1] = sel[1]
    stt = status_of(dev)
    out = pkv.paged_sparse_attention(q.to(dev), dev_i32(meta.cu_q_lens, dev),
                                     dev_i32(meta.context_lens, dev), dev_i32(table, dev),
                                     dev_i32(mine, dev), pool.to(dev), meta.scale, dev_status=stt)
    without = np.where(mine == 5, -1, mine)
    without[1] = mine[1]
    check_step(out, meta, q, pool, without)
    assert int(stt.item()) == 2


# ------------------------------------------------------------------------- attention

def check_step(out, meta, q, pool, selected):
    held, x = pool.double().numpy(), q.double().numpy()
    rows, t = [], 0
    for s, (n, c) in enumerate(zip(meta.q_lens, meta.context_lens)):
        for i in range(n):
            rows.append(ref.sparse_attention(x[t], c - n + i, meta.block_tables[s], selected[t], held,
                                             meta.scale))
            t += 1
    check_out(out, *(np.stack(r) for r in zip(*rows)), q.shape[2])


def attend(pkv, dev, meta, q, pool, selected, **kw):
    st = status_of(dev)
    out = pkv.paged_sparse_attention(q.to(dev), dev_i32(meta.cu_q_lens, dev),
                                     dev_i32(meta.context_lens, dev), dev_i32(meta.block_tables, dev),
                                     dev_i32(selected, dev), pool.to(dev), meta.scale, dev_status=st,
                                     **kw)
    return out, int(st.item())


@pytest.mark.parametrize("case", range(len(SELECTS)))
@pytest.mark.parametrize("scale", [None, 0.0, -0.3, 2.0])
def test_attention_over_selected_blocks(pkv, cuda_device, case, scale):
    meta, pool, q = select_case(case)
    if scale is not None:
        meta.scale = scale
    q = (q.float() / q.float().abs().amax(dim=(1, 2), keepdim=True) * 3).to(torch.bfloat16)
    rng = np.random.default_rng(case)
    num = SELECTS[case][5]
    sel = np.full((meta.total_q, meta.num_kv_heads, num), -1)
    t = 0
    for n, c in zip(meta.q_lens, meta.context_lens):
        for i in range(n):
            nb = (c - n + i) // 16 + 1
            for h in range(meta.num_kv_heads):
                k = min(nb, num)
                sel[t, h, :k] = np.sort(rng.choice(nb, k, replace=False))
            t += 1
    out, st = attend(pkv, cuda_device, meta, q, pool, sel)
    check_step(out, meta, q, pool, sel)
    assert st == 0
    # the same calls again, and in place: the same bits
    again, _ = attend(pkv, cuda_device, meta, q, pool, sel)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    qd = q.to(cuda_device)
    pkv.paged_sparse_attention(qd, dev_i32(meta.cu_q_lens, cuda_device),
                               dev_i32(meta.context_lens, cuda_device),
                               dev_i32(meta.block_tables, cuda_device), dev_i32(sel, cuda_device),
                               pool.to(cuda_device), meta.scale, out=qd)
    assert torch.equal(out.view(torch.int16), qd.view(torch.int16))


def test_selections_of_a_callers_own(pkv, cuda_device):
    """Any order, entries past the token's blocks, none at all, a block twice, one entry."""
    meta, pool, q = select_case(1)
    q = (q.float() / q.float().abs().amax(dim=(1, 2), keepdim=True)).to(torch.bfloat16)
    rng = np.random.default_rng(4)
    sel = np.full((2, 8, 9), -1)
    sel[0, 0] = [7, 3, 255, -1, 0, 256, 9000, 12, 2 ** 31 - 1]
    sel[0, 1, 4] = 255
    sel[0, 3] = [5, 5, 5, 2, 1, 1, 1, 1, 9]
    sel[1] = rng.integers(0, 187, (8, 9))
    out, st = attend(pkv, cuda_device, meta, q, pool, sel)
    check_step(out, meta, q, pool, sel)
    assert st == 0 and bool((out[0, 4:6] == 0).all())
    out, _ = attend(pkv, cuda_device, meta, q, pool, sel[:, :, :1])
    check_step(out, meta, q, pool, sel[:, :, :1])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_what_lies_past_the_position_does_not_matter(pkv, cuda_device, value):
    meta, pool, q = select_case(0)
    q = (q.float() / q.float().abs().amax(dim=(1, 2), keepdim=True)).to(torch.bfloat16)
    sel = np.full((4, 2, 4), -1)
    for t, c in enumerate(meta.context_lens):
        nb = -(-c // 16)
        sel[t, :, :min(nb, 4)] = np.arange(nb)[-4:]
    spoilt = pool.clone()
    for s, c in enumerate(meta.context_lens):
        if c % 16:
            spoilt[meta.block_tables[s, c // 16], :, :, c % 16:] = value
    clean, _ = attend(pkv, cuda_device, meta, q, pool, sel)
    got, st = attend(pkv, cuda_device, meta, q, spoilt, sel)
    assert torch.equal(clean.view(torch.int16), got.view(torch.int16)) and st == 0
    check_step(got, meta, q, pool, sel)


def test_all_blocks_selected_is_the_packed_attention(pkv, cuda_device):
    meta = workloads.build_step("all", 3, [1, 7, 20, 1], [700, 333, 20, 17], 16, 4, 128,
                                rng=np.random.default_rng(3))
    q, k, v, pool = workloads.make_values(meta)
    dev = cuda_device
    index, unit = pkv.block_index(meta.num_blocks, 4, 128, device=dev)
    sel = pkv.select_blocks(q.to(dev), *(dev_i32(x, dev) for x in (meta.cu_q_lens, meta.context_lens,
                                                                  meta.block_tables)), index, unit, 44)
    out, _ = attend(pkv, dev, meta, q, pool, sel.cpu().numpy())
    dense = pkv.paged_varlen_attention(q.to(dev), meta.cu_q_lens, meta.context_lens, meta.block_tables,
                                       pool.to(dev), meta.scale)
    check_step(out, meta, q, pool, sel.cpu().numpy())
    check_step(dense, meta, q, pool, sel.cpu().numpy())


# ------------------------------------------------------------------------- together

@pytest.mark.parametrize("graph", [False, True])
def test_a_beam_search_with_pages_and_sparse_attention(pkv, cuda_device, graph):
    """Steps of a search over two requests of three beams: select, fork, reserve, copy, append,
    index, select blocks, attend.  The beams' caches are kept on the host as plain lists of keys
    and values; each step's pages, slots, selection and output are those of the lists.  With
    `graph` two steps (from one set of tables to the other and back) are captured and replayed."""
    dev, rng = cuda_device, np.random.default_rng(77)
    req, beams, vocab, hq, hkv, d, width, blocks = 2, 3, 300, 8, 2, 64, 12, 90
    rows, num, scale = req * beams, 6, 0.125
    steps = 24
    pool = torch.zeros((blocks, 2, hkv, 16, d), dtype=torch.bfloat16, device=dev)
    index, unit = pkv.block_index(blocks, hkv, d, device=dev)
    tabs = [dev_i32(np.full((rows, width), -1), dev) for _ in range(2)]
    lens = [dev_i32(np.zeros(rows), dev) for _ in range(2)]
    refs, st = dev_i32(np.zeros(blocks), dev), status_of(dev)
    # prompts: one row a request, the other beams forked from it
    prompt = [90, 17]
    cu = np.concatenate([[0], np.cumsum(np.where(np.arange(rows) % beams == 0,
                                                 np.repeat(prompt, beams), 0))])
    slots, src, _ = pkv.reserve_blocks(dev_i32(cu, dev), tabs[0], lens[0], refs,
                                       num_tokens=int(cu[-1]), dev_status=st)
    assert int(src.max()) == -1
    kv = bf16(rng.standard_normal((2, int(cu[-1]), hkv, d)))
    pkv.paged_kv_append(kv[0].to(dev), kv[1].to(dev), slots, pool)
    pkv.update_block_index(pool, slots, index, unit)
    cache = [kv[:, cu[r]:cu[r + 1]].double().numpy() for r in range(rows)]
    cache = [cache[r // beams * beams] for r in range(rows)]
    first = dev_i32(np.repeat([0, beams], beams), dev)
    logits = torch.zeros((req, beams, vocab), device=dev)
    cum = torch.zeros((req, beams), device=dev)
    q = torch.zeros((rows, hq, d), dtype=torch.bfloat16, device=dev)
    k, v = (torch.zeros((rows, hkv, d), dtype=torch.bfloat16, device=dev) for _ in range(2))
    one = dev_i32(np.arange(rows + 1), dev)
    pkv.fork_sequences(first, tabs[0], lens[0], refs, tabs[1], lens[1], dev_status=st)
    side = torch.cuda.Stream(dev) if graph else None
    torch.cuda.synchronize(dev)
    beam = pkv.BoundBeamSelect(logits, cum, beams, stream=side)
    parents = beam.parents.view(-1)

    def bind(a, b):
        kw = dict(dev_status=st, stream=side)
        fork = pkv.BoundForkSequences(parents, tabs[a], lens[a], refs, tabs[b], lens[b], **kw)
        room = pkv.BoundReserveBlocks(one, tabs[b], lens[b], refs, num_tokens=rows, **kw)
        copy = pkv.BoundCopyBlocks([pool, index, unit], room.copy_src, room.copy_dst, **kw)
        idx = pkv.BoundIndexUpdate(pool, room.slot_mapping, index, unit, **kw)
        sel = pkv.BoundSelectBlocks(q, one, lens[b], tabs[b], index, unit, num, sink_blocks=1,
                                    recent_blocks=1, **kw)
        att = pkv.BoundSparseAttention(q, one, lens[b], tabs[b], sel.selected, pool, scale,
                                       torch.empty_like(q), **kw)

        def run():
            beam.run()
            fork.run()
            room.run()
            copy.run()
            pkv.paged_kv_append(k, v, room.slot_mapping, pool, dev_status=st)
            idx.run()
            sel.run()
            att.run()
        return run, room, sel, att

    bound = {1: bind(1, 0), 0: bind(0, 1)}
    graphs = {}
    if graph:
        saved = [x.clone() for x in (*tabs, *lens, refs, pool, index, unit)]
        torch.cuda.synchronize(dev)
        for a in (1, 0):
            graphs[a] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graphs[a], stream=side):
                bound[a][0]()
        torch.cuda.synchronize(dev)
        for x, y in zip((*tabs, *lens, refs, pool, index, unit), saved):
            assert torch.equal(x, y)             # captured, not run
    a = 1
    for step in range(steps):
        logits.copy_(torch.from_numpy(rng.standard_normal((req, beams, vocab)) * 2))
        cum.copy_(torch.from_numpy(rng.uniform(-1, 0, (req, beams))))
        q.copy_(bf16(rng.standard_normal((rows, hq, d))))
        k.copy_(bf16(rng.standard_normal((rows, hkv, d))))
        v.copy_(bf16(rng.standard_normal((rows, hkv, d))))
        run, room, sel, att = bound[a]
        torch.cuda.synchronize(dev)
        graphs[a].replay() if graph else run()
        torch.cuda.synchronize(dev)
        assert int(st.item()) == 0
        want = ref.beam(logits.double().cpu().numpy(), cum.cpu().numpy(), beams)
        assert beam.tokens.cpu().tolist() == want[1].tolist()
        par = parents.cpu().tolist()
        assert par == want[2].reshape(-1).tolist()
        new = torch.stack([k, v]).double().cpu().numpy()
        cache = [np.concatenate([cache[p], new[:, i:i + 1]], axis=1) for i, p in enumerate(par)]
        b = 1 - a
        table, held = tabs[b].cpu().numpy(), pool.double().cpu().numpy()
        assert lens[b].cpu().tolist() == [c.shape[1] for c in cache]
        counts = np.zeros(blocks, dtype=np.int64)
        idx, uni = index.cpu().numpy(), unit.cpu().numpy()
        out, xs = att.out, q.double().cpu().numpy()
        rows_want = []
        for r, c in enumerate(cache):
            n = c.shape[1]
            ids = table[r, :-(-n // 16)]
            np.add.at(counts, ids, 1)
            got = held[ids].transpose(1, 0, 3, 2, 4).reshape(2, -1, hkv, d)[:, :n]
            np.testing.assert_array_equal(got, c)
            for j, blk in enumerate(ids):
                w, u = ref.bounds(c[0, j * 16:j * 16 + 16].transpose(1, 0, 2))
                np.testing.assert_array_equal(idx[blk], w)
                np.testing.assert_array_equal(uni[blk], u)
            chosen = ref.select(xs[r], n - 1, table[r], idx, uni, num, 1, 1)
            np.testing.assert_array_equal(sel.selected[r].cpu().numpy(), chosen)
            rows_want.append(ref.sparse_attention(xs[r], n - 1, table[r], chosen, held, scale))
        np.testing.assert_array_equal(refs.cpu().numpy(), counts)
        check_out(out, *(np.stack(x) for x in zip(*rows_want)), d)
        a = b
    # both requests end: every block is free again
    pkv.free_sequences(dev_i32(np.arange(rows), dev), tabs[a], lens[a], refs, dev_status=st)
    assert int(refs.abs().max()) == 0 and int(st.item()) == 0


def test_calls_on_two_streams_at_once(pkv, cuda_device):
    """Selections and attentions with a workspace each, side by side on two streams."""
    dev = cuda_device
    cases = [select_case(2), select_case(4)]
    want, calls = [], []
    for (meta, pool, q), case in zip(cases, (2, 4)):
        index, unit = (torch.as_tensor(x).to(dev) for x in whole_index(pool))
        args = [q.to(dev), *(dev_i32(x, dev) for x in (meta.cu_q_lens, meta.context_lens,
                                                       meta.block_tables))]
        num, sink, recent = SELECTS[case][5:]
        kw = dict(sink_blocks=sink, recent_blocks=recent)
        pd = pool.to(dev)
        sel = pkv.select_blocks(*args, index, unit, num, **kw)
        want.append((sel, pkv.paged_sparse_attention(*args, sel, pd, meta.scale)))
        stream = torch.cuda.Stream(dev)
        a = pkv.BoundSelectBlocks(*args, index, unit, num, stream=stream, **kw)
        b = pkv.BoundSparseAttention(*args, a.selected, pd, meta.scale, torch.empty_like(args[0]),
                                     stream=stream)
        calls.append((a, b))
    torch.cuda.synchronize(dev)
    for _ in range(20):
        for a, b in calls:
            a.run()
            b.run()
    torch.cuda.synchronize(dev)
    for (a, b), (sel, out) in zip(calls, want):
        assert torch.equal(a.selected, sel) and torch.equal(b.out.view(torch.int16), out.view(torch.int16))


def test_python_refusals_on_device_tensors(pkv, cuda_device):
    dev = cuda_device
    meta, pool, q = select_case(0)
    index, unit = pkv.block_index(meta.num_blocks, 2, 64, device=dev)
    cu, ctx, table = (dev_i32(x, dev) for x in (meta.cu_q_lens, meta.context_lens, meta.block_tables))
    q, pool = q.to(dev), pool.to(dev)
    sel = dev_i32(np.zeros((4, 2, 4)), dev)
    with pytest.raises(ValueError):
        pkv.update_block_index(pool, cu, index[:, :1].contiguous(), unit[:, :1].contiguous())
    with pytest.raises(TypeError):
        pkv.update_block_index(pool, cu, index.view(torch.uint8), unit)
    with pytest.raises(ValueError):
        pkv.select_blocks(q, cu[:-1], ctx, table, index, unit, 4)
    with pytest.raises(ValueError):
        pkv.select_blocks(q[:, :7].contiguous(), cu, ctx, table, index, unit, 4)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.select_blocks(q, cu.cpu(), ctx, table, index, unit, 4)
    with pytest.raises(pkv.PkvError):
        pkv.select_blocks(q, cu, ctx, table, index, unit, 4, sink_blocks=3, recent_blocks=2)
    with pytest.raises(ValueError):
        pkv.paged_sparse_attention(q, cu, ctx, table, sel[:3], pool, 0.1)
    with pytest.raises(ValueError, match="apart"):
        both = torch.zeros((5, 8, 64), dtype=torch.bfloat16, device=dev)
        pkv.paged_sparse_attention(both[:4], cu, ctx, table, sel, pool, 0.1, out=both[1:])
    with pytest.raises(pkv.PkvError):
        pkv.paged_sparse_attention(q, cu, ctx, table, sel, pool, float("nan"))


# ------------------------------------------------------------------------- weights

@pytest.mark.parametrize("case", range(len(SELECTS)))
@pytest.mark.parametrize("keys", [2, 5, 300])
def test_weights_keep_sixteen_bits(pkv, cuda_device, case, keys):
    """A weight goes into the product with V as two bf16 parts: the first is its leading bits, at
    least (1 - 2^-8) (1 - 2^-7) of it, so the second is below 2^-6 of it and rounded by 2^-8 of
    itself.  That leaves 2^-14 of A where one bf16 part would leave 2^-8; the rest as above."""
    hq, hkv, d = SELECTS[case][:3]
    rng = np.random.default_rng(900 + case)
    n, ctx = [1] * 40, rng.integers(1, keys + 1, 40).tolist()
    meta = workloads.build_step("weights", 1, n, ctx, hq, hkv, d, rng=rng)
    pool = make_pool(rng, meta.num_blocks, hkv, d)
    q = bf16(rng.standard_normal((meta.total_q, hq, d)))
    sel = np.tile(np.arange(-(-keys // 16)), (meta.total_q, hkv, 1))
    out, st = attend(pkv, cuda_device, meta, q, pool, sel)
    assert st == 0
    held, x = pool.double().numpy(), q.double().numpy()
    rows = [ref.sparse_attention(x[t], c - 1, meta.block_tables[t], sel[t], held, meta.scale)
            for t, c in enumerate(ctx)]
    want, mag, dots = (np.stack(r) for r in zip(*rows))
    e = (d + 4) * 2.0 ** -24 * dots[..., None] + 2.0 ** -22 + 2.0 ** -14
    tol = 2.0 ** -8 * np.abs(want) + mag * (2.0 ** -14 + 2 * e)
    over = np.abs(out.double().cpu().numpy() - want) - tol
    assert (over <= 0).all(), f"worst {over.max():.3e}, {int((over > 0).sum())} of {over.size}"


@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
def test_an_infinite_value_stays_infinite(pkv, cuda_device, value):
    """V of infinity at a visible key with a weight: the output is that infinity, not NaN, also
    where the weight is a power of two (one key, or keys alike)."""
    dev = cuda_device
    meta = workloads.build_step("inf", 1, [1, 1, 1], [1, 16, 40], 8, 2, 64, rng=np.random.default_rng(2))
    pool = make_pool(np.random.default_rng(3), meta.num_blocks, 2, 64)
    pool[:, 0] = 0.5
    for s in range(3):
        pool[meta.block_tables[s, 0], 1, :, 0, 5] = value
    q = bf16(np.random.default_rng(4).standard_normal((3, 8, 64)))
    sel = np.tile(np.arange(3), (3, 2, 1))
    out, _ = attend(pkv, dev, meta, q, pool, sel)
    assert bool((out[:, :, 5] == value).all())
    assert bool(torch.isfinite(torch.cat([out[:, :, :5], out[:, :, 6:]], dim=2)).all())


# ------------------------------------------------------------------------- contexts past the table

@pytest.mark.parametrize("over", [1, 2, 3, 17])
@pytest.mark.parametrize("passes", [False, True])
def test_windows_that_cross_the_tables_last_column(pkv, cuda_device, over, passes):
    """A sequence whose context its table cannot hold has no token that is served, the first
    ones of its window neither, whatever the workspace held; the others are as ever."""
    dev = cuda_device
    hq, hkv, d, num = 8, 2, 64, 4
    n, ctx = [2, 3, 1], [300, 16 * 20 + over, 17]
    rng = np.random.default_rng(over)
    pool = make_pool(rng, 64, hkv, d)
    index, unit = whole_index(pool)
    table = rng.permutation(60).reshape(3, 20)
    q = bf16(rng.standard_normal((6, hq, d)))
    cu = np.concatenate([[0], np.cumsum(n)])
    on = [q.to(dev), *(dev_i32(x, dev) for x in (cu, ctx, table))]
    lib = pkv._load()
    one = lib.pkv_select_workspace_size(1, hkv, 20)
    import ctypes
    want = np.full((6, hkv, num), -1)
    x = q.double().numpy()
    for t, (s, pos) in {0: (0, 298), 1: (0, 299), 5: (2, 16)}.items():
        want[t] = ref.select(x[t], pos, table[s], index, unit, num, 1, 1)
    di, du = torch.as_tensor(index).to(dev), torch.as_tensor(unit).to(dev)
    for fill in (255, 0, 63):
        ws = torch.full((one if passes else 6 * one,), fill, dtype=torch.uint8, device=dev)
        sel, st = torch.full((6, hkv, num), -7, dtype=torch.int32, device=dev), status_of(dev)
        code = lib.pkv_select_blocks(
            on[0].data_ptr(), on[1].data_ptr(), on[2].data_ptr(), on[3].data_ptr(), 20, 3, 6, hq,
            di.data_ptr(), du.data_ptr(), ctypes.byref(pkv.PoolDesc(64, 16, hkv, d)), num, 1, 1,
            sel.data_ptr(), ws.data_ptr(), ws.numel(), st.data_ptr(),
            torch.cuda.current_stream(dev).cuda_stream)
        assert code == 0 and int(st.item()) == 4
        np.testing.assert_array_equal(sel.cpu().numpy(), want)
    st.zero_()
    out = torch.full_like(on[0], 7.0)
    pkv.paged_sparse_attention(*on, dev_i32(np.where(want < 0, 0, want), dev), pool.to(dev), 0.1, out=out,
                               dev_status=st)
    assert int(st.item()) == 4 and bool((out[2:5] == 7.0).all())
    assert not bool((out[[0, 1, 5]] == 7.0).any())


# ------------------------------------------------------------------------- right behind the page calls

@pytest.mark.parametrize("first", ["reserve", "fork", "free"])
def test_selection_and_attention_right_behind_a_page_call(pkv, cuda_device, first):
    """Nothing between the call that writes lengths and tables and those that read them; the
    queries are written in place by the attention before, too."""
    dev, rng = cuda_device, np.random.default_rng(31)
    rows, width, hq, hkv, d, num, scale = 24, 40, 8, 2, 64, 5, 0.125
    blocks = rows * width + 8
    pool = make_pool(rng, blocks, hkv, d)
    index, unit = whole_index(pool)
    on_pool, di, du = pool.to(dev), torch.as_tensor(index).to(dev), torch.as_tensor(unit).to(dev)
    table = rng.permutation(blocks)[:rows * width].reshape(rows, width)
    ctx = rng.integers(17, width * 16 - 40, rows)
    refs = np.zeros(blocks)
    for r in range(rows):
        refs[table[r, :ref.used(ctx[r])]] += 1
    q = bf16(rng.standard_normal((rows, hq, d))).to(dev)
    one = dev_i32(np.arange(rows + 1), dev)
    for step in range(8):
        tabs, lens, counts = dev_i32(table, dev), dev_i32(ctx, dev), dev_i32(refs, dev)
        new, new_lens = dev_i32(np.zeros((rows, width)), dev), dev_i32(np.zeros(rows), dev)
        n = rng.integers(1, 40, rows)
        cu = dev_i32(np.concatenate([[0], np.cumsum(n)]), dev)
        parents, ended = dev_i32(rng.integers(0, rows, rows), dev), dev_i32(rng.integers(0, rows, 9), dev)
        x, st = q.clone(), status_of(dev)
        if first == "reserve":
            call = pkv.BoundReserveBlocks(cu, tabs, lens, counts, num_tokens=int(n.sum()), dev_status=st)
            read = (tabs, lens)
        elif first == "fork":
            call = pkv.BoundForkSequences(parents, tabs, lens, counts, new, new_lens, dev_status=st)
            read = (new, new_lens)
        else:
            call = pkv.BoundFreeSequences(ended, tabs, lens, counts, dev_status=st)
            read = (tabs, lens)
        stt = status_of(dev)
        own = pkv.BoundSparseAttention(x, one, read[1], read[0],
                                       dev_i32(np.zeros((rows, hkv, num)), dev), on_pool, scale, x)
        sel = pkv.BoundSelectBlocks(x, one, read[1], read[0], di, du, num, dev_status=stt)
        att = pkv.BoundSparseAttention(x, one, read[1], read[0], sel.selected, on_pool, scale,
                                       torch.full_like(q, 7.0), dev_status=stt)
        torch.cuda.synchronize(dev)
        call.run()
        own.run()
        sel.run()
        att.run()
        torch.cuda.synchronize(dev)
        assert int(st.item()) == 0 and int(stt.item()) == (4 if first == "free" else 0)
        t, c, xs = read[0].cpu().numpy(), read[1].cpu().numpy(), x.double().cpu().numpy()
        gone = set(ended.cpu().tolist()) if first == "free" else set()
        assert [int(z) for z in c[sorted(gone)]] == [0] * len(gone)
        held = pool.double().numpy()
        for r in range(rows):
            if r in gone:
                assert int(sel.selected[r].max()) == -1 and bool((att.out[r] == 7.0).all())
                continue
            chosen = ref.select(xs[r], c[r] - 1, t[r], index, unit, num, 1, 2)
            np.testing.assert_array_equal(sel.selected[r].cpu().numpy(), chosen)
            want, mag, dots = ref.sparse_attention(xs[r], c[r] - 1, t[r], chosen, held, scale)
            check_out(att.out[r], want, mag, dots, d)


def test_lengths_that_fall_stay_in_bounds(pkv, cuda_device):
    """cu_q_lens that is not non-decreasing: a token behind the end of the sequence it is counted
    into has no place, so no position past the table is looked up."""
    dev = cuda_device
    rng = np.random.default_rng(6)
    pool = make_pool(rng, 64, 1, 64)
    index, unit = (torch.as_tensor(x).to(dev) for x in whole_index(pool))
    table = rng.permutation(64)[:40].reshape(4, 10)
    q = bf16(rng.standard_normal((400, 2, 64))).to(dev)
    on = [q, *(dev_i32(x, dev) for x in ([0, 300, 1, 2, 400], [160, 160, 160, 160], table))]
    st = status_of(dev)
    sel = pkv.select_blocks(*on, index, unit, 4, dev_status=st)
    assert int(st.item()) == 4 and int(sel[2:300].max()) == -1 and int(sel.max()) < 10
    st.zero_()
    out = torch.full_like(q, 7.0)
    pkv.paged_sparse_attention(*on, dev_i32(np.zeros((400, 1, 4)), dev), pool.to(dev), 0.1, out=out,
                               dev_status=st)
    assert int(st.item()) == 4 and bool((out[2:300] == 7.0).all())
