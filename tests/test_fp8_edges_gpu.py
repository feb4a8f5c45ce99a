"""GPU tests of the rotating append and the 8-bit pool at their edges: codes compared
byte for byte with a rounding of its own, scales of blocks past the context, stored
scales that are none, padding, staging arrays that do not fit, large copies.

The append's arithmetic is defined in fp32 with every operation rounded, so its codes
and scales have no tolerance.  Attention is compared with tests/fp8_ref.py within
the bounds that test_fp8_rope_gpu.py derives, or bit for bit with a second call.
"""

import numpy as np
import pytest
import torch

import fp8_ref as ref
import workloads
from fp8_bytes import E4M3, append_bytes, value_of
from test_fp8_rope_gpu import (check_attention, check_rotated, i32, make_pool, rope_inputs,
                               status_of, values_of)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv(cuda_device):
    import paged_kv_attention_append_gb300 as m
    m.build()
    return m


# ------------------------------------------------------------------------- attention

CHAINS = [  # (q_lens, ctx_lens, steps, hkv, group, d): blocks past the context in the plan
    ([1, 1, 1, 1], [15, 16, 40, 300], 20, 2, 4, 128),
    ([1, 1], [31, 700], 40, 1, 8, 64),
    ([4, 6, 2], [64, 300, 30], 7, 2, 4, 128),        # windows of two row groups share blocks
    ([3, 1], [160, 47], 9, 2, 5, 64),
]


@pytest.mark.parametrize("case", range(len(CHAINS)))
@pytest.mark.parametrize("past", [float("nan"), float("inf"), -1.0, 2.0 ** 90])
@pytest.mark.parametrize("sms", [1, 152])
def test_scales_past_the_context_do_not_matter(pkv, cuda_device, case, past, sms):
    """A chain's plan covers blocks that later steps fill.  Until then neither their bytes
    nor their scales count: the first step gives the bits it gives with small scales there."""
    ql, ctx, steps, hkv, group, d = CHAINS[case]
    dev = cuda_device
    rng = np.random.default_rng(900 + case)
    last = [c + n * (steps - 1) for n, c in zip(ql, ctx)]
    meta = workloads.build_step("chain", 90 + case, ql, last, hkv * group, hkv, d, rng=rng)
    codes, scales = make_pool(rng, meta.num_blocks, hkv, d)
    q = ref.bf16(rng.standard_normal((meta.total_q, hkv * group, d)))
    want = ref.attention(ref.f64(q), meta.cu_q_lens, ctx, meta.block_tables,
                         values_of(codes, scales), meta.scale)
    later = [int(b) for s, c in enumerate(ctx) for b in meta.block_tables[s, -(-c // 16):] if b >= 0]
    assert later
    outs = []
    for s in (2.0 ** -30, past):
        raw, sc = codes.clone().view(torch.uint8), scales.clone()
        raw[later] = 0 if s == 2.0 ** -30 else 0x7F
        sc[later] = s
        pool, st = raw.to(dev).view(torch.float8_e4m3fn), status_of(dev)
        plan = pkv.plan_step(meta.cu_q_lens, ctx, hkv * group, pool, num_sms=sms, chain_steps=steps,
                             block_tables=meta.block_tables, fp8=True)
        outs.append(pkv.paged_varlen_attention_fp8(
            q.to(dev), meta.cu_q_lens, i32(ctx, dev), meta.block_tables, pool, sc.to(dev),
            meta.scale, plan=plan, dev_status=st).cpu())
        assert int(st.item()) == 0
    check_attention(outs[0], *want, max(ctx), tensor_cores=False, scales=scales)
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))


@pytest.mark.parametrize("window", [1, 3])
def test_chain_that_fills_new_blocks(pkv, cuda_device, window):
    """Decode steps of one plan in one graph, append and attention, over a pool whose unused
    blocks hold NaN codes and NaN scales: the sequences cross into such blocks on the way,
    and every step is right."""
    dev = cuda_device
    rng = np.random.default_rng(910 + window)
    hq, hkv, d, steps, first = 8, 2, 128, 20, np.array([14, 47, 100, 300])
    n = len(first)
    last = first + window * (steps - 1)
    meta = workloads.build_step("fill", 91, [window] * n, last, hq, hkv, d, rng=rng)
    tables, nb = meta.block_tables, meta.num_blocks
    codes, scales = make_pool(rng, nb, hkv, d)
    raw = codes.view(torch.uint8)
    for s in range(n):
        held = int(first[s]) - window                  # keys cached before the first step
        for j, b in enumerate(tables[s, :-(-int(last[s]) // 16)]):
            keep = min(max(held - 16 * j, 0), 16)
            raw[int(b), :, :, keep:] = 0x7F
            if keep == 0:
                scales[int(b)] = float("nan")
    pool, sc, st = codes.to(dev), scales.to(dev), status_of(dev)
    cs = torch.from_numpy(ref.table(500, d)).to(dev)
    cu, bt = i32(meta.cu_q_lens, dev), i32(tables, dev)
    at = lambda c: np.concatenate([np.arange(x - window, x) for x in c])  # noqa: E731
    seq = np.repeat(np.arange(n), window)
    pos = at(first)
    ctx, pp = i32(first, dev), i32(pos, dev)
    sl = i32([int(tables[s, p // 16]) * 16 + p % 16 for s, p in zip(seq, pos)], dev)
    plan = pkv.plan_step(meta.cu_q_lens, first, hq, pool, chain_steps=steps, block_tables=tables,
                         fp8=True)
    ins = [rope_inputs(rng, n * window, hq, hkv, d, True, dev)[1] for _ in range(steps)]
    got = []

    def run():
        for t, (q, k, v) in enumerate(ins):
            qr = pkv.rope_kv_append_fp8(q, k, v, pp, cs, sl, pool, sc, dev_status=st)
            out = pkv.paged_varlen_attention_fp8(qr, cu, ctx, bt, pool, sc, meta.scale, plan=plan,
                                                 dev_status=st)
            got.append((qr, out, pool.clone(), sc.clone()))
            if t + 1 < steps:
                pkv.decode_advance(ctx, sl, cu, bt, pool, dev_status=st)
                pp.add_(window)

    side = torch.cuda.Stream(dev)
    torch.cuda.synchronize(dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        run()
    g.replay()
    torch.cuda.synchronize(dev)
    assert int(st.item()) == 0
    for t, (qr, out, pool_t, sc_t) in enumerate(got):
        c = first + window * t
        want = ref.attention(ref.f64(qr), meta.cu_q_lens, c, tables,
                             np.nan_to_num(values_of(pool_t.cpu(), sc_t.cpu())), meta.scale)
        check_attention(out.cpu(), *want, int(c.max()), tensor_cores=False,
                        scales=sc_t.cpu().nan_to_num())


@pytest.mark.parametrize("pmq", [-1, 1])
@pytest.mark.parametrize("group,d", [(4, 128), (8, 64)])
def test_key_scales_of_blocks_far_apart(pkv, cuda_device, group, d, pmq):
    """K scales that differ by up to 2^8 from block to block of a head, V scales too."""
    dev = cuda_device
    rng = np.random.default_rng(915)
    ql, ctx, hkv = [1, 3, 70, 1], [700, 90, 300, 17], 2
    meta = workloads.build_step("kscale", 91, ql, ctx, hkv * group, hkv, d, rng=rng, scale=0.02)
    codes, scales = make_pool(rng, meta.num_blocks, hkv, d)
    scales = scales * torch.from_numpy(np.exp2(rng.integers(-4, 5, scales.shape)).astype(np.float32))
    q = ref.bf16(rng.standard_normal((meta.total_q, hkv * group, d)))
    want = ref.attention(ref.f64(q), meta.cu_q_lens, ctx, meta.block_tables, values_of(codes, scales),
                         float(np.float32(meta.scale)))
    pool, st = codes.to(dev), status_of(dev)
    plan = pkv.plan_step(meta.cu_q_lens, ctx, hkv * group, pool, block_tables=meta.block_tables,
                         prefill_min_q=pmq, fp8=True)
    out = pkv.paged_varlen_attention_fp8(q.to(dev), meta.cu_q_lens, meta.context_lens,
                                         meta.block_tables, pool, scales.to(dev), meta.scale,
                                         plan=plan, dev_status=st)
    assert int(st.item()) == 0
    check_attention(out.cpu(), *want, max(ctx), tensor_cores=pmq == 1, scales=scales)


STAGED = [  # (q_lens, ctx_lens, hkv, group, d, num_sms, shared blocks, sequence with copies)
    ([1, 70], [200, 90], 2, 4, 128, None, 0, 1),             # written directly
    ([1, 128, 200], [30, 1000, 700], 2, 2, 64, None, 0, 2),  # whole sub-tiles staged out
    ([64, 1], [4000, 50], 1, 2, 64, 152, 0, 0),              # keys cut into many items
    ([64], [4000], 1, 2, 128, 152, 0, 0),
    ([1] * 20, [17 * 16 + 1 + i for i in range(20)], 2, 4, 128, 1, 17, 0),   # gathered prefix
    ([2] * 40, [40 * 16 + 2 + i for i in range(40)], 2, 4, 64, 9, 40, 0),
]


@pytest.mark.parametrize("case", range(len(STAGED)))
@pytest.mark.parametrize("kind", ["none", "short", "past", "negative"])
def test_rows_without_their_copies_are_not_written(pkv, cuda_device, case, kind):
    """A staging array that does not give a tensor-core sequence all its copies: reported,
    and every row that would need them stays as it was, whether it is written directly,
    merged from parts or gathered with other sequences' rows.  The others are right."""
    ql, ctx, hkv, group, d, sms, shared, bad = STAGED[case]
    dev = cuda_device
    rng = np.random.default_rng(920 + case)
    meta = workloads.build_step("stage", 92 + case, ql, ctx, hkv * group, hkv, d, rng=rng,
                                shared_prefix_blocks=shared)
    codes, scales = make_pool(rng, meta.num_blocks, hkv, d)
    q = ref.bf16(rng.standard_normal((meta.total_q, hkv * group, d)))
    plan = pkv.plan_step(meta.cu_q_lens, ctx, hkv * group, codes.to(dev), num_sms=sms,
                         block_tables=meta.block_tables, fp8=True)
    begin, n = plan.stage.cpu().numpy(), plan.fp8.staged_blocks
    assert n > 0 and begin[bad + 1] > begin[bad]
    if kind == "none":
        begin[bad + 1:] = begin[bad]
    elif kind == "short":
        begin[bad + 1:] -= 8
    elif kind == "past":
        begin[bad + 1:] += n
        begin[bad] += n
    else:
        begin[bad] = -8
    plan.stage = i32(begin, dev)
    # what an earlier call may have left there: finite partial results
    plan.workspace.view(torch.float32).fill_(1.0)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=dev)
    st = status_of(dev)
    pkv.paged_varlen_attention_fp8(q.to(dev), meta.cu_q_lens, meta.context_lens, meta.block_tables,
                                   codes.to(dev), scales.to(dev), meta.scale, plan=plan, out=out,
                                   dev_status=st)
    assert int(st.item()) == 4
    want = ref.attention(ref.f64(q), meta.cu_q_lens, meta.context_lens, meta.block_tables,
                         values_of(codes, scales), meta.scale)
    got = out.cpu()
    untouched = (got == 7.0).all(dim=2).numpy()                 # [row, head]
    if shared:
        must = np.ones(meta.total_q, dtype=bool)
    else:
        must = np.zeros(meta.total_q, dtype=bool)
        a, b = int(meta.cu_q_lens[bad]), int(meta.cu_q_lens[bad + 1])
        must[b - 1 if kind == "short" else a:b] = True          # the last token sees every key
    assert untouched[must].all()
    # every row of a head holds either its result or what it held before
    done = ~untouched
    check_attention(got[done], *(x[done] for x in want), max(ctx), tensor_cores=True, scales=scales)
    for s in range(0 if not shared else len(ql), len(ql)):
        if ql[s] < 64 or (s < bad and kind in ("none", "short")):   # not touched by the change
            assert done[int(meta.cu_q_lens[s]):int(meta.cu_q_lens[s + 1])].all()


def test_copies_past_their_limit(pkv, cuda_device):
    """72 chunks of 64 tokens at 32 000 keys each, whose copies would take 9.4 GB: some of
    them run on the split-KV kernel, and every row is right (64-bit reference on the GPU;
    the sequences read the same blocks)."""
    dev = cuda_device
    rng = np.random.default_rng(930)
    n, qn, ctx, hkv, d, hq = 72, 64, 32_000, 8, 128, 8
    nb = ctx // 16
    codes, scales = make_pool(rng, nb, hkv, d)
    pool, sc, st = codes.to(dev), scales.to(dev), status_of(dev)
    table = np.tile(rng.permutation(nb).astype(np.int32), (n, 1))
    cu = np.arange(n + 1, dtype=np.int32) * qn
    ctxs = np.full(n, ctx, dtype=np.int32)
    q = ref.bf16(rng.standard_normal((n * qn, hq, d)))
    plan = pkv.plan_step(cu, ctxs, hq, pool, block_tables=table, fp8=True)
    kept = np.diff(plan.stage.cpu().numpy()) > 0
    assert kept.any() and not kept.all() and plan.workspace.numel() < 9 << 30
    out = pkv.paged_varlen_attention_fp8(q.to(dev), cu, ctxs, table, pool, sc, d ** -0.5, plan=plan,
                                         dev_status=st)
    assert int(st.item()) == 0
    got = out.cpu()
    vals = torch.from_numpy(values_of(codes, scales))[torch.from_numpy(table[0]).long()].to(dev)
    i = torch.arange(n * qn, device=dev) % qn
    hidden = torch.arange(ctx, device=dev)[None] > (ctx - qn + i)[:, None]
    for h in range(hq):
        k, v = (vals[:, j, h].reshape(-1, d) for j in (0, 1))
        qh = q[:, h].to(dev).double()
        x = ((qh @ k.T) * d ** -0.5).masked_fill_(hidden, float("-inf"))
        w = torch.softmax(x, dim=1)
        want, wabs = w @ v, w @ v.abs()
        mag = (qh.abs() @ k.abs().T).amax(dim=1, keepdim=True) * d ** -0.5
        check_attention(got[:, h], *(t.cpu().numpy() for t in (want, wabs, mag)), ctx,
                        tensor_cores=True, scales=scales)


@pytest.mark.parametrize("ql,ctx,hkv,group,d,shared", [
    ([1] * 12, list(range(5, 2405, 200)), 8, 4, 128, 0),
    ([4, 8, 3, 1] * 3, [900, 33, 512, 2000] * 3, 2, 8, 128, 0),
    ([2] * 64, [1024 + 9 * i + 2 for i in range(64)], 8, 4, 128, 64),
    ([300, 1, 130], [900, 3000, 131], 2, 5, 64, 0),
])
def test_same_call_gives_the_same_bits(pkv, cuda_device, ql, ctx, hkv, group, d, shared):
    dev = cuda_device
    rng = np.random.default_rng(940)
    meta = workloads.build_step("twice", 94, ql, ctx, hkv * group, hkv, d, rng=rng,
                                shared_prefix_blocks=shared)
    codes, scales = make_pool(rng, meta.num_blocks, hkv, d, "any")
    pool, sc = codes.to(dev), scales.to(dev)
    q = ref.bf16(rng.standard_normal((meta.total_q, hkv * group, d))).to(dev)
    plan = pkv.plan_step(meta.cu_q_lens, ctx, hkv * group, pool, block_tables=meta.block_tables,
                         fp8=True)
    outs = []
    for k in range(6):
        if plan.workspace is not None:
            plan.workspace.fill_(0x11 * k)
        out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=dev)
        outs.append(pkv.paged_varlen_attention_fp8(q, meta.cu_q_lens, meta.context_lens,
                                                   meta.block_tables, pool, sc, meta.scale,
                                                   plan=plan, out=out))
    torch.cuda.synchronize(dev)
    assert all(torch.equal(o.view(torch.int16), outs[0].view(torch.int16)) for o in outs[1:])


@pytest.mark.parametrize("thread", [False, True])
def test_bound_planner_of_an_8_bit_pool_serves_the_attention(pkv, cuda_device, thread):
    """A serving loop that uploads what BoundPlan(fp8=True) writes, plan and staging array,
    into its own buffers: steps with and without tensor-core work, each against the
    reference."""
    dev = cuda_device
    rng = np.random.default_rng(950)
    steps = [([1, 90, 2], [333, 200, 50]), ([1, 1, 1], [334, 201, 51]), ([3, 64, 130], [337, 265, 181])]
    cu_h, ctx_h = np.zeros(4, np.int32), np.zeros(3, np.int32)
    meta = workloads.build_step("bound", 95, *steps[-1], 8, 2, 128, rng=rng)
    bt_h = meta.block_tables.astype(np.int32).copy()
    codes, scales = make_pool(rng, meta.num_blocks, 2, 128)
    pool, sc, st = codes.to(dev), scales.to(dev), status_of(dev)
    plan_h, stage_h = np.zeros(1 << 16, np.int32), np.zeros(4, np.int32)
    bp = pkv.BoundPlan(cu_h, ctx_h, 8, pool, plan_h, block_tables=bt_h, fp8=True, stage_out=stage_h,
                       spin_us=100 if thread else None)
    plan_d, stage_d = torch.zeros(1 << 18, dtype=torch.uint8, device=dev), i32(stage_h, dev)
    bt = i32(bt_h, dev)
    staged = []
    for ql, ctx in steps:
        cu_h[1:], ctx_h[:] = np.cumsum(ql), ctx
        if thread:
            bp.post()
            info, nb = bp.wait()
        else:
            info, nb = bp.run()
        plan_d[:nb] = torch.from_numpy(plan_h.view(np.uint8)[:nb]).to(dev)
        stage_d.copy_(torch.from_numpy(stage_h))
        plan = pkv.StepPlan(info, plan_h.view(np.uint8)[:nb].view(np.int32), dev, fp8=True)
        plan.dev, plan.stage, plan.fp8 = plan_d, stage_d, bp.fp8
        assert plan.workspace is None or plan.workspace.numel() >= bp.fp8.workspace_bytes
        staged.append(bp.fp8.staged_blocks)
        q = ref.bf16(rng.standard_normal((int(cu_h[-1]), 8, 128)))
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
        pkv.BoundAttentionFp8(q.to(dev), i32(cu_h, dev), i32(ctx_h, dev), bt, pool, sc, meta.scale,
                              plan, out, dev_status=st).run()
        torch.cuda.synchronize(dev)
        assert int(st.item()) == 0
        want = ref.attention(ref.f64(q), cu_h, ctx_h, bt_h, values_of(codes, scales), meta.scale)
        check_attention(out.cpu(), *want, max(ctx), tensor_cores=staged[-1] > 0, scales=scales)
    bp.close()
    assert staged[0] > 0 and staged[1] == 0 and staged[2] > 0


# ------------------------------------------------------------------------ 8-bit append

def assert_same_codes(got, want, scales, want_scales):
    assert np.array_equal(scales.cpu().numpy(), want_scales)
    g = got.cpu().view(torch.uint8).numpy()
    nan = (want & 127) == 127
    assert np.array_equal(nan, (g & 127) == 127)
    assert np.array_equal(g[~nan], want[~nan])


def grid_rows(d, scale):
    """Rows whose values over `scale` are e4m3 midpoints (ties of either parity), codes'
    own values, values just past half the smallest step and just below powers of two."""
    mid = (E4M3[1:] + E4M3[:-1]) / 2
    x = np.concatenate([[448.0], mid, E4M3, 2.0 ** -10 * np.array([1, 1.0078125, 0.9921875]),
                        np.exp2(np.arange(-8, 9.0)) * 0.99609375, [446.0]])
    x = np.concatenate([x, -x]) * scale
    x = np.concatenate([x, np.zeros(-len(x) % d)]).reshape(-1, d)
    return x


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -64, 2.0 ** 40, 2.0 ** -7])
def test_codes_of_ties_and_borders(pkv, cuda_device, d, scale):
    """New rows on the borders between two codes, into new blocks; then a larger row in
    each block, so that every code is re-expressed, ties in e4m3's subnormals among them."""
    dev = cuda_device
    x = grid_rows(d, scale)
    x = np.concatenate([x] + [x * 2.0 ** -k for k in (1, 3, 9)])
    x[:, 0] = 448.0 * scale                        # each row alone would need this scale
    n = len(x)
    rows = ref.bf16(x)
    assert np.array_equal(ref.f64(rows), x)
    rows = rows[:, None].contiguous()
    nb = n // 8 + 1
    slots = np.array([t // 8 * 16 + t % 8 for t in range(n)])
    for grow in (1.0, 2.0, 8.0, 512.0, 2.0 ** 20):
        pool, sc = pkv.fp8_pool(nb, 1, d, device=dev)
        want, want_sc = np.zeros((nb, 2, 1, 16, d), np.uint8), np.ones((nb, 1, 2), np.float32)
        r = np.stack([ref.f64(rows), -ref.f64(rows)], axis=1).astype(np.float32)
        pkv.paged_kv_append_fp8(rows.to(dev), -rows.to(dev), i32(slots, dev), pool, sc)
        want, want_sc = append_bytes(want, want_sc, r, slots.tolist())
        assert_same_codes(pool, want, sc, want_sc)
        big = ref.bf16(np.full((nb, 1, d), 448.0 * scale * grow))
        pkv.paged_kv_append_fp8(big.to(dev), big.to(dev), i32(np.arange(nb) * 16 + 9, dev), pool, sc)
        r = np.repeat(ref.f64(big)[:, None], 2, axis=1).astype(np.float32)
        want, want_sc = append_bytes(want, want_sc, r, (np.arange(nb) * 16 + 9).tolist())
        assert_same_codes(pool, want, sc, want_sc)


@pytest.mark.parametrize("kind", ["pow2", "any"])
@pytest.mark.parametrize("size", [1e-4, 1.0, 3e3])
@pytest.mark.parametrize("rot,inter,d", [(0, False, 128), (128, False, 128), (32, True, 64),
                                         (48, False, 64)])
def test_codes_of_random_rows(pkv, cuda_device, kind, size, rot, inter, d):
    """Runs of tokens that start anywhere in a block, new rows of sizes spread over 2^16
    a row: codes, scales and untouched rows to the byte."""
    dev = cuda_device
    rng = np.random.default_rng(960 + rot)
    slots, b = [], 0
    while len(slots) < 300:
        off = int(rng.integers(0, 16))
        slots += list(range(b * 16 + off, b * 16 + off + int(rng.integers(1, 40))))
        b = slots[-1] // 16 + 1
    nb, n, hkv = b, len(slots), 3
    perm = rng.permutation(nb)
    slots = [int(perm[s // 16]) * 16 + s % 16 for s in slots]
    x = rng.standard_normal((n, 2 + 2 * hkv, d)) * np.exp2(rng.uniform(-8, 8, (n, 2 + 2 * hkv, 1)))
    xb = ref.bf16(x * size)
    q, k, v = xb[:, :2], xb[:, 2:2 + hkv], xb[:, 2 + hkv:]
    before, sc = make_pool(rng, nb, hkv, d, kind)
    pool, scd, st = before.to(dev), sc.to(dev), status_of(dev)
    kr = ref.f64(k).astype(np.float32)
    if rot:
        cs = ref.table(3000, rot)
        pos = rng.integers(0, 3000, size=n)
        xd = xb.to(dev)
        out = pkv.rope_kv_append_fp8(xd[:, :2], xd[:, 2:2 + hkv], xd[:, 2 + hkv:], i32(pos, dev),
                                     torch.from_numpy(cs).to(dev), i32(slots, dev), pool, scd,
                                     interleaved=inter, dev_status=st)
        check_rotated(out, q, pos, cs, inter)
        kr = ref.rotate(ref.f64(k), pos, cs, inter, np.float32)[0]
    else:
        pkv.paged_kv_append_fp8(k.contiguous().to(dev), v.contiguous().to(dev), i32(slots, dev), pool,
                                scd, dev_status=st)
    assert int(st.item()) == 0
    rows = np.stack([kr, ref.f64(v).astype(np.float32)], axis=1)
    want = append_bytes(before.view(torch.uint8).numpy(), sc.numpy(), rows, slots)
    assert_same_codes(pool, want[0], scd, want[1])


def test_token_by_token_to_the_byte(pkv, cuda_device):
    """A block filled one token at a time, its scales growing on the way: the bytes that
    the defined sequence of re-expressions gives."""
    dev = cuda_device
    rng = np.random.default_rng(970)
    k = ref.bf16(rng.standard_normal((16, 2, 128)) * np.exp2(np.arange(16) / 2)[:, None, None])
    pool, sc = pkv.fp8_pool(2, 2, 128, device=dev)
    want, want_sc = np.zeros((2, 2, 2, 16, 128), np.uint8), np.ones((2, 2, 2), np.float32)
    rows = np.repeat(ref.f64(k)[:, None], 2, axis=1).astype(np.float32)
    for t in range(16):
        kt = k[t:t + 1].to(dev)
        pkv.paged_kv_append_fp8(kt, kt, i32([t], dev), pool, sc)
        want, want_sc = append_bytes(want, want_sc, rows[t:t + 1], [t])
        assert_same_codes(pool, want, sc, want_sc)


@pytest.mark.parametrize("stored", [0.0, -0.0, -2.0, float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("size", [0.0, 1.0])
def test_stored_scale_that_is_none(pkv, cuda_device, stored, size):
    """Kept rows under a scale that is not positive and finite stand for nothing: they
    become zeros of the new scale (NaN codes stay NaN), which is a proper one."""
    dev = cuda_device
    rng = np.random.default_rng(980)
    before, sc = make_pool(rng, 3, 2, 64)
    before.view(torch.uint8)[0, 0, 0, 1, 5] = 0x7F
    sc[0] = stored
    sc[1, 1, 0] = stored
    pool, scd, st = before.to(dev), sc.to(dev), status_of(dev)
    k = ref.bf16(size * rng.standard_normal((3, 2, 64)))
    slots = [4, 16 + 7, 32]
    pkv.paged_kv_append_fp8(k.to(dev), k.to(dev), i32(slots, dev), pool, scd, dev_status=st)
    assert int(st.item()) == 0
    rows = np.repeat(ref.f64(k)[:, None], 2, axis=1).astype(np.float32)
    want = append_bytes(before.view(torch.uint8).numpy(), sc.numpy(), rows, slots)
    assert np.array_equal(value_of(want[0][0, :, :, :4])[~np.isnan(value_of(want[0][0, :, :, :4]))] == 0,
                          np.ones(2 * 2 * 4 * 64 - 1, bool))
    assert_same_codes(pool, want[0], scd, want[1])


# ---------------------------------------------------------------------------- padding

@pytest.mark.parametrize("fp8", [False, True])
def test_padding_by_position_alone(pkv, cuda_device, fp8):
    """A token at a negative position is padding whatever its slot holds: no status, and
    nothing written.  At a position past the table the position is what is reported."""
    dev = cuda_device
    rng = np.random.default_rng(990)
    n, hq, hkv, d, nb = 40, 4, 2, 64, 4
    (q, k, v), (qd, kd, vd) = rope_inputs(rng, n, hq, hkv, d, True, dev)
    cs = ref.table(100, d)
    pos = rng.integers(0, 100, size=n)
    slots = np.arange(n)
    pad = np.array([1, 17, 30, 39])
    pos[pad] = [-1, -7, -1, -2 ** 31]
    slots[pad] = [nb * 16, 2 ** 31 - 1, 5, -1]
    before, sc = make_pool(rng, nb, hkv, d)
    if not fp8:
        before = ref.bf16(rng.standard_normal((nb, 2, hkv, 16, d)))
    for late in (False, True):
        p, s = pos.copy(), slots.copy()
        if late:
            p[20], s[20] = 100, nb * 16 + 3       # both wrong: the position is reported
        pool, scd, st = before.to(dev), sc.to(dev), status_of(dev)
        q_out = torch.full((n, hq, d), 3.0, dtype=torch.bfloat16, device=dev)
        args = (qd, kd, vd, i32(p, dev), torch.from_numpy(cs).to(dev), i32(s, dev), pool)
        if fp8:
            pkv.rope_kv_append_fp8(*args, scd, q_out=q_out, dev_status=st)
        else:
            pkv.rope_kv_append(*args, q_out=q_out, dev_status=st)
        assert int(st.item()) == (5 if late else 0)
        out = [20] if late else []
        skipped = np.array(sorted(pad.tolist() + out))
        rows = np.array([t for t in range(n) if t not in skipped])
        assert bool((q_out[skipped] == 3.0).all())
        check_rotated(q_out, q, np.clip(p, 0, 99), cs, False, rows)
        kr = ref.rotate(ref.f64(k), np.clip(p, 0, 99), cs, False, np.float32)[0]
        if fp8:
            r = np.stack([kr, ref.f64(v).astype(np.float32)], axis=1)
            live = [int(x) if t in rows else -1 for t, x in enumerate(s)]
            want = append_bytes(before.view(torch.uint8).numpy(), sc.numpy(), r, live)
            assert_same_codes(pool, want[0], scd, want[1])
        else:
            want = before.clone()
            for t in rows:
                want[s[t] // 16, 0, :, s[t] % 16] = ref.bf16(kr[t])
                want[s[t] // 16, 1, :, s[t] % 16] = v[t]
            assert torch.equal(pool.cpu().view(torch.int16), want.view(torch.int16))
