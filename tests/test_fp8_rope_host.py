"""CPU tests of the rotating append's and the 8-bit attention's entry points: every
refusal happens before anything is enqueued, and the staging array matches the plan."""

import ctypes

import numpy as np
import pytest
import torch

import fp8_ref as ref
import oracle
import paged_kv_attention_append_gb300 as pkv
import workloads

A = 0x1000                      # an aligned address that is never dereferenced
OK, NULL, SHAPE, RANGE, UNSUPPORTED, WORKSPACE, ALIGN = 0, 1, 2, 3, 4, 5, 8


@pytest.fixture(scope="module")
def lib():
    pkv.build()
    return pkv._load()


def rope_call(lib, fp8=False, **kw):
    a = dict(q=A, qs=8 * 128, k=A, ks=2 * 128, v=A, vs=2 * 128, cos_sin=A, positions=A, max_pos=10,
             rot=128, inter=0, slots=A, n=4, hq=8, q_out=A, qos=8 * 128, pool=A, scales=A, nb=4,
             bs=16, hkv=2, d=128, rope=True)
    a.update(kw)
    rope = pkv.Rope(a["cos_sin"], a["positions"], a["max_pos"], a["rot"], a["inter"])
    desc = pkv.PoolDesc(a["nb"], a["bs"], a["hkv"], a["d"])
    args = [a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"],
            ctypes.byref(rope) if a["rope"] else None, a["slots"], a["n"], a["hq"], a["q_out"],
            a["qos"], a["pool"]]
    if fp8:
        return lib.pkv_rope_kv_append_fp8(*args, a["scales"], ctypes.byref(desc), None, None)
    return lib.pkv_rope_kv_append(*args, ctypes.byref(desc), None, None)


REFUSED = [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(pool=None), NULL),
    (dict(q=None), NULL), (dict(q_out=None), NULL), (dict(cos_sin=None), NULL),
    (dict(positions=None), NULL), (dict(n=-1), SHAPE), (dict(hq=-1), SHAPE),
    (dict(rot=0), UNSUPPORTED), (dict(rot=8), UNSUPPORTED), (dict(rot=24), UNSUPPORTED),
    (dict(rot=144), UNSUPPORTED), (dict(rot=-16), UNSUPPORTED), (dict(max_pos=-1), SHAPE),
    (dict(inter=2), RANGE), (dict(ks=128), SHAPE), (dict(vs=2 * 128 + 4), SHAPE),
    (dict(qs=7 * 128), SHAPE), (dict(qos=8 * 128 + 1), SHAPE), (dict(k=A + 8), ALIGN),
    (dict(q=A + 2), ALIGN), (dict(q_out=A + 4), ALIGN), (dict(pool=A + 8), ALIGN),
    (dict(cos_sin=A + 4), ALIGN), (dict(positions=A + 2), ALIGN), (dict(slots=A + 1), ALIGN),
    (dict(d=96), UNSUPPORTED), (dict(bs=32), UNSUPPORTED), (dict(hkv=0), SHAPE),
    (dict(nb=1 << 26), UNSUPPORTED), (dict(n=0), OK), (dict(n=0, k=None), OK),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(REFUSED)))
def test_rope_refusals(lib, fp8, case):
    kw, want = REFUSED[case]
    before = pkv.kernel_launch_count()
    assert rope_call(lib, fp8, **kw) == want
    assert pkv.kernel_launch_count() == before


def test_rope_only_refusals(lib):
    assert rope_call(lib, rope=False) == NULL
    assert rope_call(lib, True, rope=False) == NULL             # q without a rotation
    assert rope_call(lib, True, scales=None) == NULL
    assert rope_call(lib, True, scales=A + 4) == ALIGN
    assert rope_call(lib, True, rope=False, hq=0, n=0) == OK


def plan_of(meta, **kw):
    info, host = pkv.plan_step(meta.cu_q_lens, meta.context_lens, meta.num_q_heads,
                               pkv.PoolDesc(meta.num_blocks, 16, meta.num_kv_heads, meta.head_dim),
                               num_sms=kw.pop("num_sms", 152), upload=False, **kw)
    return info, host


@pytest.mark.parametrize("seed", range(8))
@pytest.mark.parametrize("shared", [0, 20])
def test_stage_covers_the_tensor_core_sequences(lib, seed, shared):
    rng = np.random.default_rng(seed)
    meta = workloads.random_step(rng, max_ctx=700, num_seqs=40 if shared else None,
                                 shared_prefix_blocks=shared)
    info, host = plan_of(meta, block_tables=meta.block_tables)
    begin, fp8 = pkv.stage_fp8(info, host)
    nbytes = int(fp8.workspace_bytes)
    counts = np.diff(begin)
    assert begin[0] == 0 and (counts >= 0).all()
    for s in range(meta.num_seqs):
        nb = -(-int(meta.context_lens[s]) // 16)
        if meta.q_lens[s] >= 64:
            assert nb <= counts[s] <= nb + 7
        else:                           # only as the table of a gathered prefix
            assert counts[s] <= max(shared, 0)
    if info.num_prefill_tiles == 0:
        assert begin[-1] == 0 and nbytes == info.workspace_bytes
    else:
        slab = 2 * meta.num_kv_heads * 16 * meta.head_dim * 2
        assert nbytes >= info.workspace_bytes + int(begin[-1]) * slab
    group = meta.num_q_heads // meta.num_kv_heads
    rows = [min(int(q), 16 // group) * group for q in meta.q_lens if 0 < q < 64]
    assert fp8.max_rows <= 16 and fp8.staged_blocks == begin[-1]
    if not shared and info.num_prefill_tiles == 0:
        assert fp8.max_rows == max(rows, default=0)


@pytest.mark.parametrize("seed", range(6))
def test_fp8_plan_covers_the_same_keys(lib, seed):
    """pkv_plan_step_fp8 divides the work otherwise; what it covers is the same.  Without
    a shared prefix every (row group, KV head)'s blocks are read as often as in the bf16
    plan; a short shared prefix is streamed by each row group instead of shared."""
    rng = np.random.default_rng(100 + seed)
    meta = workloads.random_step(rng, max_ctx=900, max_q=3 if seed % 2 else None,
                                 shared_prefix_blocks=[0, 12][seed // 3])
    infos = []
    for fp8 in (False, True):
        info, host = plan_of(meta, block_tables=meta.block_tables, fp8=fp8, num_sms=4)
        assert pkv.stage_fp8(info, host)[1].max_rows <= 16
        infos.append(info)
    a, b = infos
    assert (a.kv_tokens, a.max_blocks_needed) == (b.kv_tokens, b.max_blocks_needed)
    assert b.decode_blocks == a.decode_blocks if seed < 3 else b.decode_blocks >= a.decode_blocks
    assert b.num_decode_warps <= 4 * 16


def test_upload_again_keeps_the_addresses():
    """A plan uploaded again, here for a step with fewer sequences, stays where it was: a
    captured graph holds the addresses of the plan, the staging array and the workspace."""
    metas = [workloads.build_step("fp8", 9, ql, ctx, 8, 2, 128) for ql, ctx in
             (([200, 1, 90], [400, 33, 700]), ([130, 1], [300, 40]))]
    (info0, host0), (info1, host1) = (plan_of(m, fp8=True) for m in metas)
    plan = pkv.StepPlan(info0, host0, torch.device("cpu"), fp8=True)
    begin0, _ = pkv.stage_fp8(info0, host0)
    assert np.array_equal(plan.stage.numpy(), begin0)
    kept = [t.data_ptr() for t in (plan.dev, plan.stage, plan.workspace)]
    plan.info, plan.host = info1, host1
    plan.upload()
    begin1, fp8 = pkv.stage_fp8(info1, host1)
    assert fp8.staged_blocks > 0
    assert np.array_equal(plan.stage.numpy()[:begin1.size], begin1)
    assert [t.data_ptr() for t in (plan.dev, plan.stage, plan.workspace)] == kept
    assert plan.workspace.numel() >= plan.fp8.workspace_bytes


@pytest.mark.parametrize("decodes", [1, 3, 16, 64])
@pytest.mark.parametrize("chunk,ctx", [(2048, 4608), (4096, 16384), (8192, 8192)])
def test_full_prefill_leaves_sms_to_the_split_kv_work(lib, decodes, chunk, ctx):
    """8-bit pool: with a prefill for every SM, an even number of SMs is left for the
    decodes, whose warps all fit there; more with more decodes.  A plan for a bf16 pool
    gives the prefill every SM."""
    def plan(n, **kw):
        ql, cl = [1] * n + [chunk], [4096 + 16 * i for i in range(n)] + [ctx]
        cu = np.concatenate([[0], np.cumsum(ql)])
        return pkv.plan_step(cu, cl, 32, pkv.PoolDesc(sum(cl) // 16 + len(cl), 16, 8, 128),
                             num_sms=152, upload=False, **kw)[0]
    info = plan(decodes, fp8=True)
    left = 152 - info.num_prefill_ctas
    assert left > 0 and left % 2 == 0
    assert 0 < info.num_decode_warps <= 16 * left
    assert 152 - plan(2 * decodes, fp8=True).num_prefill_ctas >= left
    assert plan(decodes).num_prefill_ctas == 152
    assert plan(0, fp8=True).num_prefill_ctas == 152


@pytest.mark.parametrize("decodes,ctx,beside", [(16, 2000, True), (8, 100, True), (64, 4000, False)])
def test_short_stream_stays_on_the_sms_a_small_prefill_leaves(lib, decodes, ctx, beside):
    """8-bit pool: the split-KV warps beside a 64-token prompt all find a free SM, unless
    the stream is long."""
    cu = np.concatenate([[0], np.cumsum([1] * decodes + [64])])
    cl = [ctx] * decodes + [64]
    info = pkv.plan_step(cu, cl, 32, pkv.PoolDesc(sum(cl) // 16 + len(cl), 16, 8, 128),
                         num_sms=152, upload=False, fp8=True)[0]
    assert info.num_prefill_ctas == 32
    assert (info.num_decode_warps <= 16 * (152 - 32)) == beside


def test_stage_refusals(lib):
    meta = workloads.build_step("s", 1, [70, 1], [70, 40], 4, 2, 64)
    info, host = plan_of(meta)
    begin = np.zeros(3, dtype=np.int32)
    out = pkv.Fp8Info()
    ptr = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    f = lib.pkv_plan_stage_fp8
    assert f(None, ctypes.byref(info), ptr(begin), ctypes.byref(out)) == NULL
    assert f(ptr(host), None, ptr(begin), ctypes.byref(out)) == NULL
    assert f(ptr(host), ctypes.byref(info), None, ctypes.byref(out)) == NULL
    assert f(ptr(host), ctypes.byref(info), ptr(begin), None) == NULL
    other = host.copy()
    other[0] ^= 1
    assert f(ptr(other), ctypes.byref(info), ptr(begin), ctypes.byref(out)) == SHAPE
    bad = pkv.PlanInfo.from_buffer_copy(info)
    bad.num_prefill_tiles += 1
    assert f(ptr(host), ctypes.byref(bad), ptr(begin), ctypes.byref(out)) == SHAPE


def attention_call(lib, info, **kw):
    a = dict(q=A, cu=A, ctx=A, bt=A, mb=64, pool=A, scales=A, scale=0.1, plan=A, stage=A, blocks=12, rows=16,
             fp8=True, out=A, ws=A, wsb=1 << 30)
    a.update(kw)
    desc = pkv.PoolDesc(100, 16, info.num_kv_heads, info.head_dim)
    fp8 = pkv.Fp8Info(a["blocks"], a["rows"], a["wsb"])
    return lib.pkv_paged_varlen_attention_fp8(
        a["q"], a["cu"], a["ctx"], a["bt"], a["mb"], a["pool"], a["scales"], ctypes.byref(desc),
        a["scale"], ctypes.byref(info), a["plan"], ctypes.byref(fp8) if a["fp8"] else None, a["stage"],
        a["out"], a["ws"], a["wsb"], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(scales=None), NULL), (dict(fp8=False), NULL), (dict(scales=A + 8), ALIGN),
    (dict(q=None), NULL), (dict(pool=None), NULL), (dict(stage=None), NULL), (dict(ws=None), NULL), (dict(blocks=0), SHAPE),
    (dict(blocks=-3), SHAPE), (dict(blocks=1 << 30), SHAPE), (dict(wsb=4096), WORKSPACE),
    (dict(mb=2), RANGE), (dict(scale=float("inf")), RANGE), (dict(scale=float("nan")), RANGE),
    (dict(ws=A + 16), ALIGN), (dict(out=A + 2), ALIGN)])
def test_attention_refusals(lib, kw, want):
    meta = workloads.build_step("s", 1, [70, 1], [70, 40], 4, 2, 64)
    info, _ = plan_of(meta)
    assert info.num_prefill_tiles > 0
    before = pkv.kernel_launch_count()
    assert attention_call(lib, info, **kw) == want
    assert pkv.kernel_launch_count() == before


def test_empty_step_is_ok(lib):
    meta = workloads.build_step("s", 1, [0], [9], 4, 2, 64)
    info, host = plan_of(meta)
    begin, fp8 = pkv.stage_fp8(info, host)
    nbytes = int(fp8.workspace_bytes)
    assert begin.tolist() == [0, 0] and nbytes == info.workspace_bytes
    assert attention_call(lib, info, q=None, pool=None, stage=None, blocks=0) == OK


@pytest.mark.parametrize("thread", [False, True])
def test_bound_planner_for_an_8_bit_pool(lib, thread):
    """BoundPlan(fp8=True) writes what plan_step(fp8=True) and stage_fp8 write, run after
    run, on the calling thread or on the planning thread."""
    meta = workloads.make_config("agent_mixed")
    desc = pkv.PoolDesc(meta.num_blocks, 16, meta.num_kv_heads, meta.head_dim)
    cu, ctx = meta.cu_q_lens.astype(np.int32).copy(), meta.context_lens.astype(np.int32).copy()
    bt = meta.block_tables.astype(np.int32).copy()
    out, stage = np.zeros(1 << 18, np.int32), np.full(len(cu), -7, np.int32)
    bp = pkv.BoundPlan(cu, ctx, meta.num_q_heads, desc, out, num_sms=152, block_tables=bt, fp8=True,
                       stage_out=stage, spin_us=50 if thread else None)
    for _ in range(2):
        if thread:
            bp.post()
            info, nb = bp.wait()
        else:
            info, nb = bp.run()
        want_info, want = plan_of(meta if ctx[-1] == meta.context_lens[-1] else
                                  workloads.StepMeta(**{**meta.__dict__, "context_lens": ctx}),
                                  block_tables=bt, fp8=True)
        begin, fp8 = pkv.stage_fp8(want_info, want)
        assert nb == want.nbytes and np.array_equal(out.view(np.uint8)[:nb], want.view(np.uint8)[:nb])
        assert np.array_equal(stage, begin) and begin[-1] > 0
        for f in ("staged_blocks", "max_rows", "workspace_bytes"):
            assert getattr(bp.fp8, f) == getattr(fp8, f)
        ctx[-1] -= 16
    bp.close()
    with pytest.raises(TypeError):
        pkv.BoundPlan(cu, ctx, meta.num_q_heads, desc, out, num_sms=152, fp8=True)
    with pytest.raises(ValueError):
        pkv.BoundPlan(cu, ctx, meta.num_q_heads, desc, out, num_sms=152, fp8=True,
                      stage_out=stage[:-1].copy())


# ------------------------------------------------- the plain forms the GPU tests compare with

@pytest.mark.parametrize("seed", range(4))
def test_plain_attention_is_the_oracle(seed):
    rng = np.random.default_rng(seed)
    meta = workloads.random_step(rng, max_ctx=90)
    q, _, _, pool = workloads.make_values(meta)
    want = oracle.paged_varlen_attention(q, meta.cu_q_lens, meta.context_lens, meta.block_tables,
                                         pool, meta.scale)
    got, wabs, mag = ref.attention(ref.f64(q), meta.cu_q_lens, meta.context_lens,
                                   meta.block_tables, ref.f64(pool), meta.scale)
    assert np.abs(got - want).max() <= 1e-12
    assert (np.abs(got) <= wabs + 1e-12).all() and (mag >= 0).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_plain_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((7, 2, 64))
    pos = rng.integers(0, 50, size=7)
    cs = ref.table(50, 32)
    y, size = ref.rotate(x, pos, cs, interleaved)
    h = x[..., :32]
    z = h[..., 0::2] + 1j * h[..., 1::2] if interleaved else h[..., :16] + 1j * h[..., 16:]
    t = z * (cs[pos, :16] + 1j * cs[pos, 16:].astype(np.float64))[:, None]
    want = np.stack([t.real, t.imag], axis=-1 if interleaved else -2).reshape(h.shape)
    assert np.abs(y[..., :32] - want).max() <= 1e-12
    assert np.array_equal(y[..., 32:], x[..., 32:]) and (np.abs(y) <= size + 1e-12).all()
    # a rotation keeps each pair's length up to the table's rounding, 2^-23 relative
    assert np.abs(np.abs(t) / np.abs(z) - 1).max() <= 2.0 ** -22


def test_plain_append_fp8():
    """Values stand within half a step of what was appended; kept rows keep theirs."""
    rng = np.random.default_rng(4)
    codes = ref.decode(ref.encode(rng.standard_normal((3, 2, 1, 16, 64)) * 100))
    scales = np.full((3, 1, 2), 0.25)
    rows = rng.standard_normal((4, 2, 1, 64)) * np.array([1, 1, 1, 5000.0])[:, None, None, None]
    new, sc, rounded = ref.append_fp8(codes, scales, rows, [5, 6, 16, 35])
    assert rounded.sum() == 2 * (2 + 1 + 4)          # block 2 grew: its rows 0-2 and the new one
    assert (sc[0] == 0.25).all() and (sc[1] < 0.25).all() and (sc[2] > 0.25).all()
    for b, off, t in ((0, 5, 0), (0, 6, 1), (1, 0, 2), (2, 3, 3)):
        held = ref.decode(ref.encode(new[b, :, 0, off])) * sc[b, 0][:, None]
        assert (np.abs(held - rows[t, :, 0]) <=
                np.maximum(2.0 ** -4 * np.abs(rows[t, :, 0]), 2.0 ** -10 * sc[b, 0][:, None])).all()
    assert np.allclose(new[2, :, 0, :3] * sc[2, 0][:, None, None],
                       codes[2, :, 0, :3] * 0.25)
    assert np.array_equal(new[0, :, 0, :5], codes[0, :, 0, :5])
    for a in (448.0, 448.0001, 447.9, 1e-30, 0.0, 3.5, 1e30):
        s = ref.pow2_scale(a)
        assert a <= 448 * s and (s == 2.0 ** -64 or a > 224 * s)
