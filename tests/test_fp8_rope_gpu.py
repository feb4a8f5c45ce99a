"""GPU tests of the rotating append, the 8-bit pool and attention over it, against
the plain 64-bit forms of tests/fp8_ref.py.

Tolerances (u = half a step relative to the value: bf16 2^-8, fp16 2^-11, fp32
2^-24, e4m3 2^-4, or 2^-10 absolute below e4m3's smallest normal 2^-6):

* a rotated element: each of two products and their sum is rounded to fp32, so it
  is off by at most 3 * 2^-24 (|a c| + |b s|) before its one rounding.
* attention, an output element with weights w: bf16 rounding of the result, 2^-8
  |out|; the rounding of each weight for the P V product, relative u_w (split-KV
  fp16 2^-11, tensor cores bf16 2^-8), so u_w sum w |v|; and the error e of each
  exponent x = scale q.k, which changes a weight by e and the sum by as much, so
  2 e sum w |v|.  e: an fp32 sum of D <= 128 terms, 128 * 2^-24 = 2^-17 of
  sum |q k| |scale| =: A, plus the fp32 roundings of x itself and of its scaling
  (4 * 2^-24 A), plus exp2's own 2^-21.  With scales that are no powers of two
  the tensor-core path rounds each K and V value to bf16 as well: e + 2^-8 A and
  2^-8 sum w |v| more.  The fp32 accumulation of O and of the sum over ctx keys adds
  at most 2 ctx 2^-24 sum w |v|.  A weight far below the row's largest meets fp16's
  smallest step, 2^-24: the largest weight (times its V scale) is held as 2^14, so
  rounding to that step is off by at most 2^-25 / 2^14 = 2^-39 of the largest, times
  a stored value of at most 448, for each of ctx keys: ctx 2^-39 448 max(V scale).
  (A near one-hot softmax over a zero in V shows it: an element of 1e-17 is then
  off by 2e-15, all of it from weights of 2^-50.)
"""

import numpy as np
import pytest
import torch

import fp8_ref as ref
import workloads

pytestmark = pytest.mark.gpu

OUT_CANARY = 0x7FC1
GUARD = 4096


@pytest.fixture(scope="module")
def pkv(cuda_device):
    import paged_kv_attention_append_gb300 as m
    m.build()
    return m


def i32(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)


def status_of(dev):
    return torch.zeros(1, dtype=torch.int32, device=dev)


def make_pool(rng, nb, hkv, d, kind="pow2"):
    """(codes uint8 torch CPU, scales float32 torch CPU): N(0, 1)-like contents."""
    x = rng.standard_normal((nb, 2, hkv, 16, d))
    amax = np.abs(x).max(axis=(3, 4))                     # [nb, 2, hkv]
    if kind == "pow2":
        s = np.exp2(np.ceil(np.log2(amax / 448.0)))
    elif kind == "any":
        s = (amax / 448.0).astype(np.float32).astype(np.float64)
    else:                                                 # blocks of very different size
        s = np.exp2(np.ceil(np.log2(amax / 448.0)))
    codes = ref.encode(x / s[..., None, None])
    if kind == "wide":                                    # the same codes, scales over 2^24
        # (V only: scaled keys would turn the softmax into a one-hot of one block)
        s[:, 1] *= np.exp2(rng.integers(-12, 13, size=(nb, hkv)))
    return codes, torch.from_numpy(s.transpose(0, 2, 1).astype(np.float32)).contiguous()


def values_of(codes, scales):
    return ref.decode(codes) * ref.f64(scales).transpose(0, 2, 1)[..., None, None]


def run_attention(pkv, dev, meta, q, codes, scales, *, num_sms=None, tables=True, pmq=None,
                  dev_tables=None, expect=0):
    """The attention through plan_step and the bound call; out and the workspace sit
    between canaries that are checked after it."""
    pool, sc = codes.to(dev), scales.to(dev)
    st = status_of(dev)
    plan = pkv.plan_step(meta.cu_q_lens, meta.context_lens, meta.num_q_heads, pool,
                         num_sms=num_sms, block_tables=meta.block_tables if tables else None,
                         prefill_min_q=pmq, fp8=True)
    n = 0 if plan.workspace is None else plan.workspace.numel()
    ws = torch.full((n + 2 * GUARD,), 0xA5, dtype=torch.uint8, device=dev)
    plan.workspace = ws[GUARD:GUARD + n]
    buf = torch.full((q.shape[0] + 6, *q.shape[1:]), OUT_CANARY, dtype=torch.int16,
                     device=dev).view(torch.bfloat16)
    out = buf[3:3 + q.shape[0]]
    pkv.paged_varlen_attention_fp8(q.to(dev), meta.cu_q_lens, meta.context_lens,
                                   i32(meta.block_tables if dev_tables is None else dev_tables, dev),
                                   pool, sc, meta.scale, plan=plan, out=out, dev_status=st)
    torch.cuda.synchronize(dev)
    assert int(st.item()) == expect
    edge = torch.cat([buf[:3], buf[-3:]]).view(torch.int16)
    assert bool((edge == OUT_CANARY).all()), "wrote outside out"
    assert bool((ws[:GUARD] == 0xA5).all()) and bool((ws[GUARD + n:] == 0xA5).all()), \
        "wrote outside the workspace"
    assert torch.equal(pool.cpu().view(torch.uint8), codes.view(torch.uint8))
    return out.cpu(), plan


def check_attention(got, want, wabs, mag, ctx_max, *, tensor_cores, exact_scales=True, scales=None):
    u_w = 2.0 ** -8 if tensor_cores else 2.0 ** -11
    e = (2.0 ** -17 + 4 * 2.0 ** -24) * mag + 2.0 ** -21
    if tensor_cores and not exact_scales:
        u_w = u_w + 2.0 ** -8
        e = e + 2.0 ** -8 * mag
    tol = 2.0 ** -8 * np.abs(want) + (u_w + 2 * e + 2 * ctx_max * 2.0 ** -24) * wabs
    if scales is not None:
        tol = tol + ctx_max * 2.0 ** -39 * 448 * float(scales[..., 1].max())
    err = np.abs(ref.f64(got) - want)
    assert np.isfinite(err).all()
    worst = float((err / np.maximum(tol, 1e-300)).max()) if err.size else 0.0
    assert worst <= 1.0, f"worst element at {worst:.2f} of its tolerance"
    return worst


def step_case(seed, **kw):
    rng = np.random.default_rng(seed)
    return rng, workloads.random_step(rng, **kw)


# ------------------------------------------------------------------------- attention

SPLIT = [  # (q_lens, ctx_lens, hkv, group, d)
    ([1], [1], 1, 1, 128),
    ([1, 1, 1, 1], [1, 15, 16, 17], 2, 4, 64),
    ([1, 1, 1], [31, 32, 33], 2, 5, 128),
    ([1] * 5, [2, 129, 640, 777, 1024], 8, 4, 128),
    ([2, 3, 1, 8], [16, 17, 100, 40], 2, 8, 128),
    ([5, 1, 0, 7], [5, 300, 90, 33], 4, 1, 64),
    ([4, 8], [260, 512], 2, 16, 128),
    ([1, 2], [1000, 2049], 1, 3, 64),
]


@pytest.mark.parametrize("case", range(len(SPLIT)))
@pytest.mark.parametrize("kind", ["pow2", "any", "wide"])
@pytest.mark.parametrize("sms", [1, 152])
def test_split_kv_rows(pkv, cuda_device, case, kind, sms):
    ql, ctx, hkv, group, d = SPLIT[case]
    rng = np.random.default_rng(100 + case)
    meta = workloads.build_step("fp8", 7 + case, ql, ctx, hkv * group, hkv, d, rng=rng)
    codes, scales = make_pool(rng, meta.num_blocks, hkv, d, kind)
    q = ref.bf16(rng.standard_normal((meta.total_q, hkv * group, d)))
    want = ref.attention(ref.f64(q), meta.cu_q_lens, ctx, meta.block_tables,
                         values_of(codes, scales), meta.scale)
    got, plan = run_attention(pkv, cuda_device, meta, q, codes, scales, num_sms=sms)
    assert plan.fp8.staged_blocks == 0
    check_attention(got, *want, max(ctx), tensor_cores=False, scales=scales)


@pytest.mark.parametrize("qmag", [1e-30, 1e-3, 30.0, 1e4])
def test_q_of_any_size(pkv, cuda_device, qmag):
    """q is scaled per row before it becomes fp16; the softmax scale undoes its size."""
    rng = np.random.default_rng(5)
    meta = workloads.build_step("fp8", 5, [1, 2], [70, 200], 8, 2, 128, rng=rng,
                                scale=1.0 / (qmag * 11.0))
    codes, scales = make_pool(rng, meta.num_blocks, 2, 128)
    x = rng.standard_normal((3, 8, 128))
    x[0, 0] = 0.0                      # a row of zeros
    x[1, 1, 5:] *= 1e-6                # a row with a few large values
    q = ref.bf16(x * qmag)
    want = ref.attention(ref.f64(q), meta.cu_q_lens, [70, 200], meta.block_tables,
                         values_of(codes, scales), np.float32(meta.scale).astype(np.float64))
    got, _ = run_attention(pkv, cuda_device, meta, q, codes, scales)
    check_attention(got, *want, 200, tensor_cores=False, scales=scales)


@pytest.mark.parametrize("scale", [0.0, -0.07, 3.0])
@pytest.mark.parametrize("pmq", [-1, 1])
def test_softmax_scale(pkv, cuda_device, scale, pmq):
    rng = np.random.default_rng(8)
    meta = workloads.build_step("fp8", 8, [70, 1, 3], [70, 150, 40], 4, 2, 64, rng=rng, scale=scale)
    codes, scales = make_pool(rng, meta.num_blocks, 2, 64)
    q = ref.bf16(rng.standard_normal((74, 4, 64)))
    want = ref.attention(ref.f64(q), meta.cu_q_lens, meta.context_lens, meta.block_tables,
                         values_of(codes, scales), float(np.float32(scale)))
    got, _ = run_attention(pkv, cuda_device, meta, q, codes, scales, pmq=pmq)
    check_attention(got, *want, 150, tensor_cores=pmq == 1, scales=scales)


TENSOR = [  # prefill-class chunks, ragged, with decodes beside them
    ([128], [128], 2, 1, 128),
    ([65, 1], [65, 40], 1, 5, 128),
    ([300, 1, 2], [450, 77, 18], 2, 4, 64),
    ([130, 64, 1], [1000, 64, 500], 4, 2, 128),
    ([257], [2050], 2, 8, 128),
]


@pytest.mark.parametrize("case", range(len(TENSOR)))
@pytest.mark.parametrize("kind", ["pow2", "any"])
@pytest.mark.parametrize("sms", [3, 152])
def test_tensor_core_chunks(pkv, cuda_device, case, kind, sms):
    ql, ctx, hkv, group, d = TENSOR[case]
    rng = np.random.default_rng(200 + case)
    meta = workloads.build_step("fp8", 17 + case, ql, ctx, hkv * group, hkv, d, rng=rng)
    codes, scales = make_pool(rng, meta.num_blocks, hkv, d, kind)
    q = ref.bf16(rng.standard_normal((meta.total_q, hkv * group, d)))
    want = ref.attention(ref.f64(q), meta.cu_q_lens, ctx, meta.block_tables,
                         values_of(codes, scales), meta.scale)
    got, plan = run_attention(pkv, cuda_device, meta, q, codes, scales, num_sms=sms)
    assert plan.fp8.staged_blocks >= sum(-(-c // 16) for n, c in zip(ql, ctx) if n >= 64)
    check_attention(got, *want, max(ctx), tensor_cores=True, scales=scales, exact_scales=kind == "pow2")


@pytest.mark.parametrize("group,n_seqs,q_len,blocks", [(4, 20, 1, 17), (2, 6, 2, 33), (8, 9, 3, 8),
                                                       (1, 3, 2, 20), (4, 40, 2, 40)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sms", [1, 9, 152])
def test_shared_prefix(pkv, cuda_device, group, n_seqs, q_len, blocks, d, sms):
    """Gathered tensor-core sub-tiles (long prefixes of many rows for the SMs) and
    streamed ones."""
    rng = np.random.default_rng(300 + blocks)
    ctx = blocks * 16 + q_len + rng.integers(0, 90, size=n_seqs)
    meta = workloads.build_step("fp8", 27, [q_len] * n_seqs, ctx, 2 * group, 2, d, rng=rng,
                                shared_prefix_blocks=blocks)
    codes, scales = make_pool(rng, meta.num_blocks, 2, d)
    q = ref.bf16(rng.standard_normal((meta.total_q, 2 * group, d)))
    want = ref.attention(ref.f64(q), meta.cu_q_lens, ctx, meta.block_tables,
                         values_of(codes, scales), meta.scale)
    got, plan = run_attention(pkv, cuda_device, meta, q, codes, scales, num_sms=sms)
    check_attention(got, *want, int(ctx.max()), tensor_cores=plan.fp8.staged_blocks > 0, scales=scales)


@pytest.mark.parametrize("group,n_seqs,q_len,blocks", [(4, 20, 1, 17), (8, 3, 1, 9), (2, 6, 3, 33)])
def test_shared_prefix_of_a_bf16_plan(pkv, cuda_device, group, n_seqs, q_len, blocks):
    """A plan made for a bf16 pool (pkv_plan_step_ex: gathered at 64 rows, else shared
    split-KV CTAs) serves an 8-bit pool with pkv_plan_stage_fp8's summary."""
    rng = np.random.default_rng(320 + blocks)
    ctx = blocks * 16 + q_len + rng.integers(0, 90, size=n_seqs)
    meta = workloads.build_step("fp8", 28, [q_len] * n_seqs, ctx, 2 * group, 2, 128, rng=rng,
                                shared_prefix_blocks=blocks)
    codes, scales = make_pool(rng, meta.num_blocks, 2, 128)
    q = ref.bf16(rng.standard_normal((meta.total_q, 2 * group, 128)))
    want = ref.attention(ref.f64(q), meta.cu_q_lens, ctx, meta.block_tables,
                         values_of(codes, scales), meta.scale)
    dev = cuda_device
    info, host = pkv.plan_step(meta.cu_q_lens, meta.context_lens, 2 * group,
                               pkv.pool_desc(codes), block_tables=meta.block_tables,
                               upload=False, device=dev)
    assert info.num_gather_rows > 0 or info.num_shared_ctas > 0
    plan = pkv.StepPlan(info, host, dev, fp8=True)
    st = status_of(dev)
    out = pkv.paged_varlen_attention_fp8(q.to(dev), meta.cu_q_lens, meta.context_lens,
                                         meta.block_tables, codes.to(dev), scales.to(dev),
                                         meta.scale, plan=plan, dev_status=st)
    torch.cuda.synchronize(dev)
    assert int(st.item()) == 0
    check_attention(out.cpu(), *want, int(ctx.max()), tensor_cores=info.num_gather_rows > 0,
                    scales=scales)


def test_summary_of_a_smaller_plan_is_reported(pkv, cuda_device):
    """fp8.max_rows below what the plan holds: the larger row groups are reported and
    their rows left as they were; the others are right."""
    dev = cuda_device
    rng = np.random.default_rng(33)
    meta = workloads.build_step("fp8", 33, [1, 4], [200, 90], 8, 2, 128, rng=rng)
    codes, scales = make_pool(rng, meta.num_blocks, 2, 128)
    q = ref.bf16(rng.standard_normal((5, 8, 128)))
    want = ref.attention(ref.f64(q), meta.cu_q_lens, meta.context_lens, meta.block_tables,
                         values_of(codes, scales), meta.scale)
    plan = pkv.plan_step(meta.cu_q_lens, meta.context_lens, 8, codes.to(dev), fp8=True)
    assert plan.fp8.max_rows == 16
    plan.fp8.max_rows = 8
    out = torch.full((5, 8, 128), 7.0, dtype=torch.bfloat16, device=dev)
    st = status_of(dev)
    pkv.paged_varlen_attention_fp8(q.to(dev), meta.cu_q_lens, meta.context_lens,
                                   meta.block_tables, codes.to(dev), scales.to(dev), meta.scale,
                                   plan=plan, out=out, dev_status=st)
    torch.cuda.synchronize(dev)
    assert int(st.item()) == 4
    assert bool((out[1:] == 7.0).all())
    check_attention(out[:1].cpu(), *(x[:1] for x in want), 200, tensor_cores=False, scales=scales)


@pytest.mark.parametrize("stage", ["none", "past", "other"])
def test_wrong_staging_array_is_reported(pkv, cuda_device, stage):
    """A staging array that does not give a tensor-core sequence its copies: reported,
    nothing outside the workspace and out is written, the other rows are right."""
    dev = cuda_device
    rng = np.random.default_rng(34)
    meta = workloads.build_step("fp8", 34, [1, 70], [200, 90], 8, 2, 128, rng=rng)
    codes, scales = make_pool(rng, meta.num_blocks, 2, 128)
    q = ref.bf16(rng.standard_normal((71, 8, 128)))
    want = ref.attention(ref.f64(q), meta.cu_q_lens, meta.context_lens, meta.block_tables,
                         values_of(codes, scales), meta.scale)
    plan = pkv.plan_step(meta.cu_q_lens, meta.context_lens, 8, codes.to(dev), fp8=True)
    n = plan.fp8.staged_blocks
    assert n == 8 and plan.stage.tolist() == [0, 0, n]
    plan.stage = i32({"none": [0, 0, 0], "past": [0, n, 2 * n], "other": [0, n, n]}[stage], dev)
    ws = torch.full((plan.workspace.numel() + 2 * GUARD,), 0xA5, dtype=torch.uint8, device=dev)
    plan.workspace = ws[GUARD:-GUARD]
    out = torch.full((71, 8, 128), 7.0, dtype=torch.bfloat16, device=dev)
    st = status_of(dev)
    pkv.paged_varlen_attention_fp8(q.to(dev), meta.cu_q_lens, meta.context_lens,
                                   meta.block_tables, codes.to(dev), scales.to(dev), meta.scale,
                                   plan=plan, out=out, dev_status=st)
    torch.cuda.synchronize(dev)
    assert int(st.item()) == 4
    assert bool((ws[:GUARD] == 0xA5).all()) and bool((ws[-GUARD:] == 0xA5).all())
    check_attention(out[:1].cpu(), *(x[:1] for x in want), 200, tensor_cores=False, scales=scales)


@pytest.mark.parametrize("q_lens", [[1] * 6, [1], [3, 2, 4], [1] * 40, [8, 1, 8, 5]])
@pytest.mark.parametrize("sms", [3, 4, 9])
def test_split_kv_beside_a_full_prefill(pkv, cuda_device, q_lens, sms):
    """The tensor-core kernel takes every SM that the plan does not leave to the split-KV
    kernel; both kernels' rows are right."""
    rng = np.random.default_rng(35)
    ql = q_lens + [330]
    ctx = [int(x) for x in rng.integers(8, 900, size=len(q_lens))] + [700]
    meta = workloads.build_step("fp8", 35, ql, ctx, 8, 2, 128, rng=rng)
    codes, scales = make_pool(rng, meta.num_blocks, 2, 128)
    q = ref.bf16(rng.standard_normal((meta.total_q, 8, 128)))
    want = ref.attention(ref.f64(q), meta.cu_q_lens, meta.context_lens, meta.block_tables,
                         values_of(codes, scales), meta.scale)
    got, plan = run_attention(pkv, cuda_device, meta, q, codes, scales, num_sms=sms)
    assert plan.info.num_prefill_ctas < sms and plan.info.num_decode_warps > 0
    n = meta.total_q - 330
    for rows, tc in ((slice(0, n), False), (slice(n, None), True)):
        check_attention(got[rows], *(x[rows] for x in want), 900, tensor_cores=tc, scales=scales)


def test_wide_windows_share_blocks(pkv, cuda_device):
    """Verify windows of more than 16 rows: two row groups read each block once."""
    rng = np.random.default_rng(31)
    meta = workloads.build_step("fp8", 31, [8, 7, 4], [700, 90, 1300], 8, 2, 128, rng=rng)
    codes, scales = make_pool(rng, meta.num_blocks, 2, 128, "any")
    q = ref.bf16(rng.standard_normal((19, 8, 128)))
    want = ref.attention(ref.f64(q), meta.cu_q_lens, meta.context_lens, meta.block_tables,
                         values_of(codes, scales), meta.scale)
    got, plan = run_attention(pkv, cuda_device, meta, q, codes, scales)
    assert plan.info.num_shared_ctas > 0
    check_attention(got, *want, 1300, tensor_cores=False, scales=scales)


@pytest.mark.parametrize("pmq", [-1, 1])
def test_stale_bytes_do_not_matter(pkv, cuda_device, pmq):
    """Rows past the context hold NaN codes, unused blocks NaN scales as well."""
    rng = np.random.default_rng(41)
    ql, ctx = [1, 3, 70, 2], [5, 23, 75, 130]
    meta = workloads.build_step("fp8", 41, ql, ctx, 8, 2, 128, rng=rng)
    codes, scales = make_pool(rng, meta.num_blocks, 2, 128)
    q = ref.bf16(rng.standard_normal((meta.total_q, 8, 128)))
    clean, _ = run_attention(pkv, cuda_device, meta, q, codes, scales, pmq=pmq)
    dirty, sc = codes.clone().view(torch.uint8), scales.clone()
    used = set()
    for s, c in enumerate(ctx):
        ids = meta.block_tables[s][:-(-c // 16)]
        used.update(int(b) for b in ids)
        if c % 16:
            dirty[int(ids[-1]), :, :, c % 16:] = 0x7F
    for b in set(range(meta.num_blocks)) - used:
        dirty[b] = 0xFF
        sc[b] = float("nan")
    got, _ = run_attention(pkv, cuda_device, meta, q, dirty.view(torch.float8_e4m3fn), sc, pmq=pmq)
    assert torch.equal(got.view(torch.int16), clean.view(torch.int16))


@pytest.mark.parametrize("seed", range(6))
def test_random_steps(pkv, cuda_device, seed):
    rng, meta = step_case(400 + seed, max_ctx=400)
    codes, scales = make_pool(rng, meta.num_blocks, meta.num_kv_heads, meta.head_dim)
    q = ref.bf16(rng.standard_normal((meta.total_q, meta.num_q_heads, meta.head_dim)))
    want = ref.attention(ref.f64(q), meta.cu_q_lens, meta.context_lens, meta.block_tables,
                         values_of(codes, scales), meta.scale)
    got, plan = run_attention(pkv, cuda_device, meta, q, codes, scales,
                              num_sms=int(rng.choice([1, 8, 152])))
    check_attention(got, *want, 400, tensor_cores=plan.fp8.staged_blocks > 0, scales=scales)


def test_long_context_and_far_blocks(pkv, cuda_device):
    """A 40 000-token context in a pool whose last blocks lie past 4 GiB."""
    dev = cuda_device
    rng = np.random.default_rng(51)
    hkv, d, nb = 8, 128, 140_000
    need = -(-40_000 // 16)
    meta = workloads.build_step("fp8", 51, [1, 1], [40_000, 77], 8, hkv, d, rng=rng)
    codes, scales = make_pool(rng, need + 5, hkv, d)
    table = np.full((2, need), -1, dtype=np.int32)
    table[0] = nb - 1 - np.arange(need)
    table[1, :5] = np.arange(5)
    pool = torch.zeros((nb, 2, hkv, 16, d), dtype=torch.uint8, device=dev)
    assert pool.numel() > 1 << 32
    sc = torch.ones((nb, hkv, 2), device=dev)
    pool[nb - need:] = codes[:need].view(torch.uint8).to(dev)
    sc[nb - need:] = scales[:need].to(dev)
    pool[:5], sc[:5] = codes[need:].view(torch.uint8).to(dev), scales[need:].to(dev)
    q = ref.bf16(rng.standard_normal((2, 8, d)))
    small = np.full((2, need), -1, dtype=np.int32)
    small[0], small[1, :5] = need - 1 - np.arange(need), need + np.arange(5)
    want = ref.attention(ref.f64(q), meta.cu_q_lens, meta.context_lens, small,
                         values_of(codes, scales), meta.scale)
    out = pkv.paged_varlen_attention_fp8(q.to(dev), meta.cu_q_lens, meta.context_lens, table,
                                         pool.view(torch.float8_e4m3fn), sc, meta.scale)
    check_attention(out.cpu(), *want, 40_000, tensor_cores=False, scales=scales)


@pytest.mark.parametrize("fp8", [False, True])
def test_far_blocks_of_append_and_tensor_cores(pkv, cuda_device, fp8):
    """A chunk appended to and attended from blocks past 4 GiB gives the bits that it
    gives in a pool of 7 blocks."""
    dev = cuda_device
    rng = np.random.default_rng(53)
    hkv, d, n, nb = 8, 128, 100, 140_000
    q, k, v = (ref.bf16(rng.standard_normal((n, h, d))).to(dev) for h in (16, hkv, hkv))
    cs, pos = pkv.rope_cos_sin(n, d, device=dev), i32(np.arange(n), dev)
    got = []
    for blocks in (7, nb):
        if fp8:
            pool, sc = pkv.fp8_pool(blocks, hkv, d, device=dev)
            assert blocks == 7 or pool.numel() > 1 << 32
        else:
            pool = torch.zeros((blocks, 2, hkv, 16, d), dtype=torch.bfloat16, device=dev)
        t = np.arange(n)
        slots = i32((blocks - 1 - t // 16) * 16 + t % 16, dev)
        table = blocks - 1 - np.arange(7, dtype=np.int32)[None]
        if fp8:
            qr = pkv.rope_kv_append_fp8(q, k, v, pos, cs, slots, pool, sc)
            out = pkv.paged_varlen_attention_fp8(qr, [0, n], [n], table, pool, sc, d ** -0.5)
        else:
            qr = pkv.rope_kv_append(q, k, v, pos, cs, slots, pool)
            out = pkv.paged_varlen_attention(qr, [0, n], [n], table, pool, d ** -0.5)
        raw = pool.view(torch.uint8)
        got.append([qr, out, raw[blocks - 7:].clone()] + ([sc[blocks - 7:].clone()] if fp8 else []))
        assert not bool(raw[:blocks - 7].any())
        del pool, raw
    assert bool(got[0][1].isfinite().all()) and bool(got[0][2].any())
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("pmq", [-1, 1])
def test_bad_block_is_reported_and_skipped(pkv, cuda_device, pmq):
    rng = np.random.default_rng(61)
    meta = workloads.build_step("fp8", 61, [66, 1], [80, 64], 4, 2, 128, rng=rng)
    codes, scales = make_pool(rng, meta.num_blocks, 2, 128)
    q = ref.bf16(rng.standard_normal((67, 4, 128)))
    bad = meta.block_tables.copy()
    bad[0, 2] = meta.num_blocks + 3
    got, plan = run_attention(pkv, cuda_device, meta, q, codes, scales, tables=False,
                              dev_tables=bad, pmq=pmq, expect=2)
    want = ref.attention(ref.f64(q), meta.cu_q_lens, meta.context_lens, meta.block_tables,
                         values_of(codes, scales), meta.scale)
    check_attention(got[66:], *(x[66:] for x in want), 64, tensor_cores=plan.fp8.staged_blocks > 0, scales=scales)


def test_side_stream_graphs_and_two_plans(pkv, cuda_device):
    """Captured on a side stream, replayed with new inputs; two graphs with a plan (and
    so a workspace) each, replayed in turn."""
    dev = cuda_device
    rng = np.random.default_rng(71)
    runs = []
    for k, (ql, ctx) in enumerate([([1, 70], [600, 200]), ([2, 1, 1], [900, 30, 400])]):
        meta = workloads.build_step("fp8", 71 + k, ql, ctx, 8, 2, 128, rng=rng)
        codes, scales = make_pool(rng, meta.num_blocks, 2, 128)
        pool, sc = codes.to(dev), scales.to(dev)
        plan = pkv.plan_step(meta.cu_q_lens, meta.context_lens, 8, pool,
                             block_tables=meta.block_tables, fp8=True)
        q = torch.zeros((meta.total_q, 8, 128), dtype=torch.bfloat16, device=dev)
        out = torch.empty_like(q)
        st = status_of(dev)
        side = torch.cuda.Stream(dev)
        side.wait_stream(torch.cuda.current_stream(dev))
        call = pkv.BoundAttentionFp8(q, i32(meta.cu_q_lens, dev), i32(meta.context_lens, dev),
                                     i32(meta.block_tables, dev), pool, sc, meta.scale, plan, out,
                                     dev_status=st, stream=side)
        torch.cuda.synchronize(dev)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call.run()
        runs.append((meta, codes, scales, q, out, st, g, call))
    for rep in range(2):
        fresh = []
        for meta, codes, scales, q, out, st, g, _ in runs:
            fresh.append(ref.bf16(rng.standard_normal(tuple(q.shape))))
            q.copy_(fresh[-1])
            out.fill_(float("nan"))
        for r in runs:
            r[6].replay()
        torch.cuda.synchronize(dev)
        for (meta, codes, scales, q, out, st, g, _), qq in zip(runs, fresh):
            assert int(st.item()) == 0
            want = ref.attention(ref.f64(qq), meta.cu_q_lens, meta.context_lens, meta.block_tables,
                                 values_of(codes, scales), meta.scale)
            check_attention(out.cpu(), *want, 900, tensor_cores=True, scales=scales)


def test_same_plan_serves_both_pools(pkv, cuda_device):
    """With power-of-two scales the pool's values are exact in bf16: the bf16
    attention on them agrees within both paths' roundings."""
    dev = cuda_device
    rng = np.random.default_rng(81)
    meta = workloads.build_step("fp8", 81, [1, 90, 2], [333, 200, 50], 8, 2, 128, rng=rng)
    codes, scales = make_pool(rng, meta.num_blocks, 2, 128)
    vals = values_of(codes, scales)
    q = ref.bf16(rng.standard_normal((93, 8, 128)))
    pool16 = ref.bf16(vals).to(dev)
    assert np.array_equal(ref.f64(pool16), vals)
    plan = pkv.plan_step(meta.cu_q_lens, meta.context_lens, 8, pool16,
                         block_tables=meta.block_tables, fp8=True)
    want = ref.attention(ref.f64(q), meta.cu_q_lens, meta.context_lens, meta.block_tables, vals,
                         meta.scale)
    args = (q.to(dev), meta.cu_q_lens, meta.context_lens, meta.block_tables)
    a = pkv.paged_varlen_attention(*args, pool16, meta.scale, plan=plan)
    b = pkv.paged_varlen_attention_fp8(*args, codes.to(dev), scales.to(dev), meta.scale, plan=plan)
    check_attention(a.cpu(), *want, 333, tensor_cores=True)
    check_attention(b.cpu(), *want, 333, tensor_cores=True, scales=scales)


# ------------------------------------------------------------------ rotating append

def rope_inputs(rng, n, hq, hkv, d, packed, dev, size=1.0):
    x = ref.bf16(size * rng.standard_normal((n, hq + 2 * hkv, d)))
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    xd = x.to(dev)
    views = (xd[:, :hq], xd[:, hq:hq + hkv], xd[:, hq + hkv:])
    return (q, k, v), (views if packed else tuple(t.contiguous() for t in views))


def check_rotated(got, x, positions, cs, inter, rows=None):
    want, size = ref.rotate(ref.f64(x), positions, cs, inter)
    tol = 2.0 ** -8 * np.abs(want) + 4 * 2.0 ** -24 * size
    err = np.abs(ref.f64(got) - want)
    if rows is not None:
        err, tol = err[rows], tol[rows]
    assert (err <= tol).all()
    # evaluated in fp32 with every operation rounded, the result is the same to the bit
    same = ref.bf16(ref.rotate(ref.f64(x), positions, cs, inter, np.float32)[0])
    a, b = got.cpu().view(torch.int16), same.view(torch.int16)
    assert torch.equal(a if rows is None else a[rows], b if rows is None else b[rows])


ROPE = [  # n, hq, hkv, d, rot, interleaved, packed
    (1, 1, 1, 64, 64, False, False),
    (1, 16, 8, 128, 128, False, True),
    (5, 3, 1, 128, 16, True, True),
    (17, 8, 2, 64, 32, True, False),
    (17, 8, 2, 64, 32, False, True),
    (33, 40, 8, 128, 128, False, True),
    (200, 5, 5, 128, 96, False, False),
    (200, 4, 4, 128, 112, True, True),
    (3000, 8, 1, 128, 128, False, False),
    (2500, 7, 1, 64, 48, True, True),
]


@pytest.mark.parametrize("case", range(len(ROPE)))
def test_rope_append_bf16(pkv, cuda_device, case):
    n, hq, hkv, d, rot, inter, packed = ROPE[case]
    dev = cuda_device
    rng = np.random.default_rng(500 + case)
    (q, k, v), (qd, kd, vd) = rope_inputs(rng, n, hq, hkv, d, packed, dev)
    max_pos = 5000
    cs = ref.table(max_pos, rot)
    pos = rng.integers(0, max_pos, size=n)
    pos[0] = max_pos - 1
    nb = n // 8 + 3
    slots = rng.permutation(nb * 16)[:n].astype(np.int32)
    skip = rng.random(n) < 0.2
    slots[skip] = -1 - rng.integers(0, 5, size=int(skip.sum()))
    before = ref.bf16(rng.standard_normal((nb, 2, hkv, 16, d)))
    pool = before.to(dev)
    st = status_of(dev)
    out = pkv.rope_kv_append(qd, kd, vd, i32(pos, dev), torch.from_numpy(cs).to(dev),
                             i32(slots, dev), pool, interleaved=inter, dev_status=st)
    torch.cuda.synchronize(dev)
    assert int(st.item()) == 0
    check_rotated(out, q, pos, cs, inter)
    want = before.clone()
    kr = ref.bf16(ref.rotate(ref.f64(k), pos, cs, inter, np.float32)[0])
    for t in range(n):
        if slots[t] >= 0:
            want[slots[t] // 16, 0, :, slots[t] % 16] = kr[t]
            want[slots[t] // 16, 1, :, slots[t] % 16] = v[t]
    assert torch.equal(pool.cpu().view(torch.int16), want.view(torch.int16))
    # k against 64 bits too
    rows = np.flatnonzero(slots >= 0)
    got_k = pool.cpu()[slots[rows] // 16, 0, :, slots[rows] % 16]
    check_rotated(got_k, k[rows], pos[rows], cs, inter)


def test_rope_in_place_padding_and_errors(pkv, cuda_device):
    dev = cuda_device
    rng = np.random.default_rng(91)
    n, hq, hkv, d, rot = 24, 4, 2, 128, 64
    (q, k, v), (qd, kd, vd) = rope_inputs(rng, n, hq, hkv, d, True, dev)
    cs = ref.table(100, rot)
    pos = rng.integers(0, 100, size=n)
    pos[3], pos[7] = -1, 100          # padding; a position past the table
    slots = np.arange(n, dtype=np.int32)
    slots[11] = 3 * 16                # past the pool
    before = ref.bf16(rng.standard_normal((3, 2, hkv, 16, d)))
    cases = [(None, 0), ([7], 5), ([11], 1)]
    for bad, code in cases:
        p, s = pos.copy(), slots.copy()
        if code != 5:
            p[7] = 99
        if code != 1:
            s[11] = 11
        if bad is None:
            p[7], s[11] = 99, 11
        pool, st = before.to(dev), status_of(dev)
        packed = torch.cat([q, k, v], dim=1).to(dev)
        qv = packed[:, :hq]
        out = pkv.rope_kv_append(qv, packed[:, hq:hq + hkv], packed[:, hq + hkv:], i32(p, dev),
                                 torch.from_numpy(cs).to(dev), i32(s, dev), pool, q_out=qv,
                                 dev_status=st)
        torch.cuda.synchronize(dev)
        assert int(st.item()) == code and out.data_ptr() == qv.data_ptr()
        skipped = [3] + ([7] if code == 5 else [])
        rows = np.array([t for t in range(n) if t not in skipped])
        safe = np.clip(p, 0, 99)
        check_rotated(qv.contiguous(), q, safe, cs, False, rows)
        assert torch.equal(qv.cpu()[skipped].view(torch.int16), q[skipped].view(torch.int16))
        assert torch.equal(packed.cpu()[:, hq:], torch.cat([k, v], dim=1))   # k and v not touched
        want = before.clone()
        kr = ref.bf16(ref.rotate(ref.f64(k), safe, cs, False, np.float32)[0])
        for t in rows:
            if s[t] < 48:
                want[s[t] // 16, 0, :, s[t] % 16] = kr[t]
                want[s[t] // 16, 1, :, s[t] % 16] = v[t]
        assert torch.equal(pool.cpu().view(torch.int16), want.view(torch.int16))


# ------------------------------------------------------------------------ 8-bit append

def check_pool(codes, scales, want_codes, want_scales, rounded, before, size=None):
    """Scales equal; rows this step rounded within half an e4m3 step of the exact
    codes (plus the rotation's fp32 error, `size` in code units); others untouched."""
    assert np.array_equal(ref.f64(scales), want_scales)
    got = ref.decode(codes)
    sat = np.clip(want_codes, -448.0, 448.0)
    tol = np.maximum(2.0 ** -4 * np.abs(sat), 2.0 ** -10)
    if size is not None:
        tol = tol + 4 * 2.0 ** -24 * size
    r = rounded[..., None]
    nan = np.isnan(sat)
    assert np.array_equal(np.isnan(got) & r, nan & r)
    with np.errstate(invalid="ignore"):
        assert ((np.abs(got - sat) <= tol) | ~r | nan).all()
    a, b = codes.cpu().view(torch.uint8).numpy(), before.view(torch.uint8).numpy()
    assert np.array_equal(a[~rounded], b[~rounded])


def fp8_case(pkv, dev, rng, slots, hq, hkv, d, nb, *, rot=0, inter=False, packed=False, size=1.0,
             kind="pow2", values=None, expect=0):
    n = len(slots)
    (q, k, v), (qd, kd, vd) = rope_inputs(rng, n, max(hq, 1), hkv, d, packed, dev, size)
    if values is not None:
        k, v = values(k.clone(), v.clone())
        kd, vd = k.to(dev), v.to(dev)
    before, sc = make_pool(rng, nb, hkv, d, kind)
    pool, scd, st = before.to(dev), sc.to(dev), status_of(dev)
    slots = np.asarray(slots, dtype=np.int32)
    mag = None
    if rot:
        cs = ref.table(4000, rot)
        pos = rng.integers(0, 4000, size=n)
        out = pkv.rope_kv_append_fp8(qd, kd, vd, i32(pos, dev), torch.from_numpy(cs).to(dev),
                                     i32(slots, dev), pool, scd, interleaved=inter, dev_status=st)
        check_rotated(out, q, pos, cs, inter)
        # scales follow the largest fp32 value; the fp32 form is exact to the bit, so the
        # reference takes the rows from it and the 64-bit form bounds the codes
        kr = ref.rotate(ref.f64(k), pos, cs, inter, np.float32)[0].astype(np.float64)
        k64, ksize = ref.rotate(ref.f64(k), pos, cs, inter)
        assert (np.abs(kr - k64) <= 3 * 2.0 ** -24 * ksize).all()
    else:
        pkv.paged_kv_append_fp8(kd, vd, i32(slots, dev), pool, scd, dev_status=st)
        kr = ref.f64(k)
    torch.cuda.synchronize(dev)
    assert int(st.item()) == expect
    rows = np.stack([kr, ref.f64(v)], axis=1)
    with np.errstate(invalid="ignore"):
        want = ref.append_fp8(ref.decode(before), ref.f64(sc), rows, slots.tolist())
    check_pool(pool, scd, *want, before)
    return pool, scd


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("slots", [
    [0], [5], [15], [16, 17, 18], list(range(16)), list(range(3, 40)), [40, 9, 25],
    [-1, 5, -1, -7, 6, -1, 7], [31, 30, 29, 28], [2, 100, 3], list(range(64, 96)) + [3, 4, 5]])
def test_fp8_append_blocks(pkv, cuda_device, d, slots):
    rng = np.random.default_rng(600 + len(slots))
    expect = 1 if any(s >= 96 for s in slots) else 0
    fp8_case(pkv, cuda_device, rng, slots, 0, 3, d, 6, expect=expect)


@pytest.mark.parametrize("size", [0.0, 1e-30, 1e-6, 0.05, 40.0, 1e6, 1e30])
@pytest.mark.parametrize("kind", ["pow2", "any"])
def test_fp8_append_scales(pkv, cuda_device, size, kind):
    """New rows far smaller and far larger than what the block holds."""
    rng = np.random.default_rng(610)
    fp8_case(pkv, cuda_device, rng, [4, 5, 17, 32, 33, 63], 0, 2, 128, 4, size=size, kind=kind)


def test_fp8_append_borders(pkv, cuda_device):
    """Largest values at and next to 448 times a power of two, and one step past it."""
    rng = np.random.default_rng(611)

    def values(k, v):
        k[:] = 0
        for t, x in enumerate([448.0, 450.0, 446.0, 3.5, 3.515625, 3.484375, 0.0, 1.75 * 2 ** -60]):
            k[t, :, 3] = x
            v[t, :, 9] = -x
        return k, v
    fp8_case(pkv, cuda_device, rng, [16 * b for b in range(8)], 0, 1, 64, 8, values=values)


def test_fp8_append_infinities_and_nan(pkv, cuda_device):
    rng = np.random.default_rng(612)

    def values(k, v):
        k[0, 0, 0], k[0, 0, 1], k[1, 0, 2] = float("inf"), float("-inf"), float("nan")
        v[2, 0, 5], v[2, 0, 6] = float("nan"), float("-inf")
        return k, v
    fp8_case(pkv, cuda_device, rng, [0, 1, 18], 0, 1, 128, 2, values=values)


@pytest.mark.parametrize("n,hq,hkv,d,rot,inter,packed", [
    (1, 4, 1, 128, 128, False, True), (40, 8, 2, 64, 64, False, False), (40, 8, 2, 64, 32, True, True),
    (300, 40, 8, 128, 128, False, True), (1500, 2, 1, 128, 96, True, True),
    (1100, 4, 2, 64, 64, False, True)])
def test_rope_append_fp8(pkv, cuda_device, n, hq, hkv, d, rot, inter, packed):
    """Runs of every kind in one step: single tokens, part blocks, whole blocks."""
    rng = np.random.default_rng(620 + n)
    slots, b = [], 0
    while len(slots) < n:
        off = int(rng.integers(0, 16)) if rng.random() < 0.6 else 0
        slots += list(range(b * 16 + off, b * 16 + off + int(rng.integers(1, 70))))
        b = slots[-1] // 16 + 1
    nb = max(slots) // 16 + 1
    perm = rng.permutation(nb)
    slots = [int(perm[s // 16]) * 16 + s % 16 for s in slots[:n]]
    fp8_case(pkv, cuda_device, rng, slots, hq, hkv, d, nb, rot=rot, inter=inter, packed=packed)


def test_fp8_append_far_tokens_of_one_block(pkv, cuda_device):
    """Tokens of one block spread past its window, linked by one in between: the later
    one is skipped and reported, nothing outside the block changes."""
    dev = cuda_device
    rng = np.random.default_rng(630)
    n = 24
    slots = [16 + 16 * t for t in range(n)]
    slots[0], slots[10], slots[20] = 0, 1, 2
    k = ref.bf16(rng.standard_normal((n, 1, 64))).to(dev)
    before, sc = make_pool(rng, n + 2, 1, 64)
    pool, scd, st = before.to(dev), sc.to(dev), status_of(dev)
    pkv.paged_kv_append_fp8(k, k, i32(slots, dev), pool, scd, dev_status=st)
    torch.cuda.synchronize(dev)
    assert int(st.item()) == 1
    a, b = pool.cpu().view(torch.uint8), before.view(torch.uint8)
    assert torch.equal(a[11], b[11]) and torch.equal(a[0, :, :, 2:], b[0, :, :, 2:])
    assert torch.equal(a[n + 1], b[n + 1])


def test_token_by_token_equals_at_once(pkv, cuda_device):
    """Powers of two: filling a block one token at a time rounds a kept row again only
    below e4m3's smallest step, so each value is within half a step of the block's
    final scale of what writing the block at once gives (2^-9 of the scale)."""
    dev = cuda_device
    rng = np.random.default_rng(640)
    k = ref.bf16(rng.standard_normal((16, 2, 128)) * np.exp2(np.arange(16) / 2)[:, None, None]).to(dev)
    a, sa = pkv.fp8_pool(2, 2, 128, device=dev)
    b, sb = pkv.fp8_pool(2, 2, 128, device=dev)
    pkv.paged_kv_append_fp8(k, k, i32(np.arange(16), dev), a, sa)
    for t in range(16):
        pkv.paged_kv_append_fp8(k[t:t + 1], k[t:t + 1], i32([t], dev), b, sb)
    torch.cuda.synchronize(dev)
    assert torch.equal(sa, sb)
    va, vb = values_of(a.cpu(), sa.cpu()), values_of(b.cpu(), sb.cpu())
    step = ref.f64(sa).transpose(0, 2, 1)[..., None, None] * 2.0 ** -9
    # a value rounded once at a finer scale and again at each growth: one step at most
    assert (np.abs(va - vb) <= np.maximum(step, 2.0 ** -3 * np.abs(va))).all()
    assert (np.abs(va - vb) > step).mean() < 0.01


# ------------------------------------------------------------------ run together

@pytest.mark.parametrize("fp8", [False, True])
def test_serving_steps(pkv, cuda_device, fp8):
    """A prompt chunk, then decode steps, as a server runs them: the rotating append,
    the attention on the rotated q, the device-side advance, positions moved on; the
    decode steps run in one captured graph and are replayed."""
    dev = cuda_device
    rng = np.random.default_rng(700 + fp8)
    hq, hkv, d, prompts, steps = 8, 2, 128, [100, 37], 3
    cs = ref.table(400, d)
    csd = torch.from_numpy(cs).to(dev)
    last = [p + steps for p in prompts]
    meta = workloads.build_step("serve", 70, prompts, prompts, hq, hkv, d, rng=rng, pool_blocks=40)
    full = workloads.build_step("serve", 70, [1, 1], last, hq, hkv, d, rng=rng, pool_blocks=40)
    tables = full.block_tables
    scale = 1.0 / np.sqrt(d)
    if fp8:
        pool, sc = pkv.fp8_pool(40, hkv, d, device=dev)
        pool.view(torch.uint8).fill_(0x7F)          # nothing of a fresh block matters
        sc.fill_(float("nan"))
    else:
        pool, sc = torch.zeros((40, 2, hkv, 16, d), dtype=torch.bfloat16, device=dev), None
    st = status_of(dev)

    def append(q, k, v, pos, slots):
        f = (lambda *a, **kw: pkv.rope_kv_append_fp8(*a, sc, **kw)) if fp8 else pkv.rope_kv_append
        return f(q, k, v, pos, csd, slots, pool, dev_status=st)

    def attend(q, cu, ctx, bt, plan):
        if fp8:
            return pkv.paged_varlen_attention_fp8(q, cu, ctx, bt, pool, sc, scale, plan=plan,
                                                  dev_status=st)
        return pkv.paged_varlen_attention(q, cu, ctx, bt, pool, scale, plan=plan, dev_status=st)

    def values():
        return values_of(pool.cpu(), sc.cpu()) if fp8 else ref.f64(pool)

    def slot(s, p):
        return int(tables[s, p // 16]) * 16 + p % 16

    # the prompts
    n = sum(prompts)
    pos = np.concatenate([np.arange(p) for p in prompts])
    slots = [slot(s, p) for s, m in enumerate(prompts) for p in range(m)]
    (q, k, v), (qd, kd, vd) = rope_inputs(rng, n, hq, hkv, d, True, dev)
    plan = pkv.plan_step(meta.cu_q_lens, prompts, hq, pool, fp8=fp8)
    qr = append(qd, kd, vd, i32(pos, dev), i32(slots, dev))
    out = attend(qr, meta.cu_q_lens, prompts, tables, plan)
    torch.cuda.synchronize(dev)
    assert int(st.item()) == 0
    q64, size = ref.rotate(ref.f64(q), pos, cs, False)
    vals = np.nan_to_num(values())
    want = ref.attention(ref.f64(qr), meta.cu_q_lens, prompts, tables, vals, scale)
    check_attention(out.cpu(), *want, max(prompts), tensor_cores=True)
    # ... and from the unrotated inputs, all in 64 bits: keys of the cache within e4m3
    k64 = ref.rotate(ref.f64(k), pos, cs, False)[0]
    held = vals[np.array(slots) // 16, 0, :, np.array(slots) % 16]
    top = np.abs(k64).max()
    assert (np.abs(held - k64) <= (2.0 ** -4 if fp8 else 2.0 ** -8) * np.abs(k64) +
            2.0 ** -9 * 2 * top / 448).all()

    # decode steps in one graph
    cu = i32([0, 1, 2], dev)
    bt = i32(tables, dev)
    chain = pkv.plan_step([0, 1, 2], [p + 1 for p in prompts], hq, pool, chain_steps=steps, fp8=fp8)
    ctx0 = np.array([p + 1 for p in prompts])
    ctx, pp = i32(ctx0, dev), i32(ctx0 - 1, dev)
    sl = i32([slot(s, c - 1) for s, c in enumerate(ctx0)], dev)
    ins = [rope_inputs(rng, 2, hq, hkv, d, True, dev) for _ in range(steps)]
    snapshot = (pool.clone(), None if sc is None else sc.clone())
    outs, rots = [], []

    def chain_run():
        outs.clear(), rots.clear()
        for _, (qd, kd, vd) in ins:
            rots.append(append(qd, kd, vd, pp, sl))
            outs.append(attend(rots[-1], cu, ctx, bt, chain))
            pkv.decode_advance(ctx, sl, cu, bt, pool, dev_status=st)
            pp.add_(1)

    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize(dev)
    with torch.cuda.graph(g, stream=side):
        chain_run()
    for rep in range(2):
        pool.copy_(snapshot[0])
        if sc is not None:
            sc.copy_(snapshot[1])
        ctx.copy_(i32(ctx0, dev))
        pp.copy_(i32(ctx0 - 1, dev))
        sl.copy_(i32([slot(s, c - 1) for s, c in enumerate(ctx0)], dev))
        g.replay()
        torch.cuda.synchronize(dev)
        assert int(st.item()) == 0
        vals = np.nan_to_num(values())
        for i in range(steps):
            c = ctx0 + i
            p = c - 1
            check_rotated(rots[i], ins[i][0][0], p, cs, False)
            # scales may have grown after step i: only the last step reads the final pool
            if i == steps - 1 or not fp8:
                want = ref.attention(ref.f64(rots[i]), [0, 1, 2], c, tables, vals, scale)
                # the bf16 pool's split-KV kernel rounds its weights to bf16, as the tensor
                # cores do (u_w = 2^-8); the 8-bit pool's to fp16
                check_attention(outs[i].cpu(), *want, int(c.max()), tensor_cores=not fp8,
                                scales=None if sc is None else sc.cpu().nan_to_num())


def test_two_streams_at_once(pkv, cuda_device):
    """Appends and attentions of two independent batches on two streams, interleaved
    without ordering between them: each has its own pool, plan and workspace."""
    dev = cuda_device
    jobs = []
    for k in range(2):
        rng = np.random.default_rng(800 + k)
        meta = workloads.build_step("two", 80 + k, [1] * 40, rng.integers(2, 900, size=40), 8, 2,
                                    128, rng=rng)
        codes, scales = make_pool(rng, meta.num_blocks, 2, 128)
        pool, sc = codes.to(dev), scales.to(dev)
        (q, kk, v), (qd, kd, vd) = rope_inputs(rng, 40, 8, 2, 128, True, dev)
        cs = ref.table(1000, 128)
        pos = meta.context_lens - 1
        side = torch.cuda.Stream(dev)
        plan = pkv.plan_step(meta.cu_q_lens, meta.context_lens, 8, pool, fp8=True)
        out, st = torch.empty((40, 8, 128), dtype=torch.bfloat16, device=dev), status_of(dev)
        app = pkv.BoundRopeAppend(qd, kd, vd, i32(pos, dev), torch.from_numpy(cs).to(dev),
                                  i32(meta.slot_mapping, dev), pool, kv_scales=sc, dev_status=st,
                                  stream=side)
        att = pkv.BoundAttentionFp8(app.q_out, i32(meta.cu_q_lens, dev), i32(meta.context_lens, dev),
                                    i32(meta.block_tables, dev), pool, sc, meta.scale, plan, out,
                                    dev_status=st, stream=side)
        jobs.append((meta, q, pos, cs, pool, sc, app, att, out, st))
    torch.cuda.synchronize(dev)
    for _ in range(5):                 # the append of the same tokens again changes nothing
        for j in jobs:
            j[6].run()
        for j in jobs:
            j[7].run()
    torch.cuda.synchronize(dev)
    for meta, q, pos, cs, pool, sc, app, att, out, st in jobs:
        assert int(st.item()) == 0
        check_rotated(app.q_out, q, pos, cs, False)
        want = ref.attention(ref.f64(app.q_out), meta.cu_q_lens, meta.context_lens,
                             meta.block_tables, values_of(pool.cpu(), sc.cpu()), meta.scale)
        check_attention(out.cpu(), *want, 900, tensor_cores=False, scales=sc.cpu())


def test_padded_batch_leaves_its_tail(pkv, cuda_device):
    """A batch padded to a fixed size: padding tokens have position and slot -1, padding
    sequences no query; their rows of q_out and every other row stay as they were."""
    dev = cuda_device
    rng = np.random.default_rng(820)
    n, pad = 5, 11
    meta = workloads.build_step("pad", 82, [1] * n, [3, 40, 17, 200, 65], 4, 2, 64, rng=rng)
    codes, scales = make_pool(rng, meta.num_blocks, 2, 64)
    pool, sc, st = codes.to(dev), scales.to(dev), status_of(dev)
    (q, k, v), (qd, kd, vd) = rope_inputs(rng, n + pad, 4, 2, 64, False, dev)
    cs = ref.table(300, 64)
    pos = np.concatenate([meta.context_lens - 1, np.full(pad, -1)])
    slots = np.concatenate([meta.slot_mapping, np.full(pad, -1)])
    q_out = torch.full((n + pad, 4, 64), 3.0, dtype=torch.bfloat16, device=dev)
    pkv.rope_kv_append_fp8(qd, kd, vd, i32(pos, dev), torch.from_numpy(cs).to(dev), i32(slots, dev),
                           pool, sc, q_out=q_out, dev_status=st)
    cu = np.concatenate([np.arange(n + 1), np.full(pad, n)]).astype(np.int32)
    ctx = np.concatenate([meta.context_lens, np.zeros(pad)]).astype(np.int32)
    bt = np.concatenate([meta.block_tables, np.full((pad, meta.max_blocks), -1)]).astype(np.int32)
    out = pkv.paged_varlen_attention_fp8(q_out[:n], cu, ctx, bt, pool, sc, meta.scale, dev_status=st)
    torch.cuda.synchronize(dev)
    assert int(st.item()) == 0
    assert bool((q_out[n:] == 3.0).all())
    check_rotated(q_out[:n], q[:n], pos[:n], cs, False)
    want = ref.attention(ref.f64(q_out[:n]), cu, ctx, bt, values_of(pool.cpu(), sc.cpu()), meta.scale)
    check_attention(out.cpu(), *want, 200, tensor_cores=False, scales=sc.cpu())


def test_python_refusals(pkv, cuda_device):
    dev = cuda_device
    pool, sc = pkv.fp8_pool(4, 2, 64, device=dev)
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device=dev)
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device=dev)
    pos, slots = i32([0, 1, 2], dev), i32([0, 1, 2], dev)
    cs = pkv.rope_cos_sin(8, 64, device=dev)
    ok = dict(q=q, k=k, v=k, positions=pos, cos_sin=cs, slot_mapping=slots, kv_pool=pool,
              kv_scales=sc)
    pkv.BoundRopeAppend(**ok).run()
    wide = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device=dev)
    bad = [dict(k=k.cpu()), dict(k=k.float()), dict(v=k[:2]), dict(k=wide[:, :, ::2], v=k),
           dict(k=wide[:, :, :64], v=k), dict(positions=pos[:2]), dict(positions=pos.long()),
           dict(slot_mapping=slots[:2]), dict(cos_sin=cs.double()), dict(cos_sin=None, positions=None),
           dict(q=q[:2]), dict(q_out=q[:, :2].contiguous()), dict(kv_scales=sc[:3]),
           dict(kv_pool=pool.view(torch.uint8)), dict(kv_scales=None), dict(kv_scales=sc.half())]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            pkv.BoundRopeAppend(**{**ok, **kw})
    for kw in (dict(cos_sin=cs[:, :24].contiguous()), dict(cos_sin=cs[:, :8].contiguous())):
        with pytest.raises(pkv.PkvError):
            pkv.BoundRopeAppend(**{**ok, **kw}).run()
    meta = workloads.build_step("r", 1, [1, 2], [20, 30], 4, 2, 64, pool_blocks=4)
    args = (torch.zeros((3, 4, 64), dtype=torch.bfloat16, device=dev), meta.cu_q_lens,
            meta.context_lens, meta.block_tables, pool)
    plan = pkv.plan_step(meta.cu_q_lens, meta.context_lens, 4, pool)      # not for an 8-bit pool
    with pytest.raises(ValueError):
        pkv.paged_varlen_attention_fp8(*args, sc, 0.1, plan=plan)
    plan = pkv.plan_step([0, 1], [20], 4, pool, fp8=True)                 # of another step
    with pytest.raises(ValueError):
        pkv.paged_varlen_attention_fp8(*args, sc, 0.1, plan=plan)
    with pytest.raises((ValueError, TypeError)):
        pkv.paged_varlen_attention_fp8(*args, sc.double(), 0.1)
    with pytest.raises((ValueError, TypeError)):
        pkv.paged_varlen_attention(*args, 0.1)
    # nothing to do is no error, and nothing is launched
    before = pkv.kernel_launch_count()
    pkv.rope_kv_append_fp8(q[:0], k[:0], k[:0], pos[:0], cs, slots[:0], pool, sc)
    pkv.paged_kv_append_fp8(k[:0], k[:0], slots[:0], pool, sc)
    assert pkv.paged_varlen_attention_fp8(q[:0], [0, 0], [5], [[0]], pool, sc, 0.1).shape == (0, 4, 64)
    assert pkv.kernel_launch_count() == before
