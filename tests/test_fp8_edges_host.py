"""CPU tests of the 8-bit pool at its edges."""

import numpy as np
import pytest
import torch

import paged_kv_attention_append_gb300 as pkv
from fp8_bytes import E4M3, code_of, value_of


@pytest.fixture(scope="module", autouse=True)
def lib():
    pkv.build()


def test_rounding_of_its_own_agrees_with_torch():
    """fp8_bytes against another implementation: every code's value, ties, neighbours."""
    all_codes = np.arange(256, dtype=np.uint8)
    v = torch.from_numpy(all_codes).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.nan_to_num(v, nan=-1), np.nan_to_num(value_of(all_codes), nan=-1))
    rng = np.random.default_rng(0)
    x = np.concatenate([(E4M3[1:] + E4M3[:-1]) / 2, np.exp2(rng.uniform(-14, 9, 20000))]).astype(np.float32)
    x = np.concatenate([x, -x, np.nextafter(x, np.float32(0)), np.nextafter(x, np.float32(1e9))])
    x = np.clip(x, -448, 448)
    assert np.array_equal(code_of(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


LIMIT = 8 << 30     # bytes of copies that a plan for an 8-bit pool may ask for, its longest
                    # sequence's aside


def staged(ql, ctx, hkv, group, d, *, fp8=True, shared=0):
    """plan and staging of a step whose sequences all read the same physical blocks"""
    nb = max(-(-c // 16) for c in ctx)
    table = np.tile(np.arange(nb, dtype=np.int32), (len(ctx), 1))
    if shared < nb:
        table[:, shared:] += nb * np.arange(1, len(ctx) + 1, dtype=np.int32)[:, None]
    cu = np.concatenate([[0], np.cumsum(ql)])
    info, host = pkv.plan_step(cu, ctx, hkv * group, pkv.PoolDesc(nb * (len(ctx) + 1), 16, hkv, d),
                               num_sms=152, block_tables=table, upload=False, fp8=fp8)
    begin, f = pkv.stage_fp8(info, host)
    return info, np.diff(begin), f


@pytest.mark.parametrize("hkv,d", [(8, 128), (2, 64), (1, 128)])
def test_copies_stay_within_their_limit(hkv, d):
    """Many short chunks late in long contexts: the plan's copies, the longest sequence's
    aside, fit 8 GiB, those that keep theirs have the most query tokens a key, and every
    sequence's keys are covered."""
    block = 64 * hkv * d
    ctx = [int(c) for c in np.linspace(0.8, 1.2, 40) * LIMIT / block / 32 * 16]
    ql = [64 + 3 * (i % 7) for i in range(40)]
    ql[3], ql[20] = 2048, 700
    info, counts, f = staged(ql, ctx, hkv, 2, d)
    need = np.array([8 * -(-c // 128) for c in ctx])
    assert (need.sum() - need.max()) * block > LIMIT
    kept = counts > 0
    assert np.array_equal(counts[kept], need[kept]) and kept[3] and kept[20] and not kept.all()
    most = need[kept].max()
    assert (f.staged_blocks - most) * block <= LIMIT < (f.staged_blocks + need.max()) * block
    assert f.workspace_bytes <= info.workspace_bytes + LIMIT + most * block
    per_key = np.array(ql) / np.array(ctx)
    assert per_key[~kept].max() <= per_key[kept].min()
    assert info.kv_tokens == sum(ctx)
    # a plan of the bf16 planner has no limit, and says what it needs
    assert staged(ql, ctx, hkv, 2, d, fp8=False)[2].staged_blocks == need.sum()


def test_a_step_at_the_limit_keeps_its_copies():
    full = LIMIT // (64 * 8 * 128) * 16                # 2^21 keys of 8 heads of 128
    info, counts, f = staged([128, 128], [full, full], 8, 1, 128)
    assert f.staged_blocks * 64 * 8 * 128 == 2 * LIMIT and info.num_decode_pieces == 0
    info, counts, f = staged([128, 256, 64], [full, full, 64], 8, 1, 128)
    assert counts.tolist() == [0, full // 16, 8] and info.num_decode_pieces > 0
    # one sequence past the limit by itself, alone and beside a short prompt
    info, counts, f = staged([128, 64], [3 * full, 64], 8, 1, 128)
    assert counts.tolist() == [3 * full // 16, 8] and info.num_decode_pieces == 0


def test_gathered_prefix_counts_towards_the_limit():
    """A prefix that the tensor cores would read for 64 decodes is streamed when the
    prompt chunk beside them leaves no room for its copies."""
    pre = 4096
    full = LIMIT // (64 * 8 * 128) * 16
    ctx = [full, full - 128 * 8] + [pre * 16 + 20] * 64
    ql = [256, 256] + [2] * 64
    info, counts, f = staged(ql[2:], ctx[2:], 8, 4, 128, shared=pre)
    assert info.num_gather_rows > 0 and f.staged_blocks == pre
    nb = full // 16
    table = np.zeros((66, nb), dtype=np.int32)
    table[:2] = np.arange(nb)
    table[2:, :pre] = nb + np.arange(pre)
    table[2:, pre:pre + 2] = nb + pre + np.arange(128).reshape(64, 2)
    cu = np.concatenate([[0], np.cumsum(ql)])
    info, host = pkv.plan_step(cu, ctx, 32, pkv.PoolDesc(nb + pre + 128, 16, 8, 128), num_sms=152,
                               block_tables=table, upload=False, fp8=True)
    begin, f = pkv.stage_fp8(info, host)
    assert info.num_gather_rows == 0
    assert (f.staged_blocks - nb) * 64 * 8 * 128 <= LIMIT and begin[2] == f.staged_blocks


def test_public_names():
    """What a caller who uploads an 8-bit pool's plan needs is exported and described."""
    assert set(pkv.__all__) <= set(dir(pkv))
    assert {"Fp8Info", "stage_fp8", "fp8_pool", "BoundPlan", "StepPlan"} <= set(pkv.__all__)
    assert "stage_fp8" in pkv.plan_step.__doc__ and pkv.stage_fp8.__doc__ and pkv.Fp8Info.__doc__


@pytest.mark.parametrize("rot", [15, 17, 31, 127, 0, -16])
def test_rotation_table_refusals(rot):
    """A table of 15 would have 16 columns at the frequencies of 15: the append would take it."""
    with pytest.raises(ValueError):
        pkv.rope_cos_sin(4, rot, device="cpu")


def test_rotation_table():
    t = pkv.rope_cos_sin(70000, 32, device="cpu").double().numpy()
    p = np.array([0, 1, 12345, 69999], dtype=np.float64)[:, None]
    a = p * 10000.0 ** (-np.arange(16) / 16)
    want = np.concatenate([np.cos(a), np.sin(a)], axis=1)
    # one rounding to fp32 of a value of at most 1, and the angle's in 64 bits (2^-53 of 2^17,
    # each of its two operations)
    assert np.abs(t[[0, 1, 12345, 69999]] - want).max() <= 2.0 ** -25 + 2.0 ** -34
    assert pkv.rope_cos_sin(0, 64, device="cpu").shape == (0, 64)
    with pytest.raises(ValueError):
        pkv.rope_cos_sin(-1, 64, device="cpu")
