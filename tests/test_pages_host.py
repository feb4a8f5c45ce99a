"""CPU tests of the page, beam and sparse calls: every refusal happens before anything is
enqueued, and the plain forms the GPU tests compare with give what hand-made cases need."""

import ctypes

import numpy as np
import pytest
import torch

import pages_ref as ref
import paged_kv_attention_append_gb300 as pkv

A = 0x1000                      # an aligned address that is never dereferenced
OK, NULL, SHAPE, RANGE, UNSUPPORTED, WORKSPACE, ALIGN = 0, 1, 2, 3, 4, 5, 8
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    pkv.build()
    return pkv._load()


COPY = dict(data=A, row=4096, arrays=1, blocks=10, src=A, dst=A, pairs=4, count=None, status=None,
            stream=None)
FORK = dict(parents=A, new=4, tables=A, ctx=A, rows=4, width=10, refs=A, blocks=100, keep=0,
            new_tables=2 * A, new_ctx=2 * A, status=None, stream=None)
FREE = dict(rows=A, listed=2, tables=A, ctx=A, num_rows=4, width=10, refs=A, blocks=100, status=None,
            stream=None)
RESERVE = dict(cu=A, tables=A, ctx=A, rows=4, width=10, refs=A, blocks=100, slots=A, tokens=4, src=A,
               dst=A, ws=A, wsb=BIG, status=None, stream=None)
COMPACT = dict(tables=A, ctx=A, rows=4, width=10, refs=A, blocks=100, new_tables=A, new_refs=A, src=A,
               dst=A, pairs=50, num=A, ws=A, wsb=BIG, status=None, stream=None)
BEAM = dict(logits=A, type=0, stride=1000, cum=A, finished=None, requests=2, beams=4, vocab=1000,
            select=4, pad=0, scores=A, tokens=A, parents=A, ws=A, wsb=BIG, stream=None)
DESC = dict(nb=10, bs=16, hkv=2, d=128)
INDEX = dict(pool=A, desc=DESC, slots=A, tokens=4, index=A, scales=A, status=None, stream=None)
SELECT = dict(q=A, cu=A, ctx=A, tables=A, width=10, seqs=2, total=4, hq=8, index=A, scales=A,
              desc=DESC, num=8, sink=1, recent=2, selected=A, ws=A, wsb=BIG, status=None, stream=None)
SPARSE = dict(q=A, cu=A, ctx=A, tables=A, width=10, seqs=2, total=4, hq=8, selected=A, num=8, pool=A,
              desc=DESC, scale=0.1, out=A, status=None, stream=None)

REFUSED = [
    ("fork_sequences", FORK, [
        (dict(new=-1), SHAPE), (dict(rows=-1), SHAPE), (dict(width=-1), SHAPE), (dict(blocks=-1), SHAPE),
        (dict(keep=2), RANGE), (dict(parents=None), NULL), (dict(tables=None), NULL),
        (dict(ctx=None), NULL), (dict(refs=None), NULL), (dict(new_tables=None), NULL),
        (dict(new_ctx=None), NULL), (dict(new_tables=A), SHAPE), (dict(new_ctx=A), SHAPE),
        (dict(parents=A + 2), ALIGN), (dict(refs=A + 1), ALIGN), (dict(new=0, rows=0), OK)]),
    ("free_sequences", FREE, [
        (dict(listed=-1), SHAPE), (dict(num_rows=-1), SHAPE), (dict(rows=None), NULL),
        (dict(tables=None), NULL), (dict(ctx=None), NULL), (dict(refs=None), NULL),
        (dict(rows=A + 2), ALIGN), (dict(listed=0, rows=None), OK)]),
    ("reserve_blocks", RESERVE, [
        (dict(rows=-1), SHAPE), (dict(tokens=-1), SHAPE), (dict(blocks=-1), SHAPE),
        (dict(rows=8193), UNSUPPORTED), (dict(blocks=1 << 28), UNSUPPORTED),
        (dict(width=1 << 28), UNSUPPORTED), (dict(cu=None), NULL), (dict(ctx=None), NULL),
        (dict(tables=None), NULL), (dict(refs=None), NULL), (dict(slots=None), NULL),
        (dict(src=None), NULL), (dict(dst=None), NULL), (dict(ws=None), NULL), (dict(ws=A + 4), ALIGN),
        (dict(slots=A + 2), ALIGN), (dict(wsb=100), WORKSPACE), (dict(rows=0), OK)]),
    ("compact_blocks", COMPACT, [
        (dict(rows=-1), SHAPE), (dict(blocks=-1), SHAPE), (dict(pairs=49), SHAPE), (dict(num=None), NULL),
        (dict(refs=None), NULL), (dict(new_refs=None), NULL), (dict(tables=None), NULL),
        (dict(new_tables=None), NULL), (dict(src=None), NULL), (dict(ws=None), NULL),
        (dict(ws=A + 8), ALIGN), (dict(wsb=100), WORKSPACE),
        (dict(blocks=2 ** 31 - 1, pairs=2 ** 30), UNSUPPORTED),
        (dict(blocks=0, pairs=0, rows=0, num=None), OK)]),
    ("beam_select", BEAM, [
        (dict(requests=-1), SHAPE), (dict(beams=0), SHAPE), (dict(vocab=0), SHAPE), (dict(select=0), SHAPE),
        (dict(stride=999), SHAPE), (dict(select=129), UNSUPPORTED), (dict(beams=1025), UNSUPPORTED),
        (dict(type=3), UNSUPPORTED), (dict(type=-1), UNSUPPORTED),
        (dict(vocab=2 ** 31 - 1, stride=2 ** 31), UNSUPPORTED), (dict(logits=None), NULL),
        (dict(cum=None), NULL), (dict(scores=None), NULL), (dict(tokens=None), NULL),
        (dict(parents=None), NULL), (dict(ws=None), NULL), (dict(logits=A + 1), ALIGN),
        (dict(logits=A + 2, type=2), ALIGN), (dict(cum=A + 2), ALIGN), (dict(ws=A + 8), ALIGN),
        (dict(wsb=63), WORKSPACE), (dict(requests=0), OK)]),
    ("update_block_index", INDEX, [
        (dict(tokens=-1), SHAPE), (dict(pool=None), NULL), (dict(slots=None), NULL),
        (dict(index=None), NULL), (dict(scales=None), NULL), (dict(pool=A + 8), ALIGN),
        (dict(index=A + 4), ALIGN), (dict(scales=A + 4), ALIGN), (dict(slots=A + 2), ALIGN),
        (dict(desc=dict(DESC, d=96)), UNSUPPORTED), (dict(desc=dict(DESC, bs=32)), UNSUPPORTED),
        (dict(desc=None), NULL), (dict(tokens=0, pool=None), OK)]),
    ("select_blocks", SELECT, [
        (dict(width=-1), SHAPE), (dict(seqs=-1), SHAPE), (dict(total=-1), SHAPE), (dict(num=0), SHAPE),
        (dict(hq=7), SHAPE), (dict(hq=0), SHAPE), (dict(hq=34), UNSUPPORTED), (dict(seqs=0), SHAPE),
        (dict(width=0), SHAPE), (dict(sink=-1), RANGE), (dict(recent=0), RANGE),
        (dict(sink=5, recent=4), RANGE), (dict(total=1 << 31), UNSUPPORTED), (dict(q=None), NULL),
        (dict(cu=None), NULL), (dict(index=None), NULL), (dict(scales=None), NULL),
        (dict(selected=None), NULL), (dict(ws=None), NULL), (dict(q=A + 8), ALIGN),
        (dict(index=A + 8), ALIGN), (dict(ws=A + 8), ALIGN), (dict(wsb=95), WORKSPACE),
        (dict(desc=dict(DESC, d=32)), UNSUPPORTED), (dict(desc=dict(DESC, nb=0)), SHAPE),
        (dict(total=0), OK),
        (dict(total=0, seqs=0, width=0), OK)]),
    ("paged_sparse_attention", SPARSE, [
        (dict(width=-1), SHAPE), (dict(num=0), SHAPE), (dict(hq=7), SHAPE), (dict(hq=34), UNSUPPORTED),
        (dict(scale=float("nan")), RANGE), (dict(scale=float("inf")), RANGE), (dict(q=None), NULL),
        (dict(ctx=None), NULL), (dict(tables=None), NULL), (dict(selected=None), NULL),
        (dict(pool=None), NULL), (dict(out=None), NULL), (dict(q=A + 8), ALIGN), (dict(out=A + 2), ALIGN),
        (dict(pool=A + 8), ALIGN), (dict(selected=A + 2), ALIGN),
        (dict(desc=dict(DESC, hkv=0)), SHAPE), (dict(total=0), OK)]),
]


@pytest.mark.parametrize("name,defaults,kw,want",
                         [(n, d, kw, w) for n, d, cases in REFUSED for kw, w in cases])
def test_refusals(lib, name, defaults, kw, want):
    kw = {k: (None if v is None else ctypes.byref(pkv.PoolDesc(*v.values()))) if k == "desc" else v
          for k, v in dict(defaults, **kw).items()}
    before = pkv.kernel_launch_count()
    assert getattr(lib, "pkv_" + name)(*kw.values()) == want
    assert pkv.kernel_launch_count() == before


@pytest.mark.parametrize("kw,want", [
    (dict(arrays=-1), SHAPE), (dict(blocks=-1), SHAPE), (dict(pairs=-1), SHAPE), (dict(data=None), NULL),
    (dict(src=None), NULL), (dict(dst=None), NULL), (dict(row=0), SHAPE), (dict(row=6), SHAPE),
    (dict(row=-4), SHAPE), (dict(row=1 << 37), SHAPE), (dict(data=A + 2), ALIGN), (dict(src=A + 2), ALIGN),
    (dict(count=A + 2), ALIGN), (dict(arrays=0), OK), (dict(pairs=0), OK), (dict(arrays=None), NULL)])
def test_copy_refusals(lib, kw, want):
    a = dict(COPY, **kw)
    arrays = (pkv.BlockArray * 1)(pkv.BlockArray(a["data"], a["row"]))
    if a["arrays"] is None:
        arrays, a["arrays"] = None, 1
    before = pkv.kernel_launch_count()
    assert lib.pkv_copy_blocks(arrays, a["arrays"], a["blocks"], a["src"], a["dst"], a["pairs"],
                               a["count"], None, None) == want
    assert pkv.kernel_launch_count() == before


def test_workspace_sizes(lib):
    assert lib.pkv_pages_workspace_size(-1, 10) == 0
    assert lib.pkv_pages_workspace_size(8192, 1 << 20) >= 16 * 8192 + 4 * (1 << 20)
    assert lib.pkv_beam_workspace_size(0, 4, 100, 4) == 0
    assert lib.pkv_beam_workspace_size(1, 4, 100, 4) >= 4 * (8 + 4 * 8)
    one = lib.pkv_select_workspace_size(1, 8, 1000)
    assert one >= 8 * 4000
    assert lib.pkv_select_workspace_size(10, 8, 1000) == 10 * one
    assert lib.pkv_select_workspace_size(1 << 20, 8, 1 << 16) <= 512 << 20   # in several passes


def test_python_refuses_what_the_library_cannot_see():
    cpu = torch.zeros((4, 10), dtype=torch.int32)
    one = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.fork_sequences(one, cpu, one, one, cpu.clone(), one.clone())
    with pytest.raises(ValueError, match="CUDA"):
        pkv.free_sequences(one, cpu, one, one)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.reserve_blocks(one, cpu, one, one, num_tokens=1)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.compact_blocks(cpu, one, one)
    with pytest.raises(TypeError, match="CUDA"):
        pkv.beam_select(torch.zeros(1, 2, 3), torch.zeros(1, 2), 2)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.copy_blocks([cpu], one, one)


# ------------------------------------------------------------------------- the plain forms

def test_plain_reserve_by_hand():
    # rows 0 and 1 share a full block and a partly filled one; row 2 starts empty
    tables = np.array([[4, 2, -1], [4, 2, -1], [-1, -1, -1]], dtype=np.int32)
    ctx, refs = np.array([20, 20, 0]), np.array([0, 0, 2, 0, 2, 0])
    slots, src, dst = ref.reserve([0, 1, 2, 19], tables, ctx, refs)
    assert src.tolist() == [2, -1, -1] and dst.tolist() == [0, -1, -1]
    assert tables.tolist() == [[4, 0, -1], [4, 2, -1], [1, 3, -1]]
    assert refs.tolist() == [1, 1, 1, 1, 2, 0] and ctx.tolist() == [21, 21, 17]
    assert slots[:3].tolist() == [4, 36, 16] and slots[-1] == 48
    # one of the holders does not write: the other copies
    tables, ctx = np.array([[4, 2], [4, 2]], dtype=np.int32), np.array([20, 20])
    refs = np.array([0, 0, 2, 0, 2, 0])
    _, src, dst = ref.reserve([0, 0, 1], tables, ctx, refs)
    assert src.tolist() == [-1, 2] and tables.tolist() == [[4, 2], [4, 0]]
    assert refs.tolist() == [1, 0, 1, 0, 2, 0]


def test_plain_compact_by_hand():
    tables, ctx = np.array([[5, 1], [5, 7]], dtype=np.int32), np.array([32, 20])
    new, counts, src, dst = ref.compact(tables, ctx, np.array([0, 1, 0, 0, 0, 2, 0, 1]))
    assert (src, dst) == ([5, 7], [0, 2])
    assert new.tolist() == [[0, 1], [0, 2]] and counts.tolist() == [2, 1, 1, 0, 0, 0, 0, 0]


def test_plain_beam_by_hand():
    x = np.log(np.array([[[1, 2, 1], [5, 2, 1]]], dtype=np.float64))   # probabilities over 4 and 8
    s, t, p, _ = ref.beam(x, [[0.0, 0.0]], 2)
    assert t.tolist() == [[0, 1]] and p.tolist() == [[1, 0]]
    assert np.allclose(np.exp(s), [[0.625, 0.5]])
    # ties: the lower beam, then the lower token; what is not finite never
    s, t, p, _ = ref.beam(np.array([[[0.0, 0.0], [0.0, 0.0], [np.nan, 0.0], [np.inf, 0.0]]]),
                          [[0.0, 0.0, 9.0, 9.0]], 5)
    assert t.tolist() == [[0, 1, 0, 1, -1]] and p.tolist() == [[0, 0, 1, 1, -1]]
    s, t, p, _ = ref.beam(np.zeros((1, 2, 3)), [[0.0, -2.0]], 2, np.array([[True, False]]), 2)
    assert t.tolist() == [[2, 0]] and p.tolist() == [[0, 1]] and s[0, 0] == 0.0


def test_plain_bounds_and_scores_by_hand():
    lo_hi, unit = ref.bounds(np.array([[[1.0, -126.9], [0.6, 3.0]]]))
    assert unit.tolist() == [1.0] and lo_hi.tolist() == [[[0, -127], [1, 3]]]
    assert ref.bounds(np.array([[[127.5]]]))[1] == 2.0
    s = ref.scores(np.array([[1.0, -1.0]]), lo_hi, np.array([1.0]))
    assert s.tolist() == [1024 * (1 + 127)]        # u = 2^-10
    # an upper bound of q . k, for any key of the block
    rng = np.random.default_rng(3)
    k, q = rng.standard_normal((2, 16, 64)), np.round(rng.standard_normal((2, 3, 64)) * 64) / 64
    b, u = ref.bounds(k)
    for h in range(2):
        top = 2.0 ** -10 * 2.0 ** np.floor(np.log2(np.abs(q[h]).max()))
        s = ref.scores(q[h], b[None, h], u[None, h])[0] * top
        assert s >= sum((k[h] @ x).max() for x in q[h]) - 1e-3


def test_select_refuses_tables_wider_than_a_pass(lib):
    kw = dict(SELECT, width=(1 << 30) + 1, desc=ctypes.byref(pkv.PoolDesc(*DESC.values())))
    before = pkv.kernel_launch_count()
    assert lib.pkv_select_blocks(*kw.values()) == UNSUPPORTED
    assert pkv.kernel_launch_count() == before
