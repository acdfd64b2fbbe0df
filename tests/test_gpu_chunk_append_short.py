"""kvq_append_chunk's form for the shortest runs, a block per sequence and one launch: what
a serving loop's single tokens and drafts take.  Each case is held to that form by the
launches that a captured call records; the other form has the same cases in
test_gpu_chunk_append.py."""

import ctypes

import numpy as np
import pytest
import torch

from bit_quantized_kv_pack_gb300 import kvq

from _runs import rotate, tokens_of
from _util import assert_cache_equal, to_np
from test_gpu_chunk_append import _append_ref, _held, _runs, _start

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _launches(f):
    """Kernels that f() records in a graph."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        f()
    n = ctypes.c_size_t(0)
    err = ctypes.CDLL("libcuda.so.1").cuGraphGetNodes(ctypes.c_void_p(graph.raw_cuda_graph()), None, ctypes.byref(n))
    assert err == 0
    return n.value


def _dev(*xs):
    return [torch.from_numpy(x).to(DEV) for x in xs]


CASES = [  # H, gq, d, bits, cap, Nr, S, hybrid, paged, cache lengths, run lengths, rotary, interleaved
    (2, 1, 128, 4, 64, 8, 0, 0, False, [66, 40], [6, 8], 128, False),       # the first drops tokens
    (2, 1, 128, 2, 96, 8, 4, 0, True, [100, 0, 107], [8, 7, 3], 64, True),  # the last is nearly full
    (4, 4, 256, 3, 64, 2, 0, 0, False, [65, 1, 9, 66], [2, 1, 0, 2], 256, False),
    (8, 1, 64, 4, 64, 5, 0, 1, True, [64, 69, 3], [8, 1, 7], 32, False),
    (1, 3, 32, 3, 96, 33, 2, 0, False, [130, 33, 20], [32, 1, 17], 32, True),
    (3, 1, 128, 4, 64, 0, 0, 1, False, [60, 64, 0], [8, 1, 5], 128, False),  # no window
    (1, 2, 64, 2, 32, 1, 0, 0, False, [33, 32, 1], [12, 1, 1], 0, False),
    (1, 1, 32, 4, 64, 100, 0, 0, False, [50, 163, 100], [32, 5, 32], 16, False),  # no longer than the window
]


@pytest.mark.parametrize("H,gq,d,bits,cap,Nr,S,hybrid,paged,kv,ql,rotary,inter", CASES)
def test_short_runs_are_the_single_appends(H, gq, d, bits, cap, Nr, S, hybrid, paged, kv, ql, rotary, inter):
    rng = np.random.default_rng(90 + d + bits)
    g, refs = _start(rng, kv, H, d, bits, cap, Nr, S, hybrid, len(kv) * (cap // 32) + 3 if paged else 0)
    table = kvq.rope_table(max(kv) + 5 * max(ql), rotary) if rotary else None
    host = to_np(table) if rotary else None
    dropped = 0
    for turn in range(4):  # later runs start from a moved ring, and meet the cache's end
        k, v, q, cu = _runs(rng, ql, H, H * gq, d, pad=turn)
        pos = [_held(r) + np.arange(n) for r, n in zip(refs, ql)]
        args = _dev(k, v, cu)
        got = kvq.kvq_append_chunk(g, *args, max(ql), q=torch.from_numpy(q).to(DEV), rope=table, interleaved=inter)
        word = kvq.kvq_read_error(g)[1]
        err, _ = _append_ref(refs, k, v, cu, host, rotary, inter)
        assert word == (kvq.KVQ_ERRBIT_CAPACITY if err else 0)
        dropped |= err
        n = sum(ql)
        want = rotate(q[:n], host, np.concatenate(pos), rotary, inter)
        assert np.array_equal(to_np(got[:n]).view(np.uint16), want.view(np.uint16))
        for b, r in enumerate(refs):
            assert_cache_equal(g, r, batches=[b])
    assert dropped
    kk, vv = kvq.kvq_read_tokens(g, None, max(_held(r) for r in refs), flags=kvq.KVQ_OUT_F32)
    for b, r in enumerate(refs):
        for x, y in (("k", kk), ("v", vv)):
            x = tokens_of(r, x, 0).astype(np.float32)
            assert np.array_equal(to_np(y[b, :, :x.shape[1]]), x)
    assert _launches(lambda: kvq.kvq_append_chunk(g, *args, max(ql), q=got, q_out=got, rope=table,
                                                  interleaved=inter)) == 1


def test_short_runs_of_a_fused_projection_in_place():
    """Columns of one projection output, positions given, queries rotated in place and into
    another tensor, rows of no run before, between and after left as they were."""
    rng = np.random.default_rng(91)
    H, gq, d, Nr, ql = 2, 3, 128, 16, [3, 5]
    Hq, total = H * gq, 15
    cu = np.array([2, 5, 10], np.int32)
    qkv = torch.from_numpy(rng.standard_normal((total, (Hq + 2 * H) * d)).astype(np.float16)).to(DEV)
    heads, before = qkv.view(total, Hq + 2 * H, d), to_np(qkv).copy()
    k, v = heads[:, Hq:Hq + H], heads[:, Hq + H:]
    pos = rng.integers(0, 5000, total).astype(np.int32)
    table, dcu, dpos = kvq.rope_table(5000, d), torch.from_numpy(cu).to(DEV), torch.from_numpy(pos).to(DEV)
    want = rotate(to_np(heads[:, :Hq]), to_np(table), pos, d, False)
    for place in (True, False):
        g, refs = _start(np.random.default_rng(6), [30, 77], H, d, 4, 512, Nr, 0, 0, 0)
        q = heads[:, :Hq].contiguous() if place else heads[:, :Hq]
        out = q if place else torch.full((total, Hq, d), 7.0, dtype=torch.float16, device=DEV)
        left = to_np(out).copy()

        def call(q_in, q_out, cache=g):
            return kvq.kvq_append_chunk(cache, k, v, dcu, max(ql), q=q_in, q_out=q_out, rope=table, positions=dpos)

        assert call(q, out) is out and kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)
        left[2:10] = want[2:10]
        assert np.array_equal(to_np(out), left)
        assert np.array_equal(to_np(qkv), before)
        assert _append_ref(refs, to_np(k), to_np(v), cu, to_np(table), d, False, pos)[0] == 0
        for b, r in enumerate(refs):
            assert_cache_equal(g, r, batches=[b])
        other, _ = _start(np.random.default_rng(6), [30, 77], H, d, 4, 512, Nr, 0, 0, 0)
        assert _launches(lambda: call(q, out, other)) == 1


def test_short_runs_flag_bad_runs_positions_and_pages():
    rng = np.random.default_rng(92)
    H, d, Nr = 2, 64, 4
    g, refs = _start(rng, [30, 60, 30, 30], H, d, 4, 512, Nr, 0, 0, 70)
    pages = g.block_table.clone()
    g.block_table[1, 1] = 70   # tokens 32 .. 63 of sequence 1: past the pool
    g.block_table[0, 1] = -1   # not reached by sequence 0
    pool = [x.clone() for x in (g.k_codes, g.v_codes, g.k_params, g.v_params)]
    k, v, q, _ = _runs(rng, [2, 3, 5, 2], H, H, d)
    table = kvq.rope_table(40, d)
    pos = rng.integers(0, 40, 12).astype(np.int32)
    pos[1], pos[3] = -7, 10 ** 9
    # sequence 2 ends before it begins, sequence 3 passes the rows there are
    cu = np.array([0, 2, 5, 4, 13], np.int32)
    dk, dv, dq, dcu, dpos = _dev(k, v, q, cu, pos)
    got = kvq.kvq_append_chunk(g, dk, dv, dcu, 9, q=dq, rope=table, positions=dpos)
    assert kvq.kvq_read_error(g)[1] == kvq.KVQ_ERRBIT_BADLEN | kvq.KVQ_ERRBIT_BADPOS | kvq.KVQ_ERRBIT_BADPAGE
    err, _ = _append_ref(refs[:2], k, v, cu[:3], to_np(table), d, False, pos)
    assert err == 0
    g.block_table.copy_(pages)  # what follows gathers through it
    assert np.array_equal(to_np(got[:5]), rotate(q[:5], to_np(table), pos[:5], d, False))
    for b in (0, 2, 3):
        assert_cache_equal(g, refs[b], batches=[b])
    # sequence 1: its window and counters as ever, nothing of the three packed tokens anywhere
    assert g.counters[:, 1].tolist() == [59, 4, int(refs[1].res_head[0]), 0]
    for x, r in ((g.k_res, refs[1].k_res), (g.v_res, refs[1].v_res)):
        assert np.array_equal(to_np(x[1]).view(np.uint16), r[0])
    mine = {int(g.block_table[0, 0])}
    for x, old in zip((g.k_codes, g.v_codes, g.k_params, g.v_params), pool):
        assert {int(p) for p in (x != old).flatten(1).any(1).nonzero().flatten()} <= mine
    assert _launches(lambda: kvq.kvq_append_chunk(g, dk, dv, dcu, 9, q=dq, q_out=got, rope=table, positions=dpos)) == 1


@pytest.mark.parametrize("H,Hq,d,n", [(2, 2, 128, 8), (4, 16, 256, 2), (8, 8, 64, 8), (1, 3, 32, 32), (8, 32, 128, 2)])
def test_the_form_changes_where_a_sequence_has_more_than_twelve_warps_of_work(H, Hq, d, n):
    """The longest bound that one launch takes, and the next: the same cache."""
    rng = np.random.default_rng(93)
    k, v, q, cu = _runs(rng, [1, n, 2], H, Hq, d, pad=2 * n)
    args = _dev(k, v, cu)
    dq = torch.from_numpy(q).to(DEV)
    caches = [_start(np.random.default_rng(4), [40, 9, 64], H, d, 4, 128, 8, 0, 0, 0)[0] for _ in range(2)]
    outs = [torch.zeros_like(dq) for _ in range(2)]
    for c, out, bound, launches in zip(caches, outs, (n, n + 256 // d), (1, 2)):
        def call(c=c, out=out, bound=bound):
            return kvq.kvq_append_chunk(c, *args, bound, q=dq, q_out=out)

        assert _launches(call) == launches
        call()
        assert kvq.kvq_read_error(c) == (kvq.KVQ_OK, 0)
    for name in ("k_codes", "v_codes", "k_params", "v_params", "k_res", "v_res", "counters"):
        assert torch.equal(getattr(caches[0], name), getattr(caches[1], name)), name
    assert torch.equal(*outs)
