"""kvq_append_chunk and kvq_read_tokens: a run of tokens leaves the cache bit for bit
as the oracle's single appends of the rotated tokens do, and reads back as the values
it stands for."""

import numpy as np
import pytest
import torch

import oracle
from bit_quantized_kv_pack_gb300 import kvq

from _runs import rotate, tokens_of
from _util import assert_cache_equal, gpu_cache, oracle_sequences, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _start(rng, lens, H, d, bits, cap, Nr, S, hybrid, pages):
    B, Lmax = len(lens), max(max(lens), 1)
    k = (rng.standard_normal((B, H, Lmax, d)) * 2).astype(np.float16)
    v = rng.standard_normal((B, H, Lmax, d)).astype(np.float16)
    seq = np.array(lens, np.int32)
    g = gpu_cache(B, H, d, bits, cap, Nr, sink=S, hybrid=hybrid, pages=pages, seed=5)
    kvq.kvq_quantize_pack(g, torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV),
                          torch.from_numpy(seq).to(DEV))
    assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)
    return g, oracle_sequences(k, v, seq, bits, cap, Nr, S, hybrid)


def _runs(rng, ql, H, Hq, d, pad=0):
    total = sum(ql) + pad
    k = (rng.standard_normal((total, H, d)) * 2).astype(np.float16)
    v = rng.standard_normal((total, H, d)).astype(np.float16)
    q = rng.standard_normal((total, Hq, d)).astype(np.float16)
    cu = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
    return k, v, q, cu


def _held(r):
    return int(r.packed_len[0] + r.res_len[0] + (r.sink_len[0] if r.desc.sink else 0))


def _append_ref(refs, k, v, cu, table, rotary, interleaved, positions=None):
    """Single appends of the rotated tokens; returns (error bits, K rows rotated)."""
    bits, kr = 0, k.copy()
    for b, r in enumerate(refs):
        n = int(cu[b + 1] - cu[b])
        rows = slice(int(cu[b]), int(cu[b + 1]))
        pos = _held(r) + np.arange(n) if positions is None else positions[rows]
        kr[rows] = rotate(k[rows], table, pos, rotary, interleaved)
        for t in range(int(cu[b]), int(cu[b + 1])):
            bits |= oracle.append(r, kr[t][None], v[t][None])
    return bits, kr


CASES = [  # H, gq, d, bits, cap, Nr, S, hybrid, paged, cache lengths, run lengths, rotary, interleaved
    (2, 4, 128, 4, 512, 16, 0, 0, False, [100, 3, 16], [7, 30, 1], 128, False),
    (2, 4, 128, 2, 512, 16, 4, 0, True, [100, 0, 20], [40, 33, 0], 128, True),
    (1, 1, 64, 3, 300, 33, 0, 0, False, [33, 32, 1], [1, 1, 1], 64, False),
    (3, 2, 64, 4, 320, 0, 0, 0, True, [0, 31, 64], [65, 1, 128], 32, False),
    (2, 3, 256, 4, 256, 7, 0, 1, False, [7, 200], [50, 8], 64, True),
    (2, 1, 32, 3, 256, 5, 2, 1, True, [60, 9, 0, 100], [0, 17, 3, 100], 32, False),
    (9, 5, 128, 4, 400, 100, 0, 0, False, [250], [260], 128, False),
    (2, 2, 128, 2, 400, 64, 0, 0, False, [64, 64], [64, 65], 0, False),
    (40, 1, 128, 4, 64, 1, 0, 0, False, [20, 1], [3, 8], 16, True),
    (1, 8, 256, 2, 4200, 128, 32, 0, True, [128], [4000], 256, False),
]


@pytest.mark.parametrize("H,gq,d,bits,cap,Nr,S,hybrid,paged,kv,ql,rotary,inter", CASES)
def test_append_chunk_is_the_single_appends(H, gq, d, bits, cap, Nr, S, hybrid, paged, kv, ql, rotary, inter):
    rng = np.random.default_rng(H * 1000 + d + bits)
    cap = -(-cap // 32) * 32 if paged else cap
    g, refs = _start(rng, kv, H, d, bits, cap, Nr, S, hybrid, len(kv) * (cap // 32) + 7 if paged else 0)
    table = kvq.rope_table(max(kv) + max(ql) + 1, rotary) if rotary else None
    host = to_np(table) if rotary else None
    for turn in range(2):  # the second run starts from a moved ring
        k, v, q, cu = _runs(rng, ql, H, H * gq, d)
        if turn:
            k, v, q = k[:len(ql)], v[:len(ql)], q[:len(ql)]
            cu = np.arange(len(ql) + 1, dtype=np.int32)
            if rotary:
                table = kvq.rope_table(max(kv) + max(ql) + 2, rotary)
                host = to_np(table)
        at = [np.arange(int(cu[b + 1] - cu[b])) + _held(r) for b, r in enumerate(refs)]
        got = kvq.kvq_append_chunk(g, *(torch.from_numpy(x).to(DEV) for x in (k, v, cu)),
                                   int(max(np.diff(cu))), q=torch.from_numpy(q).to(DEV), rope=table,
                                   interleaved=inter)
        word = kvq.kvq_read_error(g)[1]
        err, _ = _append_ref(refs, k, v, cu, host, rotary, inter)
        assert word == (kvq.KVQ_ERRBIT_CAPACITY if err else 0)  # 510 tokens pass 400 + 100 of one case
        want = rotate(q, host, np.concatenate(at), rotary, inter) if rotary else q
        assert np.array_equal(to_np(got).view(np.uint16), want.view(np.uint16))
        for b, r in enumerate(refs):
            assert_cache_equal(g, r, batches=[b])
        n = max(_held(r) for r in refs) + 3
        for flags, dt in ((0, np.float16), (kvq.KVQ_OUT_F32, np.float32)):
            for first in (None, torch.tensor([max(0, _held(r) - 9) for r in refs], dtype=torch.int32, device=DEV)):
                kk, vv = kvq.kvq_read_tokens(g, first, n, flags=flags)
                for b, r in enumerate(refs):
                    f = 0 if first is None else int(first[b])
                    for x, got_x in (("k", kk), ("v", vv)):
                        x = tokens_of(r, x, b=0)[:, f:].astype(np.float32).astype(dt)
                        y = to_np(got_x[b])
                        assert np.array_equal(y[:, :x.shape[1]], x) and not y[:, x.shape[1]:].any()


def test_append_chunk_of_one_token_is_append():
    rng = np.random.default_rng(3)
    g, _ = _start(rng, [40, 9], 4, 128, 4, 64, 16, 0, 0, 0)
    g2, _ = _start(np.random.default_rng(3), [40, 9], 4, 128, 4, 64, 16, 0, 0, 0)
    for _ in range(20):
        k, v, _, cu = _runs(rng, [1, 1], 4, 4, 128)
        k, v, cu = (torch.from_numpy(x).to(DEV) for x in (k, v, cu))
        kvq.kvq_append_chunk(g, k, v, cu, 1)
        kvq.kvq_append(g2, k, v)
        for name in ("k_codes", "v_codes", "k_params", "v_params", "k_res", "v_res", "counters"):
            assert torch.equal(getattr(g, name), getattr(g2, name)), name


@pytest.mark.parametrize("ql", [[6, 40], [300, 2]])  # one block per sequence; rows in one line
def test_append_chunk_drops_what_does_not_fit(ql):
    rng = np.random.default_rng(4)
    H, d, cap, Nr = 2, 128, 64, 8
    g, refs = _start(rng, [66, 40], H, d, 4, cap, Nr, 0, 0, 0)
    k, v, q, cu = _runs(rng, ql, H, H, d)
    table = kvq.rope_table(1000, 128)
    got = kvq.kvq_append_chunk(g, *(torch.from_numpy(x).to(DEV) for x in (k, v, cu)), max(ql),
                               q=torch.from_numpy(q).to(DEV), rope=table)
    assert kvq.kvq_read_error(g)[1] == kvq.KVQ_ERRBIT_CAPACITY
    pos = np.concatenate([_held(r) + np.arange(n) for r, n in zip(refs, ql)])
    err, _ = _append_ref(refs, k, v, cu, to_np(table), 128, False)
    assert err
    for b, r in enumerate(refs):
        assert_cache_equal(g, r, batches=[b])
    assert np.array_equal(to_np(got), rotate(q, to_np(table), pos, 128, False))


@pytest.mark.parametrize("ql", [[5, 9], [200, 150]])
def test_append_chunk_reads_a_fused_projection_in_place(ql):
    """Keys, values and queries as columns of one projection output, positions given,
    queries rotated in place, rows of no run (before, between, after) left as they were."""
    rng = np.random.default_rng(6)
    H, gq, d, Nr = 2, 3, 128, 16
    g, refs = _start(rng, [30, 77], H, d, 4, 512, Nr, 0, 0, 0)
    Hq = H * gq
    total = sum(ql) + 11
    cu = np.array([2, 2 + ql[0], 2 + sum(ql)], np.int32)
    qkv = torch.from_numpy(rng.standard_normal((total, (Hq + 2 * H) * d)).astype(np.float16)).to(DEV)
    heads = qkv.view(total, Hq + 2 * H, d)
    k, v = heads[:, Hq:Hq + H], heads[:, Hq + H:]
    pos = rng.integers(0, 5000, total).astype(np.int32)
    table = kvq.rope_table(5000, d)
    q = heads[:, :Hq].contiguous()
    before, cache_before = to_np(q).copy(), to_np(qkv).copy()
    got = kvq.kvq_append_chunk(g, k, v, torch.from_numpy(cu).to(DEV), max(ql), q=q, q_out=q, rope=table,
                               positions=torch.from_numpy(pos).to(DEV))
    assert got is q and kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)
    err, _ = _append_ref(refs, to_np(k), to_np(v), cu, to_np(table), d, False, pos)
    assert err == 0
    for b, r in enumerate(refs):
        assert_cache_equal(g, r, batches=[b])
    want = rotate(before, to_np(table), pos, d, False)
    want[:2], want[cu[2]:] = before[:2], before[cu[2]:]
    assert np.array_equal(to_np(q), want)
    assert np.array_equal(to_np(qkv), cache_before)
    # queries read where they are (strided), rotated into another tensor
    g2, _ = _start(np.random.default_rng(6), [30, 77], H, d, 4, 512, Nr, 0, 0, 0)
    out = torch.full((total, Hq, d), 7.0, dtype=torch.float16, device=DEV)
    kvq.kvq_append_chunk(g2, k, v, torch.from_numpy(cu).to(DEV), max(ql), q=heads[:, :Hq], q_out=out,
                         rope=table, positions=torch.from_numpy(pos).to(DEV))
    want[:2], want[cu[2]:] = 7.0, 7.0
    assert np.array_equal(to_np(out), want)


def test_append_chunk_flags_bad_runs_positions_and_pages():
    rng = np.random.default_rng(8)
    H, d, Nr = 2, 64, 4
    for big in (1, 200):  # both launch forms
        g, refs = _start(rng, [30, 30, 30], H, d, 4, 512, Nr, 0, 0, 0)
        k, v, q, _ = _runs(rng, [2, 3, big], H, H, d)
        dev = [torch.from_numpy(x).to(DEV) for x in (k, v, q)]
        table = kvq.rope_table(20, d)  # every position is past its end: the last row serves
        # sequence 1 ends before it begins, sequence 2 passes the rows there are
        cu = torch.tensor([0, 2, 1, 10 ** 6], dtype=torch.int32, device=DEV)
        kvq.kvq_append_chunk(g, dev[0], dev[1], cu, big, q=dev[2], rope=table)
        word = kvq.kvq_read_error(g)[1]
        assert word == kvq.KVQ_ERRBIT_BADLEN | (0 if big == 1 else kvq.KVQ_ERRBIT_BADPOS)
        if big == 1:  # a run of two is longer than max_len
            assert g.counters[0].tolist() == [26, 26, 26]
            continue
        _append_ref(refs[:1], k, v, np.array([0, 2]), to_np(table), d, False)
        for b, r in enumerate(refs):
            assert_cache_equal(g, r, batches=[b])
    g, _ = _start(rng, [60, 60], H, d, 4, 512, Nr, 0, 0, 40)
    g.block_table[1, 2] = 40  # tokens 64 .. 95 of sequence 1
    pool = g.k_codes.clone()
    k, v, q, cu = _runs(rng, [10, 30], H, H, d)
    kvq.kvq_append_chunk(g, *(torch.from_numpy(x).to(DEV) for x in (k, v, cu)), 30)
    assert kvq.kvq_read_error(g)[1] == kvq.KVQ_ERRBIT_BADPAGE
    assert g.counters[0].tolist() == [66, 86]
    changed = {int(p) for p in (pool != g.k_codes).flatten(1).any(1).nonzero().flatten()}
    assert changed <= {int(g.block_table[b, j]) for b, j in ((0, 1), (0, 2), (1, 1))}
    kk, _ = kvq.kvq_read_tokens(g, None, 100)
    assert kvq.kvq_read_error(g)[1] == kvq.KVQ_ERRBIT_BADPAGE
    assert not kk[1, :, 64:86].any() and kk[1, :, 63].any() and kk[1, :, 86:90].any()
    first = torch.tensor([-1, 0], dtype=torch.int32, device=DEV)
    kk, _ = kvq.kvq_read_tokens(g, first, 4)
    assert kvq.kvq_read_error(g)[1] == kvq.KVQ_ERRBIT_BADLEN
    assert not kk[0].any() and kk[1].any()


def test_append_and_read_replay_in_a_graph_and_run_on_another_stream():
    rng = np.random.default_rng(9)
    H, d, Nr = 2, 128, 16
    g, refs = _start(rng, [40, 90], H, d, 4, 512, Nr, 0, 0, 0)
    k, v, q, cu = _runs(rng, [3, 5], H, 2 * H, d)
    dk, dv, dq, dcu = (torch.from_numpy(x).to(DEV) for x in (k, v, q, cu))
    table = kvq.rope_table(500, d)
    out, (ko, vo) = torch.empty_like(dq), kvq.kvq_read_tokens(g, None, 200)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kvq.kvq_append_chunk(g, dk, dv, dcu, 5, q=dq, q_out=out, rope=table)
        kvq.kvq_read_tokens(g, None, 200, ko, vo)
    for turn in range(3):
        k2 = (rng.standard_normal(k.shape) * (turn + 1)).astype(np.float16)
        dk.copy_(torch.from_numpy(k2))
        graph.replay()
        _append_ref(refs, k2, v, cu, to_np(table), d, False)
    torch.cuda.synchronize()
    for b, r in enumerate(refs):
        assert_cache_equal(g, r, batches=[b])
        x = tokens_of(r, "k", 0).astype(np.float32).astype(np.float16)
        assert np.array_equal(to_np(ko[b, :, :x.shape[1]]), x)
