"""Calls on runs as a serving program makes them: one workspace, whatever it holds, for
calls of any shape; calls on two streams; graphs that share a workspace; a bounded wait
that runs out; the smallest calls.  Outputs are compared bit for bit with the same call
made alone: results do not depend on timing or on what a workspace held."""

import numpy as np
import pytest
import torch

from bit_quantized_kv_pack_gb300 import kvq

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _make(rng, lens, ql, H, gq, d, bits, page=0, Nr=16):
    B, cap = len(lens), -(-max(lens) // 32) * 32 + 32
    g = kvq.KVCache(B, H, d, bits, cap, Nr, page_size=page, num_pages=B * cap // 32 if page else 0)
    k, v = (torch.from_numpy(rng.standard_normal((B, H, max(lens), d)).astype(np.float16)).to(DEV)
            for _ in range(2))
    kvq.kvq_quantize_pack(g, k, v, torch.tensor(lens, dtype=torch.int32, device=DEV))
    q = torch.from_numpy(rng.standard_normal((sum(ql), H * gq, d)).astype(np.float16)).to(DEV)
    cu = torch.tensor([0] + list(np.cumsum(ql)), dtype=torch.int32, device=DEV)
    return g, q, cu, max(ql)


SHAPES = [  # cache lengths, run lengths, H, gq, d, bits, page
    ([5000, 33], [5, 30], 4, 4, 128, 4, 0),
    ([700, 1500, 64], [300, 7, 64], 2, 2, 64, 3, 32),
    ([900], [200], 3, 1, 256, 2, 0),
    ([2000], [1], 1, 8, 128, 2, 32),
    ([300] * 40, [3] * 40, 2, 4, 32, 4, 0),
]


def test_one_workspace_serves_calls_of_any_shape_whatever_it_holds():
    rng = np.random.default_rng(21)
    calls = [_make(rng, *s) for s in SHAPES]
    ws = torch.empty(max(kvq.kvq_chunk_workspace_bytes(g.desc, q.shape[1]) for g, q, _, _ in calls),
                     dtype=torch.uint8, device=DEV)
    alone = []
    for g, q, cu, n in calls:
        own = torch.zeros(kvq.kvq_chunk_workspace_bytes(g.desc, q.shape[1]), dtype=torch.uint8, device=DEV)
        alone.append([f(g, q, cu, n, workspace=own) for f in (kvq.kvq_chunk_attention, kvq.kvq_cross_attention)])
    for fill in (0xFF, 0x7F, None):  # NaN, large values and indices, what the last call left
        for order in (range(len(calls)), reversed(range(len(calls)))):
            for i in order:
                g, q, cu, n = calls[i]
                for f, want in zip((kvq.kvq_chunk_attention, kvq.kvq_cross_attention), alone[i]):
                    if fill is not None:
                        ws.fill_(fill)
                    assert torch.equal(f(g, q, cu, n, workspace=ws), want)
    for g, _, _, _ in calls:
        assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)


def test_calls_on_two_streams_and_graphs_that_share_a_workspace():
    rng = np.random.default_rng(22)
    a, b = _make(rng, *SHAPES[0]), _make(rng, *SHAPES[1])
    want = [kvq.kvq_chunk_attention(*x) for x in (a, b)]
    ws = [kvq.chunk_workspace_for(x[0], x[1].shape[1]) for x in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.empty_like(w) for _ in range(20)] for w in want]
    torch.cuda.synchronize()
    for i in range(20):
        for s in range(2):
            x = (a, b)[s]
            kvq.kvq_chunk_attention(*x, out=outs[s][i], workspace=ws[s], stream=streams[s])
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for os, w in zip(outs, want) for o in os)
    # two graphs over one workspace, replayed in turn on one stream
    big = max(ws, key=lambda w: w.numel())
    graphs, got = [], [torch.empty_like(w) for w in want]
    for x, o in zip((a, b), got):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[0]):
            kvq.kvq_chunk_attention(*x, out=o, workspace=big)
        graphs.append(g)
    with torch.cuda.stream(streams[0]):
        for _ in range(5):
            for o in got:
                o.zero_()
            for g in graphs:
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(got, want))
    for x in (a, b):
        assert kvq.kvq_read_error(x[0]) == (kvq.KVQ_OK, 0)


@pytest.mark.parametrize("shape", SHAPES)
def test_wait_that_runs_out_is_reported_and_the_next_call_is_right(shape):
    rng = np.random.default_rng(23)
    g, q, cu, n = _make(rng, *shape)
    ws = kvq.chunk_workspace_for(g, q.shape[1])
    want = kvq.kvq_chunk_attention(g, q, cu, n, workspace=ws)
    assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)
    kvq.kvq_testing_wait_fault(2000)
    try:
        kvq.kvq_chunk_attention(g, q, cu, n, workspace=ws)
        st, word = kvq.kvq_read_error(g)
    finally:
        kvq.kvq_testing_wait_fault(0)
    assert word & kvq.KVQ_ERRBIT_TIMEOUT
    for _ in range(2):
        assert torch.equal(kvq.kvq_chunk_attention(g, q, cu, n, workspace=ws), want)
        assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)


def test_calls_without_rows_or_with_runs_past_max_len():
    rng = np.random.default_rng(24)
    g, q, cu, n = _make(rng, *SHAPES[0])
    none = torch.zeros(3, dtype=torch.int32, device=DEV)
    for f in (kvq.kvq_chunk_attention, kvq.kvq_cross_attention):
        assert f(g, q[:0], none, 0).shape == (0,) + q.shape[1:]
        out = torch.full_like(q, 7.0)
        f(g, q, none, n, out=out)  # rows, and no run that has them
        assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0) and bool((out == 7.0).all())
        f(g, q, cu, 0, out=out)  # runs longer than max_len
        assert kvq.kvq_read_error(g)[1] == kvq.KVQ_ERRBIT_BADLEN and bool((out == 7.0).all())
    k = q[:, :4].contiguous()
    held = g.counters.clone()
    kvq.kvq_append_chunk(g, k, k, cu, 0)
    assert kvq.kvq_read_error(g)[1] == kvq.KVQ_ERRBIT_BADLEN and torch.equal(g.counters, held)
    kvq.kvq_append_chunk(g, k[:0], k[:0], none, 0)
    assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0) and torch.equal(g.counters, held)
    kk, vv = kvq.kvq_read_tokens(g, None, 0)
    assert kk.shape == vv.shape == (2, 4, 0, 128)


def test_arguments_of_another_shape_type_or_device_are_refused():
    rng = np.random.default_rng(25)
    g, q, cu, n = _make(rng, *SHAPES[0])
    small = torch.empty(64, dtype=torch.uint8, device=DEV)
    with pytest.raises(kvq.KvqError):
        kvq.kvq_chunk_attention(g, q, cu, n, workspace=small)
    for bad in (cu.cpu(), cu.long(), cu[:-1]):
        with pytest.raises(ValueError, match="cu_seqlens"):
            kvq.kvq_chunk_attention(g, q, bad, n)
    for bad in (q.cpu(), q.float(), q.transpose(0, 1), q[..., :64]):
        with pytest.raises(ValueError):
            kvq.kvq_cross_attention(g, bad, cu, n)
    with pytest.raises(ValueError):
        kvq.kvq_chunk_attention(g, q, cu, n, out=torch.empty_like(q)[:-1])
    with pytest.raises(ValueError):
        kvq.kvq_read_tokens(g, cu, 4)  # B + 1 entries
    assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)
