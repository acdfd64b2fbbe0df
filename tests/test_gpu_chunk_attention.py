"""kvq_chunk_attention and kvq_cross_attention against plain attention in 64 bits over
the oracle's cache: every value within the bound that the kernel's roundings allow
(_runs.attend), and, on normal data, a relative L2 error of at most 1e-3: a rounding to
fp16 is about 2e-4 off in the root mean square, and keys (through the score, twice that
at most here), weights, values and the output are rounded once each."""

import numpy as np
import pytest
import torch

from bit_quantized_kv_pack_gb300 import kvq

from _runs import attend, tokens_of
from _util import gpu_cache, oracle_sequences, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _cache(rng, lens, H, d, bits, cap, Nr, S, hybrid, paged, scale=1.0, k=None, v=None):
    B, Lmax = len(lens), max(max(lens), 1)
    if k is None:
        k = (rng.standard_normal((B, H, Lmax, d)) * scale).astype(np.float16)
    if v is None:
        v = rng.standard_normal((B, H, Lmax, d)).astype(np.float16)
    seq = np.array(lens, np.int32)
    g = gpu_cache(B, H, d, bits, cap, Nr, sink=S, hybrid=hybrid,
                  pages=B * (cap // 32) + 5 if paged else 0, seed=3)
    kvq.kvq_quantize_pack(g, torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV),
                          torch.from_numpy(seq).to(DEV))
    assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)
    return g, oracle_sequences(k, v, seq, bits, cap, Nr, S, hybrid)


def _want(refs, q, cu, causal):
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for b, r in enumerate(refs):
        lo, hi = int(cu[b]), int(cu[b + 1])
        k, v = tokens_of(r, "k", 0), tokens_of(r, "v", 0)
        n, T = k.shape[1], hi - lo
        seen = [n - T + i + 1 if causal else n for i in range(T)]
        out[lo:hi], bound[lo:hi] = attend(k, v, q[lo:hi].astype(np.float64), seen)
    return out, bound


def _check(got, want, bound, rel=1e-3):
    o = to_np(got.float()).astype(np.float64)
    assert np.isfinite(o).all()
    worst = float((np.abs(o - want) / bound).max()) if o.size else 0.0
    l2 = float(np.linalg.norm(o - want) / max(np.linalg.norm(want), 1e-300))
    assert worst <= 1.0, f"off by {worst:.2f} times the bound (rel L2 {l2:.2e})"
    assert rel is None or l2 <= rel, l2
    return l2


def _call(g, q, cu, causal, **kw):
    f = kvq.kvq_chunk_attention if causal else kvq.kvq_cross_attention
    return f(g, torch.from_numpy(q).to(DEV), torch.from_numpy(cu).to(DEV),
             int(max(np.diff(cu))), **kw)


CASES = [  # H, gq, d, bits, cap, Nr, S, hybrid, paged, cache lengths, run lengths
    (2, 4, 128, 4, 700, 16, 0, 0, False, [700, 1, 129], [5, 1, 40]),
    (2, 4, 128, 2, 704, 16, 4, 0, True, [700, 33, 128], [70, 33, 0]),
    (1, 3, 128, 3, 640, 130, 0, 0, False, [640, 200], [130, 200]),
    (1, 1, 64, 4, 1500, 0, 0, 0, False, [1500, 1, 64, 65], [300, 1, 64, 2]),
    (3, 2, 64, 3, 512, 33, 32, 1, True, [500, 70], [129, 12]),
    (2, 1, 64, 2, 512, 1, 0, 0, True, [511, 256], [257, 128]),
    (2, 3, 256, 4, 400, 20, 0, 0, False, [400, 64, 65], [100, 64, 3]),
    (1, 8, 256, 2, 384, 8, 2, 1, True, [300], [33]),
    (1, 1, 256, 3, 300, 0, 0, 0, False, [300, 5], [300, 5]),
    (2, 5, 32, 4, 500, 64, 0, 0, False, [500, 100], [60, 100]),
    (1, 16, 32, 3, 320, 0, 3, 0, True, [320], [40]),
    (4, 1, 32, 2, 260, 5, 0, 0, False, [260, 250, 1], [1, 200, 1]),
    (1, 71, 64, 4, 200, 10, 0, 0, False, [200], [9]),
    (5, 1, 128, 4, 2100, 128, 0, 0, False, [2000], [600]),
    (1, 4, 128, 2, 9000, 0, 0, 0, True, [8999], [3]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,gq,d,bits,cap,Nr,S,hybrid,paged,kv,ql", CASES)
def test_attention_of_runs(H, gq, d, bits, cap, Nr, S, hybrid, paged, kv, ql, causal):
    rng = np.random.default_rng(H * 100 + gq + d + bits)
    cap = -(-cap // 32) * 32 if paged else cap
    g, refs = _cache(rng, kv, H, d, bits, cap, Nr, S, hybrid, paged)
    cu = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
    q = rng.standard_normal((int(cu[-1]), H * gq, d)).astype(np.float16)
    want, bound = _want(refs, q, cu, causal)
    ws = kvq.chunk_workspace_for(g, H * gq)
    a = _call(g, q, cu, causal, workspace=ws)
    _check(a, want, bound)
    b = _call(g, q, cu, causal, workspace=ws)
    assert torch.equal(a, b), "the same call twice differs"
    c = _call(g, q, cu, causal, workspace=ws, flags=kvq.KVQ_OUT_F32)
    assert c.dtype == torch.float32
    _check(c, want, bound)
    assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)


def test_many_short_sequences():
    """More units than blocks, lengths of zero and one among them."""
    rng = np.random.default_rng(1)
    B, H, gq, d = 96, 4, 2, 64
    kv = [int(x) for x in rng.integers(1, 300, B)]
    ql = [int(x) for x in rng.integers(0, 5, B)]
    ql = [min(a, b) for a, b in zip(ql, kv)]
    g, refs = _cache(rng, kv, H, d, 4, 320, 32, 0, 0, False)
    cu = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
    q = rng.standard_normal((int(cu[-1]), H * gq, d)).astype(np.float16)
    for causal in (True, False):
        _check(_call(g, q, cu, causal), *_want(refs, q, cu, causal))
    assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)


@pytest.mark.parametrize("d,bits", [(128, 4), (64, 2), (256, 4), (32, 3)])
def test_rows_with_nothing_to_attend_over(d, bits):
    """A run longer than its cache (its first rows see nothing), an empty cache, and no
    run at all: zeros and KVQ_ERRBIT_EMPTY, other rows as ever."""
    rng = np.random.default_rng(2)
    H, gq = 2, 2
    kv, ql = [10, 0, 50, 0], [25, 3, 4, 0]
    g, refs = _cache(rng, kv, H, d, bits, 64, 8, 0, 0, False)
    cu = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
    q = rng.standard_normal((int(cu[-1]), H * gq, d)).astype(np.float16)
    for causal in (True, False):
        got = _call(g, q, cu, causal)
        assert kvq.kvq_read_error(g)[1] == kvq.KVQ_ERRBIT_EMPTY
        want, bound = _want(refs, q, cu, causal)
        _check(got, want, bound)
        assert not got[25:28].any() and (not causal or not got[:15].any())
    assert _call(g, q[:0], np.zeros(5, np.int32), True).shape == (0, H * gq, d)
    assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_large_scores_and_values(d):
    """Scores of hundreds, where one token takes all the weight, a maximum that keeps
    rising along the sequence, and groups up to fp16's largest value."""
    rng = np.random.default_rng(5)
    H, gq, n = 1, 4, 900
    k = rng.standard_normal((1, H, n, d)).astype(np.float16)
    k *= np.linspace(0.1, 16, n, dtype=np.float16)[:, None]
    v = rng.standard_normal((1, H, n, d)).astype(np.float16)
    v[0, 0, 300] *= 20000
    v[0, 0, 301, :32] = 65504
    v[0, 0, 302, :32] = np.where(np.arange(32) % 2, 65504, -65504)
    g, refs = _cache(rng, [n], H, d, 4, 1000, 16, 0, 0, False, k=k, v=v)
    cu = np.array([0, 60], np.int32)
    q = (rng.standard_normal((60, H * gq, d)) * 3).astype(np.float16)
    for causal in (True, False):
        want, bound = _want(refs, q, cu, causal)
        _check(_call(g, q, cu, causal, flags=kvq.KVQ_OUT_F32), want, bound, rel=None)


@pytest.mark.parametrize("d,bits,Nr", [(128, 4, 40), (128, 4, 0), (64, 2, 0), (256, 3, 16), (32, 4, 8),
                                       (128, 2, 16), (128, 3, 0), (256, 2, 0), (256, 4, 16), (64, 3, 8)])
def test_hidden_tokens_have_no_part(d, bits, Nr):
    """Infinities and NaN in tokens that a row does not see: the run's later tokens, and
    memory past the sequence's end (packed rows, ring slots).  The rows that see an
    infinite value get it."""
    rng = np.random.default_rng(7)
    H, gq, n, T = 2, 2, 230, 40
    k = rng.standard_normal((1, H, n, d)).astype(np.float16)
    v = rng.standard_normal((1, H, n, d)).astype(np.float16)
    g, refs = _cache(rng, [n], H, d, bits, 256, Nr, 0, 0, False, k=k, v=v)
    cu = np.array([0, T], np.int32)
    q = rng.standard_normal((T, H * gq, d)).astype(np.float16)
    want, bound = _want(refs, q, cu, True)
    bad = n - T + 25  # token 25 of the run, in the window or packed
    npk = int(g.packed_len[0])
    nan = 0x7E007E00
    for x, name in ((g.k_params, "k"), (g.v_params, "v")):
        x[0, :, npk:] = nan
        if bad < npk:
            x[0, :, bad] = nan
    for x in (g.k_res, g.v_res):
        if bad >= npk:
            x[0, :, bad - npk] = float("nan")
    got = _call(g, q, cu, True)
    o = to_np(got)
    assert np.isnan(o[25:]).all()
    _check(got[:25], want[:25], bound[:25])
    # an infinite value in one column only: +inf for rows that see it, others finite
    g, refs = _cache(rng, [n], H, d, bits, 256, Nr, 0, 0, False, k=k, v=v)
    if bad >= npk:
        g.v_res[0, 1, bad - npk, 5] = float("inf")
        o = to_np(_call(g, q, cu, True))
        assert np.isposinf(o[25:, gq:, 5]).all()
        o[25:, gq:, 5] = want[25:, gq:, 5]
        _check(torch.from_numpy(o), want, bound)


def test_rows_of_no_run_and_bad_runs_are_left_as_they_were():
    rng = np.random.default_rng(8)
    H, gq, d = 2, 4, 128
    g, refs = _cache(rng, [300, 200, 100], H, d, 4, 320, 16, 0, 0, False)
    q = rng.standard_normal((50, H * gq, d)).astype(np.float16)
    out = torch.full((50, H * gq, d), 3.0, dtype=torch.float16, device=DEV)
    cu = np.array([4, 14, 14, 30], np.int32)
    got = kvq.kvq_chunk_attention(g, torch.from_numpy(q).to(DEV), torch.from_numpy(cu).to(DEV), 20, out=out)
    assert got is out and kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)
    want, bound = _want(refs, q, cu, True)
    _check(out[4:30], want[4:30], bound[4:30])
    assert (out[:4] == 3).all() and (out[30:] == 3).all()
    # sequence 0 is longer than max_len, sequence 2 ends past the rows there are
    out.fill_(3.0)
    bad = np.array([0, 30, 40, 51], np.int32)
    kvq.kvq_chunk_attention(g, torch.from_numpy(q).to(DEV), torch.from_numpy(bad).to(DEV), 20, out=out)
    assert kvq.kvq_read_error(g)[1] == kvq.KVQ_ERRBIT_BADLEN
    want, bound = _want([refs[1]], q[30:40], np.array([0, 10]), True)
    _check(out[30:40], want, bound)
    assert (out[:30] == 3).all() and (out[40:] == 3).all()


@pytest.mark.parametrize("d", [64, 128])
def test_bad_pages_are_left_out(d):
    rng = np.random.default_rng(9)
    H, gq, n = 1, 2, 300
    g, refs = _cache(rng, [n, n], H, d, 4, 320, 8, 0, 0, True)
    g.block_table[0, 3] = -5  # packed tokens 96 .. 127
    g.block_table[0, 4] = 10 ** 6  # 128 .. 159
    cu = np.array([0, 20, 40], np.int32)
    q = rng.standard_normal((40, H * gq, d)).astype(np.float16)
    for causal in (True, False):
        got = _call(g, q, cu, causal)
        assert kvq.kvq_read_error(g)[1] == kvq.KVQ_ERRBIT_BADPAGE
        want, bound = _want(refs, q, cu, causal)
        _check(got[20:], want[20:], bound[20:])
        keep = np.r_[0:96, 160:n]
        k, v = tokens_of(refs[0], "k", 0)[:, keep], tokens_of(refs[0], "v", 0)[:, keep]
        seen = [n - 64 - (20 - i - 1 if causal else 0) for i in range(20)]
        want, bound = attend(k, v, q[:20].astype(np.float64), seen)
        _check(got[:20], want, bound)


def test_one_token_runs_match_decode():
    rng = np.random.default_rng(10)
    H, gq, d = 8, 4, 128
    g, _ = _cache(rng, [1000, 400, 77], H, d, 4, 1024, 128, 32, 0, False)
    q = rng.standard_normal((3, H * gq, d)).astype(np.float16)
    a = _call(g, q, np.arange(4, dtype=np.int32), True, flags=kvq.KVQ_OUT_F32)
    b = kvq.kvq_decode_attention(g, torch.from_numpy(q).to(DEV), flags=kvq.KVQ_OUT_F32)
    # both are within 2e-3 of the 64-bit result
    assert (a - b).abs().max().item() <= 4e-3


def test_append_then_attend_as_in_serving():
    """A prompt in three pieces and then drafts, through append and attention on one
    workspace, captured in a graph and replayed on a side stream."""
    rng = np.random.default_rng(11)
    H, gq, d, Nr, bits = 2, 4, 128, 32, 4
    start = [64, 20]
    g, refs = _cache(rng, start, H, d, bits, 1024, Nr, 4, 0, True)
    import oracle
    from _runs import rotate
    table = kvq.rope_table(2000, d)
    ws = kvq.chunk_workspace_for(g, H * gq)
    side = torch.cuda.Stream()
    for ql in ([200, 33], [1, 128], [5, 3], [2, 0]):
        total = sum(ql)
        k = rng.standard_normal((total, H, d)).astype(np.float16)
        v = rng.standard_normal((total, H, d)).astype(np.float16)
        q = rng.standard_normal((total, H * gq, d)).astype(np.float16)
        cu = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
        dk, dv, dq, dcu = (torch.from_numpy(x).to(DEV) for x in (k, v, q, cu))
        qr, out = torch.empty_like(dq), torch.empty_like(dq)
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kvq.kvq_append_chunk(g, dk, dv, dcu, max(ql), q=dq, q_out=qr, rope=table)
            kvq.kvq_chunk_attention(g, qr, dcu, max(ql), out=out, workspace=ws)
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)
        for b, r in enumerate(refs):
            n = int(r.packed_len[0] + r.res_len[0] + r.sink_len[0])
            rows = slice(int(cu[b]), int(cu[b + 1]))
            kr = rotate(k[rows], to_np(table), n + np.arange(ql[b]), d, False)
            for t in range(ql[b]):
                assert oracle.append(r, kr[t][None], v[rows][t][None]) == 0
        want, bound = _want(refs, to_np(qr), cu, True)
        _check(out, want, bound)


def test_long_cache_offsets_pass_32_bits():
    """Code rows whose byte offsets pass 2^32: 70 sequences of a large capacity, the last
    one's rows read where they are."""
    H, gq, d, cap = 8, 1, 128, 131072
    B = 70
    g = kvq.KVCache(B, H, d, 4, cap, 0)
    assert g.k_codes.numel() > 2 ** 32
    rng = np.random.default_rng(12)
    k = rng.standard_normal((1, H, 500, d)).astype(np.float16)
    v = rng.standard_normal((1, H, 500, d)).astype(np.float16)
    r = oracle_sequences(k, v, np.array([500], np.int32), 4, 512, 0)[0]
    for name in ("k_codes", "v_codes", "k_params", "v_params"):
        x = torch.from_numpy(getattr(r, name)[0, :, :500].view(np.int32 if "params" in name else np.uint8))
        getattr(g, name)[B - 1, :, :500] = x.to(DEV)
    g.counters[0, B - 1] = 500
    cu = np.zeros(B + 1, np.int32)
    cu[-1] = 6
    q = rng.standard_normal((6, H * gq, d)).astype(np.float16)
    got = _call(g, q, cu, True)
    want, bound = _want([r], q, np.array([0, 6]), True)
    _check(got, want, bound)
    kk, _ = kvq.kvq_read_tokens(g, None, 8)
    assert np.array_equal(to_np(kk[-1]), tokens_of(r, "k", 0)[:, :8].astype(np.float32).astype(np.float16))
    dk = torch.from_numpy(k[0, :, :6].transpose(1, 0, 2).copy()).to(DEV)
    kvq.kvq_append_chunk(g, dk, dk, torch.from_numpy(cu).to(DEV), 6)
    kk, _ = kvq.kvq_read_tokens(g, torch.full((B,), 500, dtype=torch.int32, device=DEV), 6)
    assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)
    # the same six tokens quantize as they did at the start
    assert np.array_equal(to_np(kk[-1]), tokens_of(r, "k", 0)[:, :6].astype(np.float32).astype(np.float16))
