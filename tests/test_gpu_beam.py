"""Beam search's selection against a plain one in 64 bits: log-softmax, scores added, all
proposals sorted, equal ones in the order of (beam, token)."""

import numpy as np
import pytest
import torch

from bit_quantized_kv_pack_gb300 import kvq

from _util import gpu_cache, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"


def plain(x, scores, n, finished=None, end=0):
    """(parent, token, score) [B][n] of logits [B][W][V], and each row's largest logit."""
    B, W, V = x.shape
    x = x.astype(np.float64)
    s = np.full((B, W, V), -np.inf)
    for b in range(B):
        for w in range(W):
            base = np.float64(scores[b, w])
            if not base < np.inf:
                continue
            if finished is not None and finished[b, w]:
                s[b, w, end] = base
                continue
            r = x[b, w]
            if np.isnan(r).any() or (r == np.inf).any() or not (r > -np.inf).any():
                continue
            m = r.max()
            s[b, w] = base + (r - (m + np.log(np.exp(r - m).sum())))
    flat = s.reshape(B, W * V)
    at = np.argsort(-flat, axis=1, kind="stable")[:, :n]
    return np.arange(B)[:, None] * W + at // V, at % V, np.take_along_axis(flat, at, 1)


def check(x, scores, n, finished=None, end=0, want_bits=0, **kw):
    g = gpu_cache(1, 1, 32, 4, 32, 0)
    t = x if torch.is_tensor(x) else torch.from_numpy(x).to(DEV)
    f = None if finished is None else torch.from_numpy(finished).to(DEV)
    parent, token, score = kvq.kvq_beam_select(t, torch.from_numpy(scores).to(DEV), n, finished=f, end_token=end,
                                               err=g.err, **kw)
    assert kvq.kvq_read_error(g)[1] == want_bits
    p, t_, s = plain(to_np(t), scores, n, finished, end)
    assert np.array_equal(to_np(token), t_), (to_np(token), t_)
    assert np.array_equal(to_np(parent), p)
    got = to_np(score).astype(np.float64)
    live = np.isfinite(s)
    assert np.array_equal(live, np.isfinite(got))
    # the sum's 2^-20 becomes as much of its logarithm, and the score is rounded once
    assert (np.abs(got[live] - s[live]) <= 2.0 ** -20 + 2.0 ** -24 * np.abs(s[live])).all()
    return parent, token, score


@pytest.mark.parametrize("B,W,V,n", [
    (1, 1, 1, 1), (1, 1, 7, 7), (2, 3, 5, 15), (1, 4, 33, 8), (3, 2, 1000, 4), (1, 4, 32000, 4), (2, 5, 50257, 10),
    (1, 32, 777, 32), (5, 7, 8191, 14), (1, 16, 24577, 32), (40, 8, 25001, 16), (1, 3, 200003, 32), (100, 1, 501, 3),
])
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_selection(B, W, V, n, dtype):
    rng = np.random.default_rng(V + W)
    x = (rng.standard_normal((B, W, V)) * 3).astype(dtype)
    check(x, (-10 * rng.random((B, W))).astype(np.float32), n)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("V", [8, 31, 127, 255, 257, 511, 769, 1002, 1025, 1793, 2047, 2049, 8193])
def test_short_rows_and_many_proposals(V, dtype):
    rng = np.random.default_rng(V)
    x = (rng.standard_normal((20, 16, V)) * 3).astype(dtype)
    x[0] = -np.sort(-x[0], axis=-1)                   # the largest side by side
    x[1, :, :V // 2] = -np.inf
    check(x, (-10 * rng.random((20, 16))).astype(np.float32), 32)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("V", [40, 3001, 60001])
def test_equal_scores_come_in_order(V, dtype):
    rng = np.random.default_rng(V)
    zero = np.zeros((2, 4), np.float32)
    check(np.zeros((2, 4, V), dtype), zero, 20)                                  # everything equal
    check(np.full((2, 4, V), -3.0, dtype), zero, 32)
    check((rng.integers(0, 3, (2, 4, V))).astype(dtype), zero, 32)               # a few values
    x = np.repeat((rng.standard_normal((2, 1, V)) * 2).astype(dtype), 4, 1)      # equal beams
    check(x, zero, 12)
    x[..., ::2] = 0.0
    x[..., 1::2] = -0.0                                                          # zeros of both signs
    check(x, zero, 9)


@pytest.mark.parametrize("V", [3001, 60001])
def test_values_in_rising_and_falling_order(V):
    up = np.arange(V, dtype=np.float32)[None, None] / 100
    zero = np.zeros((1, 2), np.float32)
    check(np.concatenate([up, up[..., ::-1]], 1).copy(), zero, 32)
    # the largest ones side by side in one thread's vectors
    x = np.zeros((1, 2, V), np.float32)
    x[0, 0, 1000:1004], x[0, 1, 2048:2056] = (5, 6, 7, 8), 9
    check(x, zero, 12)
    check(x.astype(np.float16), zero, 12)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_banned_tokens_and_beams_without_a_score(dtype):
    rng = np.random.default_rng(11)
    B, W, V = 3, 4, 5003
    x = (rng.standard_normal((B, W, V)) * 2).astype(dtype)
    scores = (-5 * rng.random((B, W))).astype(np.float32)
    x[:, :, rng.permutation(V)[:4000]] = -np.inf
    x[1, 2] = -np.inf                       # a row whose mask leaves nothing
    x[2] = -np.inf                          # a batch entry without a proposal
    x[0, :, :] = np.where(np.arange(V) < V - 3, -np.inf, x[0])  # three tokens left
    x[0, 0, V - 1] = 1.0
    check(x, scores, 20)
    first = np.full((B, W), -np.inf, np.float32)
    first[:, 0] = 0.0
    check((rng.standard_normal((B, W, V))).astype(dtype), first, 4)
    x = (rng.standard_normal((B, W, V))).astype(dtype)
    x[:] = np.finfo(dtype).min              # masks of the type's lowest value
    x[:, :, 17] = 2.0
    check(x, scores, 8)


def test_complete_beams():
    rng = np.random.default_rng(12)
    B, W, V = 4, 5, 900
    x = (rng.standard_normal((B, W, V)) * 2).astype(np.float16)
    scores = (-3 * rng.random((B, W))).astype(np.float32)
    fin = (rng.random((B, W)) < 0.5)
    fin[0], fin[1] = True, False
    x[2, :, :] = np.where(fin[2][:, None], np.nan, x[2].astype(np.float32)).astype(np.float16)  # not looked at
    for end in (0, 3, 451, V - 1):
        check(x, scores, 10, fin, end)
        check(x, scores, 10, fin.astype(np.uint8) * 255, end)
    check(x[:1, :, :2].copy(), scores[:1], 10, fin[:1], 1)  # all proposals there are
    scores[0, 2] = -np.inf
    check(x, scores, 10, fin, 7)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_nan_and_infinity_silence_their_beam_and_are_reported(dtype):
    rng = np.random.default_rng(13)
    x = (rng.standard_normal((2, 4, 30001)) * 2).astype(dtype)
    scores = (-3 * rng.random((2, 4))).astype(np.float32)
    bad = kvq.KVQ_ERRBIT_BADSCORE
    for value in (np.nan, np.inf):
        y = x.copy()
        y[0, 1, 29999] = value
        check(y, scores, 6, want_bits=bad)
        s = scores.copy()
        s[1, 3] = value
        check(x, s, 6, want_bits=bad)
    y = x.copy()
    y[0] = np.nan  # no beam of a batch entry is left
    check(y, scores, 6, want_bits=bad)


def test_rows_apart_and_rows_of_any_alignment():
    rng = np.random.default_rng(14)
    scores = (-3 * rng.random((2, 3))).astype(np.float32)
    for dtype, V, width in ((torch.float16, 1001, 1003), (torch.float16, 777, 800), (torch.float32, 515, 517)):
        wide = torch.full((2, 3, width), float("nan"), dtype=dtype, device=DEV)  # what lies between has no part
        wide[..., :V] = torch.from_numpy(rng.standard_normal((2, 3, V))).to(DEV)
        check(wide[..., :V], scores, 6)
    for dtype in (torch.float16, torch.float32):  # the last token's logits of each row, an odd vocabulary
        steps = torch.from_numpy(rng.standard_normal((4, 3, 1, 2503))).to(DEV).to(dtype)
        for at in (1, 2):
            x = steps[:, at]
            assert x.data_ptr() % 16
            check(x, scores.reshape(6, 1)[:4].copy(), 7)
    with pytest.raises(ValueError, match="one stride"):
        kvq.kvq_beam_select(torch.zeros(2, 4, 8, 50, dtype=torch.float16, device=DEV)[:, :, 1][:, :3],
                            torch.zeros(2, 3, device=DEV), 2)


def test_a_sum_far_below_its_largest_term_and_a_flat_one():
    x = np.full((1, 2, 131072), -8.0, np.float32)
    x[0, 0, 5] = 8.0
    check(x, np.zeros((1, 2), np.float32), 4)


def test_workspace_streams_and_graphs():
    """Any workspace contents; a stream of its own; two graphs that share a workspace."""
    rng = np.random.default_rng(15)
    B, W, V, n = 3, 4, 40001, 8
    xs = [torch.from_numpy((rng.standard_normal((B, W, V)) * 3).astype(np.float16)).to(DEV) for _ in range(2)]
    scores = torch.from_numpy((-3 * rng.random((B, W))).astype(np.float32)).to(DEV)
    ws = kvq.beam_workspace_for(B, W, V, n).fill_(0xFF)
    want = [[t.clone() for t in kvq.kvq_beam_select(x, scores, n, workspace=ws)] for x in xs]
    for x, w in zip(xs, want):
        for got, of in zip(plain(to_np(x), to_np(scores), n)[:2], w[:2]):
            assert np.array_equal(got, to_np(of))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = kvq.kvq_beam_select(xs[0], scores, n, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    outs = [[torch.empty_like(t) for t in want[0]] for _ in xs]
    graphs = []
    for x, o in zip(xs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kvq.kvq_beam_select(x, scores, n, out=o, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))


@pytest.mark.parametrize("end", [0, 1, 5, 9])
def test_complete_beams_without_a_score(end):
    """Nothing of an entry is live: what comes back is the first tokens, at -inf."""
    x = np.random.default_rng(16).standard_normal((3, 2, 10)).astype(np.float32)
    none = np.full((3, 2), -np.inf, np.float32)
    for n in (1, 2, 5, 10, 15):
        check(x, none, n, np.ones((3, 2), bool), end)
        mixed = none.copy()
        mixed[0, 1], mixed[1, 0] = -1.0, -2.0
        check(x, mixed, n, np.ones((3, 2), bool), end)
        check(x[:, :1].copy(), none[:, :1].copy(), min(n, 10), np.ones((3, 1), bool), end)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("V", [50, 5003, 70001])
def test_scores_whose_differences_are_below_their_last_bit(V, dtype):
    """Beams at the type's lowest score: all their proposals are equal in 53 bits.  A beam's
    come in the order of its logits, equal logits in that of their tokens."""
    rng = np.random.default_rng(V)
    B, W, n = 2, 3, 12
    x = np.round(rng.standard_normal((B, W, V)) * 8).astype(dtype) / 8  # with equal ones among the largest
    low = np.finfo(np.float32).min
    scores = np.full((B, W), low, np.float32)
    scores[:, 0] = -1.0
    fin = np.zeros((B, W), bool)
    fin[:, 0] = True
    g = gpu_cache(1, 1, 32, 4, 32, 0)
    parent, token, score = kvq.kvq_beam_select(torch.from_numpy(x).to(DEV), torch.from_numpy(scores).to(DEV), n,
                                               finished=torch.from_numpy(fin).to(DEV), end_token=3, err=g.err)
    assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)
    for b in range(B):
        order = np.argsort(-x[b, 1].astype(np.float64), kind="stable")[:n - 1]
        assert to_np(token)[b].tolist() == [3] + order.tolist()
        assert to_np(parent)[b].tolist() == [b * W] + [b * W + 1] * (n - 1)
        assert to_np(score)[b].tolist() == [-1.0] + [float(low)] * (n - 1)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_near_ties_of_beams(dtype):
    """Beams of the same logits in other places: the scores differ by what the sums' order makes.
    Each normaliser is within 2^-19, so what is left out is no better than what is chosen by more
    than 2^-18; a beam's own proposals come in the order of its logits."""
    rng = np.random.default_rng(21)
    B, W, V, n = 3, 8, 50021, 32
    row = (rng.standard_normal(V) * 3).astype(dtype)
    x = np.stack([[rng.permutation(row) for _ in range(W)] for _ in range(B)])
    scores = (-20 + 1e-6 * rng.standard_normal((B, W))).astype(np.float32)
    parent, token, score = (to_np(t) for t in kvq.kvq_beam_select(torch.from_numpy(x).to(DEV),
                                                                  torch.from_numpy(scores).to(DEV), n))
    x64 = x.astype(np.float64)
    true = scores.astype(np.float64)[..., None] + x64 - np.log(np.exp(x64).sum(-1, keepdims=True))
    for b in range(B):
        w = parent[b] - b * W
        mine = true[b, w, token[b]]
        assert len(set(zip(w, token[b]))) == n
        assert (mine[:-1] - mine[1:] >= -2.0 ** -18).all()
        left = true[b].copy()
        left[w, token[b]] = -np.inf
        assert left.max() <= mine[-1] + 2.0 ** -18
        assert (np.abs(score[b] - mine) <= 2.0 ** -19 + 2.0 ** -24 * np.abs(mine)).all()
        for i in range(W):
            of = token[b][w == i]
            assert of.tolist() == np.argsort(-x64[b, i], kind="stable")[:len(of)].tolist()
