"""Values at the edges of attention of runs: weights far below the largest, infinities and
NaN among seen tokens.  Against plain attention in 64 bits over the cache's own tokens."""

import numpy as np
import pytest
import torch

from bit_quantized_kv_pack_gb300 import kvq

from _runs import attend, tokens_of
from _util import gpu_cache, oracle_sequences, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T", [4, 140])  # the accumulators take turns; they share the tiles
@pytest.mark.parametrize("d,bits", [(64, 4), (128, 2), (256, 3)])
def test_a_long_tail_under_one_dominant_token_keeps_its_mass(d, bits, T):
    """Token 0 outweighs each of 32767 others by e^9 to e^18, values of one sign: the tail's
    part of the output is n times a weight that fp16 alone would not hold.  The weights'
    own rounding: half a step of fp16, or 2^-25 of a weight 2^7 times the row's reference."""
    rng = np.random.default_rng(40 + d)
    H, n = 160, 32768  # more heads than blocks: whole units
    k = torch.zeros(1, H, n, d, dtype=torch.float16, device=DEV)
    k[:, :, 0] = 1.0
    gen = torch.Generator(DEV).manual_seed(d)
    v = (torch.rand(1, H, n, d, generator=gen, device=DEV) + 0.5).half()
    v[:, :, 0] = 0.0
    g = gpu_cache(1, H, d, bits, n, 0)
    kvq.kvq_quantize_pack(g, k, v, torch.tensor([n], dtype=torch.int32, device=DEV))
    nats = np.linspace(9.0, 18.0, T)
    q = np.broadcast_to((nats / np.sqrt(d))[:, None, None], (T, H, d)).astype(np.float16)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    got = to_np(kvq.kvq_cross_attention(g, torch.from_numpy(q).to(DEV), cu, T, flags=kvq.KVQ_OUT_F32))
    assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)
    for h in (0, 1, 77, H - 1):
        r = oracle_sequences(*(to_np(x[:, h:h + 1]) for x in (k, v)), np.array([n], np.int32), bits, n, 0)[0]
        want, bound = attend(tokens_of(r, "k", 0), tokens_of(r, "v", 0), q[:, h:h + 1].astype(np.float64), [n] * T)
        bound += n * 2.0 ** -32 * 1.5
        err = np.abs(got[:, h:h + 1] - want)
        assert (err <= bound).all(), (h, float((err / bound).max()))


def _cache(rng, n, H, d, bits, cap, Nr, S, k, v):
    g = gpu_cache(1, H, d, bits, cap, Nr, sink=S)
    lens = np.array([n], np.int32)
    kvq.kvq_quantize_pack(g, *(torch.from_numpy(x).to(DEV) for x in (k, v, lens)))
    return g, oracle_sequences(k, v, lens, bits, cap, Nr, S)[0]


@pytest.mark.parametrize("T", [3, 700])  # the join's two forms: a block for a row; rows in one line
@pytest.mark.parametrize("d,bits", [(64, 4), (128, 3), (256, 2)])
def test_an_infinite_value_outlasts_much_larger_scores_in_other_pieces(d, bits, T):
    """Infinite values (a group whose min is infinite) at the start of a cache that several
    blocks share, under scores hundreds of nats higher from its middle on: still infinite
    in the rows that see them, NaN where both signs meet, the other columns as ever."""
    rng = np.random.default_rng(50 + d)
    H, gq, n, S = 1, 2, 24000, 4
    k = rng.standard_normal((1, H, n, d)).astype(np.float16)
    k[:, :, n // 2:] = 6.0
    v = rng.standard_normal((1, H, n, d)).astype(np.float16)
    g, r = _cache(rng, n, H, d, bits, n, 0, S, k, v)
    up, down = 0x7C00 << 16, (0xFC00 << 16) - (1 << 32)  # scale 0, min +-inf
    g.v_params[0, 0, 1, 0], g.v_params[0, 0, 2, 1] = up, down
    g.v_sink[0, 0, 1, 33] = float("inf")
    q = (rng.random((T, H * gq, d)) * 3 + 1).astype(np.float16)  # 6 sum(q) / sqrt(d): 100 nats and more
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    rows = np.unique(np.linspace(0, T - 1, 7).astype(int))
    for causal in (True, False):
        f = kvq.kvq_chunk_attention if causal else kvq.kvq_cross_attention
        got = to_np(f(g, torch.from_numpy(q).to(DEV), cu, T, flags=kvq.KVQ_OUT_F32))
        assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)
        assert np.isposinf(got[..., :32]).all() and np.isnan(got[..., 33]).all()
        assert np.isneginf(np.delete(got[..., 32:64], 1, -1)).all()
        seen = [n - T + i + 1 if causal else n for i in rows]
        want, bound = attend(tokens_of(r, "k", 0), tokens_of(r, "v", 0), q[rows].astype(np.float64), seen)
        bound += n * 2.0 ** -32 * np.abs(v).max()
        assert (np.abs(got[rows] - want) <= bound)[..., 64:].all()


@pytest.mark.parametrize("n", [90, 24000])  # whole units; pieces
@pytest.mark.parametrize("d,bits", [(32, 2), (64, 4), (128, 3), (256, 4)])
def test_a_nan_score_is_not_hidden_by_an_infinite_value(d, bits, n):
    """Rows that see a NaN key are NaN in every column, those of an infinite value too."""
    rng = np.random.default_rng(60 + d)
    H, gq, T = 2, 2, 20
    k, v = (rng.standard_normal((1, H, n, d)).astype(np.float16) for _ in range(2))
    g, r = _cache(rng, n, H, d, bits, n, 32, 0, k, v)
    bad = n - T + 12  # token 12 of the run, in the window
    g.k_res[0, 0, 32 - T + 12, 3] = float("nan")
    g.v_res[0, :, 2, 5] = float("inf")  # seen by all rows
    q = rng.standard_normal((T, H * gq, d)).astype(np.float16)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    got = to_np(kvq.kvq_chunk_attention(g, torch.from_numpy(q).to(DEV), cu, T, flags=kvq.KVQ_OUT_F32))
    assert np.isnan(got[12:, :gq]).all()
    assert np.isposinf(got[:12, :, 5]).all() and np.isposinf(got[:, gq:, 5]).all()
    want, bound = attend(tokens_of(r, "k", 0), tokens_of(r, "v", 0), q.astype(np.float64),
                         [n - T + i + 1 for i in range(T)])
    ok = np.abs(got - want) <= bound + n * 2.0 ** -32 * np.abs(v).max()
    ok[..., 5] = True
    assert bad >= n - 32 and ok[:12].all() and ok[:, gq:].all()
