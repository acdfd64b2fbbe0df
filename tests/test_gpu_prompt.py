"""Causal attention over whole prompts against a plain one in 64 bits."""

import math

import numpy as np
import pytest
import torch

from bit_quantized_kv_pack_gb300 import kvq

from _runs import HALF_STEP
from _util import gpu_cache, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"


def plain(q, k, v, rows=None, f32=False):
    """softmax(q k^T / sqrt(d)) v of one prompt, q [n][Hq][d], k and v [n][Hkv][d], causal, and
    the most that roundings may move each value: a score by E = (d + 2) 2^-23 sum |q k| / sqrt(d)
    (fp32 sums in any order, the reference's product), so a weight by e^2E - 1, its own rounding
    HALF_STEP, the exponential 2^-19, sums (n + 64) 2^-23, the output's rounding HALF_STEP;
    weights far below the reference lose 2^-32 of it each.  f32: weights in two parts (half a
    step of a half step) and an output of 2^-24."""
    n, hq, d = q.shape
    gq = hq // k.shape[1]
    rows = torch.arange(n, device=DEV) if rows is None else rows
    out = torch.empty(len(rows), hq, d, dtype=torch.float64, device=DEV)
    bound = torch.empty_like(out)
    for h in range(hq):
        kk, vv, qq = k[:, h // gq].double(), v[:, h // gq].double(), q[rows, h].double()
        hidden = torch.arange(n, device=DEV) > rows[:, None]
        s = (qq @ kk.T / math.sqrt(d)).masked_fill(hidden, -math.inf)
        mag = (qq.abs() @ kk.abs().T / math.sqrt(d)).masked_fill(hidden, 0.0).nan_to_num(posinf=0.0)
        p = torch.softmax(s, -1)
        out[:, h] = p @ vv
        E = (d + 2) * 2.0 ** -23 * mag.amax(1)
        steps = 2.0 ** -22 + 2.0 ** -24 if f32 else 2 * HALF_STEP
        rel = torch.expm1(2 * E) + steps + (n + 64) * 2.0 ** -23 + 2.0 ** -19
        most = (~hidden).double() @ vv.abs()
        bound[:, h] = rel[:, None] * (p @ vv.abs()) + 2.0 ** -31 * most + 2.0 ** -24
    return out, bound


def inputs(seed, total, hq, hkv, d, scale=1.0):
    gen = torch.Generator(DEV).manual_seed(seed)
    x = torch.randn(total, hq + 2 * hkv, d, generator=gen, device=DEV)
    x[:, hq:hq + hkv] *= scale * (0.5 + 2.0 * torch.rand(d, generator=gen, device=DEV) ** 6)
    return x.half().split([hq, hkv, hkv], 1)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# Prompts without tokens behind the others: there could be more blocks of rows than SMs, and
# a block's two lanes have rows of their own; with few, both have the same ones.
EMPTY = pytest.mark.parametrize("empty", [0, 200])


def ends(lens, empty=0):
    return ints(np.concatenate([[0], np.cumsum(list(lens) + [0] * empty)]))


def check(got, q, k, v, lens, first=0):
    at = first
    for n in lens:
        if n:
            want, bound = plain(q[at:at + n], k[at:at + n], v[at:at + n], f32=got.dtype == torch.float32)
            err = (got[at:at + n].double() - want).abs()
            assert torch.isfinite(got[at:at + n]).all()
            assert (err <= bound).all(), (n, float((err / bound).max()), (err > bound).nonzero()[:4].tolist())
        at += n


@pytest.mark.parametrize("lens", [[1], [2, 1, 3], [77], [128], [129, 64, 127, 0, 300], [513], [1025, 1]])
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 32), (4, 1, 64), (6, 2, 128), (8, 2, 128), (5, 1, 64), (3, 3, 128),
                                      (2, 2, 256), (8, 1, 256), (16, 2, 32), (71, 1, 64), (128, 1, 128)])
@EMPTY
def test_prompts(lens, hq, hkv, d, empty):
    total = sum(lens)
    q, k, v = inputs(total + d, total, hq, hkv, d)
    cu = ends(lens, empty)
    out = kvq.kvq_prompt_attention(q, k, v, cu, max(lens))
    assert out.dtype == torch.float16
    check(out, q, k, v, lens)
    exact = kvq.kvq_prompt_attention(q, k, v, cu, total, flags=kvq.KVQ_OUT_F32)  # a looser bound
    assert exact.dtype == torch.float32
    check(exact, q, k, v, lens)


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (16, 16, 64), (4, 4, 32), (3, 1, 256)])
def test_many_ragged_prompts(hq, hkv, d):
    rng = np.random.default_rng(d)
    lens = list(rng.integers(0, 700, 40))  # more than a window of sequences
    q, k, v = inputs(d, sum(lens), hq, hkv, d)
    cu = ints(np.concatenate([[0], np.cumsum(lens)]))
    check(kvq.kvq_prompt_attention(q, k, v, cu, max(lens)), q, k, v, lens)


@pytest.mark.parametrize("n,hq,hkv,d", [(9001, 8, 2, 128), (20000, 2, 1, 64), (6000, 2, 2, 128), (5000, 2, 1, 256),
                                      (4353, 1, 1, 64), (6200, 1, 1, 32)])
@EMPTY
def test_long_prompts(n, hq, hkv, d, empty):
    q, k, v = inputs(n, n, hq, hkv, d, scale=2.0)
    out = kvq.kvq_prompt_attention(q, k, v, ends([n], empty), n, flags=kvq.KVQ_OUT_F32)
    rows = torch.cat([torch.arange(300), torch.randint(300, n - 300, (400,), generator=torch.Generator().manual_seed(1)),
                      torch.arange(n - 300, n)]).to(DEV)
    want, bound = plain(q, k, v, rows, f32=True)
    err = (out[rows].double() - want).abs()
    assert (err <= bound).all(), float((err / bound).max())
    again = kvq.kvq_prompt_attention(q, k, v, ends([n], empty), n, flags=kvq.KVQ_OUT_F32)
    assert torch.equal(out, again)


@pytest.mark.parametrize("d", [32, 64, 128])
@EMPTY
def test_values_of_one_sign_add_up(d, empty):
    """Sums that are cut off fall short of these, more with each tile; rows of all numbers of
    tiles about a segment's and two segments' for each lane."""
    n = 4500
    q, k, v = inputs(d, n, 1, 1, d, scale=0.1)
    v = v.abs()
    out = kvq.kvq_prompt_attention(q, k, v, ends([n], empty), n, flags=kvq.KVQ_OUT_F32)
    want, _ = plain(q, k, v, f32=True)
    # a sum that is cut off to 24 bits is off by up to a whole step, 2^-23 (not half of one, which
    # 2^-16 in all stood for), of what it is then, half of the segment's on average, in 16 tiles
    # of 8 steps for each of the weights' parts: 2^-16; the exponentials 2^-19, scores
    # (d + 2) 2^-23 of products of at most 1 / 4: 2^-18; the rest 2^-20: under 2^-16 + 2^-17
    assert float(((out.double() - want).abs() / want).max()) < 1.5 * 2.0 ** -16


def test_layouts_and_rows_of_no_prompt():
    """Head-major and separate tensors; rows before, between and behind prompts stay as they were."""
    hq, hkv, d, total = 6, 2, 64, 500
    q, k, v = inputs(9, total, hq, hkv, d)
    cu = ints([40, 250, 250, 401])
    want = kvq.kvq_prompt_attention(q, k, v, cu, 300)
    check(want, q, k, v, [210, 0, 151], first=40)
    head_major = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    out = torch.full_like(want, 7.0)
    kvq.kvq_prompt_attention(head_major[0], k.contiguous(), head_major[2], cu, 300, out=out)
    assert torch.equal(out[40:401], want[40:401])
    assert (out[:40] == 7).all() and (out[401:] == 7).all()
    none = kvq.kvq_prompt_attention(q[:0], k[:0], v[:0], ints([0, 0]), 0)
    assert none.shape == (0, hq, d)
    out.fill_(7.0)
    kvq.kvq_prompt_attention(q, k, v, ints([0, 0, 0]), 300, out=out)
    assert (out == 7).all()
    with pytest.raises(kvq.KvqError):
        kvq.kvq_prompt_attention(q, k[:, :1].expand(-1, 2, -1), v, cu, 300)  # one key for all heads


def test_broken_entries_cost_no_other_prompt():
    hq, hkv, d, total = 4, 2, 128, 600
    q, k, v = inputs(10, total, hq, hkv, d)
    g = gpu_cache(1, 1, 32, 4, 32, 0)
    for cu, good in (([0, 100, 90, 300, 601], [(0, 100), (90, 300)]), ([-1, 50, 200, 100, 150], [(50, 200), (100, 150)]),
                     ([0, 600, 600, 600, 600], []), ([5, 5, 105, 505, 506], [(5, 105), (505, 506)])):
        out = torch.full((total, hq, d), 7.0, dtype=torch.float16, device=DEV)
        kvq.kvq_prompt_attention(q, k, v, ints(cu), 399, out=out, err=g.err)
        assert kvq.kvq_read_error(g)[1] == kvq.KVQ_ERRBIT_BADLEN, cu
        seen = torch.zeros(total, dtype=torch.bool)
        for lo, hi in good:
            one = kvq.kvq_prompt_attention(q[lo:hi], k[lo:hi], v[lo:hi], ints([0, hi - lo]), hi - lo)
            shared = torch.tensor([not any(a < hi and lo < b for a, b in good if (a, b) != (lo, hi))])
            if shared:
                assert torch.equal(out[lo:hi], one), (cu, lo)
            seen[lo:hi] = True
        assert (out[~seen.to(DEV)] == 7).all(), cu


@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 128), (2, 2, 64), (2, 1, 256), (1, 1, 32)])
@EMPTY
def test_what_a_row_does_not_see_has_no_part(hq, hkv, d, empty):
    """NaN and infinities in later tokens and in other prompts, keys and values alike."""
    lens = [70, 200, 1, 333]
    total = sum(lens)
    q, k, v = inputs(d, total, hq, hkv, d)
    cu = ends(lens, empty)
    want = kvq.kvq_prompt_attention(q, k, v, cu, 333)
    for value in (float("nan"), float("inf"), -float("inf")):
        for at in (0, 69, 70, 130, 199, 269, 270, 271, 400, 603):
            k2, v2 = k.clone(), v.clone()
            k2[at], v2[at] = value, value
            got = kvq.kvq_prompt_attention(q, k2, v2, cu, 333)
            lo, hi = next((a, a + n) for a, n in zip(np.concatenate([[0], np.cumsum(lens)]), lens) if a <= at < a + n)
            clean = torch.ones(total, dtype=torch.bool, device=DEV)
            clean[at:hi] = False
            assert torch.equal(got[clean], want[clean]), (value, at)
            assert not torch.isfinite(got[at:hi]).any(), (value, at)


@pytest.mark.parametrize("d", [64, 128, 256])
@EMPTY
def test_infinite_values_that_are_seen(d, empty):
    """Single columns: the sign of the infinity where one sign is seen, NaN where both are or
    where NaN is, from the token on; other columns as ever.  Scores near each other, so that
    no weight vanishes."""
    hq, hkv, n = 4, 2, 300
    q, k, v = inputs(d, n, hq, hkv, d)
    q, k = q * 0.25, k * 0.25
    cu = ends([n], empty)
    want = kvq.kvq_prompt_attention(q, k, v, cu, n)
    v2 = v.clone()
    v2[20, 0, 3], v2[150, 0, 7], v2[160, 1, 9] = math.inf, -math.inf, math.nan
    v2[40, 1, 11], v2[290, 1, 11] = math.inf, -math.inf
    got = kvq.kvq_prompt_attention(q, k, v2, cu, n)
    expect = want.clone()
    expect[20:, :2, 3], expect[150:, :2, 7], expect[160:, 2:, 9] = math.inf, -math.inf, math.nan
    expect[40:, 2:, 11] = math.inf
    expect[290:, 2:, 11] = math.nan
    assert np.array_equal(to_np(got), to_np(expect), equal_nan=True)


@EMPTY
def test_scores_that_are_not_finite(empty):
    n, d = 200, 64
    q, k, v = inputs(5, n, 2, 1, d)
    q, k, v = q.clone(), k.clone(), v
    cu = ends([n], empty)
    want = kvq.kvq_prompt_attention(q, k, v, cu, n)
    q[50, 1] = math.nan                                   # a query
    got = kvq.kvq_prompt_attention(q, k, v, cu, n)
    assert torch.isnan(got[50, 1]).all() and torch.equal(got[50, 0], want[50, 0])
    q[50, 1], q[:, :, 0], k[:, :, 0] = 0.0, 1.0, 0.0
    want = kvq.kvq_prompt_attention(q, k, v, cu, n)
    k[10, 0, 0] = -math.inf                               # a key that nobody attends to
    got = kvq.kvq_prompt_attention(q, k, v, cu, n)
    ref, bound = plain(q, k, v)
    assert torch.equal(got[:10], want[:10])
    assert torch.isfinite(ref).all() and ((got.double() - ref).abs() <= bound).all()
    k[0, 0, 0] = -math.inf                                # ... and the first: row 0 has no other
    got = kvq.kvq_prompt_attention(q, k, v, cu, n)
    assert torch.isnan(got[0]).all() and torch.isfinite(got[1:]).all()


def test_a_long_tail_under_one_dominant_token_keeps_its_mass():
    n, d = 16384, 64
    k = torch.zeros(n, 1, d, dtype=torch.float16, device=DEV)
    k[0] = 1.0
    gen = torch.Generator(DEV).manual_seed(2)
    v = (torch.rand(n, 1, d, generator=gen, device=DEV) + 0.5).half()
    v[0] = 0.0
    nats = torch.linspace(9, 18, n, device=DEV)
    q = (nats / math.sqrt(d)).half()[:, None, None].expand(-1, 1, d).contiguous()
    out = kvq.kvq_prompt_attention(q, k, v, ints([0, n]), n, flags=kvq.KVQ_OUT_F32)
    rows = torch.arange(200, n, 61, device=DEV)
    want, bound = plain(q, k, v, rows, f32=True)
    err = (out[rows].double() - want).abs()
    assert (err <= bound).all(), float((err / bound).max())


def test_streams_and_graphs():
    lens = [300, 45, 800]
    q, k, v = inputs(3, sum(lens), 8, 2, 128)
    cu = ints(np.concatenate([[0], np.cumsum(lens)]))
    want = kvq.kvq_prompt_attention(q, k, v, cu, 800)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    other = kvq.kvq_prompt_attention(q, k, v, cu, 800, stream=st)
    same = kvq.kvq_prompt_attention(q, k, v, cu, 800)  # at the same time
    torch.cuda.synchronize()
    assert torch.equal(other, want) and torch.equal(same, want)
    x = torch.cat([q, k, v], 1)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvq.kvq_prompt_attention(x[:, :8], x[:, 8:10], x[:, 10:], cu, 1145, out=out)
    q2, k2, v2 = inputs(4, sum(lens), 8, 2, 128)
    x.copy_(torch.cat([q2, k2, v2], 1))
    lens = [0, 1000, 100]
    cu.copy_(ints([0, 0, 1000, 1100]))
    g.replay()
    torch.cuda.synchronize()
    check(out, q2, k2, v2, lens)


@EMPTY
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_whole(empty):
    q, k, v = inputs(6, 500, 8, 2, 128)
    cu, g = ends([500], empty), gpu_cache(1, 1, 32, 4, 32, 0)
    want = kvq.kvq_prompt_attention(q, k, v, cu, 500)
    kvq.kvq_testing_wait_fault(2000)
    try:
        kvq.kvq_prompt_attention(q, k, v, cu, 500, err=g.err)
        assert kvq.kvq_read_error(g)[1] & kvq.KVQ_ERRBIT_TIMEOUT
    finally:
        kvq.kvq_testing_wait_fault(0)
    assert torch.equal(kvq.kvq_prompt_attention(q, k, v, cu, 500, err=g.err), want)
    assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 32), (4, 2, 64), (3, 1, 128), (4, 2, 256)])
@pytest.mark.parametrize("n", [300, 4500])
@EMPTY
def test_infinite_values_that_are_seen_with_fp32_output(hq, hkv, d, n, empty):
    """As with fp16 output, in tiles that every row of a block sees too, and over more than a
    segment of 2048 tokens for either lane."""
    q, k, v = inputs(d + n, n, hq, hkv, d)
    q, k = q * 0.25, k * 0.25
    cu, f32 = ends([n], empty), kvq.KVQ_OUT_F32
    want = kvq.kvq_prompt_attention(q, k, v, cu, n, flags=f32)
    v2, expect = v.clone(), want.clone()
    gq, last = hq // hkv, n - 10
    for tokens, head, column in (([(0, math.inf)], 0, 0), ([(20, math.inf)], 0, 3), ([(150, -math.inf)], 0, 7),
                                 ([(160, math.nan)], hkv - 1, 9), ([(40, math.inf), (last, -math.inf)], hkv - 1, 11),
                                 ([(n // 2, -math.inf), (n // 2 + 1, -math.inf)], 0, d - 1),
                                 ([(last, math.inf), (last + 1, math.nan)], hkv - 1, d - 2)):
        seen = None
        for at, value in tokens:
            v2[at, head, column] = value
            seen = value if seen is None or seen == value else math.nan
            expect[at:, head * gq:(head + 1) * gq, column] = seen
    got = kvq.kvq_prompt_attention(q, k, v2, cu, n, flags=f32)
    assert np.array_equal(to_np(got), to_np(expect), equal_nan=True)


@pytest.mark.parametrize("d", [32, 64])
def test_a_block_of_one_row_at_a_tile_s_end(d):
    """128 query heads on one: a block's lanes have a token each, and the last token of a whole
    number of tiles sees all of each tile."""
    for lens in ([256], [128, 256, 257], [255, 256, 129] * 60):
        q, k, v = inputs(d, sum(lens), 128, 1, d)
        q, k = q * 0.25, k * 0.25
        cu = ends(lens)
        want = kvq.kvq_prompt_attention(q, k, v, cu, max(lens), flags=kvq.KVQ_OUT_F32)
        v2, expect, at = v.clone(), want.clone(), 0
        for n in lens:
            for token, column, value in ((0, 1, math.inf), (127, 2, -math.inf), (n - 1, 3, math.nan)):
                v2[at + token, 0, column] = value
                expect[at + token:at + n, :, column] = value
            at += n
        got = kvq.kvq_prompt_attention(q, k, v2, cu, max(lens), flags=kvq.KVQ_OUT_F32)
        assert np.array_equal(to_np(got), to_np(expect), equal_nan=True)


@pytest.mark.parametrize("heads,tokens", [(1, 1), (8, 64), (3, 84), (2, 256)])
def test_units_are_found_in_any_order(heads, tokens):
    """Blocks take over units from others; that they come in rising order is not promised."""
    rng = np.random.default_rng(heads * tokens)
    lens = rng.integers(0, 5 * tokens, 200)
    lens[rng.random(200) < 0.3] = 0
    lens[:40] = 0                                     # the first window has none
    cu = np.concatenate([[0], np.cumsum(lens)])
    line = [(cu[b], n, h, t * tokens) for b, n in enumerate(lens) for t in reversed(range(-(-n // tokens)))
            for h in range(heads)]
    most = len(line)
    rising = np.arange(most)
    orders = [rising, rising[::-1], rng.permutation(most + 50), [most + 7, 0, most, most - 1, 0, 0, most // 2, 1]]
    for order in orders:
        got = kvq.kvq_testing_prompt_units(ints(cu), int(lens.max()), int(cu[-1]), heads, tokens, ints(list(order)))
        want = [line[u] if u < most else (-1, 0, 0, 0) for u in order]
        assert np.array_equal(to_np(got), np.array(want))


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@EMPTY
def test_the_stated_bound_for_values_of_one_sign(d, empty):
    """2.3e-5 of the sum, whatever the length: a segment's sums are cut off by 2^-23 of what they
    are then, half of it on average, in 256 steps (2048 tokens of 16, two parts of the weights):
    2^-16; segments add up rounded to nearest, 2^-24 each; exponentials 2^-19; scores are cut off
    likewise, in d / 16 steps, by 2^-23 of sums below 1: 2^-19; the rest 2^-20."""
    n = 9001
    q, k, v = inputs(d + 1, n, 1, 1, d, scale=0.1)
    v = v.abs() + 0.25
    out = kvq.kvq_prompt_attention(q, k, v, ends([n], empty), n, flags=kvq.KVQ_OUT_F32)
    for lo in range(0, n, 3000):
        rows = torch.arange(lo, min(n, lo + 3000), device=DEV)
        want, _ = plain(q, k, v, rows, f32=True)
        assert float(((out[rows].double() - want).abs() / want).max()) < 2.3e-5
