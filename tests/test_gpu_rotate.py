"""Rotary positions with several axes against the plain rule: fp32 products and sums, each
rounded, then one rounding to fp16 (bit for bit), and against the angles in 64 bits."""

import numpy as np
import pytest
import torch

from bit_quantized_kv_pack_gb300 import kvq

from _runs import HALF_STEP, rotate
from _util import gpu_cache, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"


def plain(x, table, pos, axis, rotary, interleaved):
    """The rule, pair by pair, on fp16 x [n][heads][d]; pos [axes][n]."""
    y = x.copy()
    for i in range(rotary // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
        c, s = table[np.clip(pos[axis[i]], 0, len(table) - 1), i].T[:, :, None]
        xa, xb = x[..., a].astype(np.float32), x[..., b].astype(np.float32)
        y[..., a] = (xa * c - xb * s).astype(np.float16)
        y[..., b] = (xb * c + xa * s).astype(np.float16)
    return y


def _inputs(rng, total, hq, hkv, d, rows, axes):
    x = rng.standard_normal((total, hq + 2 * hkv, d)).astype(np.float16)
    pos = rng.integers(0, rows, (axes, total)).astype(np.int32)
    return x, pos


@pytest.mark.parametrize("total,hq,hkv,d,rotary,axes,mixed", [
    (1, 32, 8, 128, 128, 3, False), (1, 1, 1, 32, 16, 1, False), (7, 5, 5, 64, 64, 2, True),
    (33, 12, 4, 128, 96, 3, True), (257, 9, 3, 256, 256, 4, True), (100, 40, 8, 256, 128, 3, False),
    (1001, 3, 1, 32, 32, 4, False), (6000, 8, 2, 64, 32, 2, False), (20000, 6, 2, 128, 128, 1, False),
])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_the_rule(total, hq, hkv, d, rotary, axes, mixed, interleaved):
    rng = np.random.default_rng(total + d)
    rows = 5000
    x, pos = _inputs(rng, total, hq, hkv, d, rows, axes)
    axis = [i % axes if mixed else min(i * axes * 3 // rotary, axes - 1) for i in range(rotary // 2)]
    rope = kvq.rope_table(rows, rotary, device=DEV)
    t = torch.from_numpy(x).to(DEV)
    q, k = t[:, :hq], t[:, hq:hq + hkv]  # columns of a fused projection's output
    qo, ko = kvq.kvq_rotate(q, k, rope, torch.from_numpy(pos).to(DEV), pair_axis=axis, interleaved=interleaved)
    table = to_np(rope)
    for got, of in ((qo, x[:, :hq]), (ko, x[:, hq:hq + hkv])):
        assert np.array_equal(to_np(got).view(np.uint16), plain(of, table, pos, axis, rotary, interleaved).view(np.uint16))
    assert np.array_equal(to_np(t).view(np.uint16), x.view(np.uint16))  # inputs as they were
    # the angles themselves: the table's rounding, three in fp32, one to fp16
    i = np.arange(rotary // 2)
    angle = pos[np.array(axis)].T.astype(np.float64) * 10000.0 ** (-2.0 * i / rotary)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
    xa, xb = x[:, :hq, a].astype(np.float64), x[:, :hq, b].astype(np.float64)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    want, mag = xa * c - xb * s, np.abs(xa) + np.abs(xb)
    # (2^-25: half a step of the smallest fp16 numbers)
    assert (np.abs(to_np(qo)[..., a] - want) <= HALF_STEP * np.abs(want) + 4 * 2.0 ** -24 * mag + 2.0 ** -25).all()


@pytest.mark.parametrize("d,interleaved", [(64, True), (128, False), (256, False)])
def test_rotation_in_place_of_projected_columns(d, interleaved):
    rng = np.random.default_rng(d)
    total, hq, hkv, rows = 300, 6, 2, 900
    x, pos = _inputs(rng, total, hq, hkv, d, rows, 3)
    axis = kvq.axes_of_pairs((d // 8, d // 8, d // 4), interleaved=True)
    rope = kvq.rope_table(rows, d, device=DEV)
    t = torch.from_numpy(x).to(DEV)
    q, k = t[:, :hq], t[:, hq:hq + hkv]
    kvq.kvq_rotate(q, k, rope, torch.from_numpy(pos).to(DEV), pair_axis=axis, interleaved=interleaved, q_out=q, k_out=k)
    want = x.copy()
    want[:, :hq + hkv] = plain(x[:, :hq + hkv], to_np(rope), pos, axis, d, interleaved)
    assert np.array_equal(to_np(t).view(np.uint16), want.view(np.uint16))  # values untouched


def test_one_of_both_and_no_rows():
    rng = np.random.default_rng(3)
    x, pos = _inputs(rng, 50, 4, 2, 64, 100, 1)
    rope, t, p = kvq.rope_table(100, 64, device=DEV), torch.from_numpy(x).to(DEV), torch.from_numpy(pos[0]).to(DEV)
    want = rotate(x, to_np(rope), pos[0], 64, False)
    q, none = kvq.kvq_rotate(t[:, :4], None, rope, p)
    assert none is None and np.array_equal(to_np(q).view(np.uint16), want[:, :4].view(np.uint16))
    none, k = kvq.kvq_rotate(None, t[:, 4:6], rope, p)
    assert none is None and np.array_equal(to_np(k).view(np.uint16), want[:, 4:6].view(np.uint16))
    q, k = kvq.kvq_rotate(t[:0, :4], t[:0, 4:6], rope, p[:0])
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)


def test_positions_outside_the_table_take_the_nearest_row_and_are_reported():
    rng = np.random.default_rng(4)
    x, pos = _inputs(rng, 40, 3, 1, 128, 64, 2)
    pos[1, 5], pos[0, 30], pos[1, 31] = -1, 64, 2 ** 31 - 1
    axis = kvq.axes_of_pairs((32, 32))
    rope, t, p = kvq.rope_table(64, 128, device=DEV), torch.from_numpy(x).to(DEV), torch.from_numpy(pos).to(DEV)
    g = gpu_cache(1, 1, 128, 4, 32, 0)
    q, _ = kvq.kvq_rotate(t[:, :3], None, rope, p, pair_axis=axis, err=g.err)
    assert kvq.kvq_read_error(g) == (kvq.KVQ_ERR_INVALID_ARG, kvq.KVQ_ERRBIT_BADPOS)
    want = plain(x[:, :3], to_np(rope), pos, axis, 128, False)
    assert np.array_equal(to_np(q).view(np.uint16), want.view(np.uint16))
    q2, _ = kvq.kvq_rotate(t[:, :3], None, rope, p, pair_axis=axis)  # nobody asked
    assert torch.equal(q2, q) and kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)


def test_one_axis_is_the_appends_rotation():
    """Keys rotated here and appended as they are leave the cache that the append's own
    rotation leaves, queries the same."""
    rng = np.random.default_rng(5)
    B, H, hq, d, T = 2, 2, 6, 128, 37
    x = torch.from_numpy(rng.standard_normal((B * T, hq + 2 * H, d)).astype(np.float16)).to(DEV)
    q, k, v = x[:, :hq], x[:, hq:hq + H], x[:, hq + H:]
    cu = torch.tensor([0, T, 2 * T], dtype=torch.int32, device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV).repeat(2)
    rope = kvq.rope_table(64, d, device=DEV)
    a, b = gpu_cache(B, H, d, 4, 64, 16), gpu_cache(B, H, d, 4, 64, 16)
    qa = kvq.kvq_append_chunk(a, k, v, cu, T, q=q, rope=rope)
    qb, kb = kvq.kvq_rotate(q, k, rope, pos)
    kvq.kvq_append_chunk(b, kb, v.contiguous(), cu, T)
    assert torch.equal(qa, qb)
    for n in ("k_codes", "v_codes", "k_params", "v_params", "k_res", "v_res", "counters"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n


def test_infinities_and_nan_stay_in_their_pairs():
    rng = np.random.default_rng(6)
    x, pos = _inputs(rng, 9, 2, 1, 64, 50, 1)
    pos[0] = np.arange(1, 10)  # (no sine or cosine of these is 0)
    x[3, 1, 5], x[6, 0, 40] = np.inf, np.nan
    rope, t = kvq.rope_table(50, 64, device=DEV), torch.from_numpy(x).to(DEV)
    q, _ = kvq.kvq_rotate(t[:, :2], None, rope, torch.from_numpy(pos).to(DEV))
    bad = ~np.isfinite(to_np(q))
    assert bad[3, 1, [5, 37]].all() and bad[6, 0, [8, 40]].all() and bad.sum() == 4


def test_another_stream_and_a_graph():
    rng = np.random.default_rng(7)
    x, pos = _inputs(rng, 200, 8, 2, 128, 300, 3)
    axis = kvq.axes_of_pairs((16, 24, 24))
    rope, t, p = kvq.rope_table(300, 128, device=DEV), torch.from_numpy(x).to(DEV), torch.from_numpy(pos).to(DEV)
    want, _ = kvq.kvq_rotate(t[:, :8], None, rope, p, pair_axis=axis)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got, _ = kvq.kvq_rotate(t[:, :8], None, rope, p, pair_axis=axis, stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvq.kvq_rotate(t[:, :8], None, rope, p, pair_axis=list(axis), q_out=out)
    t2 = torch.from_numpy(rng.standard_normal(x.shape).astype(np.float16)).to(DEV)
    t.copy_(t2)
    p.add_(1).remainder_(300)
    g.replay()
    torch.cuda.synchronize()
    want = plain(to_np(t2)[:, :8], to_np(rope), (pos + 1) % 300, axis, 128, False)
    assert np.array_equal(to_np(out).view(np.uint16), want.view(np.uint16))
