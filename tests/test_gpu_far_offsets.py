"""Rows whose offsets pass 32 bits: the calls around the cache give the same bytes as for
the same rows side by side."""

import pytest
import torch

from bit_quantized_kv_pack_gb300 import kvq

pytestmark = pytest.mark.gpu
DEV = "cuda"
APART = 1 << 24  # elements between rows: 300 of them are 10 GB of fp16


def apart(x, head=None):
    """x [rows][heads][d], its rows APART elements from each other, heads `head`."""
    rows, heads, d = x.shape
    room = torch.empty(rows * APART, dtype=x.dtype, device=DEV)
    y = room.as_strided(x.shape, (APART, head or d, 1))
    return y.copy_(x)


def test_rotation():
    gen = torch.Generator(DEV).manual_seed(1)
    q, k = (torch.randn(300, h, 64, generator=gen, device=DEV).half() for h in (5, 2))
    rope = kvq.rope_table(500, 64, device=DEV)
    positions = torch.randint(0, 500, (3, 300), generator=gen, device=DEV, dtype=torch.int32)
    axis = [i % 3 for i in range(32)]
    want = kvq.kvq_rotate(q, k, rope, positions, pair_axis=axis)
    far = apart(q, head=1 << 20)
    kvq.kvq_rotate(far, k, rope, positions, pair_axis=axis, q_out=far)
    assert torch.equal(far, want[0])


@pytest.mark.parametrize("empty", [0, 200])
def test_prompt(empty):
    gen = torch.Generator(DEV).manual_seed(2)
    q, k, v = (torch.randn(300, h, 128, generator=gen, device=DEV).half() for h in (4, 2, 2))
    cu = torch.tensor([0, 290, 300] + [300] * empty, dtype=torch.int32, device=DEV)
    want = kvq.kvq_prompt_attention(q, k, v, cu, 290)
    room = torch.empty(300 * APART, dtype=torch.float16, device=DEV)
    far = [room.as_strided(x.shape, (APART, 1 << 20, 1), i << 23).copy_(x) for i, x in enumerate((q, k))]
    assert torch.equal(kvq.kvq_prompt_attention(far[0], far[1], v, cu, 290), want)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_selection(dtype):
    gen = torch.Generator(DEV).manual_seed(3)
    x = torch.randn(270, 1, 5003, generator=gen, device=DEV).to(dtype)
    scores = torch.randn(270, 1, generator=gen, device=DEV)
    want = kvq.kvq_beam_select(x, scores, 3)
    got = kvq.kvq_beam_select(apart(x), scores, 3)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_caches():
    src = kvq.KVCache(3, 8, 128, 4, 1 << 22, 32)  # a sequence's codes are 2 GiB
    dst = src.twin()
    gen = torch.Generator(DEV).manual_seed(4)
    lens = [33, 0, 70]
    src.counters.copy_(torch.tensor([lens, [0, 5, 32], [0, 3, 9], [0, 0, 0]], dtype=torch.int32))
    for n in ("k_codes", "v_codes"):
        t = getattr(src, n)[:, :, :70]
        t.copy_(torch.randint(0, 256, t.shape, generator=gen, device=DEV, dtype=torch.uint8))
    for n in ("k_params", "v_params"):
        t = getattr(src, n)[:, :, :70]
        t.copy_(torch.randn(t.shape, generator=gen, device=DEV))
    for n in ("k_res", "v_res"):
        getattr(src, n).copy_(torch.randn(getattr(src, n).shape, generator=gen, device=DEV))
    index = [2, 0, 2]
    kvq.kvq_reorder(dst, src, torch.tensor(index, dtype=torch.int32, device=DEV))
    assert kvq.kvq_read_error(dst) == (kvq.KVQ_OK, 0)
    assert torch.equal(dst.counters[:3], src.counters[:3, index])
    for i, a in enumerate(index):
        for n in ("k_codes", "v_codes", "k_params", "v_params"):
            assert torch.equal(getattr(dst, n)[i, :, :lens[a]], getattr(src, n)[a, :, :lens[a]]), (n, i)
            assert not getattr(dst, n)[i, :, lens[a]:lens[a] + 40].any(), (n, i)  # as they were
    for n in ("k_res", "v_res"):
        assert torch.equal(getattr(dst, n)[0], getattr(src, n)[2])
