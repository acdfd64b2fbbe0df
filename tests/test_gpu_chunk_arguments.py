"""Arguments of the calls on runs that the documentation allows: views whose dimensions of
one entry carry odd strides, bounds on the run lengths past 32 bits."""

import numpy as np
import pytest
import torch

from bit_quantized_kv_pack_gb300 import kvq

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _odd(t, *dims):
    """t with another stride in its dimensions of one entry."""
    stride = list(t.stride())
    for i in dims:
        assert t.shape[i] == 1
        stride[i] = 3 + i
    return t.as_strided(t.shape, stride)


@pytest.mark.parametrize("total,H", [(1, 2), (5, 1), (1, 1)])
def test_strides_of_dimensions_with_one_entry_do_not_matter(total, H):
    rng = np.random.default_rng(80)
    d = 64
    dims = [i for i, n in enumerate((total, H)) if n == 1]
    k, v, q = (torch.from_numpy(rng.standard_normal((total, H, d)).astype(np.float16)).to(DEV) for _ in range(3))
    cu = torch.tensor([0, total], dtype=torch.int32, device=DEV)
    table = kvq.rope_table(10, d)
    caches = [kvq.KVCache(1, H, d, 4, 64, 2) for _ in range(3)]
    want = kvq.kvq_append_chunk(caches[0], k, v, cu, total, q=q, rope=table)
    # all three odd; then the keys alone, the values being columns of a wider tensor
    got = kvq.kvq_append_chunk(caches[1], _odd(k, *dims), _odd(v, *dims), cu, total, q=_odd(q, *dims), rope=table)
    assert torch.equal(got, want)
    wide = torch.cat([v, v], 1)[:, :H] if total == 1 else v
    q2 = _odd(q, *dims).clone(memory_format=torch.preserve_format)
    got = kvq.kvq_append_chunk(caches[2], _odd(k, *dims), wide, cu, total, q=q2, q_out=q2, rope=table)
    assert torch.equal(got, want)
    for c in caches[1:]:
        for name in ("k_codes", "v_codes", "k_params", "v_params", "k_res", "v_res", "counters"):
            assert torch.equal(getattr(c, name), getattr(caches[0], name)), name
    a = kvq.kvq_chunk_attention(caches[0], want, cu, total)
    b = kvq.kvq_chunk_attention(caches[0], _odd(want, *dims), cu, total)
    assert torch.equal(a, b)
    assert kvq.kvq_read_error(caches[0]) == (kvq.KVQ_OK, 0)


@pytest.mark.parametrize("bound", [2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 3, 2 ** 40])
def test_any_upper_bound_of_the_run_lengths_serves(bound):
    rng = np.random.default_rng(81)
    H, d, T = 2, 64, 9
    k, v, q = (torch.from_numpy(rng.standard_normal((T, H, d)).astype(np.float16)).to(DEV) for _ in range(3))
    cu = torch.tensor([0, 5, 9], dtype=torch.int32, device=DEV)
    caches = [kvq.KVCache(2, H, d, 4, 64, 2) for _ in range(2)]
    outs = []
    for c, n in zip(caches, (5, bound)):
        kvq.kvq_append_chunk(c, k, v, cu, n)
        outs.append([kvq.kvq_chunk_attention(c, q, cu, n), kvq.kvq_cross_attention(c, q, cu, n)])
        assert kvq.kvq_read_error(c) == (kvq.KVQ_OK, 0)
        for bad in (-1, -2 ** 32, -2 ** 40):
            for f in (lambda: kvq.kvq_append_chunk(c, k, v, cu, bad), lambda: kvq.kvq_cross_attention(c, q, cu, bad)):
                with pytest.raises(kvq.KvqError, match="invalid argument"):
                    f()
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert torch.equal(caches[0].counters, caches[1].counters) and torch.equal(caches[0].k_codes, caches[1].k_codes)


@pytest.mark.parametrize("T", [1, 13, 40])  # a block per sequence (up to 12 warps of work); rows in one line
def test_positions_past_31_bits_take_the_last_row_of_the_table(T):
    """A paged cache of 2^31 - 32 packed tokens (its pages are the same two) and a sink."""
    rng = np.random.default_rng(82)
    d, cap, rows = 32, 2 ** 31 - 32, 50
    c = kvq.KVCache(1, 1, d, 2, cap, 64, sink=64, page_size=32, num_pages=2)
    c.counters.copy_(torch.tensor([[cap], [0], [0], [64]], dtype=torch.int32))
    k, q = (torch.from_numpy(rng.standard_normal((T, 1, d)).astype(np.float16)).to(DEV) for _ in range(2))
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    table = kvq.rope_table(rows, d)
    got = kvq.kvq_append_chunk(c, k, k, cu, T, q=q, rope=table)
    assert kvq.kvq_read_error(c)[1] == kvq.KVQ_ERRBIT_BADPOS
    from _runs import rotate
    last = np.full(T, rows - 1)
    assert np.array_equal(got.cpu().numpy(), rotate(q.cpu().numpy(), table.cpu().numpy(), last, d, False))
    assert np.array_equal(c.k_res[0, :, :T].transpose(0, 1).cpu().numpy(),
                          rotate(k.cpu().numpy(), table.cpu().numpy(), last, d, False))
    assert c.counters[:, 0].tolist() == [cap, T, 0, 64]
