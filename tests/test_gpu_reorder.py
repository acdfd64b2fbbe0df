"""Caches whose sequences follow an index: every live byte, nothing else, for contiguous,
paged, hybrid caches with sink and window, and pages shared."""

import numpy as np
import pytest
import torch

from bit_quantized_kv_pack_gb300 import kvq

from _util import to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


ROWS = ("k_codes", "v_codes", "k_params", "v_params", "k_mode", "v_mode")
STATE = ("k_res", "v_res", "k_sink", "v_sink", "counters")


def filled(rng, c):
    """Random bytes in every array of a cache."""
    for name in (*ROWS, *STATE[:4]):
        t = getattr(c, name)
        if not t.numel():
            continue
        b = torch.from_numpy(rng.integers(0, 256, t.numel() * t.element_size(), dtype=np.uint8))
        t.copy_(b.view(t.dtype).view(t.shape).to(DEV))
    return c


def lengths(rng, c, packed):
    """Counters of a cache: packed tokens as given, windows and sinks of all kinds."""
    D = c.desc
    B = D.batch
    res = rng.integers(0, D.residual + 1, B)
    res[::2] = D.residual
    head = rng.integers(0, max(D.residual, 1), B)
    sink = rng.integers(0, D.sink + 1, B)
    c.counters.copy_(torch.from_numpy(np.stack([packed, res, head, sink]).astype(np.int32)))
    return c


def expected(dst, src, index, share=False):
    """dst's arrays after the call, by loops over sequences (numpy bytes)."""
    D, S = dst.desc, src.desc
    raw = lambda t: to_np(t).view(np.uint16 if t.dtype == torch.float16 else to_np(t).dtype)  # noqa: E731
    w = {n: raw(getattr(dst, n)).copy() for n in (*ROWS, *STATE, "block_table")}
    f = {n: raw(getattr(src, n)) for n in (*ROWS, *STATE, "block_table")}
    if share:
        for n in ROWS:
            f[n] = w[n].copy()
    for i, a in enumerate(index):
        if not 0 <= a < S.batch:
            continue
        npk, nres, head, ns = (int(x) for x in f["counters"][:, a])
        if npk > D.capacity:
            continue
        w["counters"][:3, i] = npk, nres, head
        if D.sink:
            w["counters"][3, i] = ns
        slots = [(head + j) % D.residual for j in range(nres)]
        for x in "kv":
            w[x + "_res"][i][:, slots] = f[x + "_res"][a][:, slots]
            w[x + "_sink"][i, :, :ns] = f[x + "_sink"][a, :, :ns]
        for n in ROWS:
            if not w[n].size:
                continue
            if not D.page_size:
                w[n][i, :, :npk] = f[n][a, :, :npk]
                continue
            for p in range(npk // 32 if share else 0, -(-npk // 32)):
                to, of = w["block_table"][i, p], f["block_table"][a, p]
                if 0 <= to < D.num_pages and 0 <= of < S.num_pages:
                    w[n][to, :, :min(32, npk - 32 * p)] = f[n][of, :, :min(32, npk - 32 * p)]
        if share:
            w["block_table"][i, :npk // 32] = f["block_table"][a, :npk // 32]
    return w


def check(dst, src, index, share=False, bits=0, **kw):
    want = expected(dst, src, index, share)
    before = {n: getattr(src, n).clone() for n in (*STATE, "block_table")}
    kvq.kvq_reorder(dst, src, torch.tensor(index, dtype=torch.int32, device=DEV), share_pages=share, **kw)
    torch.cuda.synchronize()
    assert kvq.kvq_read_error(dst)[1] == bits
    for n, x in want.items():
        assert np.array_equal(to_np(getattr(dst, n)).view(x.dtype), x), n
    for n, x in before.items():
        assert to_np(getattr(src, n)).tobytes() == to_np(x).tobytes(), n


@pytest.mark.parametrize("d,bits,cap,Nr,sink,hybrid", [
    (128, 4, 300, 128, 0, 0), (128, 2, 1031, 33, 4, 1), (64, 3, 257, 16, 5, 1), (32, 2, 701, 7, 3, 1),
    (32, 3, 515, 0, 0, 0), (256, 4, 200, 96, 32, 0), (256, 2, 77, 1, 0, 1), (64, 4, 0, 50, 9, 0),
    (32, 4, 4096, 1024, 256, 0),
])
def test_contiguous_caches(d, bits, cap, Nr, sink, hybrid):
    rng = np.random.default_rng(d + bits)
    B, H = 7, 3
    src = filled(rng, kvq.KVCache(B, H, d, bits, cap, Nr, sink=sink, hybrid=hybrid))
    lengths(rng, src, np.r_[0, cap, rng.integers(0, cap + 1, B - 2)])
    dst = lengths(rng, filled(rng, src.twin()), np.zeros(B))
    check(dst, src, [3, 3, 0, 1, 6, 5, 5])
    other = lengths(rng, filled(rng, src.twin(batch=11, capacity=cap + 33)), np.zeros(11))  # more and larger
    check(other, src, list(rng.integers(0, B, 11)))
    one = lengths(rng, filled(rng, src.twin(batch=1)), np.zeros(1))
    check(one, src, [1])


@pytest.mark.parametrize("d,bits,cap,Nr,sink,hybrid", [
    (128, 4, 320, 128, 0, 0), (64, 3, 256, 16, 5, 1), (32, 2, 704, 0, 3, 1), (256, 4, 96, 96, 32, 0),
])
@pytest.mark.parametrize("share", [False, True])
def test_paged_caches(d, bits, cap, Nr, sink, hybrid, share):
    rng = np.random.default_rng(d + bits + share)
    B, H, per = 6, 2, cap // 32
    src = filled(rng, kvq.KVCache(B, H, d, bits, cap, Nr, sink=sink, hybrid=hybrid, page_size=32,
                                  num_pages=2 * B * per + 3))
    lengths(rng, src, np.r_[0, cap, 31, 32, 33, rng.integers(0, cap + 1)])
    dst = src.twin(share_pages=share)
    if not share:
        filled(rng, dst)
    filled_state = filled(rng, kvq.KVCache(B, H, d, bits, 0, Nr, sink=sink))
    for n in STATE[:4]:
        getattr(dst, n).copy_(getattr(filled_state, n))
    pages = rng.permutation(2 * B * per + 3).astype(np.int32)
    src.block_table.copy_(torch.from_numpy(pages[:B * per].reshape(B, per)))
    dst.block_table.copy_(torch.from_numpy(pages[-B * per:].reshape(B, per)))
    check(dst, src, [4, 4, 1, 5, 3, 0], share)


def test_pages_of_one_pool_without_sharing():
    rng = np.random.default_rng(21)
    src = filled(rng, kvq.KVCache(2, 2, 64, 4, 128, 8, page_size=32, num_pages=40))
    lengths(rng, src, np.array([100, 64]))
    dst = src.twin(batch=5, share_pages=True)
    dst.block_table.copy_(torch.arange(10, 30, dtype=torch.int32).view(5, 4))
    kvq.kvq_reorder(dst, src, torch.tensor([0, 1, 1, 0, 0], dtype=torch.int32, device=DEV))
    for i, a in enumerate([0, 1, 1, 0, 0]):
        for p in range(4):
            rows = min(32, max(0, [100, 64][a] - 32 * p))
            for n in ROWS[:4]:
                t = getattr(src, n)
                got, of = t[10 + 4 * i + p, :, :rows], t[int(src.block_table[a, p]), :, :rows]
                assert to_np(got).tobytes() == to_np(of).tobytes()


def test_bad_indices_pages_and_capacities_cost_no_other_sequence():
    rng = np.random.default_rng(22)
    src = filled(rng, kvq.KVCache(4, 2, 64, 4, 128, 8, sink=2, page_size=32, num_pages=16))
    lengths(rng, src, np.array([100, 64, 128, 5]))
    src.block_table[0, 1] = 16
    src.block_table[1, 0] = -1
    dst = filled(rng, src.twin(capacity=96, num_pages=30))
    dst.block_table.copy_(torch.arange(12, dtype=torch.int32).view(4, 3) * 2)
    dst.block_table[2, 1] = 99
    both = kvq.KVQ_ERRBIT_BADINDEX | kvq.KVQ_ERRBIT_CAPACITY
    check(dst, src, [-1, 1, 4, 2], bits=both | kvq.KVQ_ERRBIT_BADPAGE)
    check(dst, src, [3, 3, 1, 2 ** 31 - 1], bits=kvq.KVQ_ERRBIT_BADINDEX | kvq.KVQ_ERRBIT_BADPAGE)
    assert kvq.kvq_read_error(dst) == (kvq.KVQ_OK, 0)


def test_many_sequences_streams_and_graphs():
    rng = np.random.default_rng(23)
    B = 700  # more than a block looks at together
    src = filled(rng, kvq.KVCache(B, 1, 32, 4, 64, 4))
    lengths(rng, src, rng.integers(0, 65, B))
    index = rng.integers(0, B, B)
    check(filled(rng, src.twin()), src, list(index))
    dst = filled(rng, src.twin())
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    check(dst, src, list(index[::-1]), stream=st.cuda_stream)
    # a captured step follows the indices of its replay
    at = torch.zeros(B, dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvq.kvq_reorder(dst, src, at)
    at.copy_(torch.from_numpy(index.astype(np.int32)))
    want = expected(dst, src, index)
    g.replay()
    torch.cuda.synchronize()
    for n, x in want.items():
        assert np.array_equal(to_np(getattr(dst, n)).view(x.dtype), x), n


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("writer", ["reorder", "append"])
def test_a_step_that_reads_early_sees_what_was_written_two_kernels_before(writer, paged):
    """A reorder into (or an append to) one cache, a step of another, then a step of the first
    with KVQ_STEP_EARLY_CACHE_READ: grids of a few blocks, so that all of them could run at once.
    The same calls without the flag, one after the other, give every byte of the caches, and the
    same outputs but for roundings: a step's splits add up in any order (red.add), up to 64 sums in
    fp32, 2^-23 of values below 8 each: 2^-14; and each side is rounded to fp16, 2^-11 of the value."""
    rng = np.random.default_rng(41 + paged)
    H, d, gq, cap, Nr, rounds = 1, 128, 4, 1024, 16, 24
    kw = dict(page_size=32, num_pages=200) if paged else {}
    src = kvq.KVCache(4, H, d, 4, cap, Nr, **kw)
    k, v = (torch.from_numpy(rng.standard_normal((4, H, 900, d)).astype(np.float16)).to(DEV) for _ in range(2))
    if paged:
        src.block_table.copy_(torch.arange(128, dtype=torch.int32).view(4, 32))
    kvq.kvq_quantize_pack(src, k, v, ints([40, 900, 300, 610]))
    order = [ints([int(i)]) for i in rng.integers(0, 4, rounds)]
    q, kn, vn = (torch.from_numpy(rng.standard_normal((rounds, 3, 1, n, d)).astype(np.float16)).to(DEV)
                 for n in (H * gq, H, H))
    results = []
    for flags in (kvq.KVQ_STEP_EARLY_CACHE_READ, 0):
        a, b = (src.twin(batch=1) for _ in range(2))
        for i, c in enumerate((a, b)):
            if paged:
                c.block_table.copy_(torch.arange(32 * i, 32 * i + 32, dtype=torch.int32).view(1, 32))
            kvq.kvq_reorder(c, src, ints([i]))
        ws = kvq.workspace_for(a, H * gq)
        out = torch.zeros(rounds, 2, 1, H * gq, d, dtype=torch.float16, device=DEV)
        torch.cuda.synchronize()
        for i in range(rounds):
            if writer == "reorder":
                kvq.kvq_reorder(a, src, order[i])
            else:
                kvq.kvq_append(a, kn[i, 2], vn[i, 2])
            if not flags:
                torch.cuda.synchronize()
            for j, c in enumerate((b, a)):
                kvq.kvq_decode_step(c, q[i, j], kn[i, j], vn[i, j], out[i, j], ws, flags=flags)
                if not flags:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert kvq.kvq_read_error(a) == kvq.kvq_read_error(b) == (kvq.KVQ_OK, 0)
        results.append([out] + [getattr(c, n) for c in (a, b) for n in (*ROWS, *STATE)])
    x, y = (r.pop(0).double() for r in results)
    assert ((x - y).abs() <= 2.0 ** -14 + 2.0 ** -10 * y.abs()).all()
    for x, y in zip(*results):
        assert to_np(x).tobytes() == to_np(y).tobytes()
