"""Entries of cu_seqlens that are out of order: the sequences with broken entries are
skipped, every other sequence gets its whole run, in both launch forms of the append and
in the attention, bit for bit as the oracle's single appends."""

import numpy as np
import pytest
import torch

import oracle
from bit_quantized_kv_pack_gb300 import kvq

from _runs import attend, rotate, tokens_of
from _util import assert_cache_equal, gpu_cache, oracle_sequences, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _probe(value):
    """41 sequences of 7 tokens; entry 20 (one that a search in steps of two looks at) broken."""
    cu = [7 * i for i in range(42)]
    cu[20] = value
    return cu


CASES = [  # d, max_len, cu
    (256, 200, [0, 2, 1, 10 ** 6]),
    (64, 200, [0, 10 ** 6, 40, 90]),  # entry 1 past the end: two broken, the third is right
    (128, 40, [0, 30, 10, 50]),  # rows 10 .. 29 in two runs
    (128, 7, _probe(10 ** 6)),
    (64, 7, _probe(-3)),
    (32, 7, _probe(0)),
    (256, 7, _probe(150)),
    (128, 1, [0, 1, 0, 1, 2]),  # the form of one block per sequence
]


@pytest.mark.parametrize("d,max_len,cu", CASES)
def test_entries_out_of_order(d, max_len, cu):
    rng = np.random.default_rng(70 + d)
    B, H, gq, Nr, cap, held = len(cu) - 1, 2, 2, 4, 256, 9
    total = max(x for x in cu if x < 10 ** 6) + 3
    k0, v0 = (rng.standard_normal((B, H, held, d)).astype(np.float16) for _ in range(2))
    lens = np.full(B, held, np.int32)
    g = gpu_cache(B, H, d, 4, cap, Nr)
    kvq.kvq_quantize_pack(g, *(torch.from_numpy(x).to(DEV) for x in (k0, v0, lens)))
    refs = oracle_sequences(k0, v0, lens, 4, cap, Nr)
    k, v = (rng.standard_normal((total, H, d)).astype(np.float16) for _ in range(2))
    q = rng.standard_normal((total, H * gq, d)).astype(np.float16)
    dcu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    table = kvq.rope_table(400, d)
    good = [b for b in range(B) if 0 <= cu[b] <= cu[b + 1] <= total and cu[b + 1] - cu[b] <= max_len]
    assert 0 < len(good) < B
    # a row in two runs: either's queries and output
    rows_of = [[b for b in good if cu[b] <= t < cu[b + 1]] for t in range(total)]
    qo = torch.full((total, H * gq, d), 7.0, dtype=torch.float16, device=DEV)
    kvq.kvq_append_chunk(g, *(torch.from_numpy(x).to(DEV) for x in (k, v)), dcu, max_len,
                         q=torch.from_numpy(q).to(DEV), q_out=qo, rope=table)
    assert kvq.kvq_read_error(g)[1] == kvq.KVQ_ERRBIT_BADLEN
    for b in good:
        rows = slice(cu[b], cu[b + 1])
        kr = rotate(k[rows], to_np(table), held + np.arange(cu[b + 1] - cu[b]), d, False)
        for t in range(cu[b + 1] - cu[b]):
            assert oracle.append(refs[b], kr[t][None], v[rows][t][None]) == 0
    for b in range(B):
        assert_cache_equal(g, refs[b], batches=[b])
    for t, bs in enumerate(rows_of):
        want = [rotate(q[t:t + 1], to_np(table), np.array([held + t - cu[b]]), d, False)[0] for b in bs]
        got = to_np(qo[t])
        assert any(np.array_equal(got, w) for w in want) if bs else (got == 7.0).all(), t
    out = kvq.kvq_chunk_attention(g, torch.from_numpy(q).to(DEV), dcu, max_len, out=qo.float().fill_(7.0))
    assert kvq.kvq_read_error(g)[1] == kvq.KVQ_ERRBIT_BADLEN
    for t, bs in enumerate(rows_of):
        got = to_np(out[t])
        if not bs:
            assert (got == 7.0).all()
        if len(bs) != 1:
            continue
        r, n = refs[bs[0]], held + cu[bs[0] + 1] - cu[bs[0]]
        seen = n - (cu[bs[0] + 1] - t) + 1
        want, bound = attend(tokens_of(r, "k", 0), tokens_of(r, "v", 0), q[t:t + 1].astype(np.float64), [seen])
        assert (np.abs(got - want[0]) <= bound[0]).all(), t
