"""Attention of runs where a block has many units, one after the other: what a unit's rows
exchange (maxima, sums) is not overwritten by the next unit's, whose first scores may be
ready while a warp is still in the epilogue.  Results do not depend on timing: repeats,
alone and beside a stream that keeps the memory busy, are equal bit for bit and within the
bound of the 64-bit result."""

import numpy as np
import pytest
import torch

from bit_quantized_kv_pack_gb300 import kvq

from _runs import attend, tokens_of
from _util import gpu_cache, oracle_sequences, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"

# H, gq, d, bits, Nr, cache lengths, run lengths: whole units of few tiles, of both kinds of
# row blocks (up to 128 rows: the accumulators take turns; above: they share the tiles),
# hundreds of them, so that each block has several of both in turn
CASES = [
    (8, 2, 64, 4, 16, [130, 300, 40, 260] * 12, [128, 3, 40, 256] * 12),
    (10, 1, 128, 2, 0, [200, 90, 256] * 14, [200, 20, 130] * 14),
    (6, 2, 256, 3, 8, [100, 70, 200] * 16, [64, 3, 70] * 16),
    (16, 1, 32, 4, 4, [140, 500] * 20, [140, 2] * 20),
]


@pytest.mark.parametrize("H,gq,d,bits,Nr,kv,ql", CASES)
def test_units_of_a_block_do_not_disturb_one_another(H, gq, d, bits, Nr, kv, ql):
    rng = np.random.default_rng(31 + d)
    B, L = len(kv), max(kv)
    # scores that differ much from unit to unit: a maximum in place of a sum would show
    k = (rng.standard_normal((B, H, L, d)) * rng.uniform(0.2, 4.0, (B, H, 1, 1))).astype(np.float16)
    v = rng.standard_normal((B, H, L, d)).astype(np.float16)
    lens = np.array(kv, np.int32)
    g = gpu_cache(B, H, d, bits, 512, Nr)
    kvq.kvq_quantize_pack(g, *(torch.from_numpy(x).to(DEV) for x in (k, v, lens)))
    cu = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
    q = rng.standard_normal((int(cu[-1]), H * gq, d)).astype(np.float16)
    dq, dcu = torch.from_numpy(q).to(DEV), torch.from_numpy(cu).to(DEV)
    ws = kvq.chunk_workspace_for(g, H * gq)
    want = kvq.kvq_chunk_attention(g, dq, dcu, max(ql), workspace=ws, flags=kvq.KVQ_OUT_F32)
    for b, r in list(enumerate(oracle_sequences(k[:4], v[:4], lens[:4], bits, 512, Nr)))[:4]:
        rows, n = slice(int(cu[b]), int(cu[b + 1])), kv[b]
        seen = [n - ql[b] + i + 1 for i in range(ql[b])]
        o, bound = attend(tokens_of(r, "k", 0), tokens_of(r, "v", 0), q[rows].astype(np.float64), seen)
        assert (np.abs(to_np(want[rows]) - o) <= bound).all()
    busy, other = torch.empty(1 << 26, device=DEV), torch.cuda.Stream()
    out = torch.empty_like(want)
    for turn in range(60):
        if turn % 2:
            with torch.cuda.stream(other):
                busy.add_(1.0)
        kvq.kvq_chunk_attention(g, dq, dcu, max(ql), out=out, workspace=ws)
        assert torch.equal(out, want), turn
    torch.cuda.synchronize()
    assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)
