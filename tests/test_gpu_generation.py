"""The calls around the cache together, as a generation with beams uses them: a prompt of
text and images rotated, attended and packed, handed to its beams, then steps of decode,
selection and reorder; against the same generation in 64 bits on the host."""

import copy

import numpy as np
import pytest
import torch

import oracle
from bit_quantized_kv_pack_gb300 import kvq

from _runs import attend, rotate, tokens_of
from _util import assert_cache_equal, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"


def positions(n):
    """Text, then an image of rows and columns, then text: [3][n]."""
    text, rows, cols = 7, 5, 6
    p = np.zeros((3, n), np.int32)
    p[:, :text] = np.arange(text)
    i = np.arange(min(rows * cols, n - text))
    p[:, text:text + len(i)] = text + np.stack([i * 0, i // cols, i % cols])
    rest = n - text - len(i)
    p[:, n - rest:] = p.max() + 1 + np.arange(rest)
    return p


def turned(x, table, pos, axis, rotary):
    """Each pair at its axis' position: the one-axis rule for each axis, its pairs taken."""
    y = x.copy()
    half = rotary // 2
    for a in range(len(pos)):
        z = rotate(x, table, pos[a], rotary, False)
        mine = np.flatnonzero(np.array(axis) == a)
        for m in (mine, mine + half):
            y[..., m] = z[..., m]
    return y


@pytest.mark.parametrize("share", [False, True])
def test_beams_from_a_prompt_of_text_and_images(share):
    rng = np.random.default_rng(31 + share)
    B, W, H, hq, d, V, Nr, steps = 2, 3, 2, 8, 128, 1501, 8, 6
    lens = [61, 90]
    total, cap, table_rows = sum(lens), 128, 200
    axis = list(kvq.axes_of_pairs((16, 24, 24)))
    rope = kvq.rope_table(table_rows, d, device=DEV)
    table = to_np(rope)
    x = rng.standard_normal((total, hq + 2 * H, d)).astype(np.float16)
    pos = np.concatenate([positions(n) for n in lens], 1)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)

    # the prompts: rotated in place, attended, packed
    t = torch.from_numpy(x).to(DEV)
    q, k, v = t[:, :hq], t[:, hq:hq + H], t[:, hq + H:]
    paged = dict(page_size=32, num_pages=200) if share else {}
    prompts = kvq.KVCache(B, H, d, 4, cap, Nr, **paged)
    kvq.kvq_rotate(q, k, rope, torch.from_numpy(pos).to(DEV), pair_axis=axis, q_out=q, k_out=k, err=prompts.err)
    out = kvq.kvq_prompt_attention(q, k, v, torch.from_numpy(cu).to(DEV), max(lens), flags=kvq.KVQ_OUT_F32,
                                   err=prompts.err)
    padded = [torch.zeros(B, H, max(lens), d, dtype=torch.float16, device=DEV) for _ in range(2)]
    for b in range(B):
        for y, of in zip(padded, (k, v)):
            y[b, :, :lens[b]] = of[cu[b]:cu[b + 1]].transpose(0, 1)
    if share:
        prompts.block_table.copy_(torch.arange(B * 4, dtype=torch.int32).view(B, 4))
    kvq.kvq_quantize_pack(prompts, *padded, torch.tensor(lens, dtype=torch.int32, device=DEV))
    assert kvq.kvq_read_error(prompts) == (kvq.KVQ_OK, 0)

    xr = x.copy()
    xr[:, :hq + H] = turned(x[:, :hq + H], table, pos, axis, d)
    assert np.array_equal(to_np(t).view(np.uint16), xr.view(np.uint16))
    refs = []  # a one-sequence oracle cache for each beam
    for b in range(B):
        mine = xr[cu[b]:cu[b + 1]].transpose(1, 0, 2)
        kk, vv = (mine[hq + i * H:hq + (i + 1) * H].astype(np.float64) for i in range(2))
        want, bound = attend(kk, vv, mine[:hq].transpose(1, 0, 2).astype(np.float64), np.arange(lens[b]) + 1)
        assert (np.abs(to_np(out)[cu[b]:cu[b + 1]] - want) <= bound).all()
        r = oracle.Cache(1, H, d, 4, cap, Nr)
        assert oracle.quantize_pack(r, *(np.ascontiguousarray(y[None]) for y in (mine[hq:hq + H], mine[hq + H:])),
                                    np.array([lens[b]], np.int32)) == 0
        refs += [r] * W

    # to the beams; two caches that take turns
    caches = [prompts.twin(batch=B * W, share_pages=share) for _ in range(2)]
    if share:
        own = torch.arange(8, 8 + 2 * B * W * 4, dtype=torch.int32).view(2, B * W, 4)
        for c, p in zip(caches, own):
            c.block_table.copy_(p)
    kvq.kvq_reorder(caches[0], prompts, torch.arange(B * W, dtype=torch.int32, device=DEV) // W, share_pages=share)
    scores = np.full((B, W), -np.inf, np.float32)
    scores[:, 0] = 0.0
    finished = np.zeros((B, W), np.uint8)
    head = rng.standard_normal((hq * d, V)).astype(np.float32) * 0.05
    embed = rng.standard_normal((V, hq + 2 * H, d)).astype(np.float16)
    tokens = rng.integers(0, V, (B * W,))
    ws = kvq.beam_workspace_for(B, W, V, W)
    cur = 0
    for s in range(steps):
        c, other = caches[cur], caches[1 - cur]
        new = embed[tokens]  # [B W][hq + 2 H][d]
        at = np.repeat([positions(n).max() + 1 + s for n in lens], W).astype(np.int32)
        p3 = np.broadcast_to(at, (3, B * W)).copy()
        nt = torch.from_numpy(new).to(DEV)
        q1, k1 = kvq.kvq_rotate(nt[:, :hq], nt[:, hq:hq + H], rope, torch.from_numpy(p3).to(DEV), pair_axis=axis)
        o = kvq.kvq_decode_step(c, q1, k1, nt[:, hq + H:].contiguous(), flags=kvq.KVQ_OUT_F32)
        logits = (o.flatten(1) @ torch.from_numpy(head).to(DEV)).view(B, W, V)
        par, tok, sc = kvq.kvq_beam_select(logits, torch.from_numpy(scores).to(DEV), W,
                                           finished=torch.from_numpy(finished).to(DEV), end_token=3, workspace=ws,
                                           err=c.err)
        kvq.kvq_reorder(other, c, par, share_pages=share)
        assert kvq.kvq_read_error(c) == (kvq.KVQ_OK, 0) and kvq.kvq_read_error(other) == (kvq.KVQ_OK, 0)

        nr = new.copy()
        nr[:, :hq + H] = turned(new[:, :hq + H], table, p3, axis, d)
        refs = [copy.deepcopy(r) for r in refs]
        for i, r in enumerate(refs):
            assert oracle.append(r, np.ascontiguousarray(nr[i:i + 1, hq:hq + H]),
                                 np.ascontiguousarray(nr[i:i + 1, hq + H:])) == 0
            want, bound = attend(tokens_of(r, "k", 0), tokens_of(r, "v", 0), nr[i:i + 1, :hq].astype(np.float64),
                                 [len(tokens_of(r, "k", 0)[0])])
            assert (np.abs(to_np(o)[i:i + 1] - want) <= bound + 2e-3).all()  # (the decode's own bound)
        # the selection, from the logits that the device had
        lg = to_np(logits).astype(np.float64)
        row = scores.astype(np.float64)[:, :, None] + lg - np.log(np.exp(lg - lg.max(-1, keepdims=True)).sum(
            -1, keepdims=True)) - lg.max(-1, keepdims=True)
        for b, w in np.argwhere(finished):
            row[b, w] = -np.inf
            row[b, w, 3] = scores[b, w]
        order = np.argsort(-row.reshape(B, -1), 1, kind="stable")[:, :W]
        assert np.array_equal(to_np(par), np.arange(B)[:, None] * W + order // V)
        assert np.array_equal(to_np(tok), order % V)
        got = to_np(sc)
        assert (np.abs(got - np.take_along_axis(row.reshape(B, -1), order, 1)) <= 2.0 ** -20 + 2.0 ** -24 * 60).all()
        parent = to_np(par).flatten()
        scores, tokens = got.astype(np.float32), to_np(tok).flatten()
        finished = (finished.flatten()[parent].reshape(B, W) | (to_np(tok) == 3)).astype(np.uint8)
        refs = [refs[p] for p in parent]
        cur = 1 - cur
        # every byte of the beams' caches
        for i, r in enumerate(refs):
            one = _OneSequence(caches[cur], i)
            assert_cache_equal(one, r)


class _OneSequence:
    """Sequence i of a cache, its pages gathered, as a batch of one."""

    def __init__(self, c, i):
        self.desc = kvq.CacheDesc()
        for f, _ in kvq.CacheDesc._fields_:
            setattr(self.desc, f, getattr(c.desc, f))
        self.desc.page_size = 0
        for n in ("k_codes", "v_codes", "k_params", "v_params"):
            t = getattr(c, n)
            if c.desc.page_size:
                t = t[c.block_table[i].long()].transpose(0, 1).flatten(1, 2).unsqueeze(0)
            else:
                t = t[i:i + 1]
            setattr(self, n, t.contiguous())
        for n in ("k_res", "v_res", "k_sink", "v_sink"):
            setattr(self, n, getattr(c, n)[i:i + 1])
        for j, n in enumerate(("packed_len", "res_len", "res_head", "sink_len")):
            setattr(self, n, c.counters[j, i:i + 1])
