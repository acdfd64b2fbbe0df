"""Host-side refusals of the calls around the cache (no GPU: every call here fails its
checks before anything is launched)."""

import ctypes

import pytest
import torch

from bit_quantized_kv_pack_gb300 import _build, kvq

P = ctypes.c_void_p
INVALID, UNSUPPORTED, MISALIGNED = kvq.KVQ_ERR_INVALID_ARG, kvq.KVQ_ERR_UNSUPPORTED, kvq.KVQ_ERR_MISALIGNED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kvq.load()


AXES = (ctypes.c_uint8 * 64)(*[i % 3 for i in range(64)])


def _rotate(lib, **kw):
    base = dict(q=0x100000, k=0x200000, q_out=0x300000, k_out=0x400000, q_stride_token=4096, q_stride_head=128,
                k_stride_token=1024, k_stride_head=128, q_out_stride_token=4096, q_out_stride_head=128,
                k_out_stride_token=1024, k_out_stride_head=128, num_q_heads=32, num_kv_heads=8, head_dim=128,
                total=10, rope=0x500000, rope_rows=100, rotary_dim=128, interleaved=0, axes=3, positions=0x600000,
                pair_axis=ctypes.addressof(AXES), err_word=0)
    base.update(kw)
    return lib.kvq_rotate(ctypes.byref(kvq.RotateArgs(**base)), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=0, k=0), INVALID), (dict(q_out=0), INVALID), (dict(k_out=0), INVALID), (dict(total=-1), INVALID),
    (dict(num_q_heads=0), INVALID), (dict(num_kv_heads=-1), INVALID), (dict(num_q_heads=65536), UNSUPPORTED),
    (dict(head_dim=0), INVALID), (dict(head_dim=40), INVALID), (dict(head_dim=96), UNSUPPORTED),
    (dict(head_dim=512), UNSUPPORTED), (dict(rotary_dim=0), INVALID), (dict(rotary_dim=144), INVALID),
    (dict(rotary_dim=24), UNSUPPORTED), (dict(interleaved=2), INVALID), (dict(axes=0), INVALID),
    (dict(axes=5), UNSUPPORTED), (dict(axes=2), INVALID),  # a pair has axis 2
    (dict(rope=0), INVALID), (dict(rope_rows=0), INVALID), (dict(positions=0), INVALID),
    (dict(q_stride_token=-8), INVALID), (dict(k_out_stride_head=-8), INVALID),
    (dict(q_stride_head=12), MISALIGNED), (dict(k_stride_token=1028), MISALIGNED),
    (dict(q_out_stride_token=4), MISALIGNED), (dict(q=0x100008), MISALIGNED), (dict(k_out=0x400002), MISALIGNED),
    (dict(q_out_stride_token=0), INVALID), (dict(k_out_stride_head=0), INVALID),
    (dict(rope=0x500008), MISALIGNED), (dict(positions=0x600002), MISALIGNED), (dict(err_word=0x700001), MISALIGNED),
    (dict(q_out=0x100000, q_out_stride_head=256), INVALID),  # in place, other rows
])
def test_rotate_refuses(lib, kw, expect):
    assert _rotate(lib, **kw) == expect
    assert lib.kvq_rotate(None, None) == INVALID


def _prompt(lib, **kw):
    base = dict(q=0x100000, k=0x200000, v=0x300000, q_stride_token=4096, q_stride_head=128, k_stride_token=1024,
                k_stride_head=128, v_stride_token=1024, v_stride_head=128, num_q_heads=32, num_kv_heads=8,
                head_dim=128, batch=2, cu_seqlens=0x400000, total=10, max_len=5, out=0x500000, flags=0, err_word=0)
    base.update(kw)
    return lib.kvq_prompt_attention(ctypes.byref(kvq.PromptArgs(**base)), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(out=0), INVALID),
    (dict(cu_seqlens=0), INVALID), (dict(batch=0), INVALID), (dict(total=-1), INVALID), (dict(max_len=-1), INVALID),
    (dict(num_kv_heads=0), INVALID), (dict(num_q_heads=0), INVALID), (dict(num_q_heads=12), INVALID),
    (dict(num_q_heads=129, num_kv_heads=1), UNSUPPORTED), (dict(head_dim=24), INVALID), (dict(head_dim=96), UNSUPPORTED),
    (dict(total=(1 << 30) + 1), UNSUPPORTED), (dict(batch=(1 << 20) + 1), UNSUPPORTED), (dict(flags=1), INVALID),
    (dict(q_stride_token=-8), INVALID), (dict(v_stride_head=-8), INVALID), (dict(k_stride_token=1028), MISALIGNED),
    (dict(k_stride_head=0), UNSUPPORTED), (dict(v_stride_token=0), UNSUPPORTED), (dict(q_stride_token=1 << 32), UNSUPPORTED),
    (dict(q=0x100008), MISALIGNED), (dict(v=0x300002), MISALIGNED), (dict(out=0x500008), MISALIGNED),
    (dict(cu_seqlens=0x400002), MISALIGNED), (dict(err_word=0x600002), MISALIGNED),
])
def test_prompt_attention_refuses(lib, kw, expect):
    assert _prompt(lib, **kw) == expect
    assert lib.kvq_prompt_attention(None, None) == INVALID


def _select(lib, **kw):
    base = dict(logits=0x100000, stride_row=1000, scores=0x200000, finished=0, batch=2, beams=4, vocab=1000, n=8,
                end_token=0, flags=0, parent=0x300000, token=0x400000, score=0x500000, workspace=0x600000,
                ws_bytes=1 << 30, err_word=0)
    base.update(kw)
    return lib.kvq_beam_select(ctypes.byref(kvq.BeamArgs(**base)), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(logits=0), INVALID), (dict(scores=0), INVALID), (dict(parent=0), INVALID), (dict(token=0), INVALID),
    (dict(score=0), INVALID), (dict(workspace=0), INVALID), (dict(batch=0), INVALID), (dict(beams=0), INVALID),
    (dict(vocab=0), INVALID), (dict(n=0), INVALID), (dict(n=33), UNSUPPORTED), (dict(beams=33), UNSUPPORTED),
    (dict(beams=1, vocab=7, n=8), INVALID), (dict(batch=16384, beams=4), UNSUPPORTED),
    (dict(beams=32, vocab=1 << 26, stride_row=1 << 26), UNSUPPORTED), (dict(stride_row=999), INVALID),
    (dict(flags=2), INVALID), (dict(ws_bytes=100), INVALID), (dict(finished=0x700000, end_token=1000), INVALID),
    (dict(finished=0x700000, end_token=-1), INVALID), (dict(logits=0x100001), MISALIGNED),
    (dict(logits=0x100002, flags=1), MISALIGNED),
    (dict(scores=0x200002), MISALIGNED), (dict(workspace=0x600008), MISALIGNED), (dict(score=0x500001), MISALIGNED),
    (dict(err_word=0x700002), MISALIGNED),
])
def test_beam_select_refuses(lib, kw, expect):
    assert _select(lib, **kw) == expect
    assert lib.kvq_beam_select(None, None) == INVALID


def test_beam_workspace_bytes(lib):
    for bad in ((0, 4, 1000, 4), (1, 33, 1000, 4), (1, 4, 0, 4), (1, 4, 1000, 33), (1, 1, 3, 4)):
        assert kvq.kvq_beam_workspace_bytes(*bad) == 0
    need = kvq.kvq_beam_workspace_bytes(2, 4, 1000, 8)
    assert need > 0
    assert _select(lib, ws_bytes=need - 1) == INVALID


def _desc(**kw):
    base = dict(batch=2, num_kv_heads=8, head_dim=128, bits=4, group=32, capacity=1024, residual=128, sink=4)
    base.update(kw)
    return kvq.CacheDesc(**base)


NAMES = [n for n, _ in kvq.CacheView._fields_]


def _view(addr, **same):
    return kvq.CacheView(*[P(same.get(n, addr + 0x1000 * i)) for i, n in enumerate(NAMES)])


def _at(addr, name):
    return addr + 0x1000 * NAMES.index(name)


def _reorder(lib, dst=None, src=None, same=(), index=0x900000, flags=0):
    D, S = _desc(**(dst or {})), _desc(**(src or {}))
    dv = _view(0x100000, **{n: _at(0x200000, n) for n in same})
    return lib.kvq_reorder(ctypes.byref(D), ctypes.byref(dv), ctypes.byref(S), ctypes.byref(_view(0x200000)),
                           P(index), flags, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(index=0), INVALID), (dict(index=0x900002), MISALIGNED), (dict(flags=2), INVALID),
    (dict(dst=dict(bits=2)), INVALID), (dict(dst=dict(head_dim=64)), INVALID), (dict(src=dict(num_kv_heads=4)), INVALID),
    (dict(dst=dict(residual=64)), INVALID), (dict(dst=dict(sink=0)), INVALID), (dict(dst=dict(hybrid=1)), INVALID),
    (dict(dst=dict(page_size=32, num_pages=64)), INVALID), (dict(dst=dict(batch=0)), INVALID),
    (dict(src=dict(bits=5)), UNSUPPORTED), (dict(flags=1), INVALID),  # contiguous caches have no pages to share
    (dict(dst=dict(page_size=32, num_pages=64), src=dict(page_size=32, num_pages=64), flags=1), INVALID),  # two pools
] + [(dict(same=(n,)), INVALID) for n in ("k_codes", "v_codes", "k_params", "v_params", "k_res", "v_res", "k_sink",
                                          "v_sink", "packed_len", "res_len", "res_head", "sink_len")])
def test_reorder_refuses(lib, kw, expect):
    assert _reorder(lib, **kw) == expect


def test_reorder_refuses_one_table_or_pools_of_two_sizes(lib):
    pools = ("k_codes", "v_codes", "k_params", "v_params", "k_mode", "v_mode")
    paged = dict(page_size=32, num_pages=64)
    assert _reorder(lib, paged, paged, same=(*pools, "block_table"), flags=1) == INVALID
    assert _reorder(lib, paged, dict(page_size=32, num_pages=65), same=pools, flags=1) == INVALID
    assert _reorder(lib, paged, paged, same=pools[:3], flags=1) == INVALID
    hybrid = dict(paged, hybrid=1)
    assert _reorder(lib, hybrid, hybrid, same=pools[:4], flags=1) == INVALID


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    h = torch.zeros(6, 2, 64, dtype=torch.float16)
    rope, pos = torch.zeros(9, 32, 2), torch.zeros(3, 6, dtype=torch.int32)
    with pytest.raises(ValueError, match="rope"):
        kvq.kvq_rotate(h, h, rope, pos)
    with pytest.raises(ValueError, match=r"\[total\]"):
        kvq.kvq_rotate(None, None, rope, pos)
    with pytest.raises(ValueError, match="logits"):
        kvq.kvq_beam_select(torch.zeros(1, 2, 10), torch.zeros(1, 2), 2)
    a = kvq.KVCache(2, 2, 64, 4, 64, 8, device="cpu")
    with pytest.raises(ValueError, match="index"):
        kvq.kvq_reorder(a.twin(), a, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="paged"):
        a.twin(share_pages=True)
    with pytest.raises(kvq.KvqError):
        kvq.beam_workspace_for(1, 64, 1000, 4, device="cpu")


def test_twins_have_the_shape_and_share_pools_only_when_asked():
    a = kvq.KVCache(2, 3, 64, 3, 64, 8, device="cpu", sink=5, hybrid=1, page_size=32, num_pages=9)
    b, c = a.twin(batch=4, capacity=96), a.twin(share_pages=True)
    assert (b.desc.batch, b.desc.capacity, b.desc.num_pages, b.desc.hybrid, b.desc.sink) == (4, 96, 9, 1, 5)
    assert b.k_codes.data_ptr() != a.k_codes.data_ptr() and b.block_table.shape == (4, 3)
    for n in ("k_codes", "v_codes", "k_params", "v_params", "k_mode", "v_mode"):
        assert getattr(c, n).data_ptr() == getattr(a, n).data_ptr() == getattr(c.view, n)
    assert c.desc.num_pages == 9 and (c.block_table == -1).all()
    assert c.k_res.data_ptr() != a.k_res.data_ptr() and c.block_table.data_ptr() != a.block_table.data_ptr()


def test_axes_of_pairs():
    assert list(kvq.axes_of_pairs((2, 3, 1))) == [0, 0, 1, 1, 1, 2]
    assert list(kvq.axes_of_pairs((2, 3, 1), interleaved=True)) == [0, 1, 2, 0, 1, 1]


def test_prompt_units_refuses(lib):
    good = [0x100000, 2, 10, 5, 4, 64, 0x200000, 3, 0x300000]
    for i, bad in ((0, 0), (1, 0), (2, -1), (3, -1), (4, 0), (5, 0), (6, 0), (7, 0), (8, 0), (8, 0x300008)):
        assert lib.kvq_testing_prompt_units(*[bad if i == j else x for j, x in enumerate(good)]) == INVALID


def test_calls_without_rows_need_no_device(lib):
    assert _rotate(lib, total=0, positions=0) == kvq.KVQ_OK
    assert _prompt(lib, total=0, q=0, k=0, v=0, out=0) == kvq.KVQ_OK
