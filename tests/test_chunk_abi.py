"""Host-side refusals of the calls on runs of several tokens (no GPU: every call here
fails its checks before anything is launched)."""

import ctypes

import pytest
import torch

from bit_quantized_kv_pack_gb300 import _build, kvq

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kvq.load()


def _desc(**kw):
    base = dict(batch=2, num_kv_heads=8, head_dim=128, bits=4, group=32, capacity=1000, residual=128)
    base.update(kw)
    return kvq.CacheDesc(**base)


def _view(addr=0x10000):
    return kvq.CacheView(*[P(addr + 0x1000 * i) for i in range(16)])


def _append(lib, desc=None, view=None, **kw):
    base = dict(k=0x100000, v=0x200000, kv_stride_token=1024, kv_stride_head=128, q=0x300000,
                q_out=0x400000, q_stride_token=4096, q_stride_head=128, num_q_heads=32,
                cu_seqlens=0x500000, total=10, max_len=5, rope=0x600000, rope_rows=100, rotary_dim=128,
                interleaved=0, positions=0)
    base.update(kw)
    a = kvq.AppendArgs(**base)
    view = kvq.CacheView() if view == 0 else _view()
    return lib.kvq_append_chunk(ctypes.byref(_desc(**(desc or {}))), ctypes.byref(view),
                                ctypes.byref(a), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(k=0), kvq.KVQ_ERR_INVALID_ARG), (dict(v=0), kvq.KVQ_ERR_INVALID_ARG),
    (dict(cu_seqlens=0), kvq.KVQ_ERR_INVALID_ARG), (dict(total=-1), kvq.KVQ_ERR_INVALID_ARG),
    (dict(max_len=-1), kvq.KVQ_ERR_INVALID_ARG), (dict(kv_stride_token=-8), kvq.KVQ_ERR_INVALID_ARG),
    (dict(kv_stride_head=-8), kvq.KVQ_ERR_INVALID_ARG), (dict(kv_stride_head=12), kvq.KVQ_ERR_MISALIGNED),
    (dict(kv_stride_token=1028), kvq.KVQ_ERR_MISALIGNED), (dict(q_stride_token=4), kvq.KVQ_ERR_MISALIGNED),
    (dict(q_stride_head=-128), kvq.KVQ_ERR_INVALID_ARG), (dict(q_out=0), kvq.KVQ_ERR_INVALID_ARG),
    (dict(num_q_heads=12), kvq.KVQ_ERR_INVALID_ARG), (dict(num_q_heads=0), kvq.KVQ_ERR_INVALID_ARG),
    (dict(rope=0), kvq.KVQ_ERR_INVALID_ARG), (dict(rope_rows=0), kvq.KVQ_ERR_INVALID_ARG),
    (dict(rotary_dim=-16), kvq.KVQ_ERR_INVALID_ARG), (dict(rotary_dim=144), kvq.KVQ_ERR_INVALID_ARG),
    (dict(rotary_dim=24), kvq.KVQ_ERR_UNSUPPORTED), (dict(interleaved=2), kvq.KVQ_ERR_INVALID_ARG),
    (dict(k=0x100008), kvq.KVQ_ERR_MISALIGNED), (dict(v=0x200002), kvq.KVQ_ERR_MISALIGNED),
    (dict(q=0x300004), kvq.KVQ_ERR_MISALIGNED), (dict(q_out=0x400008), kvq.KVQ_ERR_MISALIGNED),
    (dict(rope=0x600008), kvq.KVQ_ERR_MISALIGNED), (dict(cu_seqlens=0x500002), kvq.KVQ_ERR_MISALIGNED),
    (dict(positions=0x700002), kvq.KVQ_ERR_MISALIGNED),
    (dict(desc=dict(bits=5)), kvq.KVQ_ERR_UNSUPPORTED), (dict(desc=dict(batch=0)), kvq.KVQ_ERR_INVALID_ARG),
    (dict(view=0), kvq.KVQ_ERR_INVALID_ARG),
])
def test_append_chunk_refuses(lib, kw, expect):
    assert _append(lib, **kw) == expect
    assert lib.kvq_append_chunk(ctypes.byref(_desc()), ctypes.byref(_view()), None, None) == \
        kvq.KVQ_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["kvq_chunk_attention", "kvq_cross_attention"])
def test_attention_refuses(lib, name):
    D, V = _desc(), _view()
    need = kvq.kvq_chunk_workspace_bytes(D, 32)

    def call(desc=D, q=0x100000, hq=32, cu=0x200000, total=10, max_len=5, out=0x300000, ws=0x400000,
             n=need, flags=0):
        return getattr(lib, name)(ctypes.byref(desc), ctypes.byref(V), P(q), hq, P(cu), total, max_len,
                                  P(out), P(ws), n, flags, None)

    assert need > 0
    for kw in (dict(q=0), dict(hq=12), dict(hq=0), dict(cu=0), dict(total=-1), dict(max_len=-1), dict(out=0),
               dict(ws=0), dict(n=need - 1), dict(flags=1), dict(flags=4)):
        assert call(**kw) == kvq.KVQ_ERR_INVALID_ARG, kw
    for kw in (dict(q=0x100008), dict(out=0x300004), dict(ws=0x400008), dict(cu=0x200002)):
        assert call(**kw) == kvq.KVQ_ERR_MISALIGNED, kw
    assert call(desc=_desc(head_dim=96)) == kvq.KVQ_ERR_UNSUPPORTED
    assert call(total=1 << 30, max_len=1 << 30) == kvq.KVQ_ERR_UNSUPPORTED  # rows of a head pass 2^30


def test_chunk_workspace_bytes(lib):
    assert kvq.kvq_chunk_workspace_bytes(_desc(), 12) == 0
    assert kvq.kvq_chunk_workspace_bytes(_desc(bits=5), 32) == 0
    assert kvq.kvq_chunk_workspace_bytes(_desc(), 0) == 0


def test_read_tokens_refuses(lib):
    D, V = _desc(), _view()

    def call(desc=D, first=0x100000, count=4, k=0x200000, v=0x300000, flags=0):
        return lib.kvq_read_tokens(ctypes.byref(desc), ctypes.byref(V), P(first), count, P(k), P(v), flags, None)

    for kw in (dict(count=-1), dict(k=0), dict(v=0), dict(flags=1)):
        assert call(**kw) == kvq.KVQ_ERR_INVALID_ARG, kw
    for kw in (dict(first=0x100002), dict(k=0x200008), dict(v=0x300004)):
        assert call(**kw) == kvq.KVQ_ERR_MISALIGNED, kw
    assert call(desc=_desc(bits=1)) == kvq.KVQ_ERR_UNSUPPORTED


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    """The binding's own checks (shape, type, place) come before the library is called."""
    cache = kvq.KVCache(2, 2, 64, 4, 64, 8, device="cpu")
    k = torch.zeros(6, 2, 64, dtype=torch.float16)
    cu = torch.tensor([0, 2, 6], dtype=torch.int32)
    with pytest.raises(ValueError, match="cu_seqlens"):
        kvq.kvq_append_chunk(cache, k, k, cu, 4)
    with pytest.raises(ValueError, match="cu_seqlens"):
        kvq.kvq_chunk_attention(cache, k, cu, 4)
    with pytest.raises(ValueError, match=r"\[total\]"):
        kvq.kvq_cross_attention(cache, k[0], cu, 4)
    with pytest.raises(ValueError, match="first"):
        kvq.kvq_read_tokens(cache, torch.zeros(3, dtype=torch.int32), 4)
    with pytest.raises(ValueError, match="float16 or float32"):
        kvq.kvq_read_tokens(cache, None, 4, k_out=torch.zeros(2, 2, 4, 64, dtype=torch.float64))


def test_rope_table_is_the_angles_cosine_and_sine():
    t = kvq.rope_table(70000, 16, base=500.0, device="cpu").double()
    i = torch.arange(8, dtype=torch.float64)
    for pos in (0, 1, 4097, 69999):
        a = pos * 500.0 ** (-2 * i / 16)
        assert torch.equal(t[pos, :, 0].float(), a.cos().float())
        assert torch.equal(t[pos, :, 1].float(), a.sin().float())
