"""What a call makes for itself (a workspace, an output that was not given) belongs to the
stream that it runs on: memory of the current stream could be handed on while the kernels
still use it on the other one, or still be in use by work of the current stream."""

import ctypes

import pytest
import torch

from bit_quantized_kv_pack_gb300 import kvq

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, H, GQ, D = 2, 2, 4, 128


def _make(n=3000, T=40, d=D):
    g = kvq.KVCache(B, H, d, 4, 4096, 16)
    gen = torch.Generator(DEV).manual_seed(3)
    r = lambda *shape: torch.randn(*shape, generator=gen, device=DEV).half()  # noqa: E731
    kvq.kvq_quantize_pack(g, r(B, H, n, d), r(B, H, n, d), torch.full((B,), n, dtype=torch.int32, device=DEV))
    cu = torch.tensor([0, T // 4, T], dtype=torch.int32, device=DEV)
    return g, r(T, H * GQ, d), r(T, H, d), cu, r(B, H * GQ, d), r(B, H, d)


def _calls(d=D):
    """name -> f(stream): the call without outputs or workspace, and what it returns."""
    g, q, k, cu, q1, k1 = _make(d=d)
    T = int(q.shape[0])
    counters, res = g.counters.clone(), [g.k_res.clone(), g.v_res.clone()]

    def back(stream):  # the cache as it was, in the order of the stream
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            g.counters.copy_(counters)
            g.k_res.copy_(res[0])
            g.v_res.copy_(res[1])

    def append(stream):
        back(stream)
        return [kvq.kvq_append_chunk(g, k, k, cu, T, q=q, stream=stream)]

    def step(stream):
        back(stream)
        return [kvq.kvq_decode_step(g, q1, k1, k1, stream=stream)]

    return g, {
        "chunk": lambda s: [kvq.kvq_chunk_attention(g, q, cu, T, stream=s)],
        "cross": lambda s: [kvq.kvq_cross_attention(g, q, cu, T, stream=s, flags=kvq.KVQ_OUT_F32)],
        "read": lambda s: list(kvq.kvq_read_tokens(g, None, 3100, stream=s)),
        "append": append,
        "decode": lambda s: [kvq.kvq_decode_attention(g, q1, stream=s)],
        "noalloc": lambda s: [kvq.kvq_decode_attention_noalloc(g, q1, stream=s)],
        "step": step,
    }


def _stream_of(t):
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


def _taken(f, stream, monkeypatch):
    """(what f returns, the workspaces it made)"""
    made = []
    for name in ("workspace_for", "chunk_workspace_for"):
        real = getattr(kvq, name)

        def keep(*a, real=real):
            made.append(real(*a))
            return made[-1]

        monkeypatch.setattr(kvq, name, keep)
    try:
        return f(stream), made
    finally:
        monkeypatch.undo()


def _same(name, got, want):
    """Bit for bit; the decode's partial sums meet in no fixed order, and each result is
    within 2e-3 of the 64-bit one."""
    tol = 4e-3 if name in ("decode", "noalloc", "step") else 0.0
    return all(bool(((a.float() - b.float()).abs() <= tol).all()) for a, b in zip(got, want))


NAMES = ["chunk", "cross", "read", "append", "decode", "noalloc", "step"]


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_is_its_streams(name, raw, monkeypatch):
    g, calls = _calls()
    want = [t.clone() for t in calls[name](None)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    given = side
    if raw and name not in ("append", "step"):
        given = side.cuda_stream
    got, made = _taken(calls[name], given, monkeypatch)
    assert len(made) == (1 if name in ("chunk", "cross", "decode", "step") else 0)
    for t in got + made:
        assert _stream_of(t) == side.cuda_stream
    torch.cuda.synchronize()
    assert _same(name, got, want)
    # the current stream named as such, and the default stream by its handle
    for s in (torch.cuda.current_stream(), 0) if name not in ("append", "step") else (torch.cuda.current_stream(),):
        got, made = _taken(calls[name], s, monkeypatch)
        assert all(_stream_of(t) == 0 for t in got + made)
        torch.cuda.synchronize()
        assert _same(name, got, want)
    assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)


@pytest.mark.parametrize("d", [64, 128])  # the decode's two kernels
@pytest.mark.parametrize("name", NAMES)
def test_allocations_on_the_current_stream_do_not_reach_a_call_on_another(name, d):
    g, calls = _calls(d)
    want = [t.clone() for t in calls[name](None)]
    ws = kvq.chunk_workspace_for(g, H * GQ).numel(), kvq.workspace_for(g, H * GQ).numel()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    big = torch.empty(1 << 27, dtype=torch.uint8, device=DEV)
    for turn in range(20):
        with torch.cuda.stream(side):
            big.fill_(turn)  # the call's kernels wait behind this
        got = calls[name](side)
        # what the current stream allocates and fills meanwhile
        filled = [torch.full((n,), 0x7F, dtype=torch.uint8, device=DEV) for n in ws]
        filled += [torch.full_like(t, float("nan")) for t in want]
        torch.cuda.current_stream().wait_stream(side)
        assert _same(name, got, want), turn
        del got, filled
    torch.cuda.synchronize()
    assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)


def test_a_returned_output_outlives_its_use_on_the_current_stream():
    """Dropped by the caller while work of the current stream still reads it, its memory is
    not handed to the next call on the side stream before that work is done."""
    g, calls = _calls()
    want = calls["chunk"](None)[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    big = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    copies = []
    for turn in range(10):
        out = calls["chunk"](side)[0]
        torch.cuda.current_stream().wait_stream(side)
        big.fill_(turn)
        copies.append(out.clone())
        del out
        with torch.cuda.stream(side):
            torch.full_like(want, float("nan"))
    torch.cuda.synchronize()
    assert all(torch.equal(c, want) for c in copies)


@pytest.mark.parametrize("name", ["chunk", "cross", "read"])
def test_a_stream_may_be_given_as_a_pointer(name, monkeypatch):
    g, calls = _calls()
    want = [t.clone() for t in calls[name](None)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for handle, stream in ((side.cuda_stream, side.cuda_stream), (None, 0)):
        got, made = _taken(calls[name], ctypes.c_void_p(handle), monkeypatch)
        assert all(_stream_of(t) == stream for t in got + made)
        torch.cuda.synchronize()
        assert _same(name, got, want)
    assert kvq.kvq_read_error(g) == (kvq.KVQ_OK, 0)
