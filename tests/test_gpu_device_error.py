"""Errors of calls that are given no error word: kept by the library for the device, until read."""

import numpy as np
import pytest
import torch

from bit_quantized_kv_pack_gb300 import kvq

pytestmark = pytest.mark.gpu
DEV = "cuda"
CLEAN = (kvq.KVQ_OK, 0)


@pytest.fixture(autouse=True)
def clean():
    kvq.kvq_read_device_error()
    yield
    assert kvq.kvq_read_device_error() == CLEAN


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prompt(n=300):
    gen = torch.Generator(DEV).manual_seed(n)
    q, k, v = torch.randn(n, 8, 128, generator=gen, device=DEV).half().split([4, 2, 2], 1)
    return q, k, v


def test_a_wait_that_runs_out():
    q, k, v = prompt()
    cu, n = ints([0, 300]), 300
    want = kvq.kvq_prompt_attention(q, k, v, cu, n)
    assert kvq.kvq_read_device_error() == CLEAN
    kvq.kvq_testing_wait_fault(2000)
    try:
        kvq.kvq_prompt_attention(q, k, v, cu, n)
        assert kvq.kvq_read_device_error() == (kvq.KVQ_ERR_TIMEOUT, kvq.KVQ_ERRBIT_TIMEOUT)
    finally:
        kvq.kvq_testing_wait_fault(0)
    assert torch.equal(kvq.kvq_prompt_attention(q, k, v, cu, n), want)


def test_each_call_s_bits():
    q, k, v = prompt()
    kvq.kvq_prompt_attention(q, k, v, ints([0, 301]), 301)
    assert kvq.kvq_read_device_error() == (kvq.KVQ_ERR_INVALID_ARG, kvq.KVQ_ERRBIT_BADLEN)
    rope = kvq.rope_table(50, 128, device=DEV)
    kvq.kvq_rotate(q, k, rope, ints([50] * 300))
    logits = torch.zeros(1, 2, 100, device=DEV)
    logits[0, 1, 7] = float("nan")
    kvq.kvq_beam_select(logits, torch.zeros(1, 2, device=DEV), 3)
    assert kvq.kvq_read_device_error()[1] == kvq.KVQ_ERRBIT_BADPOS | kvq.KVQ_ERRBIT_BADSCORE
    # a word of one's own takes them instead
    err = ints([0])
    kvq.kvq_beam_select(logits, torch.zeros(1, 2, device=DEV), 3, err=err)
    assert err.item() == kvq.KVQ_ERRBIT_BADSCORE


def test_captured_calls_and_other_streams():
    q, k, v = prompt()
    cu, out = ints([0, 300]), torch.empty_like(q)
    kvq.kvq_prompt_attention(q, k, v, cu, 300, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvq.kvq_prompt_attention(q, k, v, cu, 300, out=out)
    g.replay()
    assert kvq.kvq_read_device_error() == CLEAN
    cu.copy_(ints([0, 301]))
    for _ in range(2):
        g.replay()
    assert kvq.kvq_read_device_error()[1] == kvq.KVQ_ERRBIT_BADLEN
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    kvq.kvq_prompt_attention(q, k, v, cu, 300, out=out, stream=st)
    assert kvq.kvq_read_device_error(stream=st)[1] == kvq.KVQ_ERRBIT_BADLEN


def test_bits_that_are_set_while_others_read_are_not_lost():
    """Two streams: each bit is read once or more, none gets lost between a read and its clear."""
    q, k, v = prompt(40)
    good, bad, out = ints([0, 40]), ints([0, 41]), torch.empty(40, 4, 128, dtype=torch.float16, device=DEV)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(50):
        kvq.kvq_prompt_attention(q, k, v, bad if i % 2 else good, 40, out=out, stream=st)
        words = [kvq.kvq_read_device_error()[1]]
        st.synchronize()
        words.append(kvq.kvq_read_device_error()[1])
        assert words[0] | words[1] == (kvq.KVQ_ERRBIT_BADLEN if i % 2 else 0)
