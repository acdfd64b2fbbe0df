"""Refusals of the binding's calls on runs that need no GPU (tests/test_chunk_abi.py has
the library's)."""

import pytest

from bit_quantized_kv_pack_gb300 import kvq


@pytest.mark.parametrize("stream", [None, 0x1000])
def test_reading_a_cache_in_host_memory_is_refused(stream):
    """Before anything is launched: its arrays' addresses are the host's."""
    cache = kvq.KVCache(2, 2, 64, 4, 64, 8, device="cpu")
    with pytest.raises(ValueError, match="CUDA memory"):
        kvq.kvq_read_tokens(cache, None, 4, stream=stream)
