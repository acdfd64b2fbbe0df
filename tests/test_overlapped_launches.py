"""Rules for kernels that may begin while the kernel before them runs, read from their sources
(a race need not show when it is run)."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_kv_pack_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu*")))


def code(path):
    """A source without its comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)


def kernels(text):
    """(name, body) of each kernel: to the next one, or the end."""
    at = [(m.start(), re.compile(r"(\w+)\s*\(").search(re.sub(r"__launch_bounds__\([^)]*\)", "", text[m.end():])).group(1))
          for m in re.finditer(r"__global__ void", text)]
    for (lo, name), hi in zip(at, [lo for lo, _ in at[1:]] + [len(text)]):
        yield name, text[lo:hi]


def test_a_kernel_that_waits_lets_the_next_begin_after_its_wait():
    """Otherwise the next one may begin before the kernel before this one is done, and
    KVQ_STEP_EARLY_CACHE_READ reads what that one still writes."""
    wait, trigger = re.compile(r"griddepcontrol\.wait|grid_dependency_wait\(\)|wait_for_previous\(\)"), "griddepcontrol.launch_dependents"
    seen = 0
    for path in SOURCES:
        for name, body in kernels(code(path)):
            waits = wait.search(body)
            if waits and trigger in body:
                assert waits.start() < body.index(trigger), (os.path.basename(path), name)
                seen += 1
    assert seen >= 4  # the step, both kernels of the attention of runs, the end of their append


def test_kernels_that_begin_early_have_no_read_only_loads():
    """Read-only loads are for data that nothing writes while the kernel runs, and these run
    before the kernel that writes it is done: a compiler may move such a load over the wait."""
    for name in ("kvq_internal.cuh", "kvq_runs.cuh", "kvq_around.cuh", "kvq_rotate.cu", "kvq_beam.cu", "kvq_reorder.cu",
                 "kvq_prompt_attn.cuh", "kvq_chunk_attn.cuh", "kvq_decode_tc.cu"):
        text = code(os.path.join(CSRC, name))
        assert not re.search(r"__ldg\(|ld\.global\.nc|__restrict__", text), name
