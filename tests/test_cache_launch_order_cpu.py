"""What the cache kernels' early launches rest on, read from their source: a kernel that may be resident while the
one ahead of it still stores must not load through the read-only path, and must wait before it signals."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_causal_gb300", "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        s = f.read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", s, flags=re.S))


@pytest.mark.parametrize("name", ["cache.cuh", "cache_rw.cu", "cache_attn.cu"])
def test_no_read_only_loads(name):
    """ld.global.nc is for data that nothing writes while the kernel lives; pools, lengths, page tables and
    activations may all be written by the kernel ahead."""
    s = code(name)
    assert not re.findall(r"\b__ldg\s*\(|ld\.global(?:\.\w+)*\.nc", s)
    assert "__restrict__" not in s          # by which the compiler would choose it itself


@pytest.mark.parametrize("name,kernels", [("cache_rw.cu", 2), ("cache_attn.cu", 2)])
def test_signal_stands_after_the_wait(name, kernels):
    bodies = re.split(r"__global__", code(name))[1:]
    assert len(bodies) == kernels
    for body in bodies:
        wait, signal = body.find("wait_for_last_kernel()"), body.find("next_kernel_may_start()")
        assert wait >= 0 and (signal < 0 or wait < signal)
