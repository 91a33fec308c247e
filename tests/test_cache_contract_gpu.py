"""The cache calls' contract on the GPU where a caller can lean on it hardest: calls with nothing between them, bytes that
mx_cache_write never writes, magnitudes and scores at the ends of what is taken, a status word with a history.
Bounds as in test_cache_gpu.py, whose helpers (and its three table widths) are used here."""
import numpy as np
import pytest
import torch

from oracle import cache as C
from test_cache_gpu import (DT, HEADS, Filled, bits, check_attn, f64, i32, make_q, ops, table_width,  # noqa: F401
                            widened)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("captured", [False, True])
def test_read_write_read_with_nothing_between(ops, fmt, captured):
    """read, write, read, attend, write, read, ... of the same positions, all small enough to be launched early and no
    other kernel between them: each sees what the last write before it left."""
    B, T, Hq, Hkv, D, page, steps = 4, 16, 8, 4, 128, 16, 24
    cache = ops.mx_cache_alloc(B, page, Hkv, D, fmt)
    table, lens = widened(i32([[2], [0], [3], [1]]), page), i32([T] * B)
    sets = [[make_q(100 + 2 * i + j, B, T, Hkv, D, "bf16", 0, mult=2.0 ** (3 * i)) for j in range(2)] for i in range(3)]
    q = make_q(7, B, T, Hq, D, "bf16", 0, mult=2.0 ** -3)
    want = []
    for k, v in sets:
        ops.mx_cache_write(cache, k, v, table, lens)
        torch.cuda.synchronize()
        kv = ops.mx_cache_read(cache, table, lens, T)
        torch.cuda.synchronize()
        want.append(kv + ops.mx_cache_attn(q, cache, table, lens))
        torch.cuda.synchronize()
    need = max(16, ops.mx_cache_attn_workspace_bytes(B, T, Hq, Hkv, D, table.shape[1] * page))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = [[torch.empty_like(x) for x in want[0][:2] + want[0]] for _ in range(steps)]

    def run():
        for i in range(steps):
            ops.mx_cache_read(cache, table, lens, T, k_out=outs[i][0], v_out=outs[i][1])      # the last step's
            ops.mx_cache_write(cache, *sets[i % 3], table, lens)
            ops.mx_cache_read(cache, table, lens, T, k_out=outs[i][2], v_out=outs[i][3])
            ops.mx_cache_attn(q, cache, table, lens, o=outs[i][4], lse=outs[i][5], workspace=ws)

    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        run = g.replay
    for _ in range(10):
        run()
        torch.cuda.synchronize()
        for i, got in enumerate(outs):
            for x, w in zip(got, want[(i - 1) % 3][:2] + want[i % 3]):
                assert torch.equal(bits(x), bits(w)), i
            for x in got:
                x.zero_()
