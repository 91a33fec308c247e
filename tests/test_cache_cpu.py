"""The key/value cache on the CPU: the oracle's E2M1 arithmetic against worked values, the oracle's
attention against a brute-force sum, the ctypes structures' layout, and every argument check that is
made before a device is touched."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from oracle import cache as C
from oracle import mx


@pytest.fixture(scope="module")
def ops():
    from block_scaled_causal_gb300 import build
    if not os.path.exists(build.LIB_PATH):
        build.build()
    from block_scaled_causal_gb300 import _binding
    return _binding


# --------------------------------------------------------------------------------------- the oracle
def test_e2m1_worked_values():
    # every midpoint goes to the even code: .25 -> 0, .75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    y = np.array([0.0, 0.25, 0.26, 0.75, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, 6.0, 7.9, -0.25, -0.3, -1.75])
    want = [0, 0, 0.5, 1, 1, 1.5, 2, 2, 3, 4, 4, 6, 6, 6, 0, -0.5, -2]
    np.testing.assert_array_equal(C.e2m1_decode(C.e2m1_encode(y)), want)
    assert C.e2m1_encode(np.array([-0.25]))[0] == 8          # the sign of zero is kept
    np.testing.assert_array_equal(C.e2m1_encode(C.e2m1_decode(np.arange(16))), np.arange(16))


def test_fp4_blocks():
    x = np.zeros((3, 64))
    x[0, 1] = 5.0                        # amax 5: e = floor(log2 5) - 2 = 0
    x[0, 33] = -0.75                     # amax .75: e = -1 - 2 = -3, -.75 * 8 = -6
    x[1, 0], x[1, 2] = 7.5, 1.0          # saturates under the floor rule, not under ceil
    x[2, 40] = np.inf
    data, sb = C.quantize(x, C.FP4)
    assert list(sb[0]) == [127, 124] and data[0, 0] == 0x60 and data[0, 16] == 0xF0
    assert list(sb[1]) == [127, 0] and data[1, 0] == 0x07 and data[1, 1] == 0x02
    assert sb[2, 1] == 0xFF and np.all(data[2, 16:] == 0x77) and sb[2, 0] == 0
    d1, s1 = C.quantize(x, C.FP4, "ceil")
    assert s1[1, 0] == 128 and C.dequantize(d1, s1, C.FP4)[1, 0] == 8.0
    assert s1[0, 0] == 127 and np.isnan(C.dequantize(data, sb, C.FP4)[2, 40])


@pytest.mark.parametrize("rule", ["floor", "ceil"])
def test_fp4_round_trip_bound(rule):
    # half a step: 2^-2 of the value above the smallest normal, a quarter of the scale below it; the floor rule
    # saturates values in (6, 8) * scale, off by at most 2 * scale
    rng = np.random.default_rng(5)
    x = rng.standard_normal((50, 128)) * np.exp(3 * rng.standard_normal((50, 1)))
    data, sb = C.quantize(x, C.FP4, rule)
    s = np.repeat(mx.e8m0_decode(sb), 32, -1)
    y, d = np.abs(x) / s, np.abs(C.dequantize(data, sb, C.FP4) - x) / s
    assert np.all(d[y < 1] <= 0.25) and np.all(d[(y >= 1) & (y <= 6)] <= 0.25 * y[(y >= 1) & (y <= 6)])
    assert np.all(y < 8) and (rule == "floor" or np.all(y <= 6))


def test_oracle_attend_is_the_sum():
    rng = np.random.default_rng(2)
    T, Hq, Hkv, D, held, n = 3, 4, 2, 64, 9, 2
    q, K, V = (rng.standard_normal(s) for s in ((T, Hq, D), (held, Hkv, D), (held, Hkv, D)))
    O, L, A, E = C.attend(q, K, V, held, n, 0.125, absent={4})
    for t in range(T):
        for h in range(Hq):
            js = [j for j in range(held - n + t + 1) if j != 4] if t < n else []
            w = [math.exp(0.125 * sum(q[t, h, d] * K[j, h // 2, d] for d in range(D))) for j in js]
            want = sum(wi * V[j, h // 2] for wi, j in zip(w, js)) / sum(w) if js else np.zeros(D)
            np.testing.assert_allclose(O[t, h], want, rtol=1e-12, atol=1e-14)
            if js:
                assert abs(L[h, t] - math.log(sum(w))) < 1e-12
            else:
                assert L[h, t] == -np.inf
    assert np.all(A >= np.abs(O)) and np.all(E >= 0)


def test_gather_crosses_pages():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((3, 2, 16, 64))
    data, sb = C.quantize(x, C.FP4)
    got = C.gather(data, sb, C.FP4, [2, -1, 0], 37, 16)
    np.testing.assert_array_equal(got[:16, 1], C.dequantize(data[2, 1], sb[2, 1], C.FP4))
    assert np.all(np.isnan(got[16:32]))
    np.testing.assert_array_equal(got[36, 0], C.dequantize(data[0, 0, 4], sb[0, 0, 4], C.FP4))


# ------------------------------------------------------------------------------- structures, refusals
def test_struct_layouts(ops):
    # LP64: 4 pointers, 4 longs, 5 ints (padded to 8)
    assert ctypes.sizeof(ops.CachePools) == 88 and ops.CachePools.format.offset == 64
    W, R, A = ops.CacheWriteParams, ops.CacheReadParams, ops.CacheAttnParams
    assert W.k.offset == 88 and W.k_stride_b.offset == 104 and W.B.offset == 152 and W.rule.offset == 164
    assert W.page_table.offset == 168 and W.max_pages.offset == 184 and W.seq_lens.offset == 192
    assert W.dev_status.offset == 208 and ctypes.sizeof(W) == 216
    assert R.B.offset == 152 and R.page_table.offset == 168 and R.starts.offset == 200 and ctypes.sizeof(R) == 216
    assert A.q.offset == 88 and A.lse.offset == 104 and A.q_stride_b.offset == 112 and A.B.offset == 160
    assert A.softmax_scale.offset == 176 and A.page_table.offset == 184 and A.max_pages.offset == 200
    assert A.seq_lens.offset == 208 and A.workspace.offset == 232 and ctypes.sizeof(A) == 248


FAKE = 0x100000   # aligned, never dereferenced: every call below is refused first


def _pools(ops, **kw):
    base = dict(k=FAKE, k_sc=FAKE, v=FAKE, v_sc=FAKE, k_page_stride=4 * 16 * 64, k_sc_page_stride=4 * 16 * 4,
                v_page_stride=4 * 16 * 64, v_sc_page_stride=4 * 16 * 4, format=ops.CACHE_MXFP4, num_pages=8,
                page_size=16, Hkv=4, D=128)
    base.update(kw)
    return ops.CachePools(**base)


POOL_CASES = [
    (dict(k=0), 1),
    (dict(v_sc=0), 1),
    (dict(k_sc=FAKE + 8), 3),
    (dict(v=FAKE + 4), 3),
    (dict(format=2), 4),
    (dict(D=96), 4),
    (dict(D=256), 4),
    (dict(page_size=24), 4),
    (dict(page_size=0), 2),
    (dict(num_pages=0), 2),
    (dict(num_pages=-1), 2),
    (dict(Hkv=-4), 2),
    (dict(k_page_stride=4 * 16 * 64 - 16), 2),       # pages would overlap
    (dict(v_sc_page_stride=4 * 16 * 4 - 16), 2),
    (dict(k_page_stride=4 * 16 * 64 + 8), 3),
    (dict(v_page_stride=1 << 36), 4),
    (dict(page_size=1 << 22, k_page_stride=1 << 30, v_page_stride=1 << 30), 4),   # 2^31 elements a page
]
COMMON = [
    (dict(B=-1), 2),
    (dict(T=-1), 2),
    (dict(dtype=2), 4),
    (dict(page_table=0), 1),
    (dict(seq_lens=0), 1),
    (dict(page_table=FAKE + 2), 3),
    (dict(seq_lens=FAKE + 1), 3),
    (dict(dev_status=FAKE + 2), 3),
    (dict(table_stride=31), 2),
    (dict(max_pages=-1), 2),
    (dict(max_pages=1 << 27, table_stride=1 << 27), 4),   # 2^31 positions
    (dict(max_pages=(1 << 26) + 1, table_stride=1 << 27), 4),   # 2^30 + 16
    (dict(B=1 << 20, T=1 << 12), 4),
    (dict(T=0), 0),
    (dict(B=0, page_table=0), 0),
]


def _strides(names):
    return {"%s_stride_%s" % (n, d): v for n in names for d, v in (("b", 2048), ("t", 512), ("h", 128))}


@pytest.mark.parametrize("pool,kw,want", [(p, {}, w) for p, w in POOL_CASES] + [({}, k, w) for k, w in COMMON] + [
    ({}, dict(k=0), 1), ({}, dict(v=FAKE + 8), 3), ({}, dict(rule=2), 4), ({}, dict(new_lens=FAKE + 2), 3),
    ({}, dict(k_stride_t=516), 3), ({}, dict(v_stride_h=12), 3)])
def test_write_refusals(ops, pool, kw, want):
    base = dict(k=FAKE, v=FAKE, B=2, T=4, dtype=0, rule=0, page_table=FAKE, table_stride=32, max_pages=32,
                seq_lens=FAKE, new_lens=FAKE, dev_status=FAKE, **_strides("kv"))
    p = ops.CacheWriteParams(cache=_pools(ops, **pool), **dict(base, **kw))
    assert ops.lib.mx_cache_write(ctypes.byref(p), None) == want


@pytest.mark.parametrize("pool,kw,want", [(p, {}, w) for p, w in POOL_CASES] + [({}, k, w) for k, w in COMMON] + [
    ({}, dict(k=0), 1), ({}, dict(v=FAKE + 8), 3), ({}, dict(starts=FAKE + 2), 3), ({}, dict(k_stride_t=516), 3),
    ({}, dict(v_stride_b=0), 2), ({}, dict(k_stride_h=0), 2)])
def test_read_refusals(ops, pool, kw, want):
    base = dict(k=FAKE, v=FAKE, B=2, T=4, dtype=0, page_table=FAKE, table_stride=32, max_pages=32, seq_lens=FAKE,
                starts=FAKE, dev_status=FAKE, **_strides("kv"))
    p = ops.CacheReadParams(cache=_pools(ops, **pool), **dict(base, **kw))
    assert ops.lib.mx_cache_read(ctypes.byref(p), None) == want


@pytest.mark.parametrize("pool,kw,want", [(p, {}, w) for p, w in POOL_CASES] + [({}, k, w) for k, w in COMMON] + [
    ({}, dict(q=0), 1), ({}, dict(o=0), 1), ({}, dict(o=FAKE + 8), 3), ({}, dict(lse=FAKE + 2), 3),
    ({}, dict(Hq=6), 2), ({}, dict(Hq=-8), 2), ({}, dict(Hq=0), 0), ({}, dict(softmax_scale=0.0), 4),
    ({}, dict(softmax_scale=float("nan")), 4), ({}, dict(softmax_scale=-1.0), 4), ({}, dict(q_stride_t=516), 3),
    ({}, dict(o_stride_h=0), 2), ({}, dict(workspace=FAKE + 8), 3), ({}, dict(new_lens=FAKE + 2), 3),
    ({}, dict(max_pages=1 << 16, table_stride=1 << 16, workspace=0), 1),
    ({}, dict(max_pages=1 << 16, table_stride=1 << 16, workspace_bytes=1 << 16), 2)])
def test_attn_refusals(ops, pool, kw, want):
    base = dict(q=FAKE, o=FAKE, lse=FAKE, B=2, T=4, Hq=8, dtype=0, softmax_scale=0.088, page_table=FAKE,
                table_stride=32, max_pages=32, seq_lens=FAKE, new_lens=FAKE, dev_status=FAKE, workspace=FAKE,
                workspace_bytes=1 << 40, **_strides("qo"))
    p = ops.CacheAttnParams(cache=_pools(ops, **pool), **dict(base, **kw))
    assert ops.lib.mx_cache_attn(ctypes.byref(p), None) == want


def test_null_params_and_status(ops):
    for f in ("mx_cache_write", "mx_cache_read", "mx_cache_attn"):
        assert getattr(ops.lib, f)(None, None) == 1
    assert ops.lib.bsc_status_string(7).decode().startswith("BSC_ERR_DEVICE_PAGE")


def test_workspace_bytes(ops):
    for bad in ((0, 1, 8, 4, 128), (1, 0, 8, 4, 128), (1, 1, 0, 4, 128), (1, 1, 8, 0, 128), (1, 1, 8, 4, 0)):
        assert ops.mx_cache_attn_workspace_bytes(*bad) == 0
    # short tables need none; long ones the same whatever their length, two slots of fp32 rows per block
    assert ops.mx_cache_attn_workspace_bytes(1, 1, 8, 4, 128, 1024) == 0
    assert ops.mx_cache_attn_workspace_bytes(1, 1, 8, 4, 128, 1 << 20) == 2 * 456 * 8 * 129 * 4
    assert ops.mx_cache_attn_workspace_bytes(8, 4, 8, 2, 64, 1 << 17) == 2 * 304 * 16 * 65 * 4
    assert ops.mx_cache_attn_workspace_bytes(8, 40, 8, 2, 64) == 2 * 304 * 32 * 65 * 4
    # sizes that no call takes: a table past the limit as one at the limit, a batch past it nothing
    assert ops.mx_cache_attn_workspace_bytes(8, 40, 8, 2, 64, (1 << 63) - 1) == 2 * 304 * 32 * 65 * 4
    assert ops.mx_cache_attn_workspace_bytes(1 << 30, 1 << 30, 1 << 30, 1, 128) == 0


def test_binding_refuses_cpu_pools(ops):
    z = lambda n: torch.zeros((2, 4, 16, n), dtype=torch.uint8)  # noqa: E731
    with pytest.raises(ValueError):
        ops.MxCache(z(64), z(4), z(64), z(4))
    with pytest.raises(ValueError):
        ops.MxCache(z(64), z(4), z(64), z(4), fmt=3)
