"""The norm, rotary positions and sparse cache attention on the CPU: structures, frequencies, the oracle against worked sums,
workspace sizes and every refusal that is made before a device is touched."""
import ctypes
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

from oracle import operands as R
from test_cache_launch_order_cpu import code
from test_cache_cpu import COMMON, FAKE, POOL_CASES, _pools, _strides, ops  # noqa: F401

NULL, SHAPE, ALIGN, UNSUPPORTED = 1, 2, 3, 4


# --------------------------------------------------------------------------------------- the oracle
def test_norm_bwd_is_the_derivative():
    rng = np.random.default_rng(0)
    s, w, dy = rng.standard_normal((2, 16)), rng.standard_normal(16), rng.standard_normal((2, 16))
    f = lambda s, w: np.sum(R.norm(s, w, 1e-3)[0] * dy)  # noqa: E731
    dx, dw, _, _ = R.norm_bwd(dy, s, w, R.norm(s, w, 1e-3)[1])
    h = 1e-6
    for i in range(2):
        for j in range(16):
            e = np.zeros_like(s)
            e[i, j] = h
            assert abs((f(s + e, w) - f(s - e, w)) / (2 * h) - dx[i, j]) < 1e-7
    for j in range(16):
        e = np.eye(16)[j] * h
        assert abs((f(s, w + e) - f(s, w - e)) / (2 * h) - dw[j]) < 1e-7


@pytest.mark.parametrize("interleaved", [0, 1])
def test_rotation_keeps_distances(interleaved):
    """q . k after rotation goes by the positions' difference; the inverse is the gradient (the transpose)."""
    rng = np.random.default_rng(1)
    x, y = rng.standard_normal((2, 1, 1, 1, 48))
    turns = np.array([2 ** 62 + 12345, 2 ** 55, 987654321012345, 77], np.uint64).repeat(2)
    r = lambda x, p, inv=False: R.rotate(x, R.angles(turns, np.array([[p]])), 1.0, interleaved, inv)[0]  # noqa: E731
    for p in (0, 1, -5, 100003, 2 ** 31 - 8):
        assert abs(np.sum(r(x, p + 7) * r(y, p)) - np.sum(r(x, 7) * y)) < 1e-12
        assert abs(np.sum(r(x, p) * y) - np.sum(x * r(y, p, True))) < 1e-12
        assert np.array_equal(r(x, p)[..., 16:], x[..., 16:])


def test_bounds_hold_and_choice():
    rng = np.random.default_rng(2)
    K = np.round(rng.standard_normal((20, 3, 64)) * 8) / 8
    codes, exps = R.page_bounds(K)
    v = codes * np.exp2(exps.astype(float) - 127)[:, None, None]
    assert np.all(v[:, 0] <= K.min(0)) and np.all(v[:, 1] >= K.max(0)) and np.abs(codes).max() <= 128
    q = rng.standard_normal((2, 64))
    assert np.all(np.maximum(q, 0).sum(0) @ v[0, 1] - np.maximum(-q, 0).sum(0) @ v[0, 0] >= (q @ K[:, 0].T).sum(0))
    codes, exps = np.zeros((6, 2, 64), np.int8), np.full(6, 127, np.uint8)
    codes[:, 1, 0] = [5, 9, 5, 9, 1, 0]
    q = np.zeros((1, 64))
    q[0, 0] = 1.0
    pick = lambda top, first, last, pages=range(6): R.choose(q, codes, exps, list(pages), 90, 16, top, first, last)  # noqa: E731
    assert pick(6, 0, 1) == [0, 1, 2, 3, 4, 5] and pick(3, 0, 1) == [1, 3, 5] and pick(4, 0, 1) == [0, 1, 3, 5]
    assert pick(2, 1, 1) == [0, 5] and pick(3, 0, 1, [0, None, 2, 3, 4, 5]) == [0, 3, 5]
    exps[4] = 0xFF
    assert pick(2, 0, 1) == [4, 5]


# -------------------------------------------------------------------------------------- frequencies
@pytest.mark.parametrize("rot", [16, 48, 128, 256])
@pytest.mark.parametrize("scaling,factor", [("PLAIN", 3.0), ("LINEAR", 4.0), ("BASE", 8.0), ("BY_PARTS", 8.0), ("BY_PARTS", 1.0)])
def test_turns(ops, rot, scaling, factor):  # noqa: F811
    getcontext().prec = 50
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097")
    base, length = Decimal(10000), 4096
    r = ops.Rope(rot, base=10000.0, scaling=getattr(ops, "ROPE_" + scaling), factor=factor, original_length=length, device="cpu")
    f = Decimal(factor)
    if scaling == "BASE":
        base = base * f ** (Decimal(rot) / Decimal(rot - 2))
    got = [int(t) % 2 ** 64 for t in r.turns.tolist()]
    for i in range(rot // 2):
        want = base ** (-Decimal(2 * i) / Decimal(rot)) / (2 * pi)
        if scaling == "LINEAR":
            want = want / f
        if scaling == "BY_PARTS":
            k = min(max((length * want - 1) / 31, Decimal(0)), Decimal(1))
            want = want * (k + (1 - k) / f)
        # a power and a few products and sums in fp64, whatever cancels in k: 2^-44 is 512 steps
        assert abs(Decimal(got[i]) / 2 ** 64 - want) <= want * Decimal(2) ** -44
    m = 0.1 * math.log(factor) + 1 if scaling == "BY_PARTS" else 1.0
    assert abs(r.magnitude - m) <= 2 ** -23 and ops.Rope(rot, magnitude=0.5, device="cpu").magnitude == 0.5


@pytest.mark.parametrize("rot", [16, 32, 96, 128, 256])
@pytest.mark.parametrize("base", [1.0, 1.7, 10000.0, 500000.0, 1e7, 1e300])
@pytest.mark.parametrize("scaling,factor", [("PLAIN", 1.0), ("LINEAR", 3.0), ("BASE", 1.3), ("BASE", 40.0), ("BY_PARTS", 1.0),
                                            ("BY_PARTS", 7.3)])
def test_turns_are_exact_to_64_bits(ops, rot, base, scaling, factor):  # noqa: F811
    """Every frequency is the formula's to 2^-64 turns (half a unit but for what 106 bits leave), so that the angle at 2^31
    tokens is within 2^-33."""
    getcontext().prec = 70
    two_pi = 2 * Decimal("3.1415926535897932384626433832795028841971693993751058209749445923078164062862")
    r = ops.Rope(rot, base=base, scaling=getattr(ops, "ROPE_" + scaling), factor=factor, original_length=8192, low_turns=0.7,
                 high_turns=33.3, device="cpu")
    b, f, low, high = Decimal(base), Decimal(factor), Decimal(0.7), Decimal(33.3)
    if scaling == "BASE":
        b = b * f ** (Decimal(rot) / Decimal(rot - 2))
    for i, t in enumerate(r.turns.tolist()):
        want = b ** (-Decimal(2 * i) / Decimal(rot)) / two_pi
        if scaling == "LINEAR":
            want = want / f
        if scaling == "BY_PARTS":
            k = min(max((8192 * want - low) / (high - low), Decimal(0)), Decimal(1))
            want = want * (k + (1 - k) / f)
        off = Decimal(t % 2 ** 64) - want * 2 ** 64
        assert abs(off) <= Decimal(0.5) + Decimal(2) ** -20, (i, off)


def test_turns_of_a_small_base(ops):  # noqa: F811
    """Frequencies of a turn and more: the fraction, to what 104 bits of the whole leave; none is left of the largest."""
    getcontext().prec = 70
    two_pi = 2 * Decimal("3.1415926535897932384626433832795028841971693993751058209749445923078164062862")
    r = ops.Rope(32, base=1e-6, device="cpu")
    for i, t in enumerate(r.turns.tolist()):
        want = Decimal(1e-6) ** (-Decimal(2 * i) / 32) / two_pi
        off = (Decimal(t % 2 ** 64) - want * 2 ** 64) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= Decimal(0.5) + Decimal(2) ** -20
    for base in (1e-300, 5e-324):
        assert len(ops.Rope(16, base=base, device="cpu").turns) == 8


@pytest.mark.parametrize("kw", [
    dict(rot=0), dict(rot=8), dict(rot=24), dict(rot=272), dict(rot=-16), dict(scaling=4), dict(scaling=-1), dict(base=0.0),
    dict(base=-1.0), dict(base=math.inf), dict(base=math.nan), dict(scaling=1, factor=0.0), dict(scaling=2, factor=math.nan),
    dict(scaling=2, factor=1e300, base=1e300), dict(scaling=3, factor=0.5, original_length=64),
    dict(scaling=3, factor=2.0, original_length=0), dict(scaling=3, factor=2.0, original_length=64, low_turns=32.0),
    dict(scaling=3, factor=2.0, original_length=64, low_turns=-1.0), dict(scaling=3, factor=2.0, original_length=math.nan)])
def test_rope_refusals(ops, kw):  # noqa: F811
    with pytest.raises(ops.BscError) as e:
        ops.Rope(**{"rot": 64, "device": "cpu", **kw})
    assert e.value.status == UNSUPPORTED


def test_magnitude_in_two_floats(ops):  # noqa: F811
    """A Rope's factor is a double, passed as its nearest float and the rest; the C call refuses a rest that is none."""
    r = ops.Rope(64, scaling=ops.ROPE_BY_PARTS, factor=8.0, original_length=8192, device="cpu")
    assert r.magnitude == 0.1 * math.log(8.0) + 1.0
    for m in (r.magnitude, 1.0, 0.7, -1.3, 0.0, 1e-40, 3e38):
        p = ops.Rope(64, magnitude=m, device="cpu").params
        assert p.magnitude == np.float32(m) and abs(p.magnitude_low) <= abs(p.magnitude) * 2.0 ** -24
        assert m == 1e-40 or abs(p.magnitude + p.magnitude_low - m) <= abs(m) * 2.0 ** -47
    x = dict(q=FAKE, q_out=FAKE, B=2, T=4, Hq=4, D=128, dtype=0, inverse=0, **_strides(("q", "q_out")))
    for low, want in ((1e-6, UNSUPPORTED), (-1e-6, UNSUPPORTED), (math.nan, UNSUPPORTED), (1e-8, ALIGN)):
        a = _angles(ops, magnitude_low=low)
        assert ops.lib.rope(ctypes.byref(ops.RopeParams(angles=a, **dict(x, q=FAKE + 8))), None) == want
    assert ops.lib.bsc_rope_magnitude(None) == 1.0


# ------------------------------------------------------------------------------- structures, sizes
def test_struct_layouts(ops):  # noqa: F811
    sizes = dict(RmsNormParams=160, RmsNormBwdParams=160, RopeConfig=48, RopeAngles=24, RopeParams=208, RopeQuantParams=176,
                 CacheWriteRopeParams=312, CacheBoundsParams=160, CacheSparseAttnParams=280)
    for n, size in sizes.items():
        assert ctypes.sizeof(getattr(ops, n)) == size, n
    assert ops.RmsNormParams.rows.offset == 64 and ops.RmsNormParams.inner.offset == 136 and ops.RmsNormParams.eps.offset == 156
    assert ops.RmsNormBwdParams.inner.offset == 128 and ops.RmsNormBwdParams.workspace.offset == 144
    assert ops.RopeParams.q.offset == 24 and ops.RopeParams.positions.offset == 152 and ops.RopeParams.B.offset == 176
    assert ops.RopeQuantParams.q_e4m3.offset == 88 and ops.RopeQuantParams.B.offset == 144
    assert ops.CacheWriteRopeParams.angles.offset == 88 and ops.CacheWriteRopeParams.q.offset == 112
    assert ops.CacheWriteRopeParams.page_table.offset == 264 and ops.CacheBoundsParams.page_table.offset == 112
    assert ops.CacheSparseAttnParams.softmax_scale.offset == 200 and ops.CacheSparseAttnParams.page_table.offset == 216


def test_workspaces(ops):  # noqa: F811
    for bad in ((0, 64), (-1, 64), (4, 0), (4, 12), (4, 16392)):
        assert ops.rms_norm_bwd_workspace_bytes(*bad) == 0
    assert ops.rms_norm_bwd_workspace_bytes(1, 16384) == 16384 * 4
    assert ops.rms_norm_bwd_workspace_bytes(1 << 39, 128) == ops.rms_norm_bwd_workspace_bytes(1 << 20, 128)
    f = ops.mx_cache_sparse_attn_workspace_bytes
    good = (2, 1, 16, 4, 128, 64, 500, 32)
    assert f(*good) >= 8 * 32 * 4 + 8 * 4
    assert f(2, 1, 16, 4, 128, 16, 20000, 32) >= 8 * 20000 * 4 + 8 * 32 * 4      # a table whose scores go through it
    for i in range(8):
        assert f(*(good[:i] + (-1,) + good[i + 1:])) == 0
    assert f(2, 1, 16, 4, 128, 64, 0, 32) >= 32                       # a table of no pages
    assert f(1 << 14, 1, 16, 4, 128, 64, 1 << 15, 32) == 0           # 2^31 scores
    assert f(1 << 20, 1, 16, 8, 128, 64, 16, 256) == 0               # 2^31 chosen pages


@pytest.mark.parametrize("i,bad", [(2, 2), (2, 6), (4, 96), (4, 256), (5, 24), (6, 1 << 25)])
def test_workspace_of_refused_sizes(ops, i, bad):  # noqa: F811
    """What mx_cache_sparse_attn refuses needs no workspace: heads that are not shared evenly, head sizes, pages, long tables."""
    good = (2, 1, 16, 4, 128, 64, 500, 32)
    assert ops.mx_cache_sparse_attn_workspace_bytes(*good) > 0
    assert ops.mx_cache_sparse_attn_workspace_bytes(*good[:i], bad, *good[i + 1:]) == 0


# -------------------------------------------------------------------------------------- refusals
def _norm(ops, **kw):
    base = dict(x=FAKE, residual=FAKE, weight=FAKE, y=FAKE, sum=FAKE, rstd=FAKE, y_e4m3=FAKE, y_sc=FAKE, rows=6, inner=2, N=64,
                dtype=0, weight_dtype=2, rule=0, eps=1e-6)
    for n in ("x", "residual", "y", "sum"):
        base.update({n + "_stride": 256, n + "_inner_stride": 64})
    return ops.RmsNormParams(**dict(base, **kw))


@pytest.mark.parametrize("kw,want", [
    (dict(x=0), NULL), (dict(weight=0), NULL), (dict(y=0, y_e4m3=0), NULL), (dict(y_sc=0), NULL), (dict(rows=-1), SHAPE),
    (dict(N=-8), SHAPE), (dict(inner=0), SHAPE), (dict(rows=0, x=0), 0), (dict(N=0, x=0), 0), (dict(N=60), UNSUPPORTED),
    (dict(N=72), UNSUPPORTED), (dict(N=16416), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
    (dict(weight_dtype=1), UNSUPPORTED), (dict(weight_dtype=3), UNSUPPORTED), (dict(rule=2), UNSUPPORTED),
    (dict(eps=-1e-6), UNSUPPORTED), (dict(eps=math.inf), UNSUPPORTED), (dict(eps=math.nan), UNSUPPORTED),
    (dict(x=FAKE + 8), ALIGN), (dict(residual=FAKE + 2), ALIGN), (dict(y=FAKE + 8), ALIGN), (dict(rstd=FAKE + 2), ALIGN),
    (dict(y_e4m3=FAKE + 8), ALIGN), (dict(x_stride=252), ALIGN), (dict(residual_inner_stride=12), ALIGN),
    (dict(y_stride=0), SHAPE), (dict(sum_inner_stride=0), SHAPE), (dict(rows=1 << 38), UNSUPPORTED), (dict(rows=(1 << 38) - 1, x=0), NULL)])
def test_norm_refusals(ops, kw, want):  # noqa: F811
    assert ops.lib.rms_norm(ctypes.byref(_norm(ops, **kw)), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dy=0), NULL), (dict(s=0), NULL), (dict(rstd=0), NULL), (dict(dx=0), NULL), (dict(dweight=0), NULL),
    (dict(workspace=0), NULL), (dict(workspace=FAKE + 8), ALIGN), (dict(d_sum=FAKE + 4), ALIGN), (dict(dweight=FAKE + 8), ALIGN),
    (dict(workspace_bytes=100), SHAPE), (dict(dx_stride=0), SHAPE), (dict(dy_stride=4), ALIGN), (dict(N=12), UNSUPPORTED),
    (dict(rows=0), 0), (dict(inner=-1), SHAPE), (dict(dtype=2), UNSUPPORTED)])
def test_norm_bwd_refusals(ops, kw, want):  # noqa: F811
    base = dict(dy=FAKE, s=FAKE, weight=FAKE, rstd=FAKE, d_sum=FAKE, dx=FAKE, dweight=FAKE, rows=6, inner=1, N=64, dtype=0,
                weight_dtype=0, workspace=FAKE, workspace_bytes=1 << 30)
    for n in ("dy", "s", "d_sum", "dx"):
        base[n + "_stride"] = 64
    p = ops.RmsNormBwdParams(**dict(base, **kw))
    assert ops.lib.rms_norm_bwd(ctypes.byref(p), None) == want


@pytest.mark.parametrize("a,want", [
    ((0, FAKE, 2, 4, 2, 64, 0, 0, FAKE), NULL), ((FAKE, 0, 2, 4, 2, 64, 0, 0, FAKE), NULL),
    ((FAKE, FAKE, 2, 4, 2, 64, 0, 0, 0), NULL), ((FAKE + 8, FAKE, 2, 4, 2, 64, 0, 0, FAKE), ALIGN),
    ((FAKE, FAKE, 2, 4, 2, 64, 0, 0, FAKE + 4), ALIGN), ((FAKE, FAKE, -1, 4, 2, 64, 0, 0, FAKE), SHAPE),
    ((FAKE, FAKE, 2, 4, 2, 48, 0, 0, FAKE), UNSUPPORTED), ((FAKE, FAKE, 2, 4, 2, 64, 2, 0, FAKE), SHAPE),
    ((FAKE, FAKE, 2, 4, 2, 64, 0, 2, FAKE), UNSUPPORTED), ((0, 0, 2, 0, 2, 64, 0, 0, 0), 0),
    ((FAKE, FAKE, 1 << 16, 1 << 15, 1, 64, 0, 0, FAKE), UNSUPPORTED), ((FAKE, FAKE, 1 << 16, 1 << 14, 1, 1024, 0, 0, FAKE), UNSUPPORTED)])
def test_dequantize_refusals(ops, a, want):  # noqa: F811
    assert ops.lib.mxfp8_dequantize(*a, None) == want


def _angles(ops, **kw):
    return ops.RopeAngles(**dict(dict(turns=FAKE, magnitude=1.0, rot=64, interleaved=0), **kw))


ANGLES = [(dict(turns=0), NULL), (dict(turns=FAKE + 4), ALIGN), (dict(rot=0), UNSUPPORTED), (dict(rot=24), UNSUPPORTED),
          (dict(rot=144), UNSUPPORTED), (dict(interleaved=2), UNSUPPORTED), (dict(magnitude=math.nan), UNSUPPORTED)]
ROPE = [(dict(q=0), NULL), (dict(positions=FAKE + 2), ALIGN), (dict(q=FAKE + 8), ALIGN), (dict(k=FAKE + 8), ALIGN),
        (dict(B=-1), SHAPE), (dict(Hkv=-1), SHAPE), (dict(T=0), 0), (dict(Hq=0), 0), (dict(D=136), UNSUPPORTED),
        (dict(D=0), UNSUPPORTED), (dict(D=272), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(B=1 << 16, T=1 << 15), UNSUPPORTED),
        (dict(Hq=(1 << 20) - 1), UNSUPPORTED), (dict(q_stride_t=516), ALIGN), (dict(k_stride_h=12), ALIGN)]


@pytest.mark.parametrize("angles,kw,want", [(a, {}, w) for a, w in ANGLES] + [({}, k, w) for k, w in ROPE] + [
    ({}, dict(q_out=0), NULL), ({}, dict(k_out=0), NULL), ({}, dict(inverse=2), UNSUPPORTED), ({}, dict(q_out_stride_b=0), SHAPE),
    ({}, dict(k_out_stride_t=0), SHAPE), ({}, dict(k_out=FAKE + 8), ALIGN)])
def test_rope_call_refusals(ops, angles, kw, want):  # noqa: F811
    base = dict(q=FAKE, k=FAKE, q_out=FAKE, k_out=FAKE, positions=FAKE, position_stride_b=1, B=2, T=4, Hq=4, Hkv=2, D=128, dtype=0,
                inverse=0, **_strides(("q", "k", "q_out", "k_out")))
    assert ops.lib.rope(ctypes.byref(ops.RopeParams(angles=_angles(ops, **angles), **dict(base, **kw))), None) == want


@pytest.mark.parametrize("angles,kw,want", [(a, {}, w) for a, w in ANGLES] + [({}, k, w) for k, w in ROPE] + [
    ({}, dict(q_e4m3=0), NULL), ({}, dict(k_sc=0), NULL), ({}, dict(q_sc=FAKE + 8), ALIGN), ({}, dict(layout=2), SHAPE),
    ({}, dict(rule=2), UNSUPPORTED), ({}, dict(D=64), UNSUPPORTED)])
def test_rope_quant_refusals(ops, angles, kw, want):  # noqa: F811
    base = dict(q=FAKE, k=FAKE, q_e4m3=FAKE, q_sc=FAKE, k_e4m3=FAKE, k_sc=FAKE, positions=FAKE, position_stride_b=1, B=2, T=4,
                Hq=4, Hkv=2, D=128, dtype=0, layout=0, rule=0, **_strides(("q", "k")))
    p = ops.RopeQuantParams(angles=_angles(ops, **angles), **dict(base, **kw))
    assert ops.lib.mxfp8_rope_quantize_qk(ctypes.byref(p), None) == want


@pytest.mark.parametrize("pool,angles,kw,want", [(p, {}, {}, w) for p, w in POOL_CASES] + [({}, a, {}, w) for a, w in ANGLES] +
                         [({}, {}, k, w) for k, w in COMMON if "B" not in k or k["B"] < 1 << 20] + [
    ({}, {}, dict(q=0), NULL), ({}, {}, dict(v=0), NULL), ({}, {}, dict(q_out=0), NULL), ({}, {}, dict(q_out=FAKE + 8), ALIGN),
    ({}, {}, dict(Hq=6), SHAPE), ({}, {}, dict(rule=2), UNSUPPORTED), ({}, {}, dict(q_out_stride_h=0), SHAPE),
    ({}, {}, dict(v_stride_t=4), ALIGN), ({}, {}, dict(new_lens=FAKE + 1), ALIGN), ({}, {}, dict(B=1 << 16, T=1 << 15), UNSUPPORTED)])
def test_write_rope_refusals(ops, pool, angles, kw, want):  # noqa: F811
    base = dict(q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, B=2, T=4, Hq=8, dtype=0, rule=0, page_table=FAKE, table_stride=32,
                max_pages=32, seq_lens=FAKE, new_lens=FAKE, dev_status=FAKE, **_strides(("q", "k", "v", "q_out")))
    p = ops.CacheWriteRopeParams(cache=_pools(ops, **pool), angles=_angles(ops, **angles), **dict(base, **kw))
    assert ops.lib.mx_cache_write_rope(ctypes.byref(p), None) == want


@pytest.mark.parametrize("pool,kw,want", [(p, {}, w) for p, w in POOL_CASES] +
                         [({}, k, w) for k, w in COMMON if "dtype" not in k and k.get("T", 0) < 4096] + [
    ({}, dict(codes=0), NULL), ({}, dict(exps=0), NULL), ({}, dict(codes=FAKE + 8), ALIGN), ({}, dict(new_lens=FAKE + 1), ALIGN),
    ({}, dict(B=1 << 28), UNSUPPORTED), ({}, dict(B=16, T=(1 << 31) - 1), UNSUPPORTED)])
def test_bounds_refusals(ops, pool, kw, want):  # noqa: F811
    base = dict(codes=FAKE, exps=FAKE, B=2, T=4, page_table=FAKE, table_stride=32, max_pages=32, seq_lens=FAKE, new_lens=FAKE,
                dev_status=FAKE)
    p = ops.CacheBoundsParams(cache=_pools(ops, **pool), **dict(base, **kw))
    if kw.get("B") == 16:
        p.cache.Hkv, p.cache.num_pages = 16, 1
    assert ops.lib.mx_cache_bounds(ctypes.byref(p), None) == want


@pytest.mark.parametrize("pool,kw,want", [(p, {}, w) for p, w in POOL_CASES] + [({}, k, w) for k, w in COMMON] + [
    ({}, dict(codes=0), NULL), ({}, dict(exps=0), NULL), ({}, dict(q=0), NULL), ({}, dict(o=0), NULL), ({}, dict(workspace=0), NULL),
    ({}, dict(codes=FAKE + 8), ALIGN), ({}, dict(blocks=FAKE + 2), ALIGN), ({}, dict(workspace=FAKE + 8), ALIGN),
    ({}, dict(Hq=6), SHAPE), ({}, dict(top=0), SHAPE), ({}, dict(last=0), SHAPE), ({}, dict(first=-1), SHAPE),
    ({}, dict(first=7), SHAPE), ({}, dict(first=2 ** 31 - 1, last=2 ** 31 - 1), SHAPE), ({}, dict(softmax_scale=0.0), UNSUPPORTED),
    ({}, dict(workspace_bytes=100), SHAPE), ({}, dict(o_stride_t=0), SHAPE), ({}, dict(q_stride_b=4), ALIGN),
    # page strides: of one [pages][2][Hkv] allocation; not of whole heads; of different numbers of them
    (dict(k_page_stride=8 * 16 * 64, k_sc_page_stride=8 * 16 * 4, v_page_stride=8 * 16 * 64, v_sc_page_stride=8 * 16 * 4),
     dict(q=0), NULL),
    (dict(k_page_stride=4 * 16 * 64 + 16), {}, UNSUPPORTED), (dict(v_page_stride=8 * 16 * 64), {}, UNSUPPORTED),
    (dict(num_pages=1, k_page_stride=16), dict(q=0), NULL),
    (dict(num_pages=1 << 29), {}, UNSUPPORTED), (dict(num_pages=(1 << 29) - 1), dict(q=0), NULL)])
def test_sparse_refusals(ops, pool, kw, want):  # noqa: F811
    base = dict(codes=FAKE, exps=FAKE, q=FAKE, o=FAKE, lse=FAKE, blocks=FAKE, B=2, T=4, Hq=8, dtype=0, softmax_scale=0.1, top=8,
                first=1, last=2, page_table=FAKE, table_stride=32, max_pages=32, seq_lens=FAKE, new_lens=FAKE, dev_status=FAKE,
                workspace=FAKE, workspace_bytes=1 << 40, **_strides("qo"))
    p = ops.CacheSparseAttnParams(cache=_pools(ops, **pool), **dict(base, **kw))
    assert ops.lib.mx_cache_sparse_attn(ctypes.byref(p), None) == want


def test_null_params(ops):  # noqa: F811
    for n in ("rms_norm", "rms_norm_bwd", "rope", "mxfp8_rope_quantize_qk", "mx_cache_write_rope", "mx_cache_bounds",
              "mx_cache_sparse_attn"):
        assert getattr(ops.lib, n)(None, None) == NULL
    assert ops.lib.bsc_rope_turns(None, None, None) == NULL


def test_binding_refuses_cpu_tensors(ops):  # noqa: F811
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    q = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16)
    r = ops.Rope(64, device="cpu")
    for f in (lambda: ops.rms_norm(x, x[0]), lambda: ops.rms_norm_bwd(x, x, x[0], x[:, 0].float()),
              lambda: ops.rope(q, q, r), lambda: ops.mxfp8_rope_quantize_qk(q, q, r),
              lambda: ops.mxfp8_dequantize(x.view(torch.uint8), x.view(torch.uint8))):
        with pytest.raises(ValueError):
            f()


@pytest.mark.parametrize("shape", [(1, 32, 2, 128), (1, 64, 1, 128), (2, 64, 2, 128), (1, 64, 2, 64)])
def test_rotated_forward_checks_k_against_v(ops, shape):  # noqa: F811
    """K and V are quantised by two calls with Rope; that they are alike is checked ahead of both."""
    r = ops.Rope(128, device="cpu")
    q, k, v = (torch.zeros(s, dtype=torch.bfloat16) for s in ((1, 64, 2, 128), (1, 64, 2, 128), shape))
    for f in (lambda: ops.forward(q, k, v, rope=r), lambda: ops.forward(q, v, k, rope=r),
              lambda: ops.forward_backward(q, k, v, q, rope=r)):
        with pytest.raises(ValueError, match="same shape"):
            f()
    meta = k.to("meta")
    with pytest.raises(ValueError, match="one device"):
        ops.forward(q, k, meta, rope=r)


def test_row_layouts(ops):  # noqa: F811
    """Rows of [..., N] by at most two strides, one split for all tensors."""
    f = ops._row_layout
    x = torch.zeros((2, 3, 5, 64))
    assert f((x, None)) == (30, 1, [(64, 0), (0, 0)])
    q = torch.zeros((2, 3, 9 * 64))[..., :320].unflatten(-1, (5, 64))
    assert f((q, x)) == (30, 5, [(576, 64), (320, 64)])
    t = torch.zeros((3, 2, 5, 64)).transpose(0, 1)                    # [2, 3, 5] by strides 320, 640, 64
    with pytest.raises(ValueError):
        f((t, q))
    assert f((t[:, :1],)) == (10, 1, [(64, 0)])
    assert f((torch.zeros((4, 128))[:, :64],)) == (4, 1, [(128, 0)])
    assert f((torch.zeros(1, 64).expand(4, 64),)) == (4, 1, [(0, 0)])
    assert f((torch.zeros((0, 64))[:, :32],))[0] == 0
    assert f((torch.zeros(64),)) == (1, 1, [(64, 0)])


@pytest.mark.parametrize("name,kernels", [("norm.cu", 3), ("rope.cu", 1), ("dequant.cu", 1), ("cache_select.cu", 2)])
def test_launch_order(name, kernels):
    """Kernels that may start while the one ahead of them still stores: their wait is before their signal and every load,
    and no load takes the read-only path."""
    import re
    s = code(name)
    assert not re.findall(r"\b__ldg\s*\(|ld\.global(?:\.\w+)*\.nc", s) and "__restrict__" not in s
    bodies = re.split(r"__global__", s)[1:]
    assert len(bodies) == kernels
    for body in bodies:
        wait, signal = body.find("wait_for_last_kernel()"), body.find("next_kernel_may_start()")
        loads = [m.start() for m in re.finditer(r"__ld\w\w\(|fetch\(|load_batch\(v|cache_page\(|seen_by\(", body)]
        assert 0 <= wait < signal and (not loads or wait < min(loads))


def test_kernels_in_place_and_early_launches():
    """The next kernel's blocks may share an SM, and its L1, only with kernels that load nothing through L1 that they store: the
    norm's rows go past L1, and a rotation whose outputs are its inputs gives no signal."""
    s = code("rope.cu")
    assert s.count("next_kernel_may_start()") == 1 and "if (a.may_signal) next_kernel_may_start();" in s
    assert "a.may_signal = (long long)grid.x * grid.y <= EARLY_BLOCKS && !in_place(a);" in s
    assert "return a.y[0] == a.x[0] || (a.x[1] && a.y[1] == a.x[1]);" in s
    s = code("norm.cu")
    assert "cp.async.cg.shared.global [%0], [%1], 16;" in s and "__ldcs" not in s
    assert s.count("__ldca(") == 3 and s.count("__ldca(reinterpret_cast<const float4*>(w)") == 2
