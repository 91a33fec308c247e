"""The key/value cache on the GPU against the fp64 oracle (oracle/cache.py): written bytes bit for bit,
values read back, attention within bounds derived below, and the calls a serving loop can make of
them: ragged and empty rows, shared and absent pages, garbage behind a sequence, other streams, graphs.
"""
import math
import threading

import numpy as np
import pytest
import torch

from block_scaled_causal_gb300 import inputs as I
from oracle import cache as C

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def ops():
    from block_scaled_causal_gb300 import _binding
    return _binding


@pytest.fixture(autouse=True, params=[0, 8192, 1 << 20], ids=["short", "wide", "long"])
def table_width(request):
    """Every test three times, with page tables just wide enough (the attention's cluster form), 8192 tokens wider
    (its list form, with parts joined through the workspace, mostly in tiles of 8 rows) and 2^20 tokens wider
    (the list in tiles of 8, 16 or 32 rows)."""
    Filled.more = request.param
    yield
    Filled.more = 0


def f64(x):
    return x.detach().cpu().double().numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rand_act(rng, shape, dtype, spread=0.0):
    """Activations with a per-row power-of-two spread."""
    x = rng.standard_normal(shape) * np.exp2(np.round(spread * rng.standard_normal(shape[:-1] + (1,))))
    return torch.tensor(x, dtype=torch.float64).to(DT[dtype])


def garbage_cache(ops, rng, pages, page, Hkv, D, fmt, gap=0):
    """An MxCache whose bytes are all random (NaN codes and 0xFF scales among them).  gap: unused
    bytes between pages, which have to stay as they are."""
    row = D // 2 if fmt == ops.CACHE_MXFP4 else D
    pools, whole = [], []
    for n in (row, D // 32, row, D // 32):
        size = Hkv * page * n
        buf = torch.tensor(rng.integers(0, 256, pages * (size + gap)), dtype=torch.uint8).cuda()
        whole.append(buf)
        pools.append(buf.view(pages, size + gap)[:, :size].unflatten(1, (Hkv, page, n)))
    return ops.MxCache(*pools, fmt=fmt), whole


class Filled:
    """Sequences of the given lengths in a cache of garbage, bytes by the oracle's quantiser."""
    more = 0

    def __init__(self, ops, seed, lens, Hkv, D, fmt, page, v_mult=None, k_mult=1.0, gap=0):
        rng = np.random.default_rng(seed)
        self.ops, self.lens, self.page = ops, lens, page
        width = max(1, max(-(-n // page) for n in lens) + 1)
        pages = len(lens) * width + 2
        self.cache, self.whole = garbage_cache(ops, rng, pages, page, Hkv, D, fmt, gap)
        perm = rng.permutation(pages)
        table = np.full((len(lens), width + Filled.more // page), -7, np.int32)    # entries that must not be read
        host = [p.cpu().numpy().copy() for p in (self.cache.k, self.cache.k_sc, self.cache.v, self.cache.v_sc)]
        self.K, self.V = [], []
        for b, n in enumerate(lens):
            used = -(-n // page)
            table[b, :used] = perm[b * width:b * width + used]
            kv = [rng.standard_normal((n, Hkv, D)) for _ in range(2)]
            kv[0] = kv[0] * k_mult
            if v_mult is not None:
                kv[1] = kv[1] * v_mult(rng, n)
            out = []
            for i, x in enumerate(kv):
                x = torch.tensor(x).to(torch.bfloat16).double().numpy()
                data, sb = C.quantize(x, fmt)
                for p in range(n):
                    pg, off = table[b, p // page], p % page
                    host[2 * i][pg, :, off], host[2 * i + 1][pg, :, off] = data[p], sb[p]
                out.append(C.dequantize(data, sb, fmt))
            self.K.append(out[0])
            self.V.append(out[1])
        for p, h in zip((self.cache.k, self.cache.k_sc, self.cache.v, self.cache.v_sc), host):
            p.copy_(torch.tensor(h))
        self.table, self.seq = torch.tensor(table).cuda(), i32(lens)


def bounds(held, D, out_eps, O, ref, A, E, vmax, tiny):
    """How far O and LSE may be from the oracle's:
    * a score is a sum of D products in fp32 (D * 2^-23 of sum |q||k|), then an exponent rounded in
      fp32: |weight error| <= es = D * 2^-23 * E + 2^-16 relative;
    * a weight is rounded to fp16 (2^-11 of it), sums run in fp32 (n * 2^-24), both against A =
      sum p |V|; numerator and denominator both carry es;
    * weights under fp16's normal range round to 2^-25 of the largest: n * 2^-25 * max |V|;
    * O is rounded once to its type (half a step)."""
    es = D * 2.0 ** -23 * E + 2.0 ** -16                     # [Hq, T]
    rel = (2.0 ** -11 + 2 * es + held * 2.0 ** -23).T[..., None]
    tol = np.abs(O) * out_eps / 2 + A * rel * (1 + out_eps) + held * 2.0 ** -25 * vmax + tiny
    return tol, es + held * 2.0 ** -23 + 2.0 ** -21 * np.abs(np.where(np.isneginf(ref), 0, ref))


def check_attn(f, q, o, lse, new, scale, layout, absent=None, cols=None):
    """O and LSE of every sequence within bounds(); cols: only these columns of O."""
    qb, ob = (f64(I.to_bshd(x, layout)) for x in (q, o))
    L = lse.cpu().double().numpy()
    cols = slice(None) if cols is None else cols
    fi = torch.finfo(o.dtype)
    for b, held in enumerate(f.lens):
        O, ref, A, E = C.attend(qb[b], f.K[b], f.V[b], held, new[b], scale, absent)
        vmax = np.nanmax(np.abs(f.V[b][..., cols]), initial=0.0)
        tol, tol_l = bounds(held, q.shape[-1], fi.eps, O[..., cols], ref, A[..., cols], E, vmax, fi.smallest_normal)
        err = np.abs(ob[b][..., cols] - O[..., cols])
        bad = ~(err <= tol)
        assert not bad.any(), (b, held, np.argwhere(bad)[:4], err[bad][:4], tol[bad][:4])
        none = np.isneginf(ref)
        assert np.array_equal(none, np.isneginf(L[b])) and np.all(ob[b][none.T] == 0)
        err = np.abs(np.where(none, 0, L[b]) - np.where(none, 0, ref))
        assert np.all(err <= tol_l), (b, err.max())


def widened(table, page):
    return torch.nn.functional.pad(table, (0, Filled.more // page), value=-7)


def make_q(seed, B, T, Hq, D, dtype, layout, mult=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((B, T, Hq, D), generator=g) * mult).to(DT[dtype])
    return I.to_layout(x, layout).cuda()


def bits(x):
    return x.contiguous().view(torch.int16 if x.element_size() == 2 else torch.int32)


# ------------------------------------------------------------------------------------------- writing
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("B,T,Hkv,D,page,dtype,layout,rule", [
    (1, 1, 1, 128, 16, "bf16", 0, 0), (3, 1, 4, 64, 48, "fp16", 1, 0), (2, 37, 3, 128, 16, "bf16", 1, 1),
    (5, 16, 2, 64, 32, "bf16", 0, 1), (2, 130, 5, 128, 64, "fp16", 0, 0)])
def test_write_bytes(ops, fmt, B, T, Hkv, D, page, dtype, layout, rule):
    rng = np.random.default_rng(B * T + D + fmt)
    cache, whole = garbage_cache(ops, rng, 60, page, Hkv, D, fmt, gap=32)
    before = [w.clone() for w in whole]
    want = [p.cpu().numpy().copy() for p in (cache.k, cache.k_sc, cache.v, cache.v_sc)]
    k, v = (rand_act(rng, (B, T, Hkv, D), dtype, 4.0 if dtype == "fp16" else 30.0) for _ in range(2))
    k[0, 0, 0, :32] = 0.0
    v[-1, -1, -1, 5] = float("nan")
    v[0, 0, 0, 40] = float("-inf")
    new = [int(rng.integers(0, T + 1)) for _ in range(B)]
    new[0] = T
    held = [n + int(rng.integers(0, 2 * page)) for n in new]
    width = max(-(-h // page) for h in held)
    table = rng.permutation(60)[:B * width].reshape(B, width).astype(np.int32)
    for i, x in enumerate((k, v)):
        for b in range(B):
            data, sb = C.quantize(f64(x[b, :new[b]]), fmt, "ceil" if rule else "floor")
            for t in range(new[b]):
                p = held[b] - new[b] + t
                want[2 * i][table[b, p // page], :, p % page] = data[t]
                want[2 * i + 1][table[b, p // page], :, p % page] = sb[t]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.mx_cache_write(cache, I.to_layout(k, layout).cuda(), I.to_layout(v, layout).cuda(), torch.tensor(table).cuda(),
                       i32(held), i32(new), layout=layout, rule=rule, dev_status=st)
    torch.cuda.synchronize()
    for got, w in zip((cache.k, cache.k_sc, cache.v, cache.v_sc), want):
        np.testing.assert_array_equal(got.cpu().numpy(), w)
    for w, b, p in zip(whole, before, (cache.k, cache.k_sc, cache.v, cache.v_sc)):   # the gaps between pages
        size = p[0].numel()
        assert torch.equal(w.view(60, -1)[:, size:], b.view(60, -1)[:, size:])
    assert int(st) == 0


@pytest.mark.parametrize("fmt", [0, 1])
def test_write_every_bf16_value(ops, fmt):
    """All 65536 bf16 patterns: alone in a block, and as elements under a larger one."""
    pat = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    lone = torch.zeros((2048, 32, 32), dtype=torch.bfloat16)
    lone[:, torch.arange(32), (torch.arange(32) * 7) % 32] = pat.view(2048, 32)
    x = torch.cat((lone.view(-1, 1, 128), pat.view(-1, 1, 128)))
    n = x.shape[0]
    cache = ops.mx_cache_alloc(-(-n // 256), 256, 1, 128, fmt)
    table = torch.arange(cache.num_pages, dtype=torch.int32, device="cuda").view(1, -1)
    for rule, name in ((0, "floor"), (1, "ceil")):
        xs = x.cuda().view(1, n, 1, 128)
        ops.mx_cache_write(cache, xs, xs.flip(1).contiguous(), table, i32([n]), rule=rule)
        torch.cuda.synchronize()
        data, sb = C.quantize(f64(x.view(n, 128)), fmt, name)
        np.testing.assert_array_equal(cache.k_sc.view(-1, 4)[:n].cpu().numpy(), sb)
        np.testing.assert_array_equal(cache.k.view(cache.num_pages * 256, -1)[:n].cpu().numpy(), data)
        np.testing.assert_array_equal(cache.v.view(cache.num_pages * 256, -1)[:n].cpu().numpy(), data[::-1])


def test_write_takes_slices_of_a_projection(ops):
    """K and V as strided slices of one fused [B, T, Hq + 2 Hkv, D] tensor, into K and V pools that are
    slices of one allocation."""
    rng = np.random.default_rng(8)
    qkv = rand_act(rng, (2, 19, 8, 128), "bf16").cuda()
    k, v = qkv[:, :, 4:6], qkv[:, :, 6:8]
    table, lens = i32([[0, 3], [2, 1]]), i32([19, 30])
    one = torch.zeros((4, 2, 2, 16, 64), dtype=torch.uint8, device="cuda")
    sc = torch.zeros((4, 2, 2, 16, 4), dtype=torch.uint8, device="cuda")
    a = ops.MxCache(one[:, 0], sc[:, 0], one[:, 1], sc[:, 1])
    b = ops.mx_cache_alloc(4, 16, 2)
    ops.mx_cache_write(a, k, v, table, lens)
    ops.mx_cache_write(b, k.contiguous(), v.contiguous(), table, lens)
    torch.cuda.synchronize()
    for x, y in ((a.k, b.k), (a.k_sc, b.k_sc), (a.v, b.v), (a.v_sc, b.v_sc)):
        assert torch.equal(x, y)
    assert int(b.k_sc.sum()) > 0


def test_write_skips_what_has_no_slot(ops):
    """Negative positions, positions past the table, page ids outside the pool: nothing is written."""
    rng = np.random.default_rng(4)
    cache, whole = garbage_cache(ops, rng, 4, 16, 2, 128, 1)
    before = [w.clone() for w in whole]
    k = rand_act(rng, (4, 5, 2, 128), "bf16").cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tab = i32([[0, 1], [4, -1], [2, 2147483647], [3, -2147483648]])
    # sequence 0: 2 held of 5 new -> positions -3..1; the others have no slot at all
    ops.mx_cache_write(cache, k, k, tab, i32([2, 16, 32, -5]), dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0x201 and ops.bsc_read_device_status(st) == 7
    data, sb = C.quantize(f64(k[0, 3:]), 1)
    np.testing.assert_array_equal(cache.k[0, :, :2].cpu().numpy(), data.transpose(1, 0, 2))
    np.testing.assert_array_equal(cache.v_sc[0, :, :2].cpu().numpy(), sb.transpose(1, 0, 2))
    cache.k[0, :, :2] = before[0].view(4, 2, 16, 64)[0, :, :2]
    assert torch.equal(whole[0], before[0])
    st.zero_()
    ops.mx_cache_write(cache, k[:1], k[:1], tab[:1], i32([40]), dev_status=st)
    assert int(st) == 0x202


# ------------------------------------------------------------------------------------------- reading
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("D,page,dtype,layout,gap", [(128, 16, "bf16", 0, 0), (64, 48, "fp16", 1, 16),
                                                     (128, 32, "fp16", 1, 0), (64, 16, "bf16", 0, 0)])
def test_read_values(ops, fmt, D, page, dtype, layout, gap):
    f = Filled(ops, 11, [1, 70, 16, 0, 33], 3, D, fmt, page, gap=gap)
    for T, starts in ((33, None), (1, [0, 69, 16, 0, 32]), (50, [-4, 40, 3, 5, -60])):
        k, v = ops.mx_cache_read(f.cache, f.table, f.seq, T, None if starts is None else i32(starts), layout, DT[dtype])
        for got, want in ((k, f.K), (v, f.V)):
            got = f64(I.to_bshd(got, layout))
            for b, n in enumerate(f.lens):
                ref = np.zeros((T, 3, D))
                for t in range(T):
                    p = (0 if starts is None else starts[b]) + t
                    if 0 <= p < n:
                        ref[t] = want[b][p]
                np.testing.assert_array_equal(got[b], f64(torch.tensor(ref).to(DT[dtype])))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_read_every_code(ops, dtype):
    """Every element code under every scale byte, rounded once."""
    for fmt in (0, 1):
        cache = ops.mx_cache_alloc(256 * 8 // 16, 16, 1, 128, fmt)
        row = cache.k.shape[-1]
        codes = torch.arange(8 * row, dtype=torch.int64).remainder(256).to(torch.uint8).view(8, row)
        cache.k.view(256, 8, row).copy_(codes.expand(256, 8, row))
        cache.k_sc.view(256, 8, 4).copy_(torch.arange(256, dtype=torch.uint8)[:, None, None].expand(256, 8, 4))
        table = torch.arange(cache.num_pages, dtype=torch.int32, device="cuda").view(1, -1)
        k, _ = ops.mx_cache_read(cache, table, i32([2048]), 2048, dtype=DT[dtype])
        data, sb = cache.k.view(2048, row).cpu().numpy(), cache.k_sc.view(2048, 4).cpu().numpy()
        want = f64(torch.tensor(C.dequantize(data, sb, fmt)).to(DT[dtype]))
        np.testing.assert_array_equal(f64(k).reshape(2048, 128), want)


def test_read_into_strided_outputs_and_bad_pages(ops):
    f = Filled(ops, 12, [40, 20], 2, 128, 1, 16)
    buf = torch.full((2, 21, 5, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, :20, 1:3], buf[:, :20, 3:5]
    f.table[0, 0] = f.cache.num_pages
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.mx_cache_read(f.cache, f.table, f.seq, 20, k_out=out[0], v_out=out[1], dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0x201
    np.testing.assert_array_equal(f64(buf[0, 16:20, 1:3]), f.K[0][16:20])
    assert float(buf[0, :16, 1:].abs().max()) == 0.0
    np.testing.assert_array_equal(f64(buf[1, :20, 3:5]), f.V[1])
    assert torch.all(buf[:, :, 0] == 3.0) and torch.all(buf[:, 20] == 3.0)
    with pytest.raises(ops.BscError):
        one = torch.empty((1, 1, 2, 128), dtype=torch.bfloat16, device="cuda")
        ops.mx_cache_read(f.cache, f.table, f.seq, 20, k_out=one.expand(2, 20, 2, 128), v_out=out[1])


# ----------------------------------------------------------------------------------------- attention
# query heads over 2 KV heads: with the tests' token counts, up to 8, 16 and many rows per KV head
HEADS = pytest.mark.parametrize("Hq", [4, 10, 40])
SHAPES = [
    # lens, T, Hq, Hkv, D, page, dtype, layout
    ([1], 1, 1, 1, 128, 16, "bf16", 0),
    ([500], 1, 16, 4, 128, 16, "bf16", 0),
    ([127, 128, 129, 1, 31, 32, 33, 16, 17], 1, 8, 2, 128, 16, "bf16", 1),
    ([300, 77, 2], 1, 6, 6, 64, 48, "fp16", 0),
    ([700, 5, 256, 64], 4, 12, 4, 128, 32, "fp16", 1),
    ([260, 40], 16, 10, 2, 64, 64, "bf16", 1),
    ([90, 33], 33, 5, 1, 128, 16, "bf16", 0),
    ([1500], 2, 7, 1, 64, 16, "bf16", 0),
    ([2100, 900], 1, 24, 1, 128, 128, "bf16", 0),
    ([130, 64, 65, 1], 7, 15, 1, 64, 48, "fp16", 1),
    ([1000, 63], 9, 8, 1, 128, 16, "fp16", 0),
]


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("lens,T,Hq,Hkv,D,page,dtype,layout", SHAPES)
def test_attn(ops, fmt, lens, T, Hq, Hkv, D, page, dtype, layout):
    f = Filled(ops, 20 + T, lens, Hkv, D, fmt, page)
    q = make_q(5, len(lens), T, Hq, D, dtype, layout)
    o, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq, layout=layout)
    torch.cuda.synchronize()
    check_attn(f, q, o, lse, [T] * len(lens), D ** -0.5, layout)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "fp16")])
@pytest.mark.parametrize("T,G,extra", [(2, 8, 5120), (8, 4, 5120), (9, 5, 5120), (3, 4, 0), (5, 6, 0), (33, 1, 0)])
def test_attn_cluster_tiles(ops, fmt, D, dtype, T, G, extra):
    """Clusters of several blocks in tiles of 16 and 32 rows: more units than 8-row tiles could have at once, or
    a table too long for their clusters; ragged, with new_lens, an absent page and NaN behind the sequence."""
    few = [600, 33, 0, 1, 17, 250, 64, 5, 129, 40, 2, 100, 31, 7, 48]
    lens = few if extra else few * 4                       # 30 or 120 (sequence, head) pairs
    f = Filled(ops, 57, lens, 2, D, fmt, 16)
    f.table = torch.nn.functional.pad(f.table, (0, extra // 16), value=-7)
    f.table[5, 3] = -1
    new = [T if b % 3 else T - 1 for b in range(len(lens))]
    q = make_q(18, len(lens), T, 2 * G, D, dtype, 0)
    o, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq, i32(new))
    gone = set(range(48, 64))
    for b in range(len(lens)):
        one = type("F", (), dict(K=[f.K[b]], V=[f.V[b]], lens=[lens[b]]))
        check_attn(one, q[b:b + 1], o[b:b + 1], lse[b:b + 1], [new[b]], D ** -0.5, 0, gone if b == 5 else None)


@HEADS
@pytest.mark.parametrize("fmt", [0, 1])
def test_attn_sharp_scores(ops, fmt, Hq):
    """Scores so wide that the running maximum keeps climbing, and so sharp that one key takes all."""
    for mult, scale in ((6.0, 0.3), (1.0, 4.0)):
        f = Filled(ops, 31, [640, 35], 2, 128, fmt, 16, k_mult=mult)
        q = make_q(6, 2, 2, Hq, 128, "bf16", 0)
        o, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq, softmax_scale=scale)
        check_attn(f, q, o, lse, [2, 2], float(np.float32(scale)), 0)


@HEADS
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("lo,hi", [(-20, 20), (-90, -60), (60, 90), (0, 30)])
def test_attn_wide_magnitudes(ops, fmt, lo, hi, Hq):
    """V tokens (and 32-element blocks of them) of very unlike magnitudes, some of them zero; each
    32-column block is held to its own magnitude."""
    def mult(rng, n):
        m = np.exp2(rng.integers(lo, hi + 1, (n, 1, 4))).repeat(32, -1)
        return m * (rng.random((n, 1, 1)) > 0.1)
    f = Filled(ops, 41, [200, 33], 2, 128, fmt, 16, v_mult=mult)
    q = make_q(7, 2, 3, Hq, 128, "bf16", 0)
    o, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq)
    for c in range(4):
        check_attn(f, q, o, lse, [3, 3], 128 ** -0.5, 0, cols=slice(32 * c, 32 * c + 32))


@HEADS
@pytest.mark.parametrize("fmt", [0, 1])
def test_attn_wide_keys(ops, fmt, Hq):
    """K blocks of very unlike magnitudes, scores kept moderate by the softmax scale."""
    rng = np.random.default_rng(3)
    f = Filled(ops, 43, [150, 48], 2, 128, fmt, 16)
    # rescale stored K blocks by powers of two: bytes stay, scales move
    shift = torch.tensor(rng.integers(-30, 12, (f.cache.num_pages, 2, 16, 4)), dtype=torch.int32).cuda()
    sc = f.cache.k_sc.int()
    f.cache.k_sc.copy_(torch.where(sc == 255, sc, (sc + shift).clamp(0, 254)).to(torch.uint8))
    host_k, host_s = f.cache.k.cpu().numpy(), f.cache.k_sc.cpu().numpy()
    f.K = [C.gather(host_k, host_s, fmt, f.table[b].cpu().numpy(), n, 16) for b, n in enumerate(f.lens)]
    q = make_q(8, 2, 2, Hq, 128, "bf16", 0)
    o, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq, softmax_scale=2e-5)
    check_attn(f, q, o, lse, [2, 2], float(np.float32(2e-5)), 0)


@HEADS
def test_attn_padded_and_empty_rows(ops, Hq):
    f = Filled(ops, 51, [100, 0, 3, 50, 2], 2, 128, 1, 16)
    q = make_q(9, 5, 4, Hq, 128, "bf16", 0)
    new = [2, 0, 4, -3, 9]                 # 9 of T = 4: clamped; 2 held with 4 new: two rows before the start
    o = torch.full_like(q, 7.0)
    o, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq, new_lens=i32(new), o=o)
    check_attn(f, q, o, lse, [2, 0, 4, 0, 4], 128 ** -0.5, 0)
    assert torch.all(torch.isneginf(lse[1])) and torch.all(torch.isneginf(lse[4, :, :2]))
    # every sequence empty
    o, lse = ops.mx_cache_attn(q, f.cache, f.table, i32([0, 0, 0, -1, 0]))
    assert torch.all(o == 0) and torch.all(torch.isneginf(lse))


@HEADS
@pytest.mark.parametrize("fmt", [0, 1])
def test_attn_absent_pages(ops, fmt, Hq):
    """A page id outside the pool is not followed: its tokens take no part, and the status says so."""
    f = Filled(ops, 52, [100], 2, 128, fmt, 16)
    q = make_q(9, 1, 2, Hq, 128, "bf16", 0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in (-1, f.cache.num_pages, 2147483647, -2147483648):
        f.table[0, 1], f.table[0, 6] = bad, bad       # 96.. is the tail page
        st.zero_()
        o, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq, dev_status=st)
        assert int(st) == 0x201
        check_attn(f, q, o, lse, [2], 128 ** -0.5, 0, absent=set(range(16, 32)) | set(range(96, 112)))
    f.table[0, :] = -1
    o, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq)
    assert torch.all(o == 0) and torch.all(torch.isneginf(lse))


@HEADS
@pytest.mark.parametrize("fmt", [0, 1])
def test_attn_length_past_the_table(ops, fmt, Hq):
    """Queries that stand past the table's end see every key it has."""
    f = Filled(ops, 53, [64], 2, 128, fmt, 16)
    q = make_q(9, 1, 2, Hq, 128, "bf16", 0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = ops.mx_cache_attn(q, f.cache, f.table[:, :4].contiguous(), i32([80]), dev_status=st)
    assert int(st) == 0x202 and ops.bsc_read_device_status(st) == 7
    for t in (0, 1):
        check_attn(f, q[:, t:t + 1], o[:, t:t + 1], lse[:, :, t:t + 1], [1], 128 ** -0.5, 0)


@HEADS
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n", [40, 45, 200])
def test_attn_rows_do_not_see_later_tokens(ops, fmt, n, Hq):
    """Row t is bit-for-bit what it is whatever the tokens after it hold, NaN and infinities included."""
    T = 5
    f = Filled(ops, 61, [n], 2, 128, fmt, 16)
    q = make_q(10, 1, T, Hq, 128, "bf16", 0)
    ref = ops.mx_cache_attn(q, f.cache, f.table, f.seq)
    fills = [float("nan"), float("inf"), 0.0, 1e30, 1e-30, 3e4, None]
    for t in range(T - 1):
        for fill in fills:
            x = torch.randn((1, T - 1 - t, 2, 128)) * 10 if fill is None else torch.full((1, T - 1 - t, 2, 128), fill)
            x = x.to(torch.bfloat16).cuda()
            ops.mx_cache_write(f.cache, x, x, f.table, f.seq)
            o, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq)
            torch.cuda.synchronize()
            assert torch.equal(bits(o[:, :t + 1]), bits(ref[0][:, :t + 1])), (t, fill)
            assert torch.equal(lse[:, :, :t + 1], ref[1][:, :, :t + 1])
        f = Filled(ops, 61, [n], 2, 128, fmt, 16)


@HEADS
@pytest.mark.parametrize("fmt", [0, 1])
def test_attn_visible_nan(ops, fmt, Hq):
    """A NaN block of V that a row sees makes that block of its output NaN, and no other; a NaN block of
    K makes the whole row NaN."""
    f = Filled(ops, 62, [90], 2, 128, fmt, 16)
    q = make_q(11, 1, 3, Hq, 128, "bf16", 0)
    clean, clean_lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq)
    pg, off = int(f.table[0, 88 // 16]), 88 % 16
    f.cache.v_sc[pg, 0, off, 1] = 255
    o, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq)
    nan = torch.isnan(o[0])                                  # [T, Hq, D]; KV head 0 serves the first half of the query heads
    want = torch.zeros_like(nan)
    want[1:, :Hq // 2, 32:64] = True                               # rows at positions 88 and 89
    assert torch.equal(nan, want)
    np.testing.assert_allclose(f64(lse), f64(clean_lse), atol=2.0 ** -16)
    keep = ~want[0]
    assert torch.equal(o[0, 0][keep], clean[0, 0][keep])
    f = Filled(ops, 62, [90], 2, 128, fmt, 16)
    f.cache.k_sc[pg, 1, off, 2] = 255
    o, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq)
    assert torch.all(torch.isnan(o[0, 1:, Hq // 2:])) and torch.all(torch.isnan(lse[0, Hq // 2:, 1:]))
    assert torch.equal(o[0, 0], clean[0, 0]) and torch.equal(o[0, :, :Hq // 2], clean[0, :, :Hq // 2])


def test_attn_shared_prefix(ops):
    """Two sequences over the same pages."""
    f = Filled(ops, 63, [64], 2, 128, 1, 16)
    q = make_q(12, 1, 1, 8, 128, "bf16", 0)
    both = torch.cat((q, q))
    o, lse = ops.mx_cache_attn(both, f.cache, f.table.expand(2, -1).contiguous(), i32([64, 48]))
    f.lens, f.K, f.V = [64, 48], [f.K[0]] * 2, [f.V[0]] * 2
    check_attn(f, both, o, lse, [1, 1], 128 ** -0.5, 0)


def test_attn_strided_and_guarded(ops):
    """q a slice of a fused projection, o a slice of a larger buffer, one row's neighbours untouched;
    a page table that is a slice of a wider one."""
    f = Filled(ops, 64, [90, 20], 2, 128, 1, 16)
    qkv = make_q(13, 2, 3, 12, 128, "bf16", 0)
    q = qkv[:, :, :8]
    buf = torch.full((2, 4, 10, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    wide = torch.full((2, f.table.shape[1] + 9), -1, dtype=torch.int32, device="cuda")
    wide[:, 4:4 + f.table.shape[1]] = f.table
    lse_buf = torch.full((2 * 8 * 3 + 64,), 9.0, device="cuda")
    ws = ops.mx_cache_attn_workspace_bytes(2, 3, 8, 2, 128)
    ws_buf = torch.full((ws + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    o, lse = ops.mx_cache_attn(q, f.cache, wide[:, 4:4 + f.table.shape[1]], f.seq, o=buf[:, :3, 1:9],
                               lse=lse_buf[32:32 + 48].view(2, 8, 3), workspace=ws_buf[2048:2048 + ws])
    torch.cuda.synchronize()
    check_attn(f, q, o, lse, [3, 3], 128 ** -0.5, 0)
    assert torch.all(buf[:, 3] == 5.0) and torch.all(buf[:, :, 0] == 5.0) and torch.all(buf[:, :, 9] == 5.0)
    assert torch.all(lse_buf[:32] == 9.0) and torch.all(lse_buf[80:] == 9.0)
    assert torch.all(ws_buf[:2048] == 0xA5) and torch.all(ws_buf[2048 + ws:] == 0xA5)


@pytest.mark.parametrize("Hq", [8, 40])
def test_streams_and_graphs(ops, Hq):
    """The same call on a side stream, twice at once on two streams, and captured and replayed on new
    inputs gives the eager call's bits; a second replay too."""
    f = Filled(ops, 65, [1200, 300], 2, 128, 1, 16)
    q, q2 = (make_q(s, 2, 2, Hq, 128, "bf16", 0) for s in (14, 15))
    ref, ref2 = (ops.mx_cache_attn(x, f.cache, f.table, f.seq) for x in (q, q2))
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    same = lambda a, b: torch.equal(bits(a[0]), bits(b[0])) and torch.equal(bits(a[1]), bits(b[1]))  # noqa: E731
    for _ in range(3):
        a = ops.mx_cache_attn(q, f.cache, f.table, f.seq, stream=s1)
        b = ops.mx_cache_attn(q2, f.cache, f.table, f.seq, stream=s2)
        torch.cuda.synchronize()
        assert same(a, ref) and same(b, ref2)
    g, x = torch.cuda.CUDAGraph(), q.clone()
    with torch.cuda.graph(g):
        out = ops.mx_cache_attn(x, f.cache, f.table, f.seq)
    for src, want in ((q, ref), (q2, ref2), (q, ref)):
        x.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert same(out, want)


@pytest.mark.parametrize("captured", [False, True])
def test_calls_in_a_row_keep_their_order(ops, captured):
    """Launches may start early, but every call sees what is ahead of it in its stream and nothing behind it: inputs,
    lengths and cache changed by slow kernels and by other calls between two attentions, across two streams too."""
    B, Hq, Hkv, D, n = 3, 8, 2, 128, 300
    f = Filled(ops, 71, [n] * B, Hkv, D, 1, 16)
    kv = [make_q(50 + i, B, 1, Hkv, D, "bf16", 0) for i in range(4)]
    qs = [make_q(60 + i, B, 1, Hq, D, "bf16", 0) for i in range(2)]
    lens2 = f.seq - 7
    x, lens = torch.zeros_like(qs[0]), f.seq.clone()
    side = torch.cuda.Stream()

    def steps(slow):
        outs = []
        main = torch.cuda.current_stream()
        for i in range(2):
            if slow:
                torch.cuda._sleep(200000)
            x.copy_(qs[i])
            lens.copy_(lens2 if i else f.seq)
            ops.mx_cache_write(f.cache, kv[2 * i], kv[2 * i + 1], f.table, lens)
            outs += ops.mx_cache_attn(x, f.cache, f.table, lens)
            x.zero_()                                         # behind the call that reads it
            lens.zero_()
            lens.copy_(f.seq)
            ops.mx_cache_write(f.cache, kv[3 - 2 * i], kv[2 - 2 * i], f.table, lens)      # and behind the attention
            outs += ops.mx_cache_read(f.cache, f.table, lens, 3, starts=lens - 3)
            side.wait_stream(main)
            if slow:
                torch.cuda._sleep(200000)
            x.copy_(qs[1 - i])
            with torch.cuda.stream(side):
                if slow:
                    torch.cuda._sleep(300000)
                ops.mx_cache_write(f.cache, kv[0], kv[1], f.table, lens)
            main.wait_stream(side)
            outs += ops.mx_cache_attn(x, f.cache, f.table, lens)
        return outs

    steps(False)             # leaves the two slots that every pass writes as every later pass finds them
    want = steps(False)
    torch.cuda.synchronize()
    want = [o.clone() for o in want]
    again = steps(False)
    torch.cuda.synchronize()
    for o, w in zip(again, want):
        assert torch.equal(o.view(torch.uint8), w.view(torch.uint8))
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = steps(True)
        for _ in range(5):
            g.replay()
    else:
        for _ in range(5):
            got = steps(True)
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        assert torch.equal(o.view(torch.uint8), w.view(torch.uint8))
    # against separate, synchronised calls
    for i in range(2):
        lens.copy_(lens2 if i else f.seq)
        ops.mx_cache_write(f.cache, kv[2 * i], kv[2 * i + 1], f.table, lens)
        torch.cuda.synchronize()
        o, lse = ops.mx_cache_attn(qs[i], f.cache, f.table, lens)
        torch.cuda.synchronize()
        assert torch.equal(bits(o), bits(want[6 * i])) and torch.equal(bits(lse), bits(want[6 * i + 1]))
        lens.copy_(f.seq)
        ops.mx_cache_write(f.cache, kv[3 - 2 * i], kv[2 - 2 * i], f.table, lens)
        torch.cuda.synchronize()
        k, v = ops.mx_cache_read(f.cache, f.table, lens, 3, starts=lens - 3)
        torch.cuda.synchronize()
        assert torch.equal(bits(k), bits(want[6 * i + 2])) and torch.equal(bits(v), bits(want[6 * i + 3]))
        ops.mx_cache_write(f.cache, kv[0], kv[1], f.table, lens)
        torch.cuda.synchronize()
        o, lse = ops.mx_cache_attn(qs[1 - i], f.cache, f.table, lens)
        torch.cuda.synchronize()
        assert torch.equal(bits(o), bits(want[6 * i + 4])) and torch.equal(bits(lse), bits(want[6 * i + 5]))


def test_two_host_threads(ops):
    """Calls of several host threads, each on its own stream, give the single call's bits."""
    f = Filled(ops, 67, [700, 90, 0], 2, 64, 0, 32)
    qs = [make_q(20 + i, 3, 1 + 8 * i, 8, 64, "fp16", 0) for i in range(3)]      # 4, 36 and 68 rows per KV head
    want = [ops.mx_cache_attn(q, f.cache, f.table, f.seq) for q in qs]
    torch.cuda.synchronize()
    got = [[] for _ in qs]

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(20):
            got[i].append(ops.mx_cache_attn(qs[i], f.cache, f.table, f.seq, stream=s))
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for outs, ref in zip(got, want):
        assert len(outs) == 20
        for o in outs:
            assert torch.equal(bits(o[0]), bits(ref[0])) and torch.equal(bits(o[1]), bits(ref[1]))


def test_two_graphs_at_once(ops):
    """Two captured calls with a workspace each, replayed at the same time on two streams."""
    f = Filled(ops, 68, [900, 40], 2, 128, 1, 16)
    xs = [make_q(30 + i, 2, 1, 8, 128, "bf16", 0) for i in range(2)]
    want = [ops.mx_cache_attn(x, f.cache, f.table, f.seq) for x in xs]
    need = max(16, ops.mx_cache_attn_workspace_bytes(2, 1, 8, 2, 128, f.table.shape[1] * 16))
    ws = [torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda") for _ in xs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x, w in zip(xs, ws):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ops.mx_cache_attn(x, f.cache, f.table, f.seq, workspace=w))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(bits(o[0]), bits(w[0])) and torch.equal(bits(o[1]), bits(w[1]))


@pytest.mark.parametrize("fmt", [0, 1])
def test_extreme_lengths(ops, fmt):
    """Lengths and starts at the ends of int32 are bad or empty positions, not addresses."""
    lo, hi = -2 ** 31, 2 ** 31 - 1
    f = Filled(ops, 69, [48, 48], 2, 128, fmt, 16)
    table = f.table[:, :3].contiguous()
    q = make_q(40, 2, 2, 4, 128, "bf16", 0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = ops.mx_cache_attn(q, f.cache, table, i32([lo, hi]), dev_status=st)
    assert torch.all(o[0] == 0) and torch.all(torch.isneginf(lse[0])) and int(st) == 0x202
    f.lens = [0, 48]
    for t in (0, 1):        # far behind the table: every key it has
        check_attn(f, q[:, t:t + 1], o[:, t:t + 1], lse[:, :, t:t + 1], [1, 1], 128 ** -0.5, 0)
    o, lse = ops.mx_cache_attn(q, f.cache, table, i32([48, 48]), i32([lo, hi]))
    f.lens = [48, 48]
    check_attn(f, q, o, lse, [0, 2], 128 ** -0.5, 0)
    k, v = ops.mx_cache_read(f.cache, table, i32([hi, lo]), 20, starts=i32([lo, hi]))
    assert not k.any() and not v.any()
    before = [p.clone() for p in (f.cache.k, f.cache.k_sc, f.cache.v, f.cache.v_sc)]
    x = make_q(41, 2, 2, 2, 128, "bf16", 0)
    st.zero_()
    ops.mx_cache_write(f.cache, x, x, table, i32([hi, lo]), i32([hi, hi]), dev_status=st)
    assert int(st) == 0x202
    for p, b in zip((f.cache.k, f.cache.k_sc, f.cache.v, f.cache.v_sc), before):
        assert torch.equal(p, b)


def test_table_without_pages(ops):
    """A page table of no columns: nothing is held, and tokens that should be are reported."""
    cache = ops.mx_cache_alloc(2, 16, 2, 128, 1)
    table = torch.empty((3, 0), dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, x = make_q(42, 3, 1, 4, 128, "bf16", 0), make_q(43, 3, 1, 2, 128, "bf16", 0)
    o, lse = ops.mx_cache_attn(q, cache, table, i32([0, 0, 0]), dev_status=st)
    assert not o.any() and torch.all(torch.isneginf(lse)) and int(st) == 0
    k, v = ops.mx_cache_read(cache, table, i32([0, 0, 0]), 5, dev_status=st)
    assert not k.any() and not v.any() and int(st) == 0
    ops.mx_cache_write(cache, x, x, table, i32([0, 1, 0]), dev_status=st)
    assert int(st) == 0x202 and not cache.k.any()
    st.zero_()
    o, lse = ops.mx_cache_attn(q, cache, table, i32([0, 1, 0]), dev_status=st)
    assert not o.any() and torch.all(torch.isneginf(lse)) and int(st) == 0x202


def test_binding_refusals(ops):
    f = Filled(ops, 66, [20], 2, 128, 1, 16)
    q = make_q(16, 1, 1, 4, 128, "bf16", 0)
    bad = [dict(q=q.float()), dict(q=q[..., :64]), dict(q=q[0]), dict(seq=f.seq.long()), dict(seq=i32([1, 2])),
           dict(table=f.table[0]), dict(layout=3), dict(o=q.half()), dict(lse=torch.empty(3, device="cuda")),
           dict(q=q.cpu()), dict(new=i32([1, 1]))]
    for kw in bad:
        a = dict(dict(q=q, table=f.table, seq=f.seq, new=None, layout=0, o=None, lse=None), **kw)
        with pytest.raises(ValueError):
            ops.mx_cache_attn(a["q"], f.cache, a["table"], a["seq"], a["new"], a["layout"], o=a["o"], lse=a["lse"])
    with pytest.raises(ops.BscError):
        ops.mx_cache_attn(q[:, :, :3].contiguous(), f.cache, f.table, f.seq)      # 3 heads over 2
    with pytest.raises(ValueError):
        ops.mx_cache_write(f.cache, q[:, :, :2], q[:, :, :2].half(), f.table, f.seq)
    with pytest.raises(ValueError):
        ops.mx_cache_write(f.cache, q[:, :, :3], q[:, :, :3], f.table, f.seq)


# ------------------------------------------------------------------------------------- used together
@pytest.mark.parametrize("fmt", [0, 1])
def test_prompt_then_decode(ops, fmt):
    """A prompt through forward() and into the cache, then six tokens one at a time and a chunk of
    three: every step against the oracle on all tokens so far."""
    B, S, Hq, Hkv, D, page = 2, 64, 8, 2, 128, 16
    rng = np.random.default_rng(77)
    total = S + 9
    q = rand_act(rng, (B, total, Hq, D), "bf16").cuda()
    k, v = (rand_act(rng, (B, total, Hkv, D), "bf16").cuda() for _ in range(2))
    cache = ops.mx_cache_alloc(B * 5, page, Hkv, D, fmt)
    table = widened(torch.tensor(rng.permutation(B * 5).reshape(B, 5), dtype=torch.int32).cuda(), page)
    ops.forward(q[:, :S].contiguous(), k[:, :S].contiguous(), v[:, :S].contiguous())
    ops.mx_cache_write(cache, k[:, :S], v[:, :S], table, i32([S] * B))
    f = type("F", (), {})()
    f.K, f.V = ([C.dequantize(*C.quantize(f64(x[b]), fmt), fmt) for b in range(B)] for x in (k, v))
    at = S
    for T in (1, 1, 1, 1, 1, 1, 3):
        lens = i32([at + T] * B)
        ops.mx_cache_write(cache, k[:, at:at + T], v[:, at:at + T], table, lens)
        o, lse = ops.mx_cache_attn(q[:, at:at + T], cache, table, lens)
        at += T
        f.lens = [at] * B
        check_attn(f, q[:, at - T:at], o, lse, [T] * B, D ** -0.5, 0)
    kk, vv = ops.mx_cache_read(cache, table, i32([at] * B), at)
    for b in range(B):
        np.testing.assert_array_equal(f64(kk[b]), f64(torch.tensor(f.K[b]).to(torch.bfloat16)))
        np.testing.assert_array_equal(f64(vv[b]), f64(torch.tensor(f.V[b]).to(torch.bfloat16)))


def test_one_decode_step_in_a_graph(ops):
    """Write and attend captured once, replayed as the sequence grows (the lengths are device data)."""
    rng = np.random.default_rng(78)
    B, Hq, Hkv, D = 2, 8, 2, 128
    cache = ops.mx_cache_alloc(2 * 3, 16, Hkv, D, 1)
    table = widened(torch.tensor(rng.permutation(6).reshape(2, 3), dtype=torch.int32).cuda(), 16)
    q, k, v = (rand_act(rng, (40, B, h, D), "bf16").cuda() for h in (Hq, Hkv, Hkv))
    lens = i32([0, 0])
    sq, sk, sv = (x[:1].transpose(0, 1).clone() for x in (q, k, v))
    ops.mx_cache_write(cache, sk, sv, table, lens)
    ops.mx_cache_attn(sq, cache, table, lens)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lens.add_(1)
        ops.mx_cache_write(cache, sk, sv, table, lens)
        o, lse = ops.mx_cache_attn(sq, cache, table, lens)
    f = type("F", (), {})()
    f.K, f.V = ([C.dequantize(*C.quantize(f64(x[:, b]), 1), 1) for b in range(B)] for x in (k, v))
    for i in range(40):
        for dst, src in ((sq, q), (sk, k), (sv, v)):
            dst.copy_(src[i:i + 1].transpose(0, 1))
        g.replay()
        f.lens = [i + 1] * B
        check_attn(f, sq, o, lse, [1, 1], D ** -0.5, 0)


def test_large_offsets(ops):
    """Pages that start past 2^32 bytes of the pool."""
    pages, page, Hkv = 9, 16, 1
    stride = (1 << 29) + 4096                       # 9 pages half a GiB apart
    buf = torch.zeros(pages * stride, dtype=torch.uint8, device="cuda")
    k = buf.view(pages, stride)[:, :page * 64].unflatten(1, (Hkv, page, 64))
    v = buf.view(pages, stride)[:, 2048:2048 + page * 64].unflatten(1, (Hkv, page, 64))
    ks, vs = (torch.zeros((pages, Hkv, page, 4), dtype=torch.uint8, device="cuda") for _ in range(2))
    big = ops.MxCache(k, ks, v, vs)
    small = ops.mx_cache_alloc(pages, page, Hkv, 128, 1)
    rng = np.random.default_rng(79)
    x = rand_act(rng, (1, pages * page, 1, 128), "bf16").cuda()
    table, lens = torch.arange(pages, dtype=torch.int32, device="cuda").flip(0).view(1, -1).contiguous(), i32([pages * page])
    q = make_q(17, 1, 1, 4, 128, "bf16", 0)
    got = []
    for c in (big, small):
        ops.mx_cache_write(c, x, x.flip(1), table, lens)
        got.append(ops.mx_cache_attn(q, c, table, lens) + ops.mx_cache_read(c, table, lens, pages * page))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert math.isfinite(float(got[0][1].sum()))
