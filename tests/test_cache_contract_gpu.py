"""The cache calls' contract on the GPU where a caller can lean on it hardest: calls with nothing between them, bytes that
mx_cache_write never writes, magnitudes and scores at the ends of what is taken, a status word with a history.
Bounds as in test_cache_gpu.py, whose helpers (and its three table widths) are used here."""
import ctypes

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


def fill_v(f, b, first, last, code, scale):
    """Element codes `code` under scale byte `scale` in V of positions first..last of sequence b, straight in the pool."""
    for p in range(first, last + 1):
        pg, off = int(f.table[b, p // f.page]), p % f.page
        f.cache.v[pg, :, off] = code
        f.cache.v_sc[pg, :, off] = scale


@HEADS
@pytest.mark.parametrize("D,n,extra", [(128, 45, 0), (64, 200, 0), (128, 200, 5120)])
@pytest.mark.parametrize("code,scale", [(0x7F, 127), (0xFF, 127), (0x7F, 0), (0xFF, 200)])
def test_rows_do_not_see_later_nan_codes(ops, D, n, extra, code, scale, Hq):
    """E4M3's NaN codes in V under a scale of their own (mx_cache_write gives such a block scale 0xFF, but the pools are
    the caller's): rows that may not see the token keep their bits, rows that see it are NaN in every column."""
    T = 5
    # the key's score may come from the other path: each within D 2^-23 sum |q||K| scale + 2^-16 of the formula's
    # (here sum |q||K| scale < 40), so the two within 2^-9
    tol = 2.0 ** -9
    f = Filled(ops, 81, [n], 2, D, 0, 16)
    f.table = torch.nn.functional.pad(f.table, (0, extra // 16), value=-7)
    q = make_q(31, 1, T, Hq, D, "bf16", 0)
    ref = ops.mx_cache_attn(q, f.cache, f.table, f.seq)
    for t in range(T - 2, -1, -1):
        fill_v(f, 0, n - T + t + 1, n - T + t + 1, code, scale)
        o, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq)
        assert torch.equal(bits(o[:, :t + 1]), bits(ref[0][:, :t + 1])), t
        assert torch.equal(bits(lse[:, :, :t + 1]), bits(ref[1][:, :, :t + 1]))
        assert torch.all(torch.isnan(o[:, t + 1:]))
        np.testing.assert_allclose(f64(lse), f64(ref[1]), rtol=0, atol=tol)


@pytest.mark.parametrize("T,G", [(2, 4), (3, 8), (12, 4)])
def test_one_nan_code_is_one_column(ops, T, G):
    """A single NaN code: its column alone, in the rows that see its token."""
    n, D = 70, 128
    f = Filled(ops, 82, [n], 2, D, 0, 16)
    q = make_q(32, 1, T, 2 * G, D, "fp16", 0)
    ref = ops.mx_cache_attn(q, f.cache, f.table, f.seq)
    p = n - 1
    f.cache.v[int(f.table[0, p // 16]), 1, p % 16, 37] = 0x7F
    o, _ = ops.mx_cache_attn(q, f.cache, f.table, f.seq)
    nan = torch.isnan(o[0])
    want = torch.zeros_like(nan)
    want[T - 1, G:, 37] = True
    assert torch.equal(nan, want)
    assert torch.equal(bits(o[:, :T - 1]), bits(ref[0][:, :T - 1]))


@HEADS
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("power", [12, 18, 20, 23, 25, 28, 31, 40, 100])
def test_large_scores(ops, fmt, power, Hq):
    """Scores so far from 0 that one fp32 step of them is many powers of e: finite, and the oracle's within what fp32
    scores allow (its bounds grow with them; the log-sum-exp is held to 2^-21 of itself)."""
    f = Filled(ops, 83, [300, 20], 2, 128, fmt, 16)
    q = make_q(33, 2, 2, Hq, 128, "bf16", 0)
    o, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq, softmax_scale=2.0 ** power)
    assert torch.all(torch.isfinite(o)) and torch.all(torch.isfinite(lse))
    check_attn(f, q, o, lse, [2, 2], 2.0 ** power, 0)


@HEADS
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("power", [10, 20, 24, 30, 60])
def test_large_scores_take_the_largest(ops, power, sign, Hq):
    """Keys that are powers of two times one vector: scores are exact, the largest is far above the others, and O is its V
    rounded once (sign -1: all scores negative, the smallest key is the largest score)."""
    n, T = 200, 2
    f = Filled(ops, 84, [n], 2, 128, 1, 16)
    best = [17, 150]                                     # per KV head; seen by every row
    k = torch.full((1, n, 2, 128), 1.0, dtype=torch.bfloat16)
    for h in range(2):
        k[0, best[h], h] = 4.0 if sign > 0 else 0.25
    v = make_q(34, 1, n, 2, 128, "bf16", 0)
    ops.mx_cache_write(f.cache, k.cuda(), v, f.table, f.seq)
    _, vv = ops.mx_cache_read(f.cache, f.table, f.seq, n)
    q = torch.full((1, T, Hq, 128), sign, dtype=torch.bfloat16, device="cuda")
    o, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq, softmax_scale=2.0 ** power)
    for h in range(2):
        want = vv[0, best[h], h].expand(T, Hq // 2, 128)
        np.testing.assert_allclose(f64(o[0, :, h * Hq // 2:(h + 1) * Hq // 2]), f64(want), rtol=2.0 ** -8, atol=0)
    s = 128.0 * 2.0 ** power * (4.0 if sign > 0 else -0.25)
    np.testing.assert_allclose(f64(lse), s, rtol=2.0 ** -21)


def test_status_keeps_the_first_code(ops):
    """One status word over a step's calls: a code that is there, another kernel's time-out among them, stays."""
    f = Filled(ops, 85, [20], 2, 128, 1, 16)
    q, x = make_q(35, 1, 1, 8, 128, "bf16", 0), make_q(36, 1, 1, 2, 128, "bf16", 0)
    bad_page = f.table.clone()
    bad_page[0, 1] = f.cache.num_pages
    short = f.table[:, :1].contiguous()                  # 16 positions of 20
    calls = [lambda t, st: ops.mx_cache_write(f.cache, x, x, t, f.seq, dev_status=st),
             lambda t, st: ops.mx_cache_read(f.cache, t, f.seq, 20, dev_status=st),
             lambda t, st: ops.mx_cache_attn(q, f.cache, t, f.seq, dev_status=st)]
    for call in calls:
        for first in (0, 0x103, 0x201, 0x202):
            for table, code in ((bad_page, 0x201), (short, 0x202)):
                st = i32([first])
                call(table, st)
                assert int(st) == (first or code)
                assert ops.bsc_read_device_status(st) == (6 if first == 0x103 else 7)
    st = i32([0])
    for call, table in zip(calls, (bad_page, short, short)):
        call(table, st)
    assert int(st) == 0x201


@HEADS
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("qp,kp,scale", [(-98, 97, 128 ** -0.5), (0, 97, 2.0 ** -96), (0, 97, 128 ** -0.5), (90, 0, 2.0 ** -90)])
def test_keys_up_to_the_bound(ops, fmt, qp, kp, scale, Hq):
    """Visible K up to 2^100 in magnitude, with q or the scale to match or scores as large as that makes them."""
    f = Filled(ops, 86, [200, 33], 2, 128, fmt, 16, k_mult=2.0 ** kp)
    assert kp == 0 or 2.0 ** 98 < max(np.abs(k).max() for k in f.K) <= 2.0 ** 100
    q = make_q(37, 2, 3, Hq, 128, "bf16", 0, mult=2.0 ** qp)
    o, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq, softmax_scale=scale)
    assert torch.all(torch.isfinite(o)) and torch.all(torch.isfinite(lse))
    check_attn(f, q, o, lse, [3, 3], float(np.float32(scale)), 0)


@HEADS
@pytest.mark.parametrize("fmt", [0, 1])
def test_tiny_queries_and_scale_over_large_keys(ops, fmt, Hq):
    """Query exponents and softmax scale together under fp32's normal range, keys that bring the scores back to 2^-5: one key
    weighs a little more than the zeros beside it."""
    n = 12
    f = Filled(ops, 87, [n], 2, 128, fmt, 16)
    sign = torch.where(torch.arange(128) % 3 == 0, -1.0, 1.0)
    k = torch.zeros((1, n, 2, 128), dtype=torch.bfloat16)
    k[0, 5] = sign * 2.0 ** 100
    v = make_q(38, 1, n, 2, 128, "bf16", 0)
    ops.mx_cache_write(f.cache, k.cuda(), v, f.table, f.seq)
    host = [x.cpu().numpy() for x in (f.cache.k, f.cache.k_sc, f.cache.v, f.cache.v_sc)]
    f.K = [C.gather(host[0], host[1], fmt, f.table[0].cpu().numpy(), n, 16)]
    f.V = [C.gather(host[2], host[3], fmt, f.table[0].cpu().numpy(), n, 16)]
    for qp, sp in ((-96, -16), (-88, -24), (-100, -12), (0, -112)):
        q = (sign * 2.0 ** qp).to(torch.bfloat16).cuda().expand(1, 1, Hq, 128)
        o, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq, softmax_scale=2.0 ** sp)
        check_attn(f, q, o, lse, [1], 2.0 ** sp, 0)


@HEADS
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n,power", [(1024, 100), (4500, 80)])
def test_values_up_to_the_bound(ops, fmt, n, power, Hq):
    """V of 2^100 over 1024 keys and of 2^80 over more, all but the first key nearly 2^4 above the reference that the first one
    sets (the most that weights and their sums grow to)."""
    f = Filled(ops, 88, [n], 2, 128, fmt, 16)
    k = torch.zeros((1, n, 2, 128), dtype=torch.bfloat16)
    k[:, 1:, :, 0] = 1.0
    v = torch.full((1, n, 2, 128), 2.0 ** power, dtype=torch.bfloat16)
    v[..., 64:] *= -0.5
    ops.mx_cache_write(f.cache, k.cuda(), v.cuda(), f.table, f.seq)
    q = torch.zeros((1, 1, Hq, 128), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    o, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq, softmax_scale=2.7)      # 3.895 in powers of two
    np.testing.assert_allclose(f64(o[..., :64]), 2.0 ** power, rtol=2.0 ** -8 + 2.0 ** -10)
    np.testing.assert_allclose(f64(o[..., 64:]), -0.5 * 2.0 ** power, rtol=2.0 ** -8 + 2.0 ** -10)
    s = float(np.float32(2.7))
    np.testing.assert_allclose(f64(lse), np.log(1 + (n - 1) * np.exp(s)), rtol=2.0 ** -14)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("Hq", [2, 6])
@pytest.mark.parametrize("n", [70, 400])
def test_many_rows_do_not_see_later_tokens(ops, fmt, Hq, n):
    """A chunk of 70 tokens, a tile of rows spread over several tiles of keys: what later tokens hold may send the tile's
    other rows through every rare path (far references, scalar keys, NaN codes), the earlier rows keep their bits."""
    T, D = 70, 128
    f = Filled(ops, 89, [n], 2, D, fmt, 16)
    q = make_q(39, 1, T, Hq, D, "bf16", 0)
    ref = ops.mx_cache_attn(q, f.cache, f.table, f.seq)
    check_attn(f, q, *ref, [T], D ** -0.5, 0)
    for t in (60, 40, 33, 9, 0):
        m = T - 1 - t
        for fill in (1e30, 1e9, 1e6, float("nan"), 1e-30, "codes"):
            if fill == "codes":
                if fmt:
                    continue
                for p in range(n - m, n, 3):
                    fill_v(f, 0, p, p, 0xFF, 127)
            else:
                x = (torch.randn((1, m, 2, D), generator=torch.Generator().manual_seed(m)) * fill).to(torch.bfloat16).cuda()
                ops.mx_cache_write(f.cache, x, x.flip(1).contiguous(), f.table, f.seq)
            o, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq)
            assert torch.equal(bits(o[:, :t + 1]), bits(ref[0][:, :t + 1])), (t, fill)
            assert torch.equal(bits(lse[:, :, :t + 1]), bits(ref[1][:, :, :t + 1])), (t, fill)


@pytest.mark.parametrize("fmt", [0, 1])
def test_write_every_fp16_value(ops, fmt):
    """All 65536 fp16 patterns: alone in a block, and as elements under a larger one."""
    pat = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.float16)
    lone = torch.zeros((2048, 32, 32), dtype=torch.float16)
    lone[:, torch.arange(32), (torch.arange(32) * 11) % 32] = pat.view(2048, 32)
    x = torch.cat((lone.view(-1, 1, 64), pat.view(-1, 1, 64)))
    n = x.shape[0]
    cache = ops.mx_cache_alloc(-(-n // 256), 256, 1, 64, fmt)
    table = widened(torch.arange(cache.num_pages, dtype=torch.int32, device="cuda").view(1, -1), 256)
    xs = x.cuda().view(1, n, 1, 64)
    for rule, name in ((0, "floor"), (1, "ceil")):
        ops.mx_cache_write(cache, xs, xs.flip(1).contiguous(), table, i32([n]), rule=rule)
        torch.cuda.synchronize()
        data, sb = C.quantize(f64(x.view(n, 64)), fmt, name)
        np.testing.assert_array_equal(cache.k_sc.view(-1, 2)[:n].cpu().numpy(), sb)
        np.testing.assert_array_equal(cache.k.view(cache.num_pages * 256, -1)[:n].cpu().numpy(), data)
        np.testing.assert_array_equal(cache.v.view(cache.num_pages * 256, -1)[:n].cpu().numpy(), data[::-1])


@HEADS
def test_attention_without_lse(ops, Hq):
    """The C call with lse = NULL gives the same O."""
    f = Filled(ops, 90, [700, 31, 0], 2, 128, 1, 16)
    q = make_q(40, 3, 2, Hq, 128, "bf16", 0)
    ref, _ = ops.mx_cache_attn(q, f.cache, f.table, f.seq)
    o = torch.full_like(q, 7.0)
    width = f.table.shape[1]
    ws = torch.empty(max(16, ops.mx_cache_attn_workspace_bytes(3, 2, Hq, 2, 128, width * 16)), dtype=torch.uint8, device="cuda")
    sb, st, sh, _ = q.stride()
    p = ops.CacheAttnParams(cache=f.cache.params, q=q.data_ptr(), o=o.data_ptr(), lse=0, B=3, T=2, Hq=Hq, dtype=0,
                            softmax_scale=128 ** -0.5, page_table=f.table.data_ptr(), table_stride=f.table.stride(0),
                            max_pages=width, seq_lens=f.seq.data_ptr(), workspace=ws.data_ptr(), workspace_bytes=ws.numel(),
                            q_stride_b=sb, q_stride_t=st, q_stride_h=sh, o_stride_b=sb, o_stride_t=st, o_stride_h=sh)
    assert ops.lib.mx_cache_attn(ctypes.byref(p), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(bits(o), bits(ref))


@pytest.mark.parametrize("fmt,dtype,layout", [(0, "bf16", 1), (1, "fp16", 0)])
def test_long_chunks(ops, fmt, dtype, layout):
    """A chunk of a prompt behind cached prefixes: more query tokens than a tile of keys has keys, some of them padding."""
    T, lens, new = 300, [300, 437, 90, 1001], [300, 211, 90, 3]
    f = Filled(ops, 91, lens, 1, 64, fmt, 48)
    q = make_q(41, 4, T, 3, 64, dtype, layout)
    o, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq, i32(new), layout=layout)
    check_attn(f, q, o, lse, new, 64 ** -0.5, layout)


def test_sizes_of_nothing(ops):
    """No sequences, no tokens, no heads: accepted, nothing is launched, outputs of that shape."""
    cache = ops.mx_cache_alloc(2, 16, 2, 64, 1)
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    for B, T, Hq in ((0, 3, 4), (2, 0, 4), (2, 1, 0)):
        table, lens = torch.zeros((B, 1), dtype=torch.int32, device="cuda"), torch.ones(B, dtype=torch.int32, device="cuda")
        o, lse = ops.mx_cache_attn(e(B, T, Hq, 64), cache, table, lens)
        assert o.shape == (B, T, Hq, 64) and lse.shape == (B, Hq, T)
        if Hq:
            ops.mx_cache_write(cache, e(B, T, 2, 64), e(B, T, 2, 64), table, lens)
            k, v = ops.mx_cache_read(cache, table, lens, T)
            assert k.shape == v.shape == (B, T, 2, 64)
    torch.cuda.synchronize()
    assert not cache.k.any() and not cache.k_sc.any()
