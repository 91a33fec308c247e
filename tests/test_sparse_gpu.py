"""Bounds of the cache's pages and the attention over the pages that a score selects, on the GPU: bounds and choices exactly
as the fp64 oracle's (oracle/operands.py), O and LSE within the dense attention's bounds."""
import numpy as np
import pytest
import torch

from block_scaled_causal_gb300 import inputs as I
from oracle import cache as C
from oracle import operands as R
from test_cache_gpu import DT, Filled, bits, bounds, f64, garbage_cache, i32, make_q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from block_scaled_causal_gb300 import _binding
    return _binding


def random_bounds(ops, cache, seed):
    """Bounds of garbage: what no page of a sequence has must not be read as if it had."""
    rng = np.random.default_rng(seed)
    b = ops.mx_cache_bounds_alloc(cache)
    b.codes.copy_(torch.tensor(rng.integers(-128, 128, b.codes.shape), dtype=torch.int8))
    b.exps.copy_(torch.tensor(rng.integers(0, 256, b.exps.shape), dtype=torch.uint8))
    return b


def all_bounds(ops, f):
    b = random_bounds(ops, f.cache, 1)
    ops.mx_cache_bounds(f.cache, b, f.table, f.seq, max(max(f.lens), 1))
    return b


def check_sparse(ops, f, b, q, out, new, layout, top, first, last, absent_pages=()):
    """Every row: the oracle's choice, and O and LSE of the tokens in it."""
    o, lse, blocks = out
    Hkv, D, page = f.cache.Hkv, f.cache.D, f.page
    qb, ob, L = f64(I.to_bshd(q, layout)), f64(I.to_bshd(o, layout)), lse.cpu().double().numpy()
    B, T, Hq = qb.shape[:3]
    G = Hq // Hkv
    codes, exps, table, got = b.codes.cpu().numpy(), b.exps.cpu().numpy(), f.table.cpu().numpy(), blocks.cpu().numpy()
    fi = torch.finfo(o.dtype)
    for i, held in enumerate(f.lens):
        for t in range(T):
            tokens = max(held - new[i] + t + 1, 0) if t < new[i] else 0
            ids = [None if not 0 <= p < f.cache.num_pages else p for p in table[i]]
            for h in range(Hkv):
                qh = qb[i, t, h * G:(h + 1) * G]
                pick = R.choose(qh, codes[:, h], exps[:, h], ids, tokens, page, top, first, last)
                assert got[i, t, h].tolist() == pick + [-1] * (top - len(pick)), (i, t, h)
                js = [j for p in pick if ids[p] is not None for j in range(p * page, min((p + 1) * page, tokens))]
                ot, lt = ob[i, t, h * G:(h + 1) * G], L[i, h * G:(h + 1) * G, t]
                if not js:
                    assert np.all(ot == 0) and np.all(np.isneginf(lt))
                    continue
                K, V = f.K[i][js][:, h:h + 1], f.V[i][js][:, h:h + 1]
                O, ref, A, E = C.attend(qh[None], K, V, len(js), 1, D ** -0.5)
                tol, tol_l = bounds(len(js), D, fi.eps, O, ref, A, E, np.abs(V).max(), fi.smallest_normal)
                assert np.all(np.abs(ot - O[0]) <= tol[0]), (i, t, h, np.abs(ot - O[0]).max())
                assert np.all(np.abs(lt - ref[:, 0]) <= tol_l[:, 0]), (i, t, h)


# ------------------------------------------------------------------------------------------- bounds
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("lens,new,T,Hkv,D,page", [
    ([1], [1], 1, 1, 128, 16), ([40, 0, 17, 64], [3, 0, 17, 33], 33, 3, 64, 16), ([200, 96, 97], [1, 1, 2], 2, 2, 128, 48),
    ([513], [300], 300, 4, 128, 256)])
def test_bounds(ops, fmt, lens, new, T, Hkv, D, page):
    f = Filled(ops, 3, lens, Hkv, D, fmt, page, k_mult=3.0, gap=32)
    b = random_bounds(ops, f.cache, 2)
    codes, exps = b.codes.cpu().numpy().copy(), b.exps.cpu().numpy().copy()
    for i, n in enumerate(lens):
        if new[i]:
            for p in range((n - new[i]) // page, -(-n // page)):
                at = f.table[i, p].item()
                codes[at], exps[at] = R.page_bounds(f.K[i][p * page:(p + 1) * page])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.mx_cache_bounds(f.cache, b, f.table, f.seq, T, i32(new), dev_status=st)
    assert st.item() == 0
    assert np.array_equal(b.exps.cpu().numpy(), exps) and np.array_equal(b.codes.cpu().numpy(), codes)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("mult", [2.0 ** -110, 2.0 ** -60, 2.0 ** 60, 2.0 ** 100, 2.0 ** 108])
def test_bounds_of_extreme_keys(ops, fmt, mult):
    f = Filled(ops, 4, [40], 2, 64, fmt, 32, k_mult=mult)
    b = all_bounds(ops, f)
    for p in range(2):
        codes, exps = R.page_bounds(f.K[0][p * 32:(p + 1) * 32])
        at = f.table[0, p].item()
        assert np.array_equal(b.exps[at].cpu().numpy(), exps) and np.array_equal(b.codes[at].cpu().numpy(), codes)


@pytest.mark.parametrize("fmt", [0, 1])
def test_bounds_of_zeros_and_nan(ops, fmt):
    f = Filled(ops, 5, [64], 2, 128, fmt, 16, k_mult=0.0)
    at = f.table[0].tolist()
    f.cache.k_sc[at[1], 0, 3, 2] = 0xFF            # a NaN block; head 1 of the page has none
    if fmt == 0:
        f.cache.k[at[2], 1, 15, 77] = 0xFF         # a NaN code
    b = all_bounds(ops, f)
    exps = b.exps.cpu().numpy()
    assert exps[at[0]].tolist() == [27, 27] and exps[at[1]].tolist() == [255, 27]
    assert exps[at[2]].tolist() == [27, 255 if fmt == 0 else 27] and torch.all(b.codes[at[:4]] == 0)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("D", [64, 128])
def test_bounds_of_shared_pages(ops, fmt, D):
    """Pages that sequences share with different numbers of tokens, in the same place of their tables or another, have the bounds
    of the most tokens: every token is 4 times as large as the one before, so that no other number of them has the same."""
    page, Hkv, T = 16, 2, 48
    f = Filled(ops, 25, [7 * page], Hkv, D, fmt, page)
    x = torch.tensor(np.random.default_rng(25).choice([-1.0, 1.0], (1, 7 * page, Hkv, D))).cuda()
    x = (x * 2.0 ** (2.0 * (torch.arange(7 * page, device="cuda") % page) - 16)[:, None, None]).bfloat16()
    ops.mx_cache_write(f.cache, x, x, f.table, f.seq)
    K = f64(ops.mx_cache_read(f.cache, f.table, f.seq, 7 * page)[0])[0].reshape(7, page, Hkv, D)
    p = f.table[0].tolist()
    lens = [1, 5, 9, 16, 17, 20, 31, 33, 36, 40, 21, 3, 12, 0, 38] * 10
    rows = [p[:3]] * 10 + [[p[3], p[2], p[4]], [p[4], p[0], p[1]], [p[2], p[5], p[3]], p[4:7], [p[1], p[3], p[5]]]
    rows = [rows[i % 15] for i in range(150)]
    new = [min(n, 9 if i < 75 else T) for i, n in enumerate(lens)]
    held = {}
    for row, n, k in zip(rows, lens, new):
        for j in range((n - k) // page, -(-n // page) if k else 0):
            held[row[j]] = max(held.get(row[j], 0), min(page, n - j * page))
    assert len(set(held.values())) > 3
    want = {q: R.page_bounds(K[p.index(q)][:n]) for q, n in held.items()}
    b = random_bounds(ops, f.cache, 26)
    others = [q for q in range(f.cache.num_pages) if q not in held]
    before = b.codes[others].clone(), b.exps[others].clone()
    for _ in range(10):
        b.codes[list(held)] = 1
        b.exps[list(held)] = 130
        ops.mx_cache_bounds(f.cache, b, i32(rows).view(150, 3), i32(lens), T, i32(new))
        for q, (codes, exps) in want.items():
            assert np.array_equal(b.exps[q].cpu().numpy(), exps) and np.array_equal(b.codes[q].cpu().numpy(), codes), (q, held[q])
    assert torch.equal(b.codes[others], before[0]) and torch.equal(b.exps[others], before[1])


# ---------------------------------------------------------------------------------------- attention
SHAPES = [([200], 1, 4, 4, 128, 16, "bf16", 0, 4, 1, 1), ([700, 33, 0, 350], 1, 16, 4, 128, 16, "bf16", 0, 8, 1, 2),
          ([300, 511], 3, 16, 2, 64, 32, "fp16", 1, 5, 0, 1), ([500, 260], 2, 5, 5, 128, 48, "fp16", 0, 6, 2, 2),
          ([640, 1], 4, 24, 2, 64, 16, "bf16", 1, 7, 0, 3), ([900], 1, 40, 1, 128, 16, "bf16", 0, 20, 3, 1),
          ([400], 1, 3, 1, 128, 16, "fp16", 0, 1, 0, 1)]


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("lens,T,Hq,Hkv,D,page,dtype,layout,top,first,last", SHAPES)
def test_sparse(ops, fmt, lens, T, Hq, Hkv, D, page, dtype, layout, top, first, last):
    f = Filled(ops, 7, lens, Hkv, D, fmt, page, k_mult=2.0)
    b = all_bounds(ops, f)
    q = make_q(1, len(lens), T, Hq, D, dtype, layout)
    new = [min(T - (i % 2 if T > 1 else 0), n) for i, n in enumerate(lens)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ops.mx_cache_sparse_attn(q, f.cache, b, f.table, f.seq, top, first, last, new_lens=i32(new), layout=layout,
                                   dev_status=st)
    assert st.item() == 0
    check_sparse(ops, f, b, q, out, new, layout, top, first, last)
    again = ops.mx_cache_sparse_attn(q, f.cache, b, f.table, f.seq, top, first, last, new_lens=i32(new), layout=layout)
    assert all(torch.equal(bits(x), bits(y)) for x, y in zip(out, again))


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T", [1, 3])
def test_all_pages_is_the_dense_attention(ops, fmt, T):
    """top at or past the pages: no score is read, and the result is mx_cache_attn's within both calls' bounds."""
    f = Filled(ops, 9, [130, 64, 7], 2, 128, fmt, 16)
    b = random_bounds(ops, f.cache, 3)
    q = make_q(2, 3, T, 8, 128, "bf16", 0)
    for top in (9, 10, 100):
        out = ops.mx_cache_sparse_attn(q, f.cache, b, f.table, f.seq, top)
        check_sparse(ops, f, b, q, out, [T, T, T], 0, top, 1, 1)
        want, lse = ops.mx_cache_attn(q, f.cache, f.table, f.seq)
        assert torch.allclose(out[1], lse, rtol=0, atol=1e-3)


def repeated(ops, entries, page, Hkv, D, fmt, distinct, seed, tail=0):
    """One sequence whose table names `distinct` pages again and again: many equal scores."""
    rng = np.random.default_rng(seed)
    f = Filled(ops, seed, [distinct * page], Hkv, D, fmt, page)
    b = all_bounds(ops, f)
    turn = rng.integers(0, distinct, entries)
    f.K, f.V = ([x[0].reshape(distinct, page, Hkv, D)[turn].reshape(entries * page, Hkv, D)] for x in (f.K, f.V))
    f.table = f.table[:, torch.tensor(turn).cuda()].contiguous()
    f.lens = [entries * page - tail]
    f.seq = i32(f.lens)
    return f, b


@pytest.mark.parametrize("entries,top,first,last", [(257, 64, 0, 1), (1000, 200, 1, 2), (4096, 33, 1, 1), (4097, 33, 1, 1),
                                                    (9000, 700, 2, 4), (10240, 50, 1, 1), (10241, 50, 1, 1),
                                                    (12000, 300, 0, 300)])
def test_ties_and_long_tables(ops, entries, top, first, last):
    """Tables up to and past what a block holds of scores (10240 pages), equal scores in the pages' order; a choice of which
    nothing is left to the scores."""
    f, b = repeated(ops, entries, 16, 2, 64, 1, 9, 11, tail=5)
    q = make_q(3, 1, 1, 4, 64, "bf16", 0)
    out = ops.mx_cache_sparse_attn(q, f.cache, b, f.table, f.seq, top, first, last)
    check_sparse(ops, f, b, q, out, [1], 0, top, first, last)


def test_queries_that_score_nothing(ops):
    """Zero queries and queries with a NaN or an infinity: every score is 0, the lowest pages are taken."""
    f = Filled(ops, 12, [320], 1, 128, 1, 16)
    b = all_bounds(ops, f)
    q = torch.zeros((1, 3, 2, 128), dtype=torch.bfloat16)
    q[0, 1, 0, 5], q[0, 2, 1, 7] = float("nan"), float("-inf")
    o, lse, blocks = ops.mx_cache_sparse_attn(q.cuda(), f.cache, b, f.table, f.seq, 4)
    assert blocks.cpu().tolist() == [[[[0, 1, 2, 19]]] * 3]
    assert torch.isfinite(o[0, 0]).all() and torch.isnan(o[0, 1, 0]).all() and torch.isfinite(o[0, 1, 1]).all()


@pytest.mark.parametrize("exps", ["all", "tiny", "huge", "zero"])
def test_bounds_that_were_never_made(ops, exps):
    """Whatever the bounds' buffers hold, the choice ends, and is the formula's."""
    f, b = repeated(ops, 1500, 16, 2, 64, 1, 30, 24)
    b = random_bounds(ops, f.cache, 25)
    if exps == "zero":
        b.codes.zero_()
        b.exps.zero_()
    elif exps != "all":
        b.exps.copy_(b.exps % 27 if exps == "tiny" else 228 + b.exps % 27)
    q = make_q(8, 1, 1, 4, 64, "bf16", 0)
    for top in (3, 64, 1400):
        out = ops.mx_cache_sparse_attn(q, f.cache, b, f.table, f.seq, top)
        check_sparse(ops, f, b, q, out, [1], 0, top, 1, 1)


def test_nan_pages_are_taken(ops):
    f = Filled(ops, 13, [320], 1, 128, 1, 16)
    f.cache.k_sc[f.table[0, 9].item(), 0, 2, 1] = 0xFF
    b = all_bounds(ops, f)
    q = make_q(4, 1, 1, 2, 128, "bf16", 0)
    o, lse, blocks = ops.mx_cache_sparse_attn(q, f.cache, b, f.table, f.seq, 3)
    assert blocks.flatten().tolist() == [0, 9, 19] and torch.isnan(o).all()


def test_absent_pages_and_lengths_past_the_table(ops):
    f = Filled(ops, 14, [320, 200], 2, 64, 0, 16)
    b = all_bounds(ops, f)
    f.table[0, 4], f.table[0, 19] = -1, f.cache.num_pages      # the second holds the newest tokens
    q = make_q(5, 2, 2, 8, 64, "bf16", 0)
    for top in (5, 30):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = ops.mx_cache_sparse_attn(q, f.cache, b, f.table, f.seq, top, dev_status=st)
        assert st.item() == 0x201
        check_sparse(ops, f, b, q, out, [2, 2], 0, top, 1, 1)
    f.table[0, 4], f.table[0, 19] = f.table[0, 3], f.table[0, 2]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    short = f.table[:, :10].contiguous()                       # 160 positions: both lengths are past them
    out = ops.mx_cache_sparse_attn(q, f.cache, b, short, f.seq, 4, dev_status=st)
    assert st.item() == 0x202 and torch.isfinite(out[0]).all() and out[2][:, :, :, -1].eq(9).all()
    st.zero_()
    ops.mx_cache_bounds(f.cache, b, short, f.seq, 200, dev_status=st)
    assert st.item() == 0x202
    none = ops.mx_cache_sparse_attn(q, f.cache, b, f.table[:, :0].contiguous(), i32([0, 0]), 4)
    assert torch.all(none[0] == 0) and torch.all(none[1] == -np.inf) and torch.all(none[2] == -1)


def test_one_allocation_and_strided_activations(ops):
    """K and V pages in one [pages][2][Hkv] allocation; q and o slices with guards that stay."""
    f = Filled(ops, 15, [250, 310], 2, 64, 1, 16)
    c = f.cache
    data, sc = (torch.stack(x, 1).contiguous() for x in ((c.k, c.v), (c.k_sc, c.v_sc)))
    f.cache = ops.MxCache(data[:, 0], sc[:, 0], data[:, 1], sc[:, 1], fmt=1)
    b = all_bounds(ops, f)
    for T in (1, 2):
        qkv = make_q(6, 2, T, 12, 64, "bf16", 0)
        q = qkv[:, :, :8]
        o = torch.full((2, T, 10, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        out = ops.mx_cache_sparse_attn(q, f.cache, b, f.table, f.seq, 6, o=o[:, :, 1:9])
        check_sparse(ops, f, b, q, out, [T, T], 0, 6, 1, 1)
        assert torch.all(o[:, :, 0] == 7) and torch.all(o[:, :, 9] == 7)
    with pytest.raises(ops.BscError):                          # pages that are no whole number of heads apart
        g = Filled(ops, 15, [100], 2, 64, 1, 16, gap=16)
        ops.mx_cache_sparse_attn(make_q(1, 1, 1, 2, 64, "bf16", 0), g.cache, random_bounds(ops, g.cache, 1), g.table, g.seq, 2)


def test_streams_and_graphs(ops):
    """On another stream, and two graphs with workspaces of their own replayed together."""
    f = Filled(ops, 16, [900, 300], 4, 128, 1, 16)
    b = all_bounds(ops, f)
    q = make_q(7, 2, 1, 16, 128, "bf16", 0)
    want = ops.mx_cache_sparse_attn(q, f.cache, b, f.table, f.seq, 12)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.mx_cache_sparse_attn(q, f.cache, b, f.table, f.seq, 12, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graphs = []
    for _ in range(2):
        outs = [torch.empty_like(t) for t in want]
        ws = torch.empty(ops.mx_cache_sparse_attn_workspace_bytes(2, 1, 16, 4, 128, 16, f.table.shape[1], 12), dtype=torch.uint8,
                         device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.mx_cache_bounds(f.cache, b, f.table, f.seq, 1)
            ops.mx_cache_sparse_attn(q, f.cache, b, f.table, f.seq, 12, o=outs[0], lse=outs[1], blocks=outs[2], workspace=ws)
        graphs.append((g, outs, torch.cuda.Stream()))
    for _ in range(3):
        for g, outs, st in graphs:
            with torch.cuda.stream(st):
                for t in outs:
                    t.zero_()
                g.replay()
    torch.cuda.synchronize()
    for _, outs, _ in graphs:
        assert all(torch.equal(x, y) for x, y in zip(outs, want))


def test_binding_refusals(ops):
    f = Filled(ops, 17, [64], 2, 64, 1, 16)
    b = ops.mx_cache_bounds_alloc(f.cache)
    other = ops.mx_cache_alloc(3, 16, 2, 64)
    q = make_q(1, 1, 1, 2, 64, "bf16", 0)
    for g in (lambda: ops.MxBounds(f.cache, b.codes.view(torch.uint8), b.exps), lambda: ops.MxBounds(f.cache, b.codes[:1], b.exps),
              lambda: ops.mx_cache_bounds(other, b, f.table, f.seq, 1),
              lambda: ops.mx_cache_sparse_attn(q, f.cache, b, f.table, f.seq, 2, blocks=torch.zeros(2, dtype=torch.int32, device="cuda")),
              lambda: ops.mx_cache_sparse_attn(q, f.cache, b, f.table, f.seq, 2, lse=torch.zeros(2, device="cuda"))):
        with pytest.raises(ValueError):
            g()
    for kw in (dict(top=0), dict(top=2, first=2), dict(top=2, last=0), dict(top=2, softmax_scale=0.0),
               dict(top=2, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ops.BscError):
            ops.mx_cache_sparse_attn(q, f.cache, b, f.table, f.seq, **kw)


# ---------------------------------------------------------------------------------- a layer's steps
def test_prompt_and_decode_steps(ops):
    """A prompt and then tokens one by one through norm, projection, rotation into the cache, bounds and sparse attention: at
    every step each part is what it is alone, given what the step before left."""
    rng = np.random.default_rng(18)
    Hq, Hkv, D, N, B, page, top = 8, 2, 128, 256, 3, 16, 3
    w = torch.tensor(rng.standard_normal((N, (Hq + 2 * Hkv) * D)) * N ** -0.5).bfloat16().cuda()
    gain = torch.tensor(1 + 0.1 * rng.standard_normal(N)).bfloat16().cuda()
    rope = ops.Rope(D, scaling=ops.ROPE_LINEAR, factor=2.0)
    cache = ops.mx_cache_alloc(3 * 8, page, Hkv, D)
    plain = ops.mx_cache_alloc(3 * 8, page, Hkv, D)
    b = ops.mx_cache_bounds_alloc(cache)
    f = Filled.__new__(Filled)
    f.cache, f.page, f.table = cache, page, torch.tensor(rng.permutation(24).reshape(3, 8).astype(np.int32)).cuda()
    held, stream = [0, 0, 0], None
    for step, (T, new) in enumerate([(70, [70, 41, 5])] + [(1, [1, 1, 1])] * 8 + [(3, [3, 0, 2])]):
        x = torch.tensor(rng.standard_normal((B, T, N))).bfloat16().cuda()
        y, stream, _ = ops.rms_norm(x, gain, residual=stream if stream is not None and stream.shape == x.shape else x)
        qkv = (y.flatten(0, 1) @ w).view(B, T, Hq + 2 * Hkv, D)
        q, k, v = qkv.split([Hq, Hkv, Hkv], 2)
        held = [h + n for h, n in zip(held, new)]
        seq, fresh = i32(held), i32(new)
        at = seq - fresh
        rq = ops.mx_cache_write_rope(cache, q, k, v, rope, f.table, seq, fresh)
        tq, tk = ops.rope(q, k, rope, at)
        for i in range(B):
            assert torch.equal(rq[i, :new[i]], tq[i, :new[i]])
        ops.mx_cache_write(plain, tk, v, f.table, seq, fresh)
        ops.mx_cache_bounds(cache, b, f.table, seq, T, fresh)
        out = ops.mx_cache_sparse_attn(rq, cache, b, f.table, seq, top, new_lens=fresh)
        f.lens = held
        got = [f64(x) for x in ops.mx_cache_read(cache, f.table, seq, max(held))]
        f.K, f.V = ([x[i, :held[i]] for i in range(B)] for x in got)
        for i in range(B):
            for p in range(-(-held[i] // page)):
                codes, exps = R.page_bounds(f.K[i][p * page:(p + 1) * page])
                pg = f.table[i, p].item()
                assert np.array_equal(b.codes[pg].cpu().numpy(), codes) and np.array_equal(b.exps[pg].cpu().numpy(), exps)
        check_sparse(ops, f, b, rq, out, new, 0, top, 1, 1)
    assert torch.equal(cache.v, plain.v) and torch.equal(cache.v_sc, plain.v_sc)
    # K rotated in 16 bits and then quantised differs by that rounding alone: half a step of bf16 moves an E2M1 byte rarely
    a, c = (f64(ops.mx_cache_read(x, f.table, i32(held), max(held))[0]) for x in (cache, plain))
    assert np.mean(a != c) < 0.02


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("interleaved", [False, True])
def test_training_step(ops, layout, interleaved):
    """forward_backward with rope is its parts: operands by mxfp8_rope_quantize_qk, gradients turned back, all bit for bit; then
    the norm's gradients from those of q, k and v through the projection run and are finite."""
    rng = np.random.default_rng(19)
    B, S, Hq, Hkv, D, N = 2, 64, 4, 2, 128, 256
    x = torch.tensor(rng.standard_normal((S * B, N))).bfloat16().cuda()
    gain = torch.ones(N, device="cuda")
    w = torch.tensor(rng.standard_normal((N, (Hq + 2 * Hkv) * D)) * N ** -0.5).bfloat16().cuda()
    y, s, rstd = ops.rms_norm(x, gain)
    lead = (B, S) if layout == 0 else (S, B)
    q, k, v = (t.contiguous() for t in (y @ w).view(*lead, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], 2))
    do = torch.tensor(rng.standard_normal(q.shape)).bfloat16().cuda()
    rope = ops.Rope(D, interleaved=interleaved)
    start = i32([3, 1000])
    o, lse, dq, dk, dv = ops.forward_backward(q, k, v, do, layout, rope=rope, positions=start)
    o2, lse2 = ops.forward(q, k, v, layout, rope=rope, positions=start)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    q8, qs, k8, ks = ops.mxfp8_rope_quantize_qk(q, k, rope, start, layout)
    vt, vsc, vtn, vtn_sc = ops.mxfp8_quantize_v_fused(v, layout)
    o3, lse3 = ops.mxfp8_causal_attn_fwd(q8, qs, k8, ks, vt, vsc, vtn, vtn_sc, layout)
    assert torch.equal(o, o3) and torch.equal(lse, lse3)
    grads = ops.bf16_attn_bwd(q8, qs, k8, ks, vtn, vtn_sc, o, lse, do, layout)
    gq, gk = ops.rope(grads[0], grads[1], rope, start, layout, inverse=True)
    assert torch.equal(dq, gq) and torch.equal(dk, gk) and torch.equal(dv, grads[2])
    leaky, _ = ops.forward(q, k, v, layout, leaky=1, rope=rope, positions=start)
    assert torch.isfinite(leaky).all()
    dqkv = torch.cat((dq, dk, dv), 2).view(S * B, -1)
    dx, dgain = ops.rms_norm_bwd(dqkv @ w.t(), s, gain, rstd, ds=x)
    assert torch.isfinite(dx).all() and torch.isfinite(dgain).all() and dgain.dtype == torch.float32
    with pytest.raises(ValueError):
        ops.forward(q, k, v, layout, positions=start)


def test_training_step_on_a_stream(ops):
    """forward_backward with rope on a given stream, behind its own inputs there, gives the current stream's bits, with all it
    allocates on the way in that stream's memory."""
    g = torch.Generator(device="cuda").manual_seed(24)
    B, S, H, D = 1, 256, 4, 128
    q, k, v, do = (torch.randn((B, S, H, D), generator=g, device="cuda").bfloat16() for _ in range(4))
    rope, s = ops.Rope(D), torch.cuda.Stream()
    want = ops.forward_backward(q, k, v, do, rope=rope)
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s):
            ins = [x.clone() for x in (q, k, v, do)]
        got = ops.forward_backward(*ins, rope=rope, stream=s)
        for n in (1 << 16, 1 << 18, 1 << 20):        # memory that the current stream may have meanwhile
            torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rotation_shifts_nothing(ops):
    """Attention goes by the difference of positions: all positions moved by one amount leave O as it is up to the operands'
    E4M3 rounding: every score is off by at most 2 * 2^-4 of scale sum |q||k| <= 2^-3 * 128^-1/2 * |q||k|."""
    g = torch.Generator().manual_seed(20)
    q, k, v = (torch.randn((1, 32, h, 128), generator=g).bfloat16().cuda() * 0.25 for h in (2, 2, 2))
    r = ops.Rope(128)
    a, la = ops.forward(q, k, v, rope=r, positions=i32([0]))
    c, lc = ops.forward(q, k, v, rope=r, positions=i32([777777]))
    nq, nk = (f64(t).reshape(32, 2, 128) for t in (q, k))
    size = 2.0 ** -3 * 128 ** -0.5 * np.linalg.norm(nq, axis=-1).max() * np.linalg.norm(nk, axis=-1).max()
    assert (la - lc).abs().max().item() <= size + 1e-3
    assert (a.float() - c.float()).abs().max().item() <= (np.exp(2 * size) - 1 + 2.0 ** -7) * v.abs().max().item()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shift", [1, 64, 777777])
def test_rotation_moves_scores_by_rounding_alone(ops, interleaved, shift):
    """Scores of several units, of Q and K at positions 0 .. 31 and all moved by one amount.  They differ by the four E4M3 roundings
    of their operands, each at most 2^-4 of an element and of random sign: by 2 * 2^-4 of the root of sum (q k)^2 in root mean
    square.  With only one of the two moved they differ by far more, whichever it is.  The attention's LSE is that of the scores."""
    g = torch.Generator().manual_seed(33)
    q, k, v = (torch.randn((1, 32, h, 128), generator=g).bfloat16().cuda() for h in (4, 4, 4))
    r = ops.Rope(128, interleaved=interleaved)

    def operands(at):
        q8, qs, k8, ks = ops.mxfp8_rope_quantize_qk(q, k, r, i32([at]))
        return tuple(f64(ops.mxfp8_dequantize(*x, 0))[0].transpose(1, 0, 2) for x in ((q8, qs), (k8, ks)))

    (q0, k0), (q1, k1) = operands(0), operands(shift)
    scores = lambda a, b: np.einsum("htd,hsd->hts", a, b)  # noqa: E731
    rms = lambda x: np.sqrt(np.mean(x * x))  # noqa: E731
    bound = 2 * 2.0 ** -4 * np.sqrt(np.mean(np.einsum("htd,hsd->hts", q0 * q0, k0 * k0)))
    s0, s1 = scores(q0, k0), scores(q1, k1)
    assert rms(s0) > 5 * bound and rms(s0 - s1) <= bound
    far = 3 if shift > 1 else 1                       # one token's turn of one of them moves the fast pairs alone
    assert rms(s0 - scores(q1, k0)) > far * bound and rms(s0 - scores(q0, k1)) > far * bound
    for at, s in ((0, s0), (shift, s1)):
        _, lse = ops.forward(q, k, v, rope=r, positions=i32([at]))
        s = np.where(np.tri(32, dtype=bool), s * 128 ** -0.5, -np.inf)
        want = np.log(np.sum(np.exp(s - s.max(-1, keepdims=True)), -1)) + s.max(-1)
        assert np.all(np.abs(lse.cpu().double().numpy()[0] - want) <= 1e-3 * np.maximum(np.abs(want), 1.0))


def test_new_bounds_bound_nothing(ops):
    """Pages whose bounds were never made are read ahead of those that score, and not taken for pages of zeros; the pages of a
    prompt are all made by one call with its length."""
    f = Filled(ops, 27, [160], 2, 64, 1, 16)
    q = make_q(28, 1, 1, 4, 64, "bf16", 0)
    b = ops.mx_cache_bounds_alloc(f.cache)
    assert torch.all(b.exps == 0xFF) and torch.all(b.codes == 0)
    made = [5, 6, 8, 9]                               # positions 80 .. 111 and 128 .. 159
    ops.mx_cache_bounds(f.cache, b, f.table, i32([112]), 32)
    ops.mx_cache_bounds(f.cache, b, f.table, f.seq, 32)
    ids = f.table[0, :10].tolist()
    assert [i for i in range(10) if torch.all(b.exps[ids[i]] < 0xFF)] == made
    out = ops.mx_cache_sparse_attn(q, f.cache, b, f.table, f.seq, 8)
    check_sparse(ops, f, b, q, out, [1], 0, 8, 1, 1)
    for h in range(2):
        assert {0, 1, 2, 3, 4, 7, 9} < set(out[2][0, 0, h].tolist())
    ops.mx_cache_bounds(f.cache, b, f.table, f.seq, 160)
    assert torch.all(b.exps[ids] < 0xFF)
    check_sparse(ops, f, b, q, ops.mx_cache_sparse_attn(q, f.cache, b, f.table, f.seq, 4), [1], 0, 4, 1, 1)


def test_large_offsets(ops):
    """Pages that start past 2^32 bytes of the pools give what pages side by side give."""
    pages, page, Hkv, apart = 9, 16, 1, 1 << 19
    big = []
    for n in (64, 4, 64, 4):
        buf = torch.zeros(((pages - 1) * apart + 1) * page * n, dtype=torch.uint8, device="cuda")
        big.append(buf.as_strided((pages, Hkv, page, n), (apart * page * n, page * n, n, 1)))
    big = ops.MxCache(*big, fmt=1)
    small = ops.mx_cache_alloc(pages, page, Hkv, 128, 1)
    g = torch.Generator().manual_seed(21)
    x = torch.randn((1, pages * page, 1, 128), generator=g).bfloat16().cuda()
    table, lens = torch.arange(pages, dtype=torch.int32, device="cuda").flip(0).view(1, -1).contiguous(), i32([pages * page])
    q, r = make_q(17, 1, pages * page, 4, 128, "bf16", 0), ops.Rope(128)
    got = []
    for c in (big, small):
        b = ops.mx_cache_bounds_alloc(c)
        rq = ops.mx_cache_write_rope(c, q, x, x.flip(1), r, table, lens)
        ops.mx_cache_bounds(c, b, table, lens, pages * page)
        got.append((rq, b.codes, b.exps) + ops.mx_cache_sparse_attn(rq[:, -1:], c, b, table, lens, 4))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert torch.isfinite(got[0][4]).all()


def test_sizes_of_nothing(ops):
    f = Filled(ops, 22, [40, 0], 2, 64, 1, 16)
    b = all_bounds(ops, f)
    q = make_q(1, 2, 1, 4, 64, "bf16", 0)
    o, lse, blocks = ops.mx_cache_sparse_attn(q[:, :0], f.cache, b, f.table, f.seq, 2)
    assert o.shape == (2, 0, 4, 64) and lse.shape == (2, 4, 0) and blocks.shape == (2, 0, 2, 2)
    o, lse, blocks = ops.mx_cache_sparse_attn(q[:0], f.cache, b, f.table[:0], f.seq[:0], 2)
    assert o.shape == (0, 1, 4, 64) and blocks.shape == (0, 1, 2, 2)
    before = b.codes.clone()
    ops.mx_cache_bounds(f.cache, b, f.table, f.seq, 0)
    ops.mx_cache_bounds(f.cache, b, f.table, f.seq, 5, i32([0, 0]))
    assert torch.equal(b.codes, before)
    r = ops.Rope(64)
    assert ops.mx_cache_write_rope(f.cache, q[:, :0], q[:, :0, :2], q[:, :0, :2], r, f.table, f.seq).shape == (2, 0, 4, 64)


def test_host_threads(ops):
    """Calls of several host threads, each on its own stream, give the single call's bits."""
    import threading
    f = Filled(ops, 23, [700, 290, 33], 2, 64, 0, 16)
    b = all_bounds(ops, f)
    qs = [make_q(30 + i, 3, 1 + i, 8, 64, "fp16", 0) for i in range(3)]
    want = [ops.mx_cache_sparse_attn(q, f.cache, b, f.table, f.seq, 7) for q in qs]
    torch.cuda.synchronize()
    got = [[] for _ in qs]

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(20):
            got[i].append(ops.mx_cache_sparse_attn(qs[i], f.cache, b, f.table, f.seq, 7, stream=s))
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for outs, ref in zip(got, want):
        assert len(outs) == 20 and all(torch.equal(x, y) for o in outs for x, y in zip(o, ref))
