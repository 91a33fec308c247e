"""Rotary positions on the GPU against the fp64 oracle (oracle/operands.py), in 16 bits, to MXFP8 and into the cache."""
import numpy as np
import pytest
import torch

from block_scaled_causal_gb300 import inputs as I
from oracle import cache as C
from oracle import operands as R
from test_cache_gpu import garbage_cache, i32

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}

# Error of one output in units of magnitude (|a| + |b|): the angle is rounded to fp32 at one half turn at most (2^-25 of
# pi radians), cosines and sines are within 2^-22, the magnitude's product and the two products and their sum 2^-24 each:
# under 2^-20 in all.
ROT = 2.0 ** -20


@pytest.fixture(scope="module")
def ops():
    from block_scaled_causal_gb300 import _binding
    return _binding


def f64(x):
    return x.detach().cpu().double().numpy()


def act(rng, B, T, H, D, dtype, layout, mult=1.0):
    x = torch.tensor(rng.standard_normal((B, T, H, D)) * mult).to(DT[dtype])
    return I.to_layout(x, layout).cuda()


def positions_of(kind, rng, B, T):
    if kind == "none":
        return None, np.broadcast_to(np.arange(T), (B, T))
    if kind == "starts":
        p = rng.integers(0, 1 << 20, B)
        return i32(p), p[:, None] + np.arange(T)
    p = rng.integers(-2 ** 31, 2 ** 31, (B, T))
    p.flat[:3] = [2 ** 31 - 1, -2 ** 31, 0][:p.size]
    return torch.tensor(p, dtype=torch.int32).cuda(), p


def expect(ops, x, rope, pos, layout, inverse=False):
    turns = rope.turns.cpu().numpy().view(np.uint64)
    return R.rotate(f64(I.to_bshd(x, layout)), R.angles(turns, pos), rope.magnitude, rope.interleaved, inverse)


def check(got, want, layout):
    fi = torch.finfo(got.dtype)
    y, size = want
    g = f64(I.to_bshd(got, layout))
    tol = np.abs(y) * fi.eps / 2 + size * ROT * 1.01 + fi.smallest_normal * fi.eps
    err = np.abs(g - y)
    assert np.all(err <= tol), (np.argwhere(~(err <= tol))[:3], err.max())


CASES = [(1, 1, 1, 1, 128, 128, "none"), (3, 1, 16, 4, 128, 64, "starts"), (2, 37, 5, 1, 64, 64, "each"),
         (1, 130, 8, 8, 96, 48, "each"), (2, 19, 3, 2, 80, 16, "starts"), (1, 9, 2, 1, 256, 256, "each"),
         (2, 5, 7, 3, 192, 176, "none"), (1, 3, 2, 2, 16, 16, "each"), (4, 11, 40, 8, 128, 112, "each")]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,layout", [("bf16", 0), ("fp16", 1)])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,rot,kind", CASES)
def test_rope(ops, B, T, Hq, Hkv, D, rot, kind, dtype, layout, interleaved):
    rng = np.random.default_rng(B * T + D)
    r = ops.Rope(rot, base=10000.0, interleaved=interleaved, scaling=ops.ROPE_BY_PARTS, factor=4.0, original_length=4096)
    q, k = act(rng, B, T, Hq, D, dtype, layout), act(rng, B, T, Hkv, D, dtype, layout)
    pos, at = positions_of(kind, rng, B, T)
    for inverse in (False, True):
        yq, yk = ops.rope(q, k, r, pos, layout, inverse=inverse)
        check(yq, expect(ops, q, r, at, layout, inverse), layout)
        check(yk, expect(ops, k, r, at, layout, inverse), layout)
    alone, none = ops.rope(q, None, r, pos, layout, inverse=True)
    assert none is None and torch.equal(alone, yq)
    q2, k2 = q.clone(), k.clone()
    a, b = ops.rope(q2, k2, r, pos, layout, inverse=True, q_out=q2, k_out=k2)
    assert a is q2 and torch.equal(q2, yq) and torch.equal(k2, yk)


def test_slices_and_special_values(ops):
    """Slices of a fused projection, rotated where they are; a NaN or an infinity stays in its pair or in what passes
    through; positions expanded over the batch."""
    rng = np.random.default_rng(1)
    qkv = act(rng, 2, 6, 8, 128, "bf16", 0)
    before = qkv.clone()
    before[0, 2, 1, 3], before[1, 4, 5, 100] = float("nan"), float("inf")
    qkv.copy_(before)
    r = ops.Rope(64)
    q, k = qkv[:, :, :5], qkv[:, :, 5:7]
    pos = torch.arange(6, dtype=torch.int32, device="cuda") * 3
    ops.rope(q, k, r, pos[None].expand(2, 6), q_out=q, k_out=k)
    want = expect(ops, before[:, :, :7], r, np.broadcast_to(np.arange(6) * 3, (2, 6)), 0)
    bad = np.argwhere(~np.isfinite(f64(qkv)))
    assert bad.tolist() == [[0, 2, 1, 3], [0, 2, 1, 35], [1, 4, 5, 100]]
    got = torch.nan_to_num(qkv[:, :, :7], 0.0, 0.0)
    w = np.where(np.isfinite(want[0]), want[0], 0)
    assert np.all(np.abs(f64(got) - w) <= np.abs(w) * 2.0 ** -8 + np.where(np.isfinite(want[1]), want[1], 0) * ROT * 1.01)
    assert torch.equal(qkv[:, :, 7], before[:, :, 7]) and torch.equal(got[..., 64:100], before[:, :, :7, 64:100])


def test_refusals(ops):
    r, q = ops.Rope(64), torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16, device="cuda")
    for f in (lambda: ops.rope(q, q.half(), r), lambda: ops.rope(q, q[:, :2], r), lambda: ops.rope(q[0], None, r),
              lambda: ops.rope(q, None, r, k_out=q), lambda: ops.rope(q, None, r, q_out=q[:, :2]), lambda: ops.rope(q.cpu(), None, r),
              lambda: ops.rope(q, None, r, torch.zeros(2, dtype=torch.int32, device="cuda")),
              lambda: ops.rope(q, None, r, torch.zeros(1, dtype=torch.int64, device="cuda")),
              lambda: ops.rope(q, None, r, torch.zeros((1, 1), dtype=torch.int32, device="cuda").expand(1, 4)),
              lambda: ops.rope(q, None, r, layout=2), lambda: ops.rope(q, None, ops.Rope(64, device="cpu"))):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: ops.rope(q, None, ops.Rope(128)), lambda: ops.mxfp8_rope_quantize_qk(q, q, r)):
        with pytest.raises(ops.BscError):
            f()
    e, none = ops.rope(q[:, :0], q[:, :0], r)
    assert e.shape == (1, 0, 2, 64)


def enclosed(data, sb, want, fmt, rule):
    """Bytes of values within the rotation's error of `want`: those of its two ends enclose them where both ends have one
    scale; each element's own error moves its block's maximum by at most as much."""
    y, size = want
    e = size * ROT * 1.01
    lo, hi = y - e, y + e
    blocks = lambda x: x.reshape(x.shape[:-1] + (-1, 32))  # noqa: E731
    near = np.maximum(np.abs(lo), np.abs(hi))
    far = np.where(lo * hi <= 0, 0, np.minimum(np.abs(lo), np.abs(hi)))
    top = np.stack([np.max(blocks(x), -1) for x in (far, near)])         # of the block's maximum: at least, at most
    probe = [np.repeat(t[..., None], 32, -1).reshape(y.shape) for t in top]
    scales = [C.quantize(p, fmt, rule)[1] for p in probe]
    assert np.all((sb == scales[0]) | (sb == scales[1]))
    sure = np.repeat((scales[0] == scales[1])[..., None], 32, -1).reshape(y.shape)

    def on_grid(x):                       # x on the grid of its block's scale: a block of x and the maximum
        z = blocks(x).copy()
        out = np.empty_like(z)
        for i in range(32):
            p = np.repeat(top[1][..., None], 32, -1)
            p[..., 0] = z[..., i]
            data, s = C.quantize(p.reshape(y.shape), fmt, rule)
            out[..., i] = blocks(C.dequantize(data, s, fmt))[..., 0]
        return out.reshape(y.shape)

    got, a, b = C.dequantize(data, sb, fmt), on_grid(lo), on_grid(hi)
    assert np.all((got >= a) & (got <= b) | ~sure)


@pytest.mark.parametrize("interleaved,rot", [(False, 128), (True, 128), (False, 48), (True, 80)])
@pytest.mark.parametrize("B,T,Hq,Hkv,dtype,layout,rule,kind", [
    (1, 1, 4, 1, "bf16", 0, 0, "none"), (2, 33, 6, 3, "fp16", 1, 1, "starts"), (1, 70, 16, 4, "bf16", 0, 0, "each")])
def test_quantised(ops, B, T, Hq, Hkv, dtype, layout, rule, kind, interleaved, rot):
    rng = np.random.default_rng(T)
    r = ops.Rope(rot, interleaved=interleaved, magnitude=1.25)
    q, k = act(rng, B, T, Hq, 128, dtype, layout, 4.0), act(rng, B, T, Hkv, 128, dtype, layout)
    pos, at = positions_of(kind, rng, B, T)
    q8, qs, k8, ks = ops.mxfp8_rope_quantize_qk(q, k, r, pos, layout, rule)
    for x, x8, sc in ((q, q8, qs), (k, k8, ks)):
        data, sb = I.to_bshd(x8, layout).cpu().numpy(), sc.permute(0, 2, 1, 3).cpu().numpy()
        enclosed(data, sb, expect(ops, x, r, at, layout), 0, "ceil" if rule else "floor")
    alone = ops.mxfp8_rope_quantize_qk(q, None, r, pos, layout, rule)
    assert torch.equal(alone[0], q8) and torch.equal(alone[1], qs) and alone[2:] == (None, None)


def test_quantised_at_position_0_is_the_quantiser(ops):
    """No turn: the bytes of mxfp8_quantize_qk_rowwise, non-finite blocks among them."""
    rng = np.random.default_rng(3)
    q = act(rng, 2, 32, 3, 128, "bf16", 0)
    q[1, 4, 2, 70] = float("inf")
    q[0, 1, 1, 5] = float("nan")
    for interleaved in (False, True):
        zero = torch.zeros((2, 32), dtype=torch.int32, device="cuda")
        got = ops.mxfp8_rope_quantize_qk(q, q, ops.Rope(32, interleaved=interleaved), zero)
        want = ops.mxfp8_quantize_qk_rowwise(q)
        # (the NaN's pair is NaN too, in the same block)
        assert torch.equal(got[1], want[1]) and torch.equal(got[0], want[0])
        assert torch.equal(got[3], want[1]) and torch.equal(got[2], want[0])


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,rot,page,dtype,layout,interleaved", [
    (1, 1, 4, 1, 128, 128, 16, "bf16", 0, False), (3, 5, 8, 2, 64, 32, 48, "fp16", 1, True),
    (2, 130, 5, 5, 128, 96, 32, "bf16", 1, False), (4, 1, 16, 4, 128, 128, 64, "fp16", 0, True)])
def test_into_the_cache(ops, fmt, B, T, Hq, Hkv, D, rot, page, dtype, layout, interleaved):
    rng = np.random.default_rng(B + T + D)
    r = ops.Rope(rot, interleaved=interleaved, base=500000.0)
    qkv = act(rng, B, T, Hq + 2 * Hkv, D, dtype, layout)
    q, k, v = qkv[..., :Hq, :], qkv[..., Hq:Hq + Hkv, :], qkv[..., Hq + Hkv:, :]
    new = [T] + [int(x) for x in rng.integers(0, T + 1, B - 1)]
    held = [n + int(x) for n, x in zip(new, rng.integers(0, 90, B))]
    if B > 1:
        held[-1] = max(new[-1] - 2, 0)                 # tokens before position 0
    width = max(1, max(-(-h // page) for h in held))
    table = torch.tensor(rng.permutation(B * width + 3)[:B * width].reshape(B, width).astype(np.int32)).cuda()
    cache, whole = garbage_cache(ops, rng, B * width + 3, page, Hkv, D, fmt, gap=32)
    other, whole2 = garbage_cache(ops, np.random.default_rng(0), B * width + 3, page, Hkv, D, fmt, gap=32)
    for a, b in zip(whole2, whole):
        a.copy_(b)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = ops.mx_cache_write_rope(cache, q, k, v, r, table, i32(held), i32(new), layout=layout, dev_status=st)
    ops.mx_cache_write(other, k, v, table, i32(held), i32(new), layout=layout)      # the same slots, K not rotated
    assert st.item() == 0
    at = np.array([[h - n + t for t in range(T)] for h, n in zip(held, new)])
    live = np.array([[t < n and h - n + t >= 0 for t in range(T)] for h, n in zip(held, new)])
    yq, yk = expect(ops, q, r, at, layout), expect(ops, k, r, at, layout)
    z = live[..., None, None]
    check(y, (yq[0] * z, yq[1] * z), layout)
    assert np.all(f64(I.to_bshd(y, layout))[~live] == 0)
    # V and everything else as mx_cache_write leaves it; K's bytes enclosed
    assert torch.equal(whole[2], whole2[2]) and torch.equal(whole[3], whole2[3])
    got_k, got_s = cache.k.cpu().numpy(), cache.k_sc.cpu().numpy()
    old_k, old_s = other.k.cpu().numpy().copy(), other.k_sc.cpu().numpy().copy()
    tb = table.cpu().numpy()
    rows = [(b, t, tb[b, at[b, t] // page], at[b, t] % page) for b, t in np.argwhere(live)]
    if rows:
        data = np.stack([got_k[p, :, o] for _, _, p, o in rows])
        sb = np.stack([got_s[p, :, o] for _, _, p, o in rows])
        enclosed(data, sb, tuple(np.stack([w[b, t] for b, t, _, _ in rows]) for w in yk), fmt, "floor")
    for _, _, p, o in rows:
        old_k[p, :, o], old_s[p, :, o] = got_k[p, :, o], got_s[p, :, o]
    assert np.array_equal(got_k, old_k) and np.array_equal(got_s, old_s)


@pytest.mark.parametrize("fmt", [0, 1])
def test_into_the_cache_without_slots(ops, fmt):
    """Page ids and lengths that the table does not have: not written, reported, q rotated all the same."""
    rng = np.random.default_rng(2)
    r = ops.Rope(64)
    q, k = act(rng, 2, 3, 4, 64, "bf16", 0), act(rng, 2, 3, 2, 64, "bf16", 0)
    for table, held, code in (([[0, 7], [1, 2]], [17, 20], 0x201), ([[0, 1], [2, 3]], [34, 20], 0x202), ([[-1, -1], [0, 1]], [20, 3], 0x201)):
        cache, whole = garbage_cache(ops, rng, 5, 16, 2, 64, fmt)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        y = ops.mx_cache_write_rope(cache, q, k, k, r, i32(table), i32(held), dev_status=st)
        assert st.item() == code
        check(y, expect(ops, q, r, np.array([[h - 3 + t for t in range(3)] for h in held]), 0), 0)


def test_streams_and_graph(ops):
    rng = np.random.default_rng(9)
    r, q, k = ops.Rope(128), act(rng, 2, 64, 8, 128, "bf16", 0), act(rng, 2, 64, 2, 128, "bf16", 0)
    want = ops.rope(q, k, r) + ops.mxfp8_rope_quantize_qk(q, k, r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.rope(q, k, r, stream=side) + ops.mxfp8_rope_quantize_qk(q, k, r, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = ops.rope(q, k, r) + ops.mxfp8_rope_quantize_qk(q, k, r)
    for t in got:
        t.zero_()
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_large_offsets(ops):
    """Tokens that start past 2^32 bytes, at positions of their own: those of a call on the last tokens alone."""
    T, H = 70000, 256                                  # 2.3e9 elements
    q = torch.empty((1, T, H, 128), dtype=torch.bfloat16, device="cuda")
    q[:, -40:].normal_()
    q[:, :-40] = 1.0
    r = ops.Rope(128)
    tail = q[:, -40:].clone()
    start = i32([T - 40])
    q8, qs, _, _ = ops.mxfp8_rope_quantize_qk(q, None, r)
    want = ops.mxfp8_rope_quantize_qk(tail, None, r, start)
    assert torch.equal(q8[:, -40:], want[0]) and torch.equal(qs[:, :, -40:], want[1])
    y, _ = ops.rope(q, None, r, q_out=q)
    assert y is q and torch.equal(q[:, -40:], ops.rope(tail, None, r, start)[0])
    assert torch.equal(q[:, 1000], ops.rope(torch.ones_like(q[:, :1]), None, r, i32([1000]))[0][:, 0])


def test_few_tokens_share_their_heads(ops):
    """A token's heads go to one warp or to several: the same bits."""
    rng = np.random.default_rng(12)
    r = ops.Rope(64)
    q, k = act(rng, 1, 3000, 33, 64, "bf16", 0), act(rng, 1, 3000, 7, 64, "bf16", 0)
    yq, yk = ops.rope(q, k, r)
    for t in (0, 7, 2999):
        a, b = ops.rope(q[:, t:t + 1], k[:, t:t + 1], r, i32([t]))
        assert torch.equal(a, yq[:, t:t + 1]) and torch.equal(b, yk[:, t:t + 1])


@pytest.mark.parametrize("D,pad", [(64, 8), (128, 8)])
def test_in_place_ahead_of_attention(ops, D, pad):
    """Q rotated in place by a few blocks, in rows that share 32-byte sectors, and read by the attention right behind: bit for
    bit what comes of a copy, eager and captured."""
    rng = np.random.default_rng(31)
    B, T, Hq, Hkv, page = 4, 2, 8, 2, 16
    cache, table = ops.mx_cache_alloc(B * 4, page, Hkv, D), torch.arange(B * 4, dtype=torch.int32).view(B, 4).cuda()
    lens, r = i32([50, 2, 33, 64]), ops.Rope(D)
    k, v = (act(rng, B, T, Hkv, D, "bf16", 0) for _ in "kv")
    x = act(rng, B, T, Hq, D, "bf16", 0)
    base = torch.zeros(B * T * Hq * (D + pad) + 8, dtype=torch.bfloat16, device="cuda")[8:].view(B, T, Hq, D + pad)[..., :D]
    assert base.data_ptr() % 32 == 16 and base.stride(2) * 2 % 32 == 16
    at = lens - T

    def step(q, write):
        y = ops.mx_cache_write_rope(cache, q, k, v, r, table, lens, q_out=q) if write else \
            ops.rope(q, None, r, at, q_out=q)[0]
        return ops.mx_cache_attn(y, cache, table, lens)

    copy = x.clone()
    want = step(copy, True)
    torch.cuda.synchronize()
    for write in (True, False):
        for _ in range(30):
            base.copy_(x)
            got = step(base, write)
            assert torch.equal(base, copy) and all(torch.equal(a, b) for a, b in zip(got, want))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = []
            for _ in range(20):
                base.copy_(x)
                outs += step(base, write)
        for _ in range(5):
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, want[i % 2]) for i, a in enumerate(outs))


def test_no_heads_of_q(ops):
    """K beside a Q of no heads would not be rotated: refused; alone, or with no tokens, there is nothing to miss."""
    q, k = (torch.ones((2, 3, h, 64), dtype=torch.bfloat16, device="cuda") for h in (0, 2))
    r, cache = ops.Rope(64), ops.mx_cache_alloc(4, 16, 2, 64)
    k128, r128 = torch.ones((2, 3, 2, 128), dtype=torch.bfloat16, device="cuda"), ops.Rope(128)
    table, lens = i32([[0, 1], [2, 3]]), i32([3, 3])
    for f in (lambda: ops.rope(q, k, r), lambda: ops.mxfp8_rope_quantize_qk(k128[:, :, :0], k128, r128),
              lambda: ops.mx_cache_write_rope(cache, q, k, k, r, table, lens)):
        with pytest.raises(ValueError, match="at least one head"):
            f()
    assert ops.rope(q, None, r)[0].shape == q.shape and ops.rope(q, k[:, :, :0], r)[1].shape == q.shape
    assert ops.rope(k[:, :0], k[:, :0], r)[1].shape == (2, 0, 2, 64)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("magnitude", [1.0, 0.1 * np.log(8.0) + 1, 0.7])
def test_cosines_are_rounded_about_once(ops, interleaved, magnitude):
    """Pairs (a, 2048) for which a cos - 2048 sin all but cancels: the product by a power of two is exact, the sum is rounded
    where it is small, so what is left are the cosine's and sine's own errors.  One rounding of each is 0.289 units of its last
    place in root mean square (0.29 and 5% are allowed), and at most 0.72 in [1/2, 1), 0.8 here, for what a sum of two parts
    that is rounded at the end has beyond its half."""
    rng = np.random.default_rng(37)
    B, T, rot = 4, 2048, 128
    r = ops.Rope(rot, base=500000.0, interleaved=interleaved, magnitude=magnitude)
    pos = rng.integers(-2 ** 31, 2 ** 31, (B, T))
    angle = R.angles(r.turns.cpu().numpy().view(np.uint64), pos)
    c, s = np.cos(angle), np.sin(angle)
    b = np.full_like(c, 2048.0)
    a = np.rint(b * s / c)
    exact = magnitude * (a * c - b * s)
    few = (np.abs(a) <= 2048) & (np.abs(exact) < 2.0 ** -6)
    assert few.sum() > 3000
    i = np.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    x = np.zeros((B, T, 1, rot))
    x[:, :, 0, ia], x[:, :, 0, ib] = np.where(few, a, 0), np.where(few, b, 0)
    q = torch.tensor(x).half().cuda()
    y = f64(ops.rope(q, None, r, torch.tensor(pos, dtype=torch.int32).cuda())[0])[:, :, 0, ia]
    err, a, b, exact = np.abs(y - exact)[few], a[few], b[few], exact[few]
    last = lambda v: np.spacing(np.abs(magnitude * v[few]).astype(np.float32)).astype(np.float64)  # noqa: E731
    out = np.abs(exact) * 2.0 ** -11 + 2.0 ** -25                 # the output's rounding, half a step
    unit = 2.0 ** -24 * (2 if magnitude > 1 else 1)
    assert np.all(err <= 0.8 * unit * (np.abs(a) + b) + out)
    size = np.mean((0.29 * last(c) * a) ** 2 + (0.29 * last(s) * b) ** 2 + out ** 2)
    assert np.sqrt(np.mean(err ** 2) / size) <= 1.05, np.sqrt(np.mean(err ** 2) / size)
