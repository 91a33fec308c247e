"""rms_norm, its gradients and mxfp8_dequantize on the GPU against the fp64 oracle (oracle/operands.py)."""
import numpy as np
import pytest
import torch

from oracle import mx
from oracle import operands as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5

# Relative error of rstd * s * w in fp32.  The mean of N <= 16384 squares: a thread adds at most 32 of them in turn, then at
# most 10 levels of a tree, every partial sum positive: 2^-24 * 43, halved by the square root; rsqrt and the three
# products are within 2^-22 * 2: in all under 2^-19.
Y_REL = 2.0 ** -19


@pytest.fixture(scope="module")
def ops():
    from block_scaled_causal_gb300 import _binding
    return _binding


def f64(x):
    return x.detach().cpu().double().numpy()


def rand(rng, shape, dtype, mult=1.0):
    return torch.tensor(rng.standard_normal(shape) * mult).to(DT[dtype]).cuda()


def half_step(y, t):
    fi = torch.finfo(t)
    return np.abs(y) * fi.eps / 2 + fi.smallest_normal * fi.eps


def check_rows(got, want, t):
    tol = half_step(want, t) * (1 + Y_REL) + np.abs(want) * Y_REL
    err = np.abs(f64(got).reshape(want.shape) - want)
    assert np.all(err <= tol), (np.argwhere(~(err <= tol))[:3], err.max())


def check_mx(codes, sc, y, rule):
    """Every byte is that of some value within Y_REL of y: the bytes of y (1 -+ Y_REL) enclose it.  A scale may be that
    of either end."""
    N = y.shape[-1]
    codes, sc = codes.cpu().numpy().reshape(-1, N), sc.cpu().numpy().reshape(-1, N // 32)
    ends = [mx.mx_quantize(y * (1 + d), 32, rule) for d in (-Y_REL, Y_REL)]
    assert np.all((sc == ends[0][1]) | (sc == ends[1][1]))
    got = mx.mx_dequantize(codes, sc, 32)
    vals = [mx.mx_dequantize(c, s, 32) for c, s in ends]
    sure = np.repeat(ends[0][1] == ends[1][1], 32, -1)       # where the scale is beyond doubt the byte lies between the ends'
    lo, hi = np.minimum(*vals), np.maximum(*vals)
    assert np.all((got >= lo) & (got <= hi) | ~sure)


SIZES = [(1, 8), (3, 24), (2, 32), (5, 40), (130, 64), (67, 128), (9, 136), (33, 256), (17, 264), (4, 512), (300, 520),
         (3, 1024), (2, 1032), (7, 2048), (321, 2560), (2, 4096), (3, 4104), (2, 8192), (3, 8200), (2, 16384),
         # more rows than SMs: other cuts of a row
         (154, 32), (200, 72), (153, 128), (170, 136), (160, 1024), (155, 4104), (153, 8192), (157, 16384)]


@pytest.mark.parametrize("rows,N", SIZES)
@pytest.mark.parametrize("dtype,weight,residual", [("bf16", "bf16", True), ("fp16", "fp32", False), ("bf16", "fp32", False),
                                                   ("fp16", "fp16", True)])
def test_forward(ops, rows, N, dtype, weight, residual):
    rng = np.random.default_rng(rows * N)
    x, w = rand(rng, (rows, N), dtype, 3.0), rand(rng, (N,), weight)
    r = rand(rng, (rows, N), dtype) if residual else None
    y, s, rstd = ops.rms_norm(x, w, EPS, residual=r)
    want_s = (x.float() + r.float()).to(x.dtype) if residual else x
    assert torch.equal(s, want_s)
    want, want_r = R.norm(f64(s), f64(w), EPS)
    check_rows(y, want, x.dtype)
    assert np.all(np.abs(f64(rstd) - want_r) <= Y_REL * want_r)
    if N % 32 == 0:
        for rule in (0, 1):
            y2, s2, rstd2, y8, sc = ops.rms_norm(x, w, EPS, residual=r, y8_out=True, rule=rule)
            assert torch.equal(y2, y) and torch.equal(s2, s) and torch.equal(rstd2, rstd)
            check_mx(y8, sc, want, "ceil" if rule else "floor")
            none, _, _, z8, zsc = ops.rms_norm(x, w, EPS, residual=r, y8_out=True, y_out=False, rule=rule)
            assert none is None and torch.equal(z8, y8) and torch.equal(zsc, sc)


@pytest.mark.parametrize("rows,N", SIZES + [(2000, 128), (700, 2560), (5000, 16)])
@pytest.mark.parametrize("dtype,weight,residual", [("bf16", "bf16", True), ("fp16", "fp32", False)])
def test_backward(ops, rows, N, dtype, weight, residual):
    """dx: the row's sum as in the forward, and a few products and a difference: 2^-18 of the terms' sizes.  dw: a block adds
    at most rows terms in turn and the blocks' shares are at most 2432 / 16 + 16 sums: (rows + 180) 2^-24 of sum |terms|,
    and 2^-22 for each term's own products."""
    rng = np.random.default_rng(rows + N)
    s, dy, w = rand(rng, (rows, N), dtype, 2.0), rand(rng, (rows, N), dtype), rand(rng, (N,), weight)
    ds = rand(rng, (rows, N), dtype) if residual else None
    _, rstd = R.norm(f64(s), f64(w), EPS)
    rstd = torch.tensor(rstd, dtype=torch.float32).cuda()
    dx, dw = ops.rms_norm_bwd(dy, s, w, rstd, ds=ds)
    want, want_w, size, size_w = R.norm_bwd(f64(dy), f64(s), f64(w), f64(rstd), None if ds is None else f64(ds))
    err = np.abs(f64(dx) - want)
    tol = half_step(want, s.dtype) + 2.0 ** -18 * size * 1.01
    assert np.all(err <= tol), (np.argwhere(~(err <= tol))[:3], err.max())
    err = np.abs(f64(dw) - want_w)
    tol = half_step(want_w, w.dtype) + ((rows + 180) * 2.0 ** -24 + 2.0 ** -22) * size_w * 1.01
    assert np.all(err <= tol), (np.argwhere(~(err <= tol))[:3], err.max())
    dx2, dw2 = ops.rms_norm_bwd(dy, s, w, rstd, ds=ds)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    into = dy.clone()
    dx3, dw3 = ops.rms_norm_bwd(into, s, w, rstd, ds=ds, dx=into)
    assert dx3 is into and torch.equal(into, dx) and torch.equal(dw3, dw)


@pytest.mark.parametrize("N", [64, 512, 2560, 8192])
@pytest.mark.parametrize("size,grad,eps", [(2.0 ** 54, 2.0 ** -50, EPS), (2.0 ** 40, 2.0 ** -62, EPS), (2.0 ** -54, 2.0 ** 26, 0.0),
                                           (2.0 ** -50, 2.0 ** 40, 0.0), (2.0 ** 54, 2.0 ** 60, 0.0)])
def test_gradients_of_large_and_small_rows(ops, N, size, grad, eps):
    """Gradients that bf16 holds, of rows whose rstd^2 times the mean leaves fp32's range: test_backward's bound."""
    rng = np.random.default_rng(N)
    s, dy, w = rand(rng, (9, N), "bf16", size), rand(rng, (9, N), "bf16", grad), rand(rng, (N,), "fp32")
    s = torch.where(s.abs() <= 4 * size, s, 0.0).bfloat16()
    _, _, rstd = ops.rms_norm(s, w, eps)
    assert np.all(np.abs(f64(rstd) * np.sqrt(np.mean(f64(s) ** 2, -1) + eps) - 1) <= Y_REL)
    dx, _ = ops.rms_norm_bwd(dy, s, w, rstd)
    want, _, terms, _ = R.norm_bwd(f64(dy), f64(s), f64(w), f64(rstd))
    err = np.abs(f64(dx) - want)
    assert np.all(err <= half_step(want, s.dtype) + 2.0 ** -18 * terms * 1.01), err.max() / np.abs(want).max()


def test_slices_and_in_place(ops):
    """The heads of a slice of a fused projection, normed where they are; what lies between stays."""
    rng = np.random.default_rng(5)
    qkv = rand(rng, (2, 7, 9, 128), "bf16")
    q, before, w = qkv[:, :, :5], qkv.clone(), rand(rng, (128,), "fp32")
    want, _ = R.norm(f64(before[:, :, :5]).reshape(-1, 128), f64(w), EPS)
    y, s, rstd = ops.rms_norm(q, w, EPS, y=q)
    assert y is q and s is q and rstd.shape == (2, 7, 5)
    check_rows(q, want, q.dtype)
    assert torch.equal(qkv[:, :, 5:], before[:, :, 5:])
    # the residual stream brought up to date where it is, and gradients of strided rows
    x, r = rand(rng, (6, 80), "fp16")[:, :64], rand(rng, (6, 72), "fp16")
    stream, tail = r[:, :64], r[:, 64:].clone()
    want_s = (x.float() + stream.float()).half()
    y, s, rstd = ops.rms_norm(x, w[:64].contiguous(), EPS, residual=stream, sum_out=stream)
    assert s is stream and torch.equal(stream, want_s) and torch.equal(r[:, 64:], tail)
    dy = rand(rng, (6, 128), "fp16")[:, 64:]
    dx, dw = ops.rms_norm_bwd(dy, stream, w[:64].contiguous(), rstd)
    want = R.norm_bwd(f64(dy), f64(stream), f64(w[:64]), f64(rstd))
    assert np.all(np.abs(f64(dx) - want[0]) <= half_step(want[0], torch.float16) + 2.0 ** -18 * want[2])
    # a row for all
    z, _, _ = ops.rms_norm(x[:1].expand(6, 64), w[:64].contiguous(), EPS)
    assert torch.equal(z[5], z[0])


def test_rows_that_are_not_ordinary(ops):
    x = torch.zeros((7, 64), dtype=torch.bfloat16)
    x[1, 3] = float("nan")
    x[2, 4] = float("inf")
    x[3] = 2.0 ** 55
    x[4] = 2.0 ** -70
    x[5, ::2] = -0.0
    x[6] = torch.linspace(-1, 1, 64)
    w = torch.ones(64, dtype=torch.bfloat16)
    y, _, rstd, y8, sc = ops.rms_norm(x.cuda(), w.cuda(), EPS, y8_out=True)
    y, y8, sc = y.cpu().float(), y8.cpu(), sc.cpu()
    assert torch.all(y[0] == 0) and torch.all(sc[0] == 0) and torch.all(y8[0] == 0)
    assert torch.isnan(y[1]).all() and torch.all(sc[1] == 0xFF) and torch.all(y8[1] == 0x7F)
    assert torch.isnan(y[2, 4]) and torch.all(y[2, :4] == 0) and sc[2].tolist() == [0xFF, 0]
    assert torch.all(y[3] == 1) and torch.all(torch.signbit(y[5, ::2])) and rstd.isfinite()[[0, 3, 4, 5, 6]].all()
    check_rows(y[[4, 6]], R.norm(f64(x[[4, 6]]), np.ones(64), EPS)[0], torch.bfloat16)


def test_sum_without_a_residual(ops):
    """The C call writes s = x where it is given a place for it and no residual."""
    import ctypes
    x, w, s, y = (torch.randn(n, device="cuda").bfloat16() for n in ((5, 64), (64,), (5, 64), (5, 64)))
    p = ops.RmsNormParams(x=x.data_ptr(), weight=w.data_ptr(), y=y.data_ptr(), sum=s.data_ptr(), rows=5, x_stride=64, y_stride=64,
                          sum_stride=64, inner=1, N=64, dtype=0, weight_dtype=0, rule=0, eps=EPS)
    assert ops.lib.rms_norm(ctypes.byref(p), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(s, x) and torch.equal(y, ops.rms_norm(x, w, EPS)[0])


def test_nothing_to_do(ops):
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    y, s, rstd = ops.rms_norm(w.new_empty((0, 64)), w)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    dx, dw = ops.rms_norm_bwd(w.new_empty((0, 64)), w.new_empty((0, 64)), w, rstd)
    assert dx.shape == (0, 64) and torch.all(dw == 0)
    given = torch.ones_like(w)
    ops.rms_norm_bwd(w.new_empty((0, 64)), w.new_empty((0, 64)), w, rstd, dweight=given)
    assert torch.all(given == 0)
    assert ops.rms_norm(w, w)[0].shape == (64,) and ops.rms_norm(w, w)[2].shape == ()


def test_refusals(ops):
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda"), torch.ones(64, dtype=torch.bfloat16, device="cuda")
    r = torch.zeros(4, device="cuda")
    for f in (lambda: ops.rms_norm(x.float(), w), lambda: ops.rms_norm(x, w.half()), lambda: ops.rms_norm(x, w[:32]),
              lambda: ops.rms_norm(x, w, residual=x[:2]), lambda: ops.rms_norm(x, w, sum_out=x),
              lambda: ops.rms_norm(x, w, y_out=False), lambda: ops.rms_norm(x, w, rstd=r[:2]), lambda: ops.rms_norm(x.cpu(), w),
              lambda: ops.rms_norm(x.t().contiguous().t(), w), lambda: ops.rms_norm_bwd(x, x, w, r.half()),
              lambda: ops.rms_norm_bwd(x, x, w, r, ds=x.half()), lambda: ops.mxfp8_dequantize(x, x),
              lambda: ops.mxfp8_dequantize(x.view(torch.uint8), x.view(torch.uint8)[:, :2], layout=0),
              lambda: ops.mxfp8_dequantize(x.view(torch.uint8).view(1, 4, 4, 32), x.view(torch.uint8)[0, :16].view(1, 4, 4, 1)),
              lambda: ops.mxfp8_dequantize(x.view(torch.uint8).view(1, 4, 4, 32), x.view(torch.uint8)[0, :16].view(1, 4, 4, 1), 2)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: ops.rms_norm(x[:, :60].contiguous(), w[:60]), lambda: ops.rms_norm(x, w, -1.0),
              lambda: ops.rms_norm(x[:, :24].contiguous(), w[:24], y8_out=True),
              lambda: ops.rms_norm_bwd(x, x, w, r, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ops.BscError):
            f()


def test_streams_and_graphs(ops):
    """The same bits on another stream and from two graphs, each with a workspace of its own, replayed together."""
    rng = np.random.default_rng(8)
    x, dy, w = rand(rng, (500, 2048), "bf16"), rand(rng, (500, 2048), "bf16"), rand(rng, (2048,), "bf16")
    y, s, rstd = ops.rms_norm(x, w, residual=dy)
    want = (y, s, rstd) + ops.rms_norm_bwd(dy, s, w, rstd, ds=x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.rms_norm(x, w, residual=dy, stream=side)
    got += ops.rms_norm_bwd(dy, got[1], w, got[2], ds=x, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        outs = [torch.empty_like(t) for t in want]
        ws = torch.empty(ops.rms_norm_bwd_workspace_bytes(500, 2048), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.rms_norm(x, w, residual=dy, y=outs[0], sum_out=outs[1], rstd=outs[2])
            ops.rms_norm_bwd(dy, outs[1], w, outs[2], ds=x, dx=outs[3], dweight=outs[4], workspace=ws)
        graphs.append((g, outs, torch.cuda.Stream()))
    for _ in range(3):
        for g, outs, st in graphs:
            with torch.cuda.stream(st):
                for t in outs:
                    t.zero_()
                g.replay()
    torch.cuda.synchronize()
    for _, outs, _ in graphs:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape,layout", [((2, 5, 3, 128), 0), ((5, 2, 3, 64), 1), ((7, 1, 1, 32), 1), ((1, 300, 5, 96), 0)])
def test_dequantize(ops, dtype, shape, layout):
    """Every code under every scale byte in turn: element * 2^e is exact in fp32, one rounding to the type."""
    rng = np.random.default_rng(3)
    x = torch.tensor(rng.integers(0, 256, shape), dtype=torch.uint8)
    B, S, H, D = shape if layout == 0 else (shape[1], shape[0]) + shape[2:]
    sc = torch.tensor(np.resize(rng.permutation(256), (B, H, S, D // 32)), dtype=torch.uint8)
    y = ops.mxfp8_dequantize(x.cuda(), sc.cuda(), layout, DT[dtype])
    xb = (x if layout == 0 else x.transpose(0, 1)).numpy()
    with np.errstate(over="ignore"):
        want = mx.mx_dequantize(xb, sc.permute(0, 2, 1, 3).contiguous().numpy(), 32)
        want = torch.tensor(np.where(np.isnan(want), np.nan, want)).float().to(DT[dtype])
    got = (y if layout == 0 else y.transpose(0, 1)).cpu()
    assert torch.equal(torch.nan_to_num(got, 7.0), torch.nan_to_num(want, 7.0))
    flat = ops.mxfp8_dequantize(x.cuda(), sc.cuda().reshape(shape[:-1] + (D // 32,)), None, DT[dtype])
    want = mx.mx_dequantize(x.numpy(), sc.reshape(shape[:-1] + (D // 32,)).numpy(), 32)
    assert torch.equal(torch.nan_to_num(flat.cpu(), 7.0), torch.nan_to_num(torch.tensor(want).float().to(DT[dtype]), 7.0))


def test_quantise_and_back(ops):
    """The rowwise quantiser's operands read back."""
    x = torch.randn((2, 64, 3, 128), generator=torch.Generator().manual_seed(1)).bfloat16()
    for layout in (0, 1):
        t = x if layout == 0 else x.transpose(0, 1).contiguous()
        y = ops.mxfp8_dequantize(*ops.mxfp8_quantize_qk_rowwise(t.cuda(), layout), layout)
        codes, sc = mx.mx_quantize(f64(t), 32, "floor")
        assert np.array_equal(f64(y), mx.mx_dequantize(codes, sc, 32))


def test_large_offsets(ops):
    """Rows that start past 2^32 elements: those of a call on the last rows alone, bit for bit."""
    rows, N = 540000, 8192                             # 4.4e9 elements
    x = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    x[-300:].normal_()
    x[:-300] = 1.0
    w = torch.randn(N, device="cuda")
    y, _, rstd, y8, sc = ops.rms_norm(x, w, EPS, y8_out=True)
    want = ops.rms_norm(x[-300:], w, EPS, y8_out=True)
    for a, b in zip((y, rstd, y8, sc), (want[0],) + want[2:]):
        assert torch.equal(a[-300:], b)
    assert torch.equal(y[0], y[rows - 301])
    dx, _ = ops.rms_norm_bwd(y, x, w, rstd, dx=y)
    assert dx is y and torch.equal(dx[-300:], ops.rms_norm_bwd(want[0], x[-300:], w, want[2])[0])
    del x, dx, y
    z = ops.mxfp8_dequantize(y8, sc, None)
    assert torch.equal(z[-300:], ops.mxfp8_dequantize(want[3], want[4], None)) and torch.equal(z[0], z[rows - 301])


def test_host_threads(ops):
    """Calls of several host threads, each on its own stream, give the single call's bits."""
    import threading
    xs = [torch.randn((n, 1024), device="cuda").bfloat16() for n in (1, 300, 2000)]
    w = torch.randn(1024, device="cuda").bfloat16()

    def both(x, stream=None):
        y, s, rstd = ops.rms_norm(x, w, EPS, residual=x, stream=stream)
        return (y, s, rstd) + ops.rms_norm_bwd(y, s, w, rstd, ds=x, stream=stream)

    want = [both(x) for x in xs]
    torch.cuda.synchronize()
    got = [[] for _ in xs]

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(20):
            got[i].append(both(xs[i], s))
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for outs, ref in zip(got, want):
        assert len(outs) == 20 and all(torch.equal(a, b) for o in outs for a, b in zip(o, ref))
