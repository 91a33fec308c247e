"""What stands around the attention: the norm before its projections, rotary positions of its Q and K, and reading
only a few pages of a long cache.

Each kind of pass has a plain form in elementary torch operations and the form a user calls:

* "norm": root-mean-square norm of rows, s = x + residual held in the activations' type, y = s rstd w; y in 16
  bits, or in MXFP8 and read back as values (rms_norm, mxfp8_dequantize); or its gradients (rms_norm_bwd);
* "rope": rotary positions of Q and K: in 16 bits, and their gradients (rope); to MXFP8 rows, read back as values
  (mxfp8_rope_quantize_qk, mxfp8_dequantize); on the way into the key/value cache, read back as values
  (mx_cache_write_rope, mx_cache_read);
* "sparse": a decode step over a long cache: the bounds of the pages that hold the newest tokens are brought up to
  date, then every query and KV head attends the pages that its score selects (mx_cache_bounds,
  mx_cache_sparse_attn).

The cache: pages k, v [pages][Hkv][page_size][D * bits / 8] and one E8M0 scale per 32 elements along D, k_sc, v_sc
[pages][Hkv][page_size][D / 32].  4 bits are E2M1, the even element in the low nibble; 8 bits are E4M3.  Scale rule:
e = clamp(floor(log2 amax) - emax, -127, 127), elements rounded to nearest even and saturated.
"""
import functools
import math
import random

import torch

own = False

BSHD, SBHD = 0, 1
#: element width in bits, largest binade, largest value, mantissa bits, exponent of the smallest normal
FORMATS = {"fp4": (4, 2, 6.0, 1, 0), "fp8": (8, 8, 448.0, 3, -6)}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------------------------------- cases
def listed():
    def norm(name, **kw):
        return dict(dict(name=name, kind="norm", dtype="bf16", weight="bf16", rows=1, N=2048, residual=True, form="act"), **kw)

    def rope(name, **kw):
        return dict(dict(name=name, kind="rope", form="act", dtype="bf16", layout=BSHD, B=1, T=1, Hq=16, Hkv=4, D=128, rot=128,
                         interleaved=False, base=10000.0, scaling="plain", factor=1.0, positions="from 0", fmt="fp4",
                         page=16, length=512, ragged=False), **kw)

    def sparse(name, **kw):
        return dict(dict(name=name, kind="sparse", fmt="fp4", dtype="bf16", layout=BSHD, B=1, T=1, Hq=16, Hkv=4, D=128,
                         length=32768, ragged=False, page=64, top=32, first=1, last=2), **kw)

    return [
        # the norm of a decode step's only token: nothing but latency
        norm("norm, one token"),
        # a batch of prompts through the norm ahead of 8-bit projections
        norm("norm, prompts to MXFP8", rows=8192, N=4096, form="mx"),
        # the norm of each head of Q before it is rotated, fp32 weights, fp16 activations
        norm("norm, heads", dtype="fp16", weight="fp32", rows=262144, N=128, residual=False),
        # a training step's gradients, the residual stream's own gradient added, a width that is no power of two
        norm("norm, gradients", rows=16384, N=2560, form="grad"),
        # Q and K of a long training sequence, forward and back
        rope("rope, training 32K", T=32768),
        # half of each head rotated, neighbouring pairs, packed sequences with positions of their own, fp16
        rope("rope, half a head, packed", dtype="fp16", layout=SBHD, B=3, T=1021, Hq=20, Hkv=5, D=96, rot=48,
             interleaved=True, positions="each"),
        # a context eight times the trained one, straight to the operands of the 8-bit attention
        rope("rope to MXFP8, 8K", form="mx", T=8192, Hkv=16, base=500000.0, scaling="by parts", factor=8.0,
             positions="starts"),
        # one decode step of a small batch: q rotated, k and v into the cache
        rope("rope into the cache, a token each", form="cache", B=8, length=3001, ragged=True),
        # a chunk of prompts behind cached prefixes, 8 bits
        rope("rope into the cache, prompts", form="cache", fmt="fp8", layout=SBHD, B=4, T=4096, Hkv=8, length=20011,
             page=64, ragged=True, scaling="linear", factor=4.0),
        # one decode step of one long conversation: a sixteenth of its pages is read
        sparse("sparse, one of 32K"),
        # a serving batch of unlike lengths, 8 bits, small pages
        sparse("sparse, 32 ragged", fmt="fp8", B=32, length=16384, ragged=True, page=32, top=48, last=4),
        # a draft of three tokens, half-width heads, eight query heads to a KV head
        sparse("sparse, draft of 3", dtype="fp16", layout=SBHD, B=5, T=3, Hq=32, D=64, length=24007, ragged=True, page=48,
               top=21, first=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "rope", "rope", "rope", "sparse", "sparse"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if kind == "norm":
        form = rng.choice(["act", "act", "mx", "grad"])
        n = _log(rng, 4, 1024) * 8 if form != "mx" else _log(rng, 1, 256) * 32
        return dict(kind=kind, dtype=dtype, weight=rng.choice([dtype, "fp32"]), rows=_log(rng, 1, min(262144, (1 << 25) // n)),
                    N=n, residual=rng.random() < 0.6, form=form)
    Hkv, D = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128, 128])
    c = dict(kind=kind, dtype=dtype, layout=rng.choice([BSHD, SBHD]), B=_log(rng, 1, 64), T=1, Hkv=Hkv, D=D,
             Hq=Hkv * rng.choice([1, 2, 3, 4, 5, 8]), page=16 * rng.choice([1, 2, 3, 4, 8]), fmt=rng.choice(["fp4", "fp8"]),
             length=_log(rng, 1, 32768), ragged=rng.random() < 0.6)
    if kind == "rope":
        c.update(form=rng.choice(["act", "act", "mx", "cache"]), T=_log(rng, 1, 8192), interleaved=rng.random() < 0.4,
                 base=rng.choice([10000.0, 500000.0]), scaling=rng.choice(["plain", "linear", "base", "by parts"]),
                 factor=rng.choice([2.0, 4.0, 8.0, 3.5]), positions=rng.choice(["from 0", "starts", "each"]))
        if c["form"] == "mx":
            c.update(D=128, dtype="bf16")
        elif c["form"] == "act":
            c["D"] = rng.choice([64, 80, 96, 128, 128, 192, 256])
        c["rot"] = rng.choice([c["D"], c["D"], 16 * rng.randint(1, c["D"] // 16)])
        if c["form"] == "cache":
            c["T"] = min(c["T"], c["length"])
        while c["B"] * c["T"] * (c["Hq"] + c["Hkv"]) * c["D"] > 1 << 25:      # about half of the largest listed case
            c["B"], c["T"] = (c["B"] // 2, c["T"]) if c["B"] > 1 else (1, c["T"] // 2)
        return c
    c.update(T=rng.choice([1, 1, 1, 2, 4]), top=_log(rng, 4, 96), first=rng.choice([0, 1, 1, 2]), last=rng.choice([1, 2]))
    while c["B"] * c["Hkv"] * c["length"] > 1 << 20:
        c["B"], c["length"] = (c["B"] // 2, c["length"]) if c["B"] > 1 else (1, c["length"] // 2)
    while c["B"] * c["T"] * c["Hkv"] * c["top"] * c["page"] > 1 << 18 and c["top"] > 4:
        c["top"] = max(4, c["top"] // 2)
    return c


def _lengths(case):
    """(tokens held, new tokens) of every sequence: fixed by the case, so that its work is."""
    r = random.Random(1000003 * case["B"] + 97 * case["length"] + case["T"])
    held, new = [], []
    for b in range(case["B"]):
        n = case["length"]
        if case["ragged"] and b:                       # the first one has the full length
            n = max(1, int(n * math.exp(r.uniform(-3.0, 0.0))))
        t = min(case["T"], n)
        if case["kind"] == "rope" and case["ragged"] and b:
            t = r.randint(1, t)
        held.append(n)
        new.append(t)
    return held, new


def work(case):
    if case["kind"] == "norm":
        rows, N, w = case["rows"], case["N"], 4 if case["weight"] == "fp32" else 2
        r = 2 if case["residual"] else 0
        if case["form"] == "grad":                     # dy, s, the residual's gradient in; dx out; weights and theirs
            return {"bytes": rows * (N * (4 + r + 2) + 4) + 2 * N * w, "flops": rows * N * 12}
        out = 2 if case["form"] == "act" else 1 + 1 / 32 + 1 + 1 / 32 + 2       # MXFP8 written, read back, values out
        return {"bytes": rows * (N * (2 + 2 * r + out) + 4) + N * w, "flops": rows * N * 5}
    D, Hq, Hkv, T = case["D"], case["Hq"], case["Hkv"], case["T"]
    if case["kind"] == "rope" and case["form"] != "cache":
        n = case["B"] * T * (Hq + Hkv) * D
        act = {"bytes": 8 * n, "flops": 6 * n}         # there and back
        return act if case["form"] == "act" else {"bytes": n * (2 + 2 * (1 + 1 / 32) + 2), "flops": 6 * n}
    held, new = _lengths(case)
    row = D * FORMATS[case["fmt"]][0] // 8 + D // 32   # a token's K or V of one head in the cache
    if case["kind"] == "rope":
        return {"bytes": sum(new) * (Hq * 2 * D + Hkv * (4 * D + 2 * row)) + case["B"] * T * (Hq * 2 * D + Hkv * 4 * D)
                + sum(new) * Hkv * 2 * row, "flops": sum(new) * (Hq * 3 + Hkv * 12) * D}
    page, top = case["page"], case["top"]
    pages = [-(-h // page) for h in held]
    read = sum(min(h, top * page) for h in held)       # of each KV head, if a draft's queries all agree
    fresh = sum((h - 1) // page - (h - n) // page + 1 for h, n in zip(held, new))
    return {"bytes": Hkv * (sum(pages) * (2 * D + 1) + fresh * (page * row + 2 * D + 1) + read * 2 * row)
            + case["B"] * T * (Hq * (4 * D + 4) + Hkv * top * 4),
            "flops": sum(n * (Hq * 4 * D * min(h, top * page) + Hkv * 4 * D * p) for h, n, p in zip(held, new, pages))}


# ------------------------------------------------------------------------------- the plain quantiser
def _floor_log2(a):
    return torch.frexp(a)[1] - 1


@functools.cache
def _powers():
    """2 ** e at index e + 127, e in [-127, 127]."""
    return torch.exp2(torch.arange(-127, 128, dtype=torch.float64, device="cuda")).float()


def _pow2(e):
    return _powers()[e + 127]


@functools.cache
def _decoded(fmt):
    """The element values of every byte, [256][elements per byte]."""
    bits, emax, most, mbits, emin = FORMATS[fmt]
    byte = torch.arange(256, device="cuda")
    code = byte[:, None] if fmt == "fp8" else torch.stack((byte & 15, byte >> 4), -1)
    field, m = (code >> mbits) & ((1 << (bits - 1 - mbits)) - 1), code & ((1 << mbits) - 1)
    a = (m + torch.where(field > 0, 1 << mbits, 0)) * _pow2(field.clamp(min=1) - 1 + emin - mbits)
    return torch.where((code >> (bits - 1)) > 0, -a, a)


def _quantise(x, fmt):
    """Element codes [..., D] and scale bytes [..., D / 32] of x [..., D]."""
    bits, emax, most, mbits, emin = FORMATS[fmt]
    x = x.float().unflatten(-1, (-1, 32))
    amax = x.abs().amax(-1)
    e = torch.where(amax > 0, (_floor_log2(amax) - emax).clamp(-127, 127), -127)
    a = x.abs() * _pow2(-e)[..., None]
    step = _pow2(_floor_log2(a).clamp(min=emin) - mbits)
    a = (torch.round(a / step) * step).clamp(max=most)
    ex = torch.where(a > 0, _floor_log2(a), emin).clamp(min=emin)
    code = (ex - emin) * (1 << mbits) + (a / _pow2(ex - mbits)).int()
    code = code + (torch.signbit(x).int() << (bits - 1))
    return code.to(torch.uint8).flatten(-2), (e + 127).to(torch.uint8)


def _pack(code, fmt):
    return code if fmt == "fp8" else code[..., 0::2] | (code[..., 1::2] << 4)


def _values(data, sc, fmt):
    """fp32 values of stored bytes [..., D * bits / 8] with scale bytes [..., D / 32]."""
    a = _decoded(fmt)[data.int()].flatten(-2)
    return (a.unflatten(-1, (-1, 32)) * _powers()[sc.int()][..., None]).flatten(-2)


# ------------------------------------------------------------------------------------------- inputs
def _in_layout(x, layout):
    return x if layout == BSHD else x.transpose(0, 1).contiguous()


def _pools(case, pages):
    row = case["D"] * FORMATS[case["fmt"]][0] // 8
    return [torch.zeros((pages, case["Hkv"], case["page"], n), dtype=torch.uint8, device="cuda")
            for n in (row, case["D"] // 32, row, case["D"] // 32)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    st, t = dict(case=dict(case)), TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if case["kind"] == "norm":
        rows, N = case["rows"], case["N"]
        loud = 1 + 7 * (torch.rand(N, generator=g, device="cuda") < 0.02)      # the few channels that activations have
        st["x"] = (normal(rows, N) * loud).to(t)
        st["r"] = (normal(rows, N) * 2 * loud).to(t) if case["residual"] else None
        st["w"] = (1 + 0.2 * normal(N)).to(TYPES[case["weight"]])
        if case["form"] == "grad":                     # what the forward pass kept, and the gradients that arrive
            x = st["x"].float()
            st["rstd"] = torch.rsqrt((x * x).mean(-1) + EPS)
            st["dy"] = (normal(rows, N) * 0.1).to(t)
            st["ds"] = (normal(rows, N) * 0.1).to(t) if case["residual"] else None
        return st

    B, T, Hq, Hkv, D, page, layout = (case[n] for n in ("B", "T", "Hq", "Hkv", "D", "page", "layout"))
    if case["kind"] == "rope":
        for name, H in (("q", Hq), ("k", Hkv), ("v", Hkv), ("dq", Hq), ("dk", Hkv)):
            if name in ("q", "k") or (name == "v") == (case["form"] == "cache") and case["form"] != "mx":
                st[name] = _in_layout(normal(B, T, H, D).to(t), layout)
        if case["positions"] == "from 0":
            st["positions"] = None
        elif case["positions"] == "starts":
            st["positions"] = torch.randint(0, 120000, (B,), generator=g, device="cuda").int()
        else:                                          # packed sequences: each one's positions start again
            at = torch.arange(T, device="cuda").int()
            cut = torch.randint(0, T, (B, 1), generator=g, device="cuda").int()
            st["positions"] = torch.where(at < cut, at + 1000, at - cut)
        if case["form"] != "cache":
            return st
    held, new = _lengths(case)
    width = max(-(-n // page) for n in held)
    pages = B * width + 1                              # the last page is no sequence's
    st["table"] = torch.randperm(pages - 1, generator=g, device="cuda").int().view(B, width)
    st["lens"], st["new"] = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (held, new))
    st["pools"] = _pools(case, pages)
    if case["kind"] == "rope":
        return st
    for b in range(B):                                 # what earlier calls have written: neighbours are alike
        at = st["table"][b].long()
        for i in range(2):
            x = (normal(width, Hkv, page, D) + normal(width, Hkv, 1, D)).to(t)
            code, sc = _quantise(x, case["fmt"])
            st["pools"][2 * i][at] = _pack(code, case["fmt"])
            st["pools"][2 * i + 1][at] = sc
    st["q"] = _in_layout(normal(B, T, Hq, D).to(t), layout)
    st["codes"] = torch.zeros((pages, Hkv, 2, D), dtype=torch.int8, device="cuda")
    st["exps"] = torch.zeros((pages, Hkv), dtype=torch.uint8, device="cuda")
    for b in range(B):                                 # the bounds of the full pages, from earlier steps
        at = st["table"][b].long()
        K = _values(st["pools"][0][at], st["pools"][1][at], case["fmt"])
        st["codes"][at], st["exps"][at] = _bounds(K, torch.ones((), dtype=torch.bool, device="cuda"))
    return st


# ---------------------------------------------------------------------------------------- the passes
def _norm_plain(st):
    x, r, w = st["x"], st["r"], st["w"].float()
    if st["case"]["form"] == "grad":
        x, rstd, dy = x.float(), st["rstd"][:, None], st["dy"].float()
        hat, gw = x * rstd, dy * w
        dx = rstd * (gw - hat * (gw * hat).mean(-1, keepdim=True))
        if st["ds"] is not None:
            dx = dx + st["ds"].float()
        return dx.to(st["x"].dtype), (dy * hat).sum(0).to(st["w"].dtype)
    s = x if r is None else (x.float() + r.float()).to(x.dtype)     # the stream is held in the activations' type
    a = s.float()
    rstd = torch.rsqrt((a * a).mean(-1, keepdim=True) + EPS)
    y = a * rstd * w
    if st["case"]["form"] == "mx":
        y = _values(*_quantise(y, "fp8"), "fp8")
    out = (y.to(x.dtype), rstd.flatten())
    return out if r is None else out + (s,)


def _norm_own(st, ops):
    form = st["case"]["form"]
    if form == "grad":
        return ops.rms_norm_bwd(st["dy"], st["x"], st["w"], st["rstd"], ds=st["ds"])
    if form == "act":
        y, s, rstd = ops.rms_norm(st["x"], st["w"], EPS, residual=st["r"])
    else:
        _, s, rstd, y8, sc = ops.rms_norm(st["x"], st["w"], EPS, residual=st["r"], y8_out=True, y_out=False)
        y = ops.mxfp8_dequantize(y8, sc, dtype=st["x"].dtype)
    return (y, rstd) if st["r"] is None else (y, rstd, s)


def _frequencies(case):
    """Radians per token of each pair, in 64 bits, and the factor on what is rotated."""
    rot, base, factor = case["rot"], case["base"], case["factor"]
    if case["scaling"] == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] != "by parts":
        return f, 1.0
    keep = ((f * 8192 / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)    # pairs of many turns in 8192 tokens stay
    return f * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1


def _angles(case, pos):
    f, m = _frequencies(case)
    a = pos.double()[..., None] * f
    return (torch.cos(a) * m).float()[:, :, None], (torch.sin(a) * m).float()[:, :, None]


def _rotate(x, cos, sin, case):
    """x [B, T, H, D] in fp32; cos, sin [B, T, 1, rot / 2]."""
    rot, x = case["rot"], x.float()
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _as_bshd(x, case):
    return x if case["layout"] == BSHD else x.transpose(0, 1)


def _rope_plain(st):
    case, t = st["case"], st["q"].dtype
    q, k = (_as_bshd(st[n], case) for n in "qk")
    at = torch.arange(case["T"], device=q.device)
    if case["form"] == "cache":
        pos = (st["lens"] - st["new"])[:, None] + at
    elif st["positions"] is None:
        pos = at[None]
    else:
        pos = st["positions"] if st["positions"].dim() == 2 else st["positions"][:, None] + at
    cos, sin = _angles(case, pos)
    q, k = _rotate(q, cos, sin, case), _rotate(k, cos, sin, case)
    if case["form"] == "act":
        back = tuple(_rotate(_as_bshd(st[n], case), cos, -sin, case) for n in ("dq", "dk"))
        return tuple(_in_layout(x.to(t), case["layout"]) for x in (q, k) + back)
    if case["form"] == "mx":
        return tuple(_in_layout(_values(*_quantise(x, "fp8"), "fp8").to(t), case["layout"]) for x in (q, k))
    live = at < st["new"][:, None]
    slot = pos.long().clamp(0, st["table"].shape[1] * case["page"] - 1)
    page = torch.gather(st["table"].long(), 1, slot // case["page"])
    off, to = slot % case["page"], torch.where(live, page, st["pools"][0].shape[0] - 1)   # padding: to no sequence's page
    outs = [torch.where(live[..., None, None], q, 0.0)]
    for_k, for_v = (_quantise(x, case["fmt"]) for x in (k, _as_bshd(st["v"], case)))
    kp, ks, vp, vs = st["pools"]
    kp[to, :, off], ks[to, :, off] = _pack(for_k[0], case["fmt"]), for_k[1]
    vp[to, :, off], vs[to, :, off] = _pack(for_v[0], case["fmt"]), for_v[1]
    outs += [torch.where((pos < st["lens"][:, None])[..., None, None], _values(p[page, :, off], s[page, :, off], case["fmt"]),
                         0.0) for p, s in ((kp, ks), (vp, vs))]
    return tuple(_in_layout(x.to(t), case["layout"]) for x in outs)


def _rope_own(st, ops):
    case, layout = st["case"], st["case"]["layout"]
    if "rope" not in st:                               # the handle that a program keeps: a frequency per pair
        kind = {"plain": ops.ROPE_PLAIN, "linear": ops.ROPE_LINEAR, "base": ops.ROPE_BASE, "by parts": ops.ROPE_BY_PARTS}
        st["rope"] = ops.Rope(case["rot"], base=case["base"], interleaved=case["interleaved"], scaling=kind[case["scaling"]],
                              factor=case["factor"], original_length=8192)
    if case["form"] == "act":
        return ops.rope(st["q"], st["k"], st["rope"], st["positions"], layout) + \
            ops.rope(st["dq"], st["dk"], st["rope"], st["positions"], layout, inverse=True)
    if case["form"] == "mx":
        q, qs, k, ks = ops.mxfp8_rope_quantize_qk(st["q"], st["k"], st["rope"], st["positions"], layout)
        return ops.mxfp8_dequantize(q, qs, layout=layout), ops.mxfp8_dequantize(k, ks, layout=layout)
    cache, t = _cache(st, ops), st["q"].dtype
    if "starts" not in st:                             # kept beside the lengths
        st["starts"] = st["lens"] - st["new"]
    q = ops.mx_cache_write_rope(cache, st["q"], st["k"], st["v"], st["rope"], st["table"], st["lens"], new_lens=st["new"],
                                layout=layout)
    return (q,) + tuple(ops.mx_cache_read(cache, st["table"], st["lens"], case["T"], starts=st["starts"], layout=layout,
                                          dtype=t))


def _cache(st, ops):
    if "cache" not in st:                              # the handle that a program keeps beside its pages
        st["cache"] = ops.MxCache(*st["pools"], fmt=ops.CACHE_MXFP4 if st["case"]["fmt"] == "fp4" else ops.CACHE_MXFP8)
    return st["cache"]


def _bounds(K, live):
    """Codes [..., 2, D] and exponent bytes [...] of the keys K [..., tokens, D] that are `live` [..., tokens, 1]."""
    lo = torch.where(live, K, math.inf).amin(-2)
    hi = torch.where(live, K, -math.inf).amax(-2)
    amax = torch.maximum(lo.abs(), hi.abs()).amax(-1)
    e = (_floor_log2(amax.clamp(min=2.0 ** -120)) - 6).clamp(-100, 100)
    f = _pow2(-e)[..., None]
    codes = torch.stack((torch.floor(lo * f), torch.ceil(hi * f)), -2)
    return codes.to(torch.int8), (e + 127).to(torch.uint8)


def _sparse_plain(st):
    case = st["case"]
    B, T, Hq, Hkv, D, page, top, fmt = (case[n] for n in ("B", "T", "Hq", "Hkv", "D", "page", "top", "fmt"))
    kp, ks, vp, vs = st["pools"]
    codes, exps, table, lens, new = st["codes"], st["exps"], st["table"].long(), st["lens"], st["new"]
    width, last_page = table.shape[1], kp.shape[0] - 1
    # the pages that hold the newest tokens
    j = ((lens - new) // page)[:, None] + torch.arange((T - 1) // page + 2, device=table.device)
    live = j * page < lens[:, None]
    at = torch.where(live, torch.gather(table, 1, j.clamp(max=width - 1).long()), last_page)
    token = j[..., None] * page + torch.arange(page, device=table.device)
    K = _values(kp[at], ks[at], fmt)
    c, e = _bounds(K, (token < lens[:, None, None])[:, :, None, :, None] | ~live[..., None, None, None])
    codes[at] = torch.where(live[..., None, None, None], c, codes[last_page])
    exps[at] = torch.where(live[..., None], e, exps[last_page])
    # every page's score for every query and KV head: whole numbers times powers of two, exact in 32 bits
    q = _as_bshd(st["q"], case).float().unflatten(2, (Hkv, -1))                      # [B][T][Hkv][G][D]
    ul = torch.stack((q.clamp(min=0).sum(3), (-q).clamp(min=0).sum(3)), 3)             # [B][T][Hkv][2][D]
    big = ul.amax((-2, -1), keepdim=True)
    ul = torch.round(ul * _pow2((6 - _floor_log2(big)).clamp(-127, 127))).clamp(max=127.0)
    lo, hi = (codes[table][..., i, :].float().permute(0, 2, 3, 1) for i in (0, 1))    # [B][Hkv][D][W]
    u, low = ul[..., 0, :].transpose(1, 2), ul[..., 1, :].transpose(1, 2)              # [B][Hkv][T][D]
    score = torch.matmul(u, hi) - torch.matmul(low, lo)                               # [B][Hkv][T][W]
    score = score * _powers()[exps[table].int()].transpose(1, 2)[:, :, None]
    t = torch.arange(T, device=table.device)
    p = torch.where(t < new[:, None], (lens - new)[:, None] + t, -1)                   # [B][T]
    n = (p // page + 1)[:, None, :, None]
    w = torch.arange(width, device=table.device)
    forced = (w < case["first"]) | (w >= n - case["last"])
    score = torch.where(w < n, torch.where(forced, math.inf, score), -math.inf)
    pick = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :top]
    pick = torch.sort(torch.where(pick < n, pick, width), dim=-1).values
    pick = torch.cat((pick, pick.new_full(pick.shape[:-1] + (max(0, top - width),), width)), -1)   # [B][Hkv][T][top]
    # attention over them
    safe = pick.clamp(max=width - 1)
    at = torch.gather(table[:, None, None].expand(B, Hkv, T, width), 3, safe)
    h = torch.arange(Hkv, device=table.device)[None, :, None, None]
    K, V = (_values(x[at, h], s[at, h], fmt).flatten(3, 4) for x, s in ((kp, ks), (vp, vs)))     # [B][Hkv][T][top page][D]
    pos = (safe[..., None] * page + torch.arange(page, device=table.device)).flatten(3)
    seen = (pick < width)[..., None].expand(pick.shape + (page,)).flatten(3) & (pos <= p[:, None, :, None])
    s = torch.matmul(q.transpose(1, 2), K.transpose(3, 4)) * D ** -0.5                # [B][Hkv][T][G][top page]
    s = torch.where(seen[:, :, :, None], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    x = torch.exp(s - m)
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, V) / torch.where(total > 0, total, 1.0)
    o = o.transpose(1, 2).reshape(B, T, Hq, D).to(st["q"].dtype)
    lse = (torch.log(total) + m)[..., 0].permute(0, 1, 3, 2).reshape(B, Hq, T)
    blocks = torch.where(pick < width, pick, -1).int().transpose(1, 2).contiguous()
    return _in_layout(o, case["layout"]), lse, blocks, codes, exps


def _sparse_own(st, ops):
    case, cache = st["case"], _cache(st, ops)
    if "bounds" not in st:                             # likewise, on the caller's two buffers
        st["bounds"] = ops.MxBounds(cache, st["codes"], st["exps"])
    ops.mx_cache_bounds(cache, st["bounds"], st["table"], st["lens"], case["T"], new_lens=st["new"])
    o, lse, blocks = ops.mx_cache_sparse_attn(st["q"], cache, st["bounds"], st["table"], st["lens"], case["top"],
                                              first=case["first"], last=case["last"], new_lens=st["new"],
                                              layout=case["layout"])
    return o, lse, blocks, st["codes"], st["exps"]


def run(st):
    kind = st["case"]["kind"]
    if not own:
        return _norm_plain(st) if kind == "norm" else _rope_plain(st) if kind == "rope" else _sparse_plain(st)
    from block_scaled_causal_gb300 import ops
    return _norm_own(st, ops) if kind == "norm" else _rope_own(st, ops) if kind == "rope" else _sparse_own(st, ops)


# -------------------------------------------------------------------------------- exactly, in 64 bits
def _grid(fmt):
    """The format's values at codes 0, 1, 2, ... of the positive half, in 64 bits."""
    if fmt == "fp4":
        return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    return torch.tensor([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)],
                        dtype=torch.float64, device="cuda")


def _nearest(x, fmt):
    """What x [..., D] is held as: the nearest grid value times the block's power of two, ties to the even code."""
    grid = _grid(fmt)
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -200)))
    e = torch.where(torch.exp2(e + 1) <= amax, e + 1, e)
    e = torch.where(torch.exp2(e) > amax, e - 1, e) - math.floor(math.log2(float(grid[-1])))
    scale = torch.exp2(torch.where(amax > 0, e.clamp(-127, 127), torch.full_like(e, -127.0)))
    y = (b.abs() / scale).clamp(max=float(grid[-1])).contiguous()
    hi = torch.searchsorted(grid, y).clamp(max=grid.numel() - 1)       # first code at or above
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - y, y - grid[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (torch.copysign(grid[code], b) * scale).reshape(x.shape)


def _held(st, which, b, n):
    """The first n tokens of sequence b, [n][Hkv][D] in 64 bits, from the bytes."""
    fmt, page = st["case"]["fmt"], st["case"]["page"]
    data, sc = st["pools"][2 * which], st["pools"][2 * which + 1]
    at = st["table"][b, : -(-n // page)].long()
    data, sc = (x[at].permute(0, 2, 1, 3).flatten(0, 1)[:n] for x in (data, sc))
    if fmt == "fp4":
        data = torch.stack((data % 16, torch.div(data, 16, rounding_mode="floor")), -1).flatten(-2)
    half = 8 if fmt == "fp4" else 128
    grid = torch.cat((_grid(fmt), torch.zeros(1, dtype=torch.float64, device="cuda")))[:half]
    data = data.long()
    x = torch.where(data >= half, -grid[data % half], grid[data % half])
    return x * torch.exp2(sc.double() - 127).repeat_interleave(32, -1)


def _exact_norm(st):
    case, w = st["case"], st["w"].double()
    x, t = st["x"].double(), st["x"].dtype
    if case["form"] == "grad":
        rstd, dy = st["rstd"].double(), st["dy"].double()
        hat = torch.einsum("rn,r->rn", x, rstd)
        c = torch.einsum("rn,rn,n->r", dy, hat, w) / case["N"]
        dx = torch.einsum("rn,n,r->rn", dy, w, rstd) - torch.einsum("rn,r,r->rn", hat, c, rstd)
        return (dx if st["ds"] is None else dx + st["ds"].double()), torch.einsum("rn,rn->n", dy, hat)
    s = x if st["r"] is None else (x + st["r"].double()).to(t).double()
    rstd = 1 / torch.sqrt(torch.einsum("rn,rn->r", s, s) / case["N"] + EPS)
    y = torch.einsum("rn,r,n->rn", s, rstd, w)
    if case["form"] == "mx":
        y = _nearest(y, "fp8")
    return (y, rstd) if st["r"] is None else (y, rstd, s)


def _exact_rope(st):
    """Pairs as complex numbers, turned by exp(i angle)."""
    case = st["case"]
    B, T, rot = case["B"], case["T"], case["rot"]
    f, m = _frequencies(case)
    pos = torch.zeros((B, T), dtype=torch.float64, device="cuda")
    for b in range(B):
        start = 0
        if case["form"] == "cache":
            start = int(st["lens"][b]) - int(st["new"][b])
        elif st["positions"] is not None and st["positions"].dim() == 1:
            start = int(st["positions"][b])
        pos[b] = torch.arange(T, device="cuda") + start
    if case["form"] != "cache" and st["positions"] is not None and st["positions"].dim() == 2:
        pos = st["positions"].double()
    turn = torch.polar(torch.full_like(pos[..., None] * f, m), pos[..., None] * f)[:, :, None]

    def turned(x, turn):
        x = (x if case["layout"] == BSHD else x.transpose(0, 1)).double().contiguous()
        pair = x[..., :rot].unflatten(-1, (-1, 2) if case["interleaved"] else (2, -1))
        pair = pair if case["interleaved"] else pair.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        x[..., :rot] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
        return x

    def laid(x):
        return x if case["layout"] == BSHD else x.transpose(0, 1).contiguous()

    q, k = turned(st["q"], turn), turned(st["k"], turn)
    if case["form"] == "act":
        return tuple(laid(x) for x in (q, k, turned(st["dq"], turn.conj()), turned(st["dk"], turn.conj())))
    if case["form"] == "mx":
        return laid(_nearest(q, "fp8")), laid(_nearest(k, "fp8"))
    v = (st["v"] if case["layout"] == BSHD else st["v"].transpose(0, 1)).double()
    k, v = _nearest(k, case["fmt"]), _nearest(v, case["fmt"])
    for b in range(B):
        for x in (q, k, v):
            x[b, int(st["new"][b]):] = 0
    return laid(q), laid(k), laid(v)


def _exact_sparse(st):
    """One sequence, query and KV head after another; the pages by whole-number scores."""
    case = st["case"]
    B, T, Hq, Hkv, D, page, top = (case[n] for n in ("B", "T", "Hq", "Hkv", "D", "page", "top"))
    G = Hq // Hkv
    q_all = (st["q"] if case["layout"] == BSHD else st["q"].transpose(0, 1)).double()
    o = torch.zeros((B, T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device="cuda")
    held, new = _lengths(case)
    for b in range(B):
        K, V = _held(st, 0, b, held[b]), _held(st, 1, b, held[b])
        pages = -(-held[b] // page)
        at = st["table"][b, :pages].long()
        codes, exps = st["codes"][at].double(), st["exps"][at].double()
        for i in range((held[b] - new[b]) // page, pages):             # bounds of the pages with the newest tokens
            k = K[i * page: (i + 1) * page]
            lo, hi = k.amin(0), k.amax(0)
            e = torch.floor(torch.log2(torch.maximum(lo.abs(), hi.abs()).amax(-1).clamp(min=2.0 ** -94))) - 6
            codes[i, :, 0], codes[i, :, 1] = torch.floor(lo / torch.exp2(e)[:, None]), torch.ceil(hi / torch.exp2(e)[:, None])
            exps[i] = e + 127
        for t in range(new[b]):
            n = held[b] - new[b] + t + 1
            seen = -(-n // page)
            q = q_all[b, t].view(Hkv, G, D)
            u, low = q.clamp(min=0).sum(1), (-q).clamp(min=0).sum(1)
            big = torch.maximum(u, low).amax(-1, keepdim=True)
            unit = torch.exp2(torch.floor(torch.log2(big)) - 6)
            u, low = (torch.round(x / unit).clamp(max=127) for x in (u, low))
            score = torch.einsum("hd,phd->hp", u, codes[:seen, :, 1]) - torch.einsum("hd,phd->hp", low, codes[:seen, :, 0])
            score = score * torch.exp2(exps[:seen] - 127).T
            score[:, : case["first"]] = math.inf
            score[:, max(0, seen - case["last"]):] = math.inf
            pick = torch.argsort(score, dim=-1, descending=True, stable=True)[:, :top]
            token = torch.zeros((Hkv, seen), dtype=torch.bool, device="cuda").scatter(1, pick, True)
            token = token.repeat_interleave(page, 1)[:, :n]
            s = torch.einsum("hgd,nhd->hgn", q, K[:n]) / math.sqrt(D)
            s = torch.where(token[:, None], s, -math.inf)
            z = torch.logsumexp(s, -1)
            o[b, t] = torch.einsum("hgn,nhd->hgd", torch.exp(s - z[..., None]), V[:n]).reshape(Hq, D)
            lse[b, :, t] = z.reshape(Hq)
    return (o if case["layout"] == BSHD else o.transpose(0, 1).contiguous()), lse, None, None, None


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "rope": _exact_rope, "sparse": _exact_sparse}[case["kind"]](st)
