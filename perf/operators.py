"""The key/value cache in MXFP4 and MXFP8: writing it, reading it back, and attention over it.

Three kinds of pass, each with a plain form in elementary torch operations and the form a user calls:

* "append": the new tokens of every sequence are quantised into their pages and read back as values
  (mx_cache_write, then mx_cache_read of the same positions);
* "read": cached tokens come back as bf16 or fp16 (mx_cache_read);
* "attend": T new queries per sequence attend the cached keys at and before their own position
  (mx_cache_attn), T = 1 for an ordinary decode step.

The cache: pages k, v [pages][Hkv][page_size][D * bits / 8] and one E8M0 scale per 32 elements along
D, k_sc, v_sc [pages][Hkv][page_size][D / 32].  4 bits are E2M1, the even element in the low nibble;
8 bits are E4M3.  Scale rule: e = clamp(floor(log2 amax) - emax, -127, 127), elements rounded to
nearest even and saturated.
"""
import functools
import math
import random

import torch

own = False

BSHD, SBHD = 0, 1
#: element width in bits, largest binade, largest value, mantissa bits, exponent of the smallest normal
FORMATS = {"fp4": (4, 2, 6.0, 1, 0), "fp8": (8, 8, 448.0, 3, -6)}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------------------- cases
def listed():
    def attend(name, **kw):
        return dict(dict(name=name, kind="attend", fmt="fp4", dtype="bf16", layout=BSHD, B=1, T=1, Hq=16, Hkv=4, D=128,
                         length=512, ragged=False, page=16, pattern="none"), **kw)

    def append(name, **kw):
        return dict(dict(name=name, kind="append", fmt="fp4", dtype="bf16", layout=BSHD, B=1, T=1, Hkv=4, D=128,
                         length=512, ragged=False, page=16, pattern="none"), **kw)

    def read(name, **kw):
        return dict(append(name, **kw), kind="read")

    return [
        # the first steps of one short conversation: nothing but latency
        attend("attend, one short", length=500),
        # one long conversation: a single row per query head, the keys split over the whole card
        attend("attend, one of 32K", length=32768, page=64),
        # a serving batch of unlike lengths, small pages
        attend("attend, 32 ragged", B=32, length=16384, ragged=True),
        # no shared heads and 8 bits: the most bytes
        attend("attend, 8 bits, 16 heads", fmt="fp8", B=16, Hkv=16, length=16384, page=128, pattern="heavy1pct"),
        # a draft of four tokens checked at once, fp16 activations
        attend("attend, draft of 4", dtype="fp16", B=16, T=4, length=8191, ragged=True, page=32),
        # a short chunk of a prompt behind a cached prefix, sequence-major activations
        attend("attend, chunk of 16", fmt="fp8", layout=SBHD, B=4, T=16, length=8209, page=64, pattern="every7x16"),
        # half-width heads, eight query heads to a key head, odd batch
        attend("attend, heads of 64", B=23, Hq=32, Hkv=4, D=64, length=4099, ragged=True, page=48),
        # one decode step of a small batch
        append("append, a token each", B=8, length=3001, ragged=True),
        # a long prompt goes into the cache at once
        append("append, prompt of 32K", T=32768, length=32768, page=64),
        # prompts of unlike lengths behind cached prefixes, 8 bits, sequence-major activations
        append("append, 8 ragged prompts", fmt="fp8", layout=SBHD, B=8, T=2048, Hkv=16, length=5003, ragged=True,
               page=32, pattern="heavy1pct"),
        # a short shared prefix
        read("read, short prefix", dtype="fp16", fmt="fp8", B=2, T=257, Hkv=4, length=400),
        # long prefixes of a batch
        read("read, 4 of 16K", B=4, T=16384, Hkv=16, length=16384, page=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    c = dict(kind=rng.choice(["attend", "attend", "append", "read"]), fmt=rng.choice(["fp4", "fp4", "fp8"]),
             dtype=rng.choice(["bf16", "bf16", "fp16"]), layout=rng.choice([BSHD, SBHD]), B=_log(rng, 1, 64), T=1,
             Hkv=rng.choice([1, 2, 4, 8, 16]), D=rng.choice([64, 128, 128]), length=_log(rng, 1, 32768),
             ragged=rng.random() < 0.6, page=16 * rng.choice([1, 2, 3, 4, 8, 16]),
             pattern=rng.choice(["none", "every7x16", "heavy1pct"]))
    most = (1 << 20) if c["fmt"] == "fp8" or c["kind"] != "attend" else (1 << 21)
    while c["B"] * c["Hkv"] * c["length"] > most:      # no more token-heads than the listed cases have
        c["B"] = max(1, c["B"] // 2) if c["B"] > 1 else 1
        if c["B"] == 1:
            c["length"] = min(c["length"], most // c["Hkv"])
    if c["kind"] == "attend":
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 5, 8])
        c["T"] = rng.choice([1, 1, 1, 2, 3, 4, 7, 8, 16])
    else:
        c["T"] = rng.choice([1, _log(rng, 1, c["length"]), c["length"]])
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
        if case["kind"] == "append" and case["ragged"] and b:
            t = r.randint(1, t)
        held.append(n)
        new.append(t)
    return held, new


def work(case):
    bits = FORMATS[case["fmt"]][0]
    held, new = _lengths(case)
    D, Hkv = case["D"], case["Hkv"]
    row = 2 * (D * bits // 8 + D // 32)                # a token's K and V of one head in the cache
    if case["kind"] == "append":                       # values in, cache out, cache in, values out
        return {"bytes": sum(new) * Hkv * 2 * (2 * 2 * D + row), "flops": sum(new) * Hkv * 2 * D * 4}
    if case["kind"] == "read":
        n = sum(min(case["T"], h) for h in held)
        return {"bytes": n * Hkv * row + case["B"] * case["T"] * Hkv * 2 * 2 * D, "flops": n * Hkv * 2 * D}
    Hq, T = case["Hq"], case["T"]
    seen = sum(sum(h - n + t + 1 for t in range(n)) for h, n in zip(held, new))
    return {"bytes": sum(held) * Hkv * row + case["B"] * T * Hq * (4 * D + 4), "flops": 4 * D * Hq * seen}


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
def _tokens(case, g, B, T):
    """K and V of T tokens, [B][T][Hkv][D] in 16 bits: normal, with the case's heavy V tokens."""
    shape = (B, T, case["Hkv"], case["D"])
    k = torch.randn(shape, generator=g, device="cuda")
    v = torch.randn(shape, generator=g, device="cuda")
    s = torch.arange(T, device="cuda")
    if case["pattern"] == "every7x16":
        v = v * torch.where((s + 1) % 7 == 0, 16.0, 1.0)[:, None, None]
    elif case["pattern"] == "heavy1pct":
        heavy = torch.rand(T, generator=g, device="cuda") < 0.01
        v = v * torch.where(heavy, 64.0, 1.0)[:, None, None]
    t = TYPES[case["dtype"]]
    return k.to(t), v.to(t)


def _in_layout(x, layout):
    return x if layout == BSHD else x.transpose(0, 1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    held, new = _lengths(case)
    B, T, Hkv, D, page, fmt = (case[n] for n in ("B", "T", "Hkv", "D", "page", "fmt"))
    width = max(-(-n // page) for n in held)
    pages = B * width + 1                              # the last page is no sequence's
    table = torch.randperm(pages - 1, generator=g, device="cuda").int().view(B, width)
    lens, fresh = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (held, new))
    row = D * FORMATS[fmt][0] // 8
    u8 = dict(dtype=torch.uint8, device="cuda")
    st = dict(case=dict(case), fmt=fmt, layout=case["layout"], T=T, page=page, table=table, lens=lens, new=fresh,
              starts=lens - fresh)
    if case["kind"] == "append":
        st["pools"] = [torch.zeros((pages, Hkv, page, n), **u8) for n in (row, D // 32, row, D // 32)]
        st["k"], st["v"] = (_in_layout(x, case["layout"]) for x in _tokens(case, g, B, T))
        return st
    if case["kind"] == "read":
        st["starts"] = torch.zeros_like(lens)
    pools = [torch.zeros((pages, Hkv, page, n), **u8) for n in (row, D // 32, row, D // 32)]
    for b in range(B):                                 # what earlier calls have written
        at = table[b].long()
        for i, x in enumerate(_tokens(case, g, 1, width * page)):
            code, sc = _quantise(x[0].view(width, page, Hkv, D).transpose(1, 2), fmt)
            pools[2 * i][at] = _pack(code, fmt)
            pools[2 * i + 1][at] = sc
    st["pools"] = pools
    if case["kind"] == "attend":
        q = torch.randn((B, T, case["Hq"], D), generator=g, device="cuda").to(TYPES[case["dtype"]])
        st["q"] = _in_layout(q, case["layout"])
    return st


# ---------------------------------------------------------------------------------------- the passes
def _slots(st, first, count):
    """Position, page and place in the page of `count` tokens of every sequence, the first at `first`."""
    pos = first[:, None].long() + torch.arange(count, device=first.device)
    safe = pos.clamp(0, st["table"].shape[1] * st["page"] - 1)
    at = torch.gather(st["table"].long(), 1, safe // st["page"])
    return pos, at, safe % st["page"]


def _read_plain(st, dtype):
    pos, at, off = _slots(st, st["starts"], st["T"])
    live = ((pos >= 0) & (pos < st["lens"][:, None]))[..., None, None]
    k, ks, v, vs = st["pools"]
    out = [_values(p[at, :, off], s[at, :, off], st["fmt"]) for p, s in ((k, ks), (v, vs))]
    return tuple(_in_layout(torch.where(live, x, 0.0).to(dtype), st["layout"]) for x in out)


def _append_plain(st):
    pos, at, off = _slots(st, st["starts"], st["T"])
    live = torch.arange(st["T"], device=pos.device) < st["new"][:, None]
    at = torch.where(live, at, st["pools"][0].shape[0] - 1)   # padding goes to the page that is no sequence's
    for i, x in enumerate((st["k"], st["v"])):
        x = x if st["layout"] == BSHD else x.transpose(0, 1)
        code, sc = _quantise(x, st["fmt"])
        st["pools"][2 * i][at, :, off] = _pack(code, st["fmt"])
        st["pools"][2 * i + 1][at, :, off] = sc
    return _read_plain(st, st["k"].dtype)


def _attend_plain(st):
    q = st["q"] if st["layout"] == BSHD else st["q"].transpose(0, 1)
    B, T, Hq, D = q.shape
    k, ks, v, vs = st["pools"]
    Hkv = k.shape[1]
    S = st["table"].shape[1] * st["page"]
    pos, at, off = _slots(st, torch.zeros_like(st["lens"]), S)
    K, V = (_values(p[at, :, off], s[at, :, off], st["fmt"]).transpose(1, 2) for p, s in ((k, ks), (v, vs)))
    q = q.float().view(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    s = torch.matmul(q, K.transpose(2, 3)) * D ** -0.5
    t = torch.arange(T, device=q.device)
    last = torch.where(t < st["new"][:, None], st["starts"][:, None] + t, -1)      # [B][T]
    last = last[:, None, :, None].expand(B, 1, T, Hq // Hkv).reshape(B, 1, -1, 1)
    seen = pos[:, None, None, :] <= last
    s = torch.where(seen, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, V) / torch.where(total > 0, total, 1.0)
    lse = torch.log(total) + top
    o = o.view(B, Hkv, T, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    lse = lse.view(B, Hkv, T, Hq // Hkv).permute(0, 1, 3, 2).reshape(B, Hq, T)
    return _in_layout(o.to(st["q"].dtype), st["layout"]), lse


def run(st):
    kind = st["case"]["kind"]
    if not own:
        if kind == "append":
            return _append_plain(st)
        return _read_plain(st, TYPES[st["case"]["dtype"]]) if kind == "read" else _attend_plain(st)
    from block_scaled_causal_gb300 import ops
    if "cache" not in st:                              # the handle that a program keeps beside its pages
        st["cache"] = ops.MxCache(*st["pools"], fmt=ops.CACHE_MXFP4 if st["fmt"] == "fp4" else ops.CACHE_MXFP8)
    cache = st["cache"]
    if kind == "attend":
        return ops.mx_cache_attn(st["q"], cache, st["table"], st["lens"], new_lens=st["new"], layout=st["layout"])
    if kind == "append":
        ops.mx_cache_write(cache, st["k"], st["v"], st["table"], st["lens"], new_lens=st["new"], layout=st["layout"])
    return ops.mx_cache_read(cache, st["table"], st["lens"], st["T"], starts=st["starts"], layout=st["layout"],
                             dtype=TYPES[st["case"]["dtype"]])


# -------------------------------------------------------------------------------- exactly, in 64 bits
def _grid(fmt):
    """The format's values at codes 0, 1, 2, ... of the positive half, in 64 bits."""
    out = []
    for code in range(8 if fmt == "fp4" else 127):
        if fmt == "fp4":
            out.append([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0][code])
        else:
            out.append((code & 7) * 2.0 ** -9 if code < 8 else (8 + (code & 7)) * 2.0 ** ((code >> 3) - 10))
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def _nearest(x, fmt):
    """What x [..., D] is held as: the nearest grid value times the block's power of two, ties to the even code."""
    grid = _grid(fmt)
    x = x.double()
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    # grid[-1] lies in the top binade: the block's maximum is brought to that binade
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
    fmt, page = st["fmt"], st["page"]
    data, sc = st["pools"][2 * which], st["pools"][2 * which + 1]
    at = st["table"][b, : -(-n // page)].long()
    data, sc = (x[at].permute(0, 2, 1, 3).flatten(0, 1)[:n] for x in (data, sc))
    if fmt == "fp4":
        data = torch.stack((data % 16, torch.div(data, 16, rounding_mode="floor")), -1).flatten(-2)
    half = 8 if fmt == "fp4" else 128
    data = data.long()
    grid = torch.cat((_grid(fmt), torch.full((half - _grid(fmt).numel(),), math.nan, dtype=torch.float64,
                                             device="cuda")))
    x = grid[data % half]
    x = torch.where(data >= half, -x, x)
    return x * torch.exp2(sc.double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    st = prepare(case, seed)
    held, new = _lengths(case)
    B, T, D = case["B"], case["T"], case["D"]
    if case["kind"] != "attend":
        outs = []
        for i in range(2):
            o = torch.zeros((B, T, case["Hkv"], D), dtype=torch.float64, device="cuda")
            for b in range(B):
                if case["kind"] == "append":
                    x = st["kv"[i]]
                    x = x[b] if case["layout"] == BSHD else x[:, b]
                    o[b, : new[b]] = _nearest(x[: new[b]], st["fmt"])
                else:
                    n = min(T, held[b])
                    o[b, :n] = _held(st, i, b, n)
            outs.append(o if case["layout"] == BSHD else o.transpose(0, 1).contiguous())
        return tuple(outs)
    Hq, Hkv = case["Hq"], case["Hkv"]
    G = Hq // Hkv
    o = torch.zeros((B, T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        K, V = _held(st, 0, b, held[b]), _held(st, 1, b, held[b])
        q = (st["q"][b] if case["layout"] == BSHD else st["q"][:, b]).double()
        for t in range(new[b]):
            n = held[b] - new[b] + t + 1
            s = torch.einsum("hgd,nhd->hgn", q[t].view(Hkv, G, D), K[:n]) / math.sqrt(D)
            z = torch.logsumexp(s, -1)
            o[b, t] = torch.einsum("hgn,nhd->hgd", torch.exp(s - z[..., None]), V[:n]).reshape(Hq, D)
            lse[b, :, t] = z.reshape(Hq)
    return (o if case["layout"] == BSHD else o.transpose(0, 1).contiguous()), lse
