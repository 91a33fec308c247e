"""Test infrastructure only: plain CPU fp64 oracle for what makes and chooses the attention's operands: the
root-mean-square norm and its gradients, rotary positions, and the choice of a cache's pages.

Nothing in the product path may import this module.
"""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------------------------------------------ the norm
def norm(s, w, eps):
    """s [rows, N] (as held), w [N] -> (y, rstd)."""
    rstd = 1 / np.sqrt(np.mean(s * s, -1) + eps)
    return s * rstd[:, None] * w, rstd


def norm_bwd(dy, s, w, rstd, ds=None):
    """-> (dx, dw, and for error bounds: |terms| of dx, |terms| of dw)."""
    hat, g = s * rstd[:, None], dy * w
    c = np.mean(g * hat, -1, keepdims=True)
    dx = rstd[:, None] * (g - hat * c) + (0 if ds is None else ds)
    size = rstd[:, None] * (np.abs(g) + np.abs(hat) * np.mean(np.abs(g * hat), -1, keepdims=True))
    return dx, (dy * hat).sum(0), size + (0 if ds is None else np.abs(ds)), np.abs(dy * hat).sum(0)


# --------------------------------------------------------------------------------- rotary positions
def angles(turns, pos):
    """Radians of positions pos (int array) for turns (uint64: turns per token times 2^64), exact to fp64."""
    with np.errstate(over="ignore"):
        t = np.asarray(pos).astype(np.int64).astype(np.uint64)[..., None] * np.asarray(turns, np.uint64)
    return t.astype(np.int64).astype(np.float64) * (np.pi / 2.0 ** 63)


def rotate(x, angle, magnitude, interleaved, inverse=False):
    """x [B, T, H, D]; angle [B, T, rot/2].  Returns (y, |terms| of y)."""
    rot = 2 * angle.shape[-1]
    c, s = (magnitude * f(angle)[:, :, None] for f in (np.cos, np.sin))
    if inverse:
        s = -s
    i = np.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = x[..., ia], x[..., ib]
    y, size = x.copy(), np.abs(x)
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    size[..., ia] = size[..., ib] = magnitude * (np.abs(a) + np.abs(b))
    return y, size


# ------------------------------------------------------------------------------- a cache's pages
def page_bounds(K):
    """K [tokens, H, D] of one page -> (codes [H, 2, D], exponent bytes [H])."""
    H, D = K.shape[1:]
    codes, exps = np.zeros((H, 2, D), np.int8), np.full(H, 0xFF, np.uint8)
    for h in range(H):
        k = K[:, h]
        top = np.max(np.abs(k)) if np.all(np.isfinite(k)) else np.inf
        if top >= 2.0 ** 107:
            continue
        e = max(int(np.frexp(max(top, 2.0 ** -200))[1]) - 1 - 6, -100)
        codes[h, 0] = np.floor(np.ldexp(k.min(0), -e))
        codes[h, 1] = np.ceil(np.ldexp(k.max(0), -e))
        exps[h] = e + 127
    return codes, exps


def query_codes(q):
    """q [G, D] of one KV head's query heads -> whole numbers u, l [D]."""
    if not np.all(np.isfinite(q)):
        return np.zeros(q.shape[1]), np.zeros(q.shape[1])
    u, l = np.maximum(q, 0).sum(0), np.maximum(-q, 0).sum(0)
    top = max(u.max(), l.max())
    if top < 2.0 ** -126:
        return np.zeros_like(u), np.zeros_like(l)
    f = min(6 - (int(np.frexp(top)[1]) - 1), 127)
    return tuple(np.minimum(np.rint(np.ldexp(x, f)), 127) for x in (u, l))


def choose(q, codes, exps, pages, tokens, page_size, top, first, last):
    """The pages of one query row and KV head, ascending.  codes [*, 2, D], exps [*] of this head by page id; pages: the
    sequence's ids (a bad one is None)."""
    n = -(-tokens // page_size)
    if n <= top:
        return list(range(n))
    u, l = query_codes(q)
    keys = []
    for i in range(n):
        if i < first or i >= n - last:
            rank, score = 3, 0.0
        elif pages[i] is None:
            rank, score = 0, 0.0
        elif exps[pages[i]] == 0xFF:
            rank, score = 2, 0.0
        else:
            c = codes[pages[i]].astype(np.float64)
            rank, score = 1, float(np.ldexp(u @ c[1] - l @ c[0], min(max(int(exps[pages[i]]), 27), 227) - 127))
        keys.append((-rank, -score, i))
    return sorted(i for _, _, i in sorted(keys)[:top])
