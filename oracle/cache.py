"""Test infrastructure only: plain CPU fp64 oracle for the block-scaled key/value cache and the
attention that reads it.

Nothing in the product path may import this module.

* Format: rowwise MX blocks of 32 elements along D for K and V, E4M3 elements (MXFP8, oracle/mx.py)
  or E2M1 elements (MXFP4).  OCP Microscaling v1.0: E2M1 has one sign, two exponent bits (bias 1)
  and one fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6; emax_elem = 2; two elements per byte, the even
  one in the low nibble.  The scale rule is the one oracle/mx.py writes out, with 2 and 6 in the
  place of 8 and 448.
* Pages: pools [pages, Hkv, page_size, ...]; position p of a sequence is slot p % page_size of its
  page p // page_size.
* Attention: query t of n at position p = held - n + t sees j <= p;
  s_j = scale <q, K_j>, LSE = ln sum exp s_j, O = sum exp(s_j - LSE) V_j.
"""
from __future__ import annotations

import numpy as np

from oracle import mx

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
FP8, FP4 = 0, 1


def e2m1_encode(y):
    """Nibbles of finite fp64 values: nearest E2M1 magnitude (ties to the even code), saturating."""
    y = np.asarray(y, dtype=np.float64)
    a = np.minimum(np.abs(y), 6.0)
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    lo = np.searchsorted(mid, a, side="left")       # a value on a midpoint goes to the lower code ...
    on_mid = np.isin(a, mid)
    code = lo + (on_mid & (lo % 2 == 1))            # ... unless that one is odd
    return (code | (np.signbit(y).astype(np.int64) << 3)).astype(np.uint8)


def e2m1_decode(n):
    n = np.asarray(n, dtype=np.int64)
    return np.where(n & 8, -1.0, 1.0) * E2M1[n & 7]


def quantize(x, fmt, rule="floor"):
    """x [..., D] -> (bytes [..., D or D/2], scale bytes [..., D/32])."""
    if fmt == FP8:
        return mx.mx_quantize(x, 32, rule)
    x = np.asarray(x, dtype=np.float64)
    xb = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32))
    finite = np.all(np.isfinite(xb), axis=-1)
    amax = np.max(np.abs(np.where(np.isfinite(xb), xb, 0.0)), axis=-1)
    fl = np.frexp(np.where(amax > 0, amax, 1.0))[1].astype(np.int64) - 1
    e = fl - 2
    if rule == "ceil":
        e = e + (np.where(amax > 0, amax, 1.0) > np.ldexp(1.5, fl)).astype(np.int64)
    e = np.clip(np.where(amax > 0, e, -127), -127, 127)
    y = np.ldexp(np.where(finite[..., None], xb, 0.0), -e[..., None])
    n = np.where(finite[..., None], e2m1_encode(y), np.uint8(7)).reshape(x.shape)
    sb = np.where(finite, e + 127, 0xFF).astype(np.uint8)
    return (n[..., 0::2] | (n[..., 1::2] << 4)).astype(np.uint8), sb


def dequantize(data, sb, fmt):
    """fp64 values [..., D]; NaN where the scale byte is 0xFF."""
    if fmt == FP8:
        return mx.mx_dequantize(data, sb, 32)
    n = np.stack((data & 15, data >> 4), -1).reshape(data.shape[:-1] + (2 * data.shape[-1],))
    v = e2m1_decode(n)
    return (v.reshape(v.shape[:-1] + (v.shape[-1] // 32, 32)) * mx.e8m0_decode(sb)[..., None]).reshape(v.shape)


def gather(data, sb, fmt, pages, count, page_size):
    """Positions 0..count-1 of one sequence as values [count, Hkv, D] (`pages`: its page ids); rows of a
    page id that the pool does not have are NaN."""
    D = sb.shape[-1] * 32
    out = np.full((count, data.shape[1], D), np.nan)
    for p in range(count):
        page = int(pages[p // page_size])
        if 0 <= page < data.shape[0]:
            out[p] = dequantize(data[page, :, p % page_size], sb[page, :, p % page_size], fmt)
    return out


def attend(q, K, V, held, n, scale, absent=None):
    """One sequence.  q [T, Hq, D]; K, V [>= held, Hkv, D]; absent: positions that are not attended.

    Returns O [T, Hq, D], LSE [Hq, T], and what error bounds need: A = sum p_j |V_j| (as O) and
    E = max_j scale * sum_d |q_d K_jd| (as LSE)."""
    T, Hq, D = q.shape
    Hkv = K.shape[1]
    G = Hq // Hkv
    O, A = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    L, E = np.full((Hq, T), -np.inf), np.zeros((Hq, T))
    for t in range(min(n, T)):
        lim = held - n + t + 1
        js = [j for j in range(max(lim, 0)) if absent is None or j not in absent]
        if not js:
            continue
        for h in range(Hq):
            k, v = K[js, h // G], V[js, h // G]
            with np.errstate(invalid="ignore", over="ignore"):
                s = scale * (k @ q[t, h])
                m = np.max(s)
                p = np.exp(s - m)
                z = p.sum()
                O[t, h], A[t, h] = (p / z) @ v, (p / z) @ np.abs(v)
                L[h, t] = m + np.log(z)
                E[h, t] = scale * np.max(np.abs(k) @ np.abs(q[t, h]))
    return O, L, A, E
