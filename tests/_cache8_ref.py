"""Plain 64-bit forms of the 8-bit cache and of rotary positions, and how far a kernel may be off.

Codes: nearest e4m3, ties to even; the scale a power of two, so x / scale is exact and both sides have to
give the same bits.

Attention over codes and scales, beside the terms of _target_ref.attention (u = 2^-24, n keys, dh products a
score, the result rounded to bf16, weights to 2^-8: a code has 4 bits, so hi is off by 2^-4 of
a weight at most and lo by 2^-4 of that): bf16 rows on the tensor cores are two codes in units
of 2^e, amax <= 448 * 2^e, amax > 224 * 2^e. lo is a code of 16 times the rest and ends at steps of 2^-9 / 16, so
a value is off by 2^-14 2^e < 2^-14 amax / 224 at most where hi + lo / 16 is not exact, and a score by that times
sum_d |k_d| scale. A weight's lo ends at the same steps, where the largest weight of a row is 2^1 at least:
2^-15 of the largest p_j s_j, and so sum_j |v_j / s_j| times that, over the sum of p.

Rotary: the reduced angle is off by 2^-32 turns of the product's cut and 2^-25 of its size, pi at most, in 32
bits (and 2^-52 * position in the table), cosine and sine by 2 units of 2^-24, two products, a sum,
the factor: 2^-21 (|a| + |b|) f covers them (2^-22 the angle, 2^-23 the functions and the rest), then one rounding
to bf16 2^-8, to fp32 2^-24.
"""
import math

import numpy as np
import torch

import _target_ref as R

LOW, HIGH, TOP = -64, 63, 448.0


def scale_for(top):
    """The least 2^e, LOW <= e <= HIGH, with top <= 448 2^e."""
    e = LOW
    while e < HIGH and top > TOP * 2.0 ** e:
        e += 1
    return 2.0 ** e


def held(x, scale):
    """Nearest e4m3 to x / scale, ties to even, as a value (without the scale); not finite: NaN."""
    y = np.asarray(x, dtype=np.float64) / scale
    with np.errstate(invalid="ignore"):
        size = np.minimum(np.abs(y), TOP)
        step = 2.0 ** (np.floor(np.log2(np.maximum(size, 2.0 ** -6))) - 3)
        z = np.copysign(np.rint(size / step) * step, y)
    return np.where(np.isfinite(np.asarray(x, dtype=np.float64)), z, np.nan)


def write_block(codes, scale, first, new):
    """Rows `new` into a page of one head from row `first` on: (codes, scale) after it. codes: values
    without the scale [page, dh]."""
    fin = np.abs(new[np.isfinite(new)])
    s = scale_for(fin.max() if fin.size else 0.0)
    out = codes.copy()
    if first:
        s = max(s, scale)
        out[:first] = held(codes[:first] * scale, s)
    out[first:first + len(new)] = held(new, s)
    return out, s


def values(codes, scale):
    """Codes [layers, pages, heads, page, dh] and scales as values in 64 bits."""
    return R.to64(codes.float()) * R.to64(scale)[..., None, None]


def attention(q, k, v, vs, scale, bf16, tc):
    """q [dh]; k, v [n, dh] values; vs [n] scales of V's pages."""
    o, tol = R.attention(q, k, v, scale, bf16)
    if not tc or k.shape[0] == 0:
        return o, tol
    with np.errstate(invalid="ignore", over="ignore"):
        s = k @ q * scale
        p = np.exp(s - s.max())
        mag = p @ np.abs(v) / p.sum()
        fine = 2.0 ** -15 * (p * vs).max() * np.sum(np.abs(v) / vs[:, None], 0) / p.sum()
        ds = 2.0 ** -14 * np.abs(q).max() / 224 * np.abs(k).sum(1).max() * scale
    return o, tol + fine + 4 * ds * mag


def pages(q, pk, pv, vs, table, lens, scale, bf16, tc, requests=None):
    """q [n, rows, Hq, dh]; pk, pv values [pages, Hkv, page, dh]; vs [pages, Hkv]: as _target_ref.pages."""
    q = R.to64(q)
    n, rows, hq, dh = q.shape
    hkv, page = pk.shape[1], pk.shape[2]
    o, tol = np.zeros(q.shape), np.zeros(q.shape)
    for i in range(n):
        r = i if requests is None else requests[i]
        ids = table[r][:-(-lens[r] // page)]
        k = pk[ids].transpose(1, 0, 2, 3).reshape(hkv, -1, dh)
        v = pv[ids].transpose(1, 0, 2, 3).reshape(hkv, -1, dh)
        s = np.repeat(vs[ids].T, page, axis=1).reshape(hkv, -1)
        for t in range(rows):
            m = max(0, lens[r] - rows + t + 1)
            for h in range(hq):
                g = h // (hq // hkv)
                o[i, t, h], tol[i, t, h] = attention(q[i, t, h], k[g, :m], v[g, :m], s[g, :m], scale, bf16, tc)
    return o, tol


def frequencies(dim, base, kind, factor=1.0, original=0, fast=0.0, slow=0.0, attention=0.0):
    """w_i in 64 bits and f, from hf_rotary_table's description."""
    if kind == "ntk":
        base = base * factor ** (dim / (dim - 2))
    w = [base ** (-2 * i / dim) for i in range(dim // 2)]
    if kind == "linear":
        w = [x / factor for x in w]
    if kind == "yarn":
        lo, hi = (dim * math.log(original / (2 * math.pi * t)) / (2 * math.log(base)) for t in (fast or 32.0, slow or 1.0))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), dim - 1)
        r = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(dim // 2)]
        w = [x * (1 - y) + x / factor * y for x, y in zip(w, r)]
    if kind == "bands":
        t = [min(max((original * x / (2 * math.pi) - (slow or 1.0)) / ((fast or 4.0) - (slow or 1.0)), 0.0), 1.0) for x in w]
        w = [x * y + x / factor * (1 - y) for x, y in zip(w, t)]
    return np.array(w), attention or (0.1 * math.log(factor) + 1 if kind == "yarn" else 1.0)


def rotary(x, pos, w, f, interleaved, bf16):
    """x [T, heads, dh] -> (y, how far off it may be)."""
    x = R.to64(x)
    half = len(w)
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    angle = np.asarray(pos, dtype=np.float64)[:, None, None] * w
    c, s = np.cos(angle) * f, np.sin(angle) * f
    y, tol = x.copy(), np.zeros(x.shape)
    u, v = a * c - b * s, b * c + a * s
    # the table's own 2^-52 of an angle, and this one's
    off = (2.0 ** -21 + np.abs(angle) * 2.0 ** -51) * abs(f) * (np.abs(a) + np.abs(b))
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = u, v
        tol[..., 0:2 * half:2], tol[..., 1:2 * half:2] = off, off
    else:
        y[..., :half], y[..., half:2 * half] = u, v
        tol[..., :half], tol[..., half:2 * half] = off, off
    half_step = 2.0 ** -8 if bf16 else 2.0 ** -24
    return y, tol + np.where(tol > 0, half_step * np.abs(y) + 2.0 ** -148, 0)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")
