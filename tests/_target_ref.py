"""Plain 64-bit forms of the target-side calls, and how far a kernel may be off.

Attention: o = sum_j p_j v_j / sum_j p_j. With u = 2^-24, an error of ds in each
score (scores are fp32 sums of dh products: ds <= (dh + 4) u sum_d |q_d k_d| scale)
changes a weight by a factor within 1 +- 2 ds, exponentials and sums of n keys by
(n + 16) u more; bf16 rounds each weight (2^-8) and the result (2^-8 |o|) once. All of
it acts on sum_j p_j |v_j| / sum_j p_j at most.
"""
import numpy as np
import torch

U = 2.0 ** -24


def attention(q, k, v, scale, bf16):
    """q [dh], k and v [n, dh] in 64 bits -> (o, how far off it may be)."""
    if k.shape[0] == 0:
        return np.zeros(q.shape[0]), np.zeros(q.shape[0])
    s = k @ q * scale
    with np.errstate(invalid="ignore", over="ignore"):
        p = np.exp(s - s.max())
        p = p / p.sum()
        o, mag = p @ v, p @ np.abs(v)
    ds = (q.shape[0] + 4) * U * float(np.max(np.abs(k) @ np.abs(q))) * scale
    half = 2.0 ** -8 if bf16 else U
    return o, (4 * ds + (k.shape[0] + 16) * U + (half if bf16 else 0)) * mag + half * np.abs(o) + 1e-30


def to64(t):
    return t.detach().double().cpu().numpy()


def check_attention(got, want, tol, what=""):
    """Elementwise, non-finite values in the same places."""
    got, want, tol = np.asarray(got), np.asarray(want), np.asarray(tol)
    fin = np.isfinite(want)
    assert np.array_equal(fin, np.isfinite(got)), f"{what}: non-finite values in other places"
    d = np.abs(got[fin] - want[fin])
    bad = d > tol[fin]
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} values off, worst {float((d / tol[fin]).max()):.2f} of the bound"


def prompt(q, k, v, offsets, scale, bf16):
    """q [T, Hq, dh], k and v [T, Hkv, dh] tensors -> (o, tol) [T, Hq, dh]; rows of no sequence are NaN."""
    q, k, v = to64(q), to64(k), to64(v)
    T, hq, dh = q.shape
    G = hq // k.shape[1]
    o, tol = np.full(q.shape, np.nan), np.zeros(q.shape)
    for a, b in zip(offsets, offsets[1:]):
        for i in range(a, b):
            for h in range(hq):
                o[i, h], tol[i, h] = attention(q[i, h], k[a:i + 1, h // G], v[a:i + 1, h // G], scale, bf16)
    return o, tol


def pages(q, pk, pv, table, lens, scale, bf16, requests=None):
    """q [n, rows, Hq, dh]; pk, pv [pages, Hkv, page, dh] of one layer."""
    q, pk, pv = to64(q), to64(pk), to64(pv)
    n, rows, hq, dh = q.shape
    hkv, page = pk.shape[1], pk.shape[2]
    o, tol = np.zeros(q.shape), np.zeros(q.shape)
    for i in range(n):
        r = i if requests is None else requests[i]
        ids = table[r][:-(-lens[r] // page)]
        k = pk[ids].transpose(1, 0, 2, 3).reshape(hkv, -1, dh)
        v = pv[ids].transpose(1, 0, 2, 3).reshape(hkv, -1, dh)
        for t in range(rows):
            m = max(0, lens[r] - rows + t + 1)
            for h in range(hq):
                g = h // (hq // hkv)
                o[i, t, h], tol[i, t, h] = attention(q[i, t, h], k[g, :m], v[g, :m], scale, bf16)
    return o, tol


class Cache:
    """The page tables as lists, one call after the other (the rules of hf_pages)."""

    def __init__(self, layers, n_pages, hkv, page, dh, requests, columns, k=None, v=None):
        self.page, self.columns = page, columns
        self.k = np.zeros((layers, n_pages, hkv, page, dh)) if k is None else k
        self.v = np.zeros_like(self.k) if v is None else v
        self.rows = [[] for _ in range(requests)]
        self.lens = [0] * requests
        self.refs = [0] * n_pages

    def _distinct(self, rs):
        return len(set(rs)) == len(rs) and all(0 <= r < len(self.lens) for r in rs)

    def extend(self, rs, counts):
        if not self._distinct(rs) or min(counts, default=0) < 0:
            return "BAD"
        if any(self.lens[r] + c > self.columns * self.page for r, c in zip(rs, counts)):
            return "FULL"
        refs0 = list(self.refs)
        plan, free = [], [i for i, x in enumerate(refs0) if x == 0]
        for r, c in zip(rs, counts):
            copy = c > 0 and self.lens[r] % self.page > 0 and refs0[self.rows[r][-1]] > 1
            plan.append((r, c, copy, -(-(self.lens[r] + c) // self.page) - len(self.rows[r])))
        if sum(x[2] + x[3] for x in plan) > len(free):
            return "FULL"
        for r, c, copy, new in plan:
            if copy:
                old, to = self.rows[r][-1], free.pop(0)
                self.k[:, to], self.v[:, to] = self.k[:, old], self.v[:, old]
                self.refs[old] -= 1
                self.refs[to] = 1
                self.rows[r][-1] = to
            for _ in range(new):
                to = free.pop(0)
                self.refs[to] = 1
                self.rows[r].append(to)
            self.lens[r] += c
        return ""

    def write(self, rs, offsets, k, v, layer=0):
        for r, a, b in zip(rs, offsets, offsets[1:]):
            for t in range(a, b):
                at = self.lens[r] - b + t
                p = self.rows[r][at // self.page]
                self.k[layer:layer + k.shape[0], p, :, at % self.page] = k[:, t]
                self.v[layer:layer + k.shape[0], p, :, at % self.page] = v[:, t]

    def fork(self, source, into):
        if not self._distinct(into) or any(not 0 <= s < len(self.lens) for s in source) or set(source) & set(into):
            return "BAD"
        if any(self.lens[r] for r in into):
            return "BAD"
        for s, r in zip(source, into):
            self.rows[r], self.lens[r] = list(self.rows[s]), self.lens[s]
            for p in self.rows[s]:
                self.refs[p] += 1
        return ""

    def truncate(self, rs, keep):
        if not self._distinct(rs) or any(not 0 <= x <= self.lens[r] for r, x in zip(rs, keep)):
            return "BAD"
        for r, x in zip(rs, keep):
            n = -(-x // self.page)
            for p in self.rows[r][n:]:
                self.refs[p] -= 1
            self.rows[r], self.lens[r] = self.rows[r][:n], x
        return ""

    def compact(self):
        used = [i for i, x in enumerate(self.refs) if x > 0]
        high = [i for i in used if i >= len(used)]
        holes = [i for i in range(len(used)) if self.refs[i] <= 0]
        for a, b in zip(high, holes):
            self.k[:, b], self.v[:, b] = self.k[:, a], self.v[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.rows = [[b if p == a else p for p in row] for row in self.rows]
        return len(used)


def verify(x, y, tok, nd, u, noise, temp):
    """One request: (n_accepted, tokens, the tokens that rounding could make next as well)."""
    S, V = len(tok), x.shape[1]

    def soft(z):
        z = z / temp
        z = np.exp(z - z.max())
        return z / z.sum()

    a = 0
    if temp == 0:
        while a < nd and int(np.argmax(x[a])) == tok[a]:
            a += 1
        new, near = int(np.argmax(x[a])), set()
    else:
        def q(s):
            return soft(y[s]) if y is not None else np.eye(V)[tok[s]]
        while a < nd and u[a] * q(a)[tok[a]] < soft(x[a])[tok[a]]:
            a += 1
        p = soft(x[a])
        w = np.maximum(p - q(a), 0) if a < nd else p
        if not (w > 0).any():
            w = p
        s = w / noise
        new = int(np.argmax(s))
        # the kernel's weights: each probability within 2^-18 of its own (an exponent of at most
        # about 40 in 24 bits, a sum, a quotient), so a score within 2^-18 (p + q) / noise
        err = 2.0 ** -18 * (p + (q(a) if a < nd else 0)) / noise
        near = {int(i) for i in np.nonzero(s + err >= s[new] - err[new])[0]}
    return a + 1, list(tok[:a]) + [new] + [-1] * (S - a), near


def bf16(t):
    return t.to(torch.bfloat16)
