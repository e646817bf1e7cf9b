"""The 8-bit cache on the GPU against plain forms in 64 bits (_cache8_ref.py, which also derives
the tolerances)."""
import random

import numpy as np
import pytest
import torch

import _cache8_ref as C
import _target_ref as R

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def hf():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from speculative_decoding_drafter_hf_gb300 import build
    build.build()
    import speculative_decoding_drafter_hf_gb300 as m
    return m


def _randn(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(DT[dtype])


def _tc(dtype, dh):
    return dtype == "bf16" and dh in (64, 128)


# ------------------------------------------------------------------ attention
ATTEND = [  # dtype, Hq, Hkv, dh, page, rows, shared, own lengths (None: an empty request)
    ("bf16", 4, 2, 128, 16, 1, 0, [1]),
    ("bf16", 8, 2, 128, 16, 8, 0, [3, 8, 9, 1000, None]),
    ("bf16", 8, 2, 128, 32, 8, 128, [0, 1, 8, 30, 700, None]),
    ("bf16", 4, 2, 64, 64, 5, 640, [5, 64, 1]),
    ("bf16", 5, 1, 128, 8, 7, 8, [2, 50, 77]),
    ("bf16", 10, 2, 64, 128, 2, 256, [300, 5]),
    ("bf16", 16, 1, 128, 16, 16, 2048, [40, 100]),
    ("bf16", 64, 1, 64, 16, 3, 32, [33, 4]),
    ("bf16", 15, 5, 128, 64, 1, 0, [129, 1, 128, 127]),
    ("bf16", 2, 2, 128, 128, 64, 128, [64, 30]),
    ("bf16", 4, 4, 128, 64, 1, 4096, [1] * 9),
    ("bf16", 32, 8, 128, 32, 1, 4096, [1, 700, 33]),
    ("bf16", 24, 8, 64, 8, 1, 0, [3000, 5]),
    ("bf16", 64, 1, 128, 32, 64, 64, [70, 64]),                  # as many rows as there are: 4096 of a head
    ("bf16", 6, 3, 128, 16, 9, 48, [200, 9, 8, 0]),              # a last head without a neighbour
    ("bf16", 21, 3, 64, 8, 7, 16, [100, 1]),                     # row tiles of 49 rows
    ("bf16", 8, 2, 128, 16, 8, 64, [40]),                        # the prefix's row tile is the entry's own
    ("bf16", 8, 2, 64, 16, 8, 64, [7]),
    ("bf16", 4, 2, 64, 32, 1, 64, [40]),
    ("bf16", 12, 2, 128, 32, 8, 64, [40, 100]),                  # row tiles of 48 rows beside a prefix's of 60
    ("bf16", 12, 2, 64, 32, 8, 64, [40, 100, None]),
    ("bf16", 4, 4, 32, 16, 4, 32, [20, 3]),
    ("bf16", 3, 1, 80, 32, 2, 64, [20, 90]),
    ("bf16", 2, 1, 256, 16, 64, 16, [64, 100]),
    ("f32", 4, 2, 64, 16, 8, 64, [3, 8, 9, 300, None]),
    ("f32", 8, 2, 128, 64, 3, 0, [130, 1]),
    ("f32", 3, 3, 48, 8, 1, 8, [1, 20]),
]


def _pool(shape, seed):
    """Codes and scales of a pool: heads and pages of different sizes."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(torch.randn(shape[:3], generator=g))[..., None, None]
    top = x.abs().amax((-1, -2))
    scale = torch.tensor([C.scale_for(float(t)) for t in top.flatten()]).view(top.shape)
    return (x / scale[..., None, None]).to(torch.float8_e4m3fn), scale


def _shared_cache(hkv, dh, page, shared, own, seed, layers=1):
    """A cache whose requests share `shared` tokens, pages in shuffled places; unused rows hold NaN."""
    rng = random.Random(seed)
    n_shared = shared // page
    counts = [0 if x is None else -(-x // page) for x in own]
    total = n_shared + sum(counts) + 3
    ids = list(range(total))
    rng.shuffle(ids)
    (k, ks), (v, vs) = (_pool((layers, total, hkv, page, dh), seed + s) for s in (1, 2))
    columns = n_shared + max(counts) + 1
    rows, lens, refs, at = [], [], [0] * total, n_shared
    used = torch.zeros((total, page), dtype=torch.bool)
    for x, c in zip(own, counts):
        row = [] if x is None else ids[:n_shared] + ids[at:at + c]
        at += c
        lens.append(0 if x is None else shared + x)
        for j, p in enumerate(row):
            refs[p] += 1
            used[p, :max(0, min(page, lens[-1] - j * page))] = True
        rows.append(row)
    for t in (k, v):
        t.view(torch.uint8).permute(1, 3, 0, 2, 4)[~used] = 0x7f
    for t in (ks, vs):
        t[:, ~used.any(1)] = float("nan")
    table = [row + [-1] * (columns - len(row)) for row in rows]
    return (k, v, ks, vs), table, lens, refs


def _on_gpu(hf, pool, table, lens, refs, dtype):
    return hf.Pages8(*(t.cuda() for t in pool), C.ints(table), C.ints(lens), C.ints(refs), dtype=DT[dtype])


def _want(q, pool, table, lens, dtype, layer=0, scale=None, req=None):
    k, v, ks, vs = pool
    dh = q.shape[-1]
    return C.pages(q, C.values(k, ks)[layer], C.values(v, vs)[layer], R.to64(vs)[layer], table, lens, scale or dh ** -0.5,
                   dtype == "bf16", _tc(dtype, dh), req)


@pytest.mark.parametrize("dtype,hq,hkv,dh,page,rows,shared,own", ATTEND)
def test_attend(hf, dtype, hq, hkv, dh, page, rows, shared, own):
    pool, table, lens, refs = _shared_cache(hkv, dh, page, shared, own, 7, layers=2)
    c = _on_gpu(hf, pool, table, lens, refs, dtype)
    n = len(own)
    pad = 16 // (4 if dtype == "f32" else 2)
    x = _randn((n, rows, hq + pad, dh), dtype, 9, 2.0)
    q = x[:, :, :hq]
    out = torch.full((n, rows, hq, dh), 7.0, dtype=DT[dtype], device="cuda")
    ws = c.attend_workspace(q, shared)
    ws.fill_(255)  # NaN everywhere: the workspace needs no values
    got = c.attend(x.cuda()[:, :, :hq], layer=1, shared=shared, out=out, workspace=ws)
    assert got is out
    want, tol = _want(q, pool, table, lens, dtype, layer=1)
    R.check_attention(R.to64(out), want, tol, "attend")
    assert not c.check()
    # the same without the prefix in common: the keys are the same ones
    again = c.attend(x.cuda()[:, :, :hq], layer=1)
    R.check_attention(R.to64(again), want, tol, "attend, nothing shared")
    assert not c.check()


@pytest.mark.parametrize("shared", [0, 32])
def test_attend_many_entries(hf, shared):
    """More entries than requests: a list that repeats them, some of them empty, some long."""
    own = [3, 17, 200, None, 64, 1, 33, 700, 16]
    pool, table, lens, refs = _shared_cache(2, 64, 16, shared, own, 8)
    c = _on_gpu(hf, pool, table, lens, refs, "bf16")
    rng = random.Random(5)
    req = [0] + [rng.randrange(len(own)) for _ in range(339)]
    q = _randn((340, 2, 4, 64), "bf16", 5)
    o = R.to64(c.attend(q.cuda(), C.ints(req), shared=shared))
    want, tol = _want(q, pool, table, lens, "bf16", req=req)
    R.check_attention(o, want, tol)
    assert not c.check()


@pytest.mark.parametrize("dtype,dh", [("bf16", 128), ("f32", 64)])
def test_attend_strange_entries_pages_and_prefixes(hf, dtype, dh):
    pool, table, lens, refs = _shared_cache(2, dh, 16, 64, [5, 60, 33, 9], 3)
    q = _randn((5, 3, 8, dh), dtype, 5)
    c = _on_gpu(hf, pool, table, lens, refs, dtype)
    req = [2, 0, 2, 3, 1]
    want, tol = _want(q, pool, table, lens, dtype, scale=0.11, req=req)
    for shared in (0, 64):
        R.check_attention(R.to64(c.attend(q.cuda(), C.ints(req), shared=shared, scale=0.11)), want, tol)
        assert not c.check()
    o = R.to64(c.attend(q.cuda(), C.ints([2, -1, 2, 4, 1]), scale=0.11))
    assert (o[1] == 0).all() and (o[3] == 0).all()
    for i in (0, 2, 4):
        R.check_attention(o[i], want[i], tol[i])
    assert c.check() == hf.CallStatus.BAD
    # lengths that fit neither the table nor the prefix
    for bad in (10 ** 6, -5, 40):
        c = _on_gpu(hf, pool, table, [lens[0], bad, lens[2], lens[3]], refs, dtype)
        o = R.to64(c.attend(q[:4].cuda(), shared=64))
        want, tol = _want(q[:4], pool, table, [lens[0], 0, lens[2], lens[3]], dtype)
        R.check_attention(o, want, tol)
        assert c.check() == hf.CallStatus.BAD
    # page ids out of range: reported, the others as before
    want, tol = _want(q[:4], pool, table, lens, dtype)
    for bad in (-1, -2, len(refs), 1 << 30):
        t = [list(r) for r in table]
        t[1][5] = bad
        c = _on_gpu(hf, pool, t, lens, refs, dtype)
        for shared in (0, 64):
            o = R.to64(c.attend(q[:4].cuda(), shared=shared))
            for i in (0, 2, 3):
                R.check_attention(o[i], want[i], tol[i])
            assert c.check() == hf.CallStatus.BAD
    # a prefix in other pages; an empty first entry; all empty
    t = [list(r) for r in table]
    t[2][3], t[2][4] = t[2][4], t[2][3]
    c = _on_gpu(hf, pool, t, lens, refs, dtype)
    o = R.to64(c.attend(q[:4].cuda(), shared=64))
    for i in (0, 1, 3):
        R.check_attention(o[i], want[i], tol[i])
    assert c.check() == hf.CallStatus.BAD
    c = _on_gpu(hf, pool, table, [0] + lens[1:], refs, dtype)
    assert (c.attend(q[:4].cuda(), shared=64) == 0).all()
    assert c.check() == hf.CallStatus.BAD
    c = _on_gpu(hf, pool, table, [0] * 4, refs, dtype)
    assert (c.attend(q[:4].cuda(), shared=64) == 0).all() and not c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads", [1, 2])
def test_attend_nan_codes_stay_with_the_rows_that_see_them(hf, dtype, heads):
    pool, table, lens, refs = _shared_cache(heads, 128, 16, 32, [90, 60], 6)
    p, k, v = table[0][-2], pool[0].view(torch.uint8), pool[1].view(torch.uint8)  # request 0's tokens 112 .. 121
    k[0, p, :, 8] = 0xff      # token 120, every value
    v[0, p, 0, 6, 5] = 0x7f   # token 118, one value
    q = _randn((2, 8, 4 * heads, 128), dtype, 11)
    c = _on_gpu(hf, pool, table, lens, refs, dtype)
    want, tol = _want(q, pool, table, lens, dtype)
    for shared in (0, 32):
        R.check_attention(R.to64(c.attend(q.cuda(), shared=shared)), want, tol)
    assert np.isnan(want).any() and not c.check()


@pytest.mark.parametrize("dh,page,odd_page", [(128, 32, False), (64, 64, False), (128, 16, True)])
def test_attend_a_long_prefix_of_many_rows(hf, dh, page, odd_page):
    """The prefix goes through bf16 rows: entries without tokens of their own (their first rows see part of the
    prefix), an empty one, one that names no request, and NaN codes at the prefix's end."""
    own = [5, 0, 200, None, 1, 40] + [3] * 10
    pool, table, lens, refs = _shared_cache(1, dh, page, 2304, own, 21)
    if odd_page:
        last = table[0][2304 // page - 1]
        pool[0].view(torch.uint8)[0, last, 0, page - 2] = 0x7f  # key 2302
        pool[1].view(torch.uint8)[0, last, 0, page - 3, 5] = 0xff  # one value of token 2301
    c = _on_gpu(hf, pool, table, lens, refs, "bf16")
    q = _randn((16, 8, 8, dh), "bf16", 22)
    want, tol = _want(q, pool, table, lens, "bf16")
    R.check_attention(R.to64(c.attend(q.cuda(), shared=2304)), want, tol)
    assert not c.check()
    if odd_page:
        assert np.isnan(want).any() and np.isfinite(want[1, 0]).all()
    o = R.to64(c.attend(q.cuda(), C.ints([0, 1, 2, 3, -7, 5] + list(range(6, 16))), shared=2304))
    assert (o[4] == 0).all() and c.check() == hf.CallStatus.BAD
    o[4] = want[4]
    R.check_attention(o, want, tol)
    # a page of the prefix out of range is reported; an empty first entry leaves zeros
    t = [list(r) for r in table]
    for r in t:
        if r[0] >= 0:
            r[3] = len(refs)
    c = _on_gpu(hf, pool, t, lens, refs, "bf16")
    c.attend(q.cuda(), shared=2304)
    assert c.check() == hf.CallStatus.BAD
    c = _on_gpu(hf, pool, table, [0] + lens[1:], refs, "bf16")
    assert (c.attend(q.cuda(), shared=2304) == 0).all() and c.check() == hf.CallStatus.BAD


def test_attend_a_long_prefix_of_many_entries(hf):
    """More entries than a CTA plans for by itself, over a prefix that goes through bf16 rows."""
    own = [3, 17, 90, None, 64, 1]
    pool, table, lens, refs = _shared_cache(2, 64, 128, 2048, own, 23)
    c = _on_gpu(hf, pool, table, lens, refs, "bf16")
    rng = random.Random(6)
    req = [0] + [rng.randrange(len(own)) for _ in range(299)]
    q = _randn((300, 2, 4, 64), "bf16", 24)
    want, tol = _want(q, pool, table, lens, "bf16", req=req)
    R.check_attention(R.to64(c.attend(q.cuda(), C.ints(req), shared=2048)), want, tol)
    assert not c.check()


def test_attend_scales_far_apart(hf):
    """Pages of scales from 2^-64 to 2^40 side by side, scores that differ by hundreds, and rows of very
    different sizes: the weights keep their bits."""
    pool, table, lens, refs = _shared_cache(1, 128, 16, 0, [700, 333], 12)
    for i, e in enumerate([-64, -30, 40, 0, 3, -7]):
        pool[3][0, table[0][7 * i]] = 2.0 ** e
    pool[2][0, table[0][3]] = 2.0 ** 5
    q = _randn((2, 4, 4, 128), "bf16", 13) * torch.tensor([2.0 ** -20, 1.0, 30.0, 2.0 ** -100], dtype=torch.bfloat16)[:, None]
    q[1, 2] = 0
    c = _on_gpu(hf, pool, table, lens, refs, "bf16")
    want, tol = _want(q, pool, table, lens, "bf16")
    R.check_attention(R.to64(c.attend(q.cuda())), want, tol)


def test_attend_rows_that_are_not_finite(hf):
    pool, table, lens, refs = _shared_cache(2, 128, 16, 0, [70, 200], 14)
    q = _randn((2, 3, 8, 128), "bf16", 15)
    want, tol = _want(q, pool, table, lens, "bf16")
    bad = q.clone()
    bad[0, 1, 3, 7], bad[1, 2, 0, 100] = float("nan"), float("inf")
    c = _on_gpu(hf, pool, table, lens, refs, "bf16")
    o = R.to64(c.attend(bad.cuda()))
    assert np.isnan(o[0, 1, 3]).all() and np.isnan(o[1, 2, 0]).all()
    o[0, 1, 3], o[1, 2, 0] = want[0, 1, 3], want[1, 2, 0]
    R.check_attention(o, want, tol)


def test_attend_on_another_stream_captured_and_two_at_once(hf):
    pool, table, lens, refs = _shared_cache(4, 128, 32, 64, [500, 33, 260], 16)
    c = _on_gpu(hf, pool, table, lens, refs, "bf16")
    q = _randn((3, 5, 8, 128), "bf16", 17).cuda()
    want, tol = _want(q, pool, table, lens, "bf16")
    first = c.attend(q, shared=64)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [c.attend(q, shared=64, stream=s) for s in (s1, s2) for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)  # (no result hangs on timing)
    R.check_attention(R.to64(first), want, tol)
    ws, out = c.attend_workspace(q, 64), torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.attend(q, shared=64, out=out, workspace=ws)
    for _ in range(3):
        out.fill_(3)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and not c.check()


def test_attend_a_long_prefix_replayed_and_two_at_once(hf):
    """The launches of a long prefix of many rows run into each other (the entries' own keys beside the prefix): with
    rows that change just before, in a graph, and on two streams at once."""
    own = [700, 3, 90, 1] * 12
    pool, table, lens, refs = _shared_cache(2, 128, 32, 2304, own, 29)
    c = _on_gpu(hf, pool, table, lens, refs, "bf16")
    qs = [_randn((48, 2, 8, 128), "bf16", 30 + i).cuda() for i in range(3)]
    firsts = []
    for q in qs:
        first = c.attend(q, shared=2304)
        torch.cuda.synchronize()
        firsts.append(first.clone())
    want, tol = _want(qs[0], pool, table, lens, "bf16")
    R.check_attention(R.to64(firsts[0]), want, tol)
    q, out, ws = torch.empty_like(qs[0]), torch.empty_like(qs[0]), c.attend_workspace(qs[0], 2304)
    ws.fill_(255)
    for i in (0, 1, 2, 1, 0, 2):  # no wait between the calls; the rows are written by the kernel just before
        q.copy_(qs[i])
        c.attend(q, shared=2304, out=out, workspace=ws)
        got = out.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, firsts[i])
    graph = torch.cuda.CUDAGraph()
    kept = [torch.empty_like(out) for _ in range(3)]
    with torch.cuda.graph(graph):
        for i in range(3):
            q.copy_(qs[i])
            c.attend(q, shared=2304, out=out, workspace=ws)
            kept[i].copy_(out)
    for _ in range(3):
        for k in kept:
            k.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(k, f) for k, f in zip(kept, firsts))
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(i, c.attend(qs[i], shared=2304, stream=streams[i % 2])) for _ in range(6) for i in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, firsts[i]) for i, o in outs) and not c.check()


def test_attend_waits_that_run_out(hf):
    from speculative_decoding_drafter_hf_gb300 import _binding as B
    pool, table, lens, refs = _shared_cache(2, 128, 16, 32, [90, 60], 18)
    c = _on_gpu(hf, pool, table, lens, refs, "bf16")
    q = _randn((2, 2, 8, 128), "bf16", 19)
    want, tol = _want(q, pool, table, lens, "bf16")
    try:
        B.hf_debug_set_wait_limit(None, 0)
        c.attend(q.cuda(), shared=32)
        assert c.check() == hf.CallStatus.TIMEOUT
    finally:
        B.hf_debug_set_wait_limit(None, -1)
    R.check_attention(R.to64(c.attend(q.cuda(), shared=32)), want, tol)
    assert not c.check()
    # through bf16 rows as well
    pool, table, lens, refs = _shared_cache(1, 128, 64, 2304, [5] * 16, 25)
    c = _on_gpu(hf, pool, table, lens, refs, "bf16")
    q = _randn((16, 8, 8, 128), "bf16", 26)
    want, tol = _want(q, pool, table, lens, "bf16")
    try:
        B.hf_debug_set_wait_limit(None, 0)
        c.attend(q.cuda(), shared=2304)
        assert c.check() == hf.CallStatus.TIMEOUT
    finally:
        B.hf_debug_set_wait_limit(None, -1)
    R.check_attention(R.to64(c.attend(q.cuda(), shared=2304)), want, tol)
    assert not c.check()


def test_attend_queries_of_every_size(hf):
    """Rows from the smallest to the largest bf16 values, with a scale to go with them."""
    pool, table, lens, refs = _shared_cache(1, 64, 16, 0, [100], 27)
    for size, scale in ((2.0 ** -133, 1e38), (2.0 ** -120, 1e35), (1e37, 1e-38)):
        q = (torch.randn((1, 2, 4, 64), generator=torch.Generator().manual_seed(28)) * size * 8).to(torch.bfloat16)
        c = _on_gpu(hf, pool, table, lens, refs, "bf16")
        want, tol = _want(q, pool, table, lens, "bf16", scale=scale)
        R.check_attention(R.to64(c.attend(q.cuda(), scale=scale)), want, tol)


# ------------------------------------------------------------------ writing and reading
class Cache(R.Cache):
    """The page tables as lists, with codes (values without their scale) and scales."""

    def __init__(self, layers, n_pages, hkv, page, dh, requests, columns):
        super().__init__(layers, n_pages, hkv, page, dh, requests, columns)
        self.scale = {x: np.ones((layers, n_pages, hkv)) for x in "kv"}

    def extend(self, rs, counts):
        before = [list(row) for row in self.rows]
        said = super().extend(rs, counts)
        for was, row in zip(before, self.rows):
            if was and row[len(was) - 1] != was[-1]:  # a copy
                for x in "kv":
                    self.scale[x][:, row[len(was) - 1]] = self.scale[x][:, was[-1]]
        return said

    def write8(self, rs, offsets, new, layer=0):
        for x, rows in new.items():
            codes = self.k if x == "k" else self.v
            for i, r in enumerate(rs):
                t, at = offsets[i], self.lens[r] - (offsets[i + 1] - offsets[i])
                while at < self.lens[r]:
                    p, r0 = self.rows[r][at // self.page], at % self.page
                    m = min(self.page - r0, self.lens[r] - at)
                    for l in range(rows.shape[0]):
                        for h in range(rows.shape[2]):
                            codes[layer + l, p, h], self.scale[x][layer + l, p, h] = C.write_block(
                                codes[layer + l, p, h], self.scale[x][layer + l, p, h], r0, rows[l, t:t + m, h])
                    t, at = t + m, at + m

    def tokens(self, x, r, first, count):
        codes = self.k if x == "k" else self.v
        at = [(self.rows[r][t // self.page], t % self.page) for t in range(first, first + count)]
        out = [codes[:, p, :, o] * self.scale[x][:, p][..., None] for p, o in at]
        return np.stack(out, 1) if out else np.zeros((codes.shape[0], 0, *codes.shape[2:3], codes.shape[4]))


def _same(got, want, what):
    assert np.array_equal(R.to64(got), want, equal_nan=True), what


def _check_cache(c, ref):
    """Every row that a request holds, its scales, and the tables."""
    assert c.lens.tolist() == ref.lens and c.refs.tolist() == ref.refs
    for r, row in enumerate(ref.rows):
        assert c.table[r, :len(row)].tolist() == row
        for j, p in enumerate(row):
            m = min(ref.page, ref.lens[r] - j * ref.page)
            for x, codes, scale in (("k", c.k, c.k_scale), ("v", c.v, c.v_scale)):
                _same(scale[:, p], ref.scale[x][:, p], f"scale of {x}")
                _same(codes[:, p, :, :m].float(), (ref.k if x == "k" else ref.v)[:, p, :, :m], f"codes of {x}")


@pytest.mark.parametrize("dtype,hkv,dh,page,layers", [
    ("bf16", 2, 128, 16, 3), ("bf16", 3, 64, 8, 1), ("bf16", 1, 80, 32, 2), ("f32", 2, 64, 16, 2), ("f32", 1, 256, 128, 1),
    ("bf16", 2, 256, 128, 1), ("f32", 5, 16, 64, 1), ("bf16", 9, 48, 8, 2),
])
def test_rounds(hf, dtype, hkv, dh, page, layers):
    """Requests that grow by prompts and by rounds of a few rows, fork, lose rows and leave; the pool is
    compacted: codes, scales and tables bit by bit, and what is read back."""
    rng = random.Random(page * dh)
    n, columns, n_pages = 5, 6, 40
    c = hf.Pages8.empty(layers, n_pages, hkv, page, dh, n, columns, dtype=DT[dtype])
    ref = Cache(layers, n_pages, hkv, page, dh, n, columns)
    for step in range(14):
        rs = [r for r in range(n) if rng.random() < 0.8]
        rng.shuffle(rs)
        counts = [rng.choice([0, 1, 2, 7, page, page + 3, 2 * page - 1]) for _ in rs]
        counts = [min(x, columns * page - ref.lens[r]) for r, x in zip(rs, counts)]
        if not rs:
            continue
        if ref.extend(rs, counts) == "":
            c.extend(C.ints(counts), C.ints(rs))
            ends = [sum(counts[:i]) + 3 for i in range(len(rs) + 1)]  # (rows that nobody owns around them)
            T = ends[-1] + 2
            size = 2.0 ** rng.randint(-4, 4)
            new = {x: _randn((layers, T, hkv + 1, dh), dtype, step * 2 + (x == "v"), size) for x in "kv"}
            ref.write8(rs, ends, {x: R.to64(y[:, :, :hkv]) for x, y in new.items()})
            gk, gv = (new[x].cuda()[:, :, :hkv] for x in "kv")
            c.write(gk, gv, C.ints(ends), C.ints(rs))
        _check_cache(c, ref)
        if step % 3 == 1:
            keep = [rng.randint(0, ref.lens[r]) for r in rs]
            ref.truncate(rs, keep)
            c.truncate(C.ints(keep), C.ints(rs))
        empty = [r for r in range(n) if ref.lens[r] == 0]
        full = [r for r in range(n) if ref.lens[r]]
        if step % 3 == 2 and empty and full:
            ref.fork([full[0]], [empty[0]])
            c.fork(C.ints([full[0]]), C.ints([empty[0]]))
        if step % 5 == 4:
            live = sum(x > 0 for x in ref.refs)
            high, hole = [i for i in range(live, n_pages) if ref.refs[i]], [i for i in range(live) if not ref.refs[i]]
            ref.compact()
            for x in "kv":
                ref.scale[x][:, hole] = ref.scale[x][:, high]
            c.compact()
        _check_cache(c, ref)
        # what is read back: any stretch, in any order, twice too
        req = [rng.randrange(n) for _ in range(7)]
        first = [rng.randint(0, ref.lens[r]) for r in req]
        count = [rng.randint(0, ref.lens[r] - f) for r, f in zip(req, first)]
        ends = [1 + sum(count[:i]) for i in range(8)]
        k, v = c.read(C.ints(first), C.ints(ends), C.ints(req), total=ends[-1] + 1)
        for x, got in (("k", k), ("v", v)):
            want = np.zeros(got.shape)
            for i, r in enumerate(req):
                want[:, ends[i]:ends[i + 1]] = ref.tokens(x, r, first[i], count[i])
            _same(got, R.to64(torch.tensor(want).to(DT[dtype])), "read")
        assert not c.check()


def test_fork_copies_the_scales(hf):
    """extend copies a shared, partly filled page: a write to the copy leaves the other's codes and scale."""
    ref = Cache(2, 9, 2, 16, 64, 2, 3)
    c = hf.Pages8.empty(2, 9, 2, 16, 64, 2, 3)
    for rs, size in (([0], 1.0), ([1], 300.0)):
        counts = [20 if rs == [0] else 2]
        ref.extend(rs, counts)
        c.extend(C.ints(counts), C.ints(rs))
        new = _randn((2, counts[0], 2, 64), "bf16", 3 + rs[0], size)
        ref.write8(rs, [0, counts[0]], {"k": R.to64(new), "v": R.to64(new)})
        c.write(new.cuda(), new.cuda(), C.ints([0, counts[0]]), C.ints(rs))
        if rs == [0]:
            ref.fork([0], [1])
            c.fork(C.ints([0]), C.ints([1]))
    _check_cache(c, ref)
    assert (ref.scale["k"][:, ref.rows[1][1]] > ref.scale["k"][:, ref.rows[0][1]]).all() and not c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_values_at_the_ends(hf, dtype):
    """Zeros, the smallest and largest values, ties, infinities and NaN."""
    page, dh = 8, 16
    rows = torch.zeros((8, dh), dtype=torch.float64)
    rows[0, :8] = torch.tensor([448.0, 1.0625, 1.1875, -1.0625, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, -0.0], dtype=torch.float64)
    rows[1, :3] = torch.tensor([449.0, 448.0, 464.0], dtype=torch.float64)     # a scale of 2
    rows[2, :4] = torch.tensor([float("inf"), float("nan"), -float("inf"), 7.0], dtype=torch.float64)
    rows[3, :2] = torch.tensor([3e38, 1.0], dtype=torch.float64)               # held to 448 2^63
    rows[4, :2] = torch.tensor([2.0 ** -100, 2.0 ** -73], dtype=torch.float64)  # below the least scale
    rows[5] = float("nan")
    x = rows.to(DT[dtype])
    want = R.to64(x)
    for i in range(8):  # each row alone in a page
        c = hf.Pages8.empty(1, 1, 1, page, dh, 1, 1, dtype=DT[dtype])
        c.k_scale.fill_(float("nan"))  # a page that nobody wrote
        c.extend(C.ints([1]))
        r = x[i].view(1, 1, 1, dh).cuda()
        c.write(r, r, C.ints([0, 1]))
        codes, s = C.write_block(np.zeros((page, dh)), 1.0, 0, want[i:i + 1])
        _same(c.k[0, 0, 0, :1].float(), codes[:1], f"row {i}")
        assert float(c.k_scale[0, 0, 0]) == s == float(c.v_scale[0, 0, 0])
        k, _ = c.read(C.ints([0]), C.ints([0, 1]), total=1)
        _same(k.view(1, dh), R.to64(torch.tensor(codes[:1] * s).to(DT[dtype])), f"row {i} read")
        assert not c.check()
    # negative zero keeps its sign
    c = hf.Pages8.empty(1, 1, 1, page, dh, 1, 1, dtype=DT[dtype])
    c.extend(C.ints([1]))
    c.write(x[0].view(1, 1, 1, dh).cuda(), x[0].view(1, 1, 1, dh).cuda(), C.ints([0, 1]))
    assert int(c.k.view(torch.uint8)[0, 0, 0, 0, 7]) == 0x80


def test_reading_at_the_ends_of_the_scales(hf):
    """Every code at the least, a middle and the largest scale, as fp32 and as bf16 rows."""
    codes = torch.arange(256, dtype=torch.uint8).view(1, 1, 1, 16, 16)
    for dtype in (torch.float32, torch.bfloat16):
        for e in (-64, 0, 7, 8, 63):
            k = codes.cuda().view(torch.float8_e4m3fn)
            s = torch.full((1, 1, 1), 2.0 ** e, device="cuda")
            c = hf.Pages8(k, k.clone(), s, s.clone(), C.ints([[0]]), C.ints([16]), C.ints([1]), dtype=dtype)
            got, again = c.read(C.ints([0]), C.ints([0, 16]), total=16)
            _same(got.view(16, 16), R.to64(codes.view(torch.float8_e4m3fn).float().view(16, 16)) * 2.0 ** e, f"2^{e}")
            assert torch.equal(got.nan_to_num(0.5), again.nan_to_num(0.5)) and not c.check()


def test_writes_and_reads_replayed(hf):
    """A captured round (extend, write, read back) replayed: it reads the lists and rows of its own time."""
    page, hkv, dh = 8, 2, 64
    c = hf.Pages8.empty(2, 30, hkv, page, dh, 3, 8)
    ref = Cache(2, 30, hkv, page, dh, 3, 8)
    counts, ends = C.ints([3, 3, 3]), C.ints([0, 3, 6, 9])
    x = torch.zeros((2, 9, hkv, dh), dtype=torch.bfloat16, device="cuda")
    first, k, v = C.ints([0, 0, 0]), torch.zeros_like(x), torch.zeros_like(x)
    c.write(x, x, C.ints([0]))  # (nothing; the calls have been made once before the capture)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.extend(counts)
        c.write(x, x, ends)
        c.read(first, ends, k=k, v=v)
    for step in range(6):
        x.copy_(_randn(x.shape, "bf16", 30 + step, 2.0 ** (step % 3)))
        first.copy_(C.ints(ref.lens))
        graph.replay()
        torch.cuda.synchronize()
        ref.extend([0, 1, 2], [3, 3, 3])
        ref.write8([0, 1, 2], [0, 3, 6, 9], {"k": R.to64(x), "v": R.to64(x)})
        _check_cache(c, ref)
        want = np.concatenate([ref.tokens("k", r, 3 * step, 3) for r in range(3)], 1)
        _same(k, R.to64(torch.tensor(want).to(torch.bfloat16)), "read")
        assert torch.equal(k, v) and not c.check()


def test_bad_entries_of_write_and_read(hf):
    c = hf.Pages8.empty(1, 12, 2, 8, 64, 4, 3)
    c.extend(C.ints([10, 5, 0, 24]))
    x = _randn((1, 39, 2, 64), "bf16", 1).cuda()
    ends = C.ints([0, 10, 15, 15, 39])
    c.write(x, x, ends)
    assert not c.check()
    state = lambda: [t.clone() for t in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)]
    before = state()
    y = _randn((1, 39, 2, 64), "bf16", 2).cuda()

    def unchanged():
        assert c.check() == hf.CallStatus.BAD
        assert all(torch.equal(a, b) for a, b in zip(before, state()))

    c.write(y, y, C.ints([0, 10, 9, 20]), C.ints([0, 1, 3]))       # bounds that decrease
    unchanged()
    c.write(y, y, C.ints([0, 11]), C.ints([0]))                    # more rows than tokens
    unchanged()
    c.write(y, y, C.ints([0, 2, 4]), C.ints([1, 1]))               # twice
    unchanged()
    c.write(y, y, C.ints([-3, 2, 40]), C.ints([0, 3]))             # bounds out of range
    unchanged()
    c.write(y, y, C.ints([0, 2, 4]), C.ints([-1, 4]))              # no such request
    unchanged()
    t = c.table.clone()
    c.table[0, 1] = 12                                             # no such page
    c.write(y, y, C.ints([0, 2]), C.ints([0]))
    unchanged()
    c.table.copy_(t)
    # a good entry beside a bad one
    c.write(y, y, C.ints([0, 99, 99]), C.ints([0, 1]))
    assert c.check() == hf.CallStatus.BAD
    for first, ends, req in (([3], [0, 8], [0]), ([-1], [0, 1], [0]), ([0], [0, 1], [4]), ([0, 0], [5, 3, 9], [0, 1]),
                             ([0], [-2, 1], [0]), ([0], [0, 41], [3])):
        k = torch.full((1, 40, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        v = k.clone()
        c.read(C.ints(first), C.ints(ends), C.ints(req), k=k, v=v)
        assert c.check() == hf.CallStatus.BAD and (k == 5).all() and (v == 5).all()
    # a good entry beside a bad one, and by layer
    k = torch.full((40, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    c.read(C.ints([0, 2]), C.ints([0, 30, 33]), C.ints([1, 3]), layer=0, k=k, v=v)
    assert c.check() == hf.CallStatus.BAD and (k[:30] == 5).all() and (k[33:] == 5).all()
    k2, _ = c.read(C.ints([2]), C.ints([0, 3]), C.ints([3]), total=3)
    assert torch.equal(k[30:33], k2[0])


def test_as_many_requests_as_there_can_be(hf):
    """A cache of 4096 requests written in one call, and read back by more entries than requests."""
    n, page, dh = 4096, 8, 16
    c = hf.Pages8.empty(1, 5000, 1, page, dh, n, 2, dtype=torch.float32)
    rng = random.Random(3)
    counts = [rng.choice([0, 1, 3, 9]) if i % 4 else 2 for i in range(n)]
    ref = Cache(1, 5000, 1, page, dh, n, 2)
    assert ref.extend(list(range(n)), counts) == ""
    c.extend(C.ints(counts))
    ends = np.concatenate([[0], np.cumsum(counts)]).tolist()
    x = _randn((1, ends[-1], 1, dh), "f32", 31, 3.0)
    ref.write8(list(range(n)), ends, {"k": R.to64(x), "v": R.to64(x)})
    c.write(x.cuda(), x.cuda(), C.ints(ends))
    req = [rng.randrange(n) for _ in range(6000)]
    first = [rng.randint(0, ref.lens[r]) for r in req]
    count = [ref.lens[r] - f for r, f in zip(req, first)]
    at = np.concatenate([[0], np.cumsum(count)]).tolist()
    k, v = c.read(C.ints(first), C.ints(at), C.ints(req), total=at[-1])
    want = np.concatenate([ref.tokens("k", r, f, m) for r, f, m in zip(req, first, count)], 1)
    _same(k, R.to64(torch.tensor(want).float()), "read")
    assert torch.equal(k, v) and not c.check()


def test_write_and_read_beyond_32_bits(hf):
    """A pool and rows past 2^32 elements: 2 layers of 2.2 GB."""
    L, pages, hkv, page, dh = 2, 17000, 8, 128, 128
    c = hf.Pages8.empty(L, pages, hkv, page, dh, 2, 20000 // 4 * 4)
    c.refs[:16990] = 1
    c.extend(C.ints([200, 130]))
    assert c.table[0, :2].tolist() == [16990, 16991]
    x = _randn((2, 330, hkv, dh), "bf16", 3).cuda()
    c.write(x, x, C.ints([0, 200, 330]))
    k, v = c.read(C.ints([0, 0]), C.ints([0, 200, 330]), total=330)
    top = 2.0 ** -4 * 1.0001
    assert ((k.float() - x.float()).abs() <= top * x.float().abs() + 2.0 ** -10 * 2.0 ** -6).all() and torch.equal(k, v)
    q = _randn((2, 1, hkv, dh), "bf16", 4)
    o = R.to64(c.attend(q.cuda(), layer=1))
    for i, (a, b) in enumerate(((0, 200), (200, 330))):
        kk = R.to64(k[1, a:b])
        for h in range(hkv):
            vs = np.repeat(R.to64(c.v_scale[1, c.table[i, :2].long(), h]), page)[:b - a]
            want, tol = C.attention(R.to64(q[i, 0, h]), kk[:, h], kk[:, h], vs, dh ** -0.5, True, True)
            R.check_attention(o[i, 0, h], want, tol)
    assert not c.check()


def test_a_layer_as_a_loop_runs_it(hf):
    """Rotary positions, the rows into the cache, attention over it: a prompt, then rounds of verified rows
    of which some are taken back. Next to plain forms of each step on the same inputs."""
    hq, hkv, dh, page = 8, 2, 128, 16
    c = hf.Pages8.empty(1, 24, hkv, page, dh, 2, 8)
    ref = Cache(1, 24, hkv, page, dh, 2, 8)
    rot = hf.Rotary(dh, scaling="yarn", factor=4.0, original=64)
    w, f = C.frequencies(dh, 1e6, "yarn", factor=4.0, original=64)
    stream = torch.cuda.Stream()
    keep = None
    for step, counts in enumerate(([40, 3], [4, 4], [4, 4], [1, 4])):
        if keep:
            ref.truncate([0, 1], keep)
            c.truncate(C.ints(keep), stream=stream)
        at = list(ref.lens)
        pos = [a + i for a, m in zip(at, counts) for i in range(m)]
        T, ends = sum(counts), [0, counts[0], sum(counts)]
        qkv = _randn((T, hq + 2 * hkv, dh), "bf16", 50 + step)
        g = qkv.cuda()
        torch.cuda.synchronize()
        q, k = rot(g[:, :hq], g[:, hq:hq + hkv], C.ints(pos), stream=stream)
        torch.cuda.synchronize()
        for got, src in ((q, qkv[:, :hq]), (k, qkv[:, hq:hq + hkv])):
            want, tol = C.rotary(src, pos, w, f, False, True)
            R.check_attention(R.to64(got), want, tol, "rotary")
        ref.extend([0, 1], counts)
        c.extend(C.ints(counts), stream=stream)
        v = g[:, hq + hkv:].contiguous()
        torch.cuda.synchronize()
        c.write(k, v, C.ints(ends), layer=0, stream=stream)
        torch.cuda.synchronize()
        ref.write8([0, 1], ends, {"k": R.to64(k)[None], "v": R.to64(v)[None]})
        _check_cache(c, ref)
        if step:
            rows = min(counts)
            mine = torch.stack([q[ends[i + 1] - rows:ends[i + 1]] for i in range(2)])
            torch.cuda.synchronize()
            o = c.attend(mine, stream=stream)
            torch.cuda.synchronize()
            pk, pv = ref.k * ref.scale["k"][..., None, None], ref.v * ref.scale["v"][..., None, None]
            want, tol = C.pages(mine, pk[0], pv[0], ref.scale["v"][0], ref.rows, ref.lens, dh ** -0.5, True, True)
            R.check_attention(R.to64(o), want, tol, "attend")
        keep = [ref.lens[0] - 1, ref.lens[1] - 2] if step else None
    assert not c.check()
