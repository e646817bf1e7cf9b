"""Calls on the 8-bit cache that test_gpu_cache8.py does not make."""
import random

import numpy as np
import pytest
import torch

import _cache8_ref as C
import _target_ref as R
from test_gpu_cache8 import _on_gpu, _randn, _shared_cache, _want, hf  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hkv,dh,page,shared", [(5, 128, 64, 32768), (3, 64, 128, 65536), (5, 64, 16, 16384)])
def test_a_long_prefix_of_an_odd_number_of_heads(hf, hkv, dh, page, shared):
    """A CTA that goes from an item of the last head, which has no neighbour and leaves one row tile idle, to items of two
    heads: the idle one must not take the next item's scales before they are there."""
    pool, table, lens, refs = _shared_cache(hkv, dh, page, shared, [700, 3, 1000, 260], 31)
    c = _on_gpu(hf, pool, table, lens, refs, "bf16")
    q = _randn((4, 2, 3 * hkv, dh), "bf16", 32)
    want, tol = _want(q, pool, table, lens, "bf16")
    first = c.attend(q.cuda(), shared=shared)
    R.check_attention(R.to64(first), want, tol)
    for _ in range(20):
        assert torch.equal(c.attend(q.cuda(), shared=shared), first)
    assert not c.check()


@pytest.mark.parametrize("n,rows", [(16, 8), (4, 2)])
def test_a_page_of_the_prefix_out_of_range_reads_as_zeros(hf, n, rows):
    """Through bf16 rows (16 x 8 rows of 8 heads) as through codes: what the workspace held before does not come in."""
    shared, page = 2304, 32
    pool, table, lens, refs = _shared_cache(1, 128, page, shared, [5, 200] + [3] * (n - 2), 41)
    t = [list(r) for r in table]
    for r in t:
        r[3], r[40] = len(refs), -5
    c = _on_gpu(hf, pool, t, lens, refs, "bf16")
    q = _randn((n, rows, 8, 128), "bf16", 42)
    ws = c.attend_workspace(q, shared)
    ws.fill_(255)
    out = c.attend(q.cuda(), shared=shared, workspace=ws)
    assert c.check() == hf.CallStatus.BAD
    for x in pool[:2]:
        x.view(torch.uint8)[:, [table[0][3], table[0][40]]] = 0
    want, tol = _want(q, pool, table, lens, "bf16")
    R.check_attention(R.to64(out), want, tol)


@pytest.mark.parametrize("dtype,dh,n,rows,shared", [("bf16", 128, 3, 2, 0), ("bf16", 128, 16, 8, 2304), ("bf16", 80, 3, 2, 32),
                                                    ("f32", 64, 3, 2, 0)])
def test_pages_without_a_scale_count_as_the_least(hf, dtype, dh, n, rows, shared):
    """Scales that no write has set, whatever they are, by every kernel alike: reading back, codes, bf16 rows, CUDA cores."""
    pool, table, lens, refs = _shared_cache(1, dh, 32, shared, [100] * n, 43)
    for t in pool[2:]:
        for p, x in ((table[0][0], float("nan")), (table[0][1], 0.0), (table[0][2], -1.0), (table[1][-2], float("inf")), (table[1][-3], 2.0 ** 64)):
            t[:, p] = x
    c = _on_gpu(hf, pool, table, lens, refs, dtype)
    q = _randn((n, rows, 8, dh), dtype, 44)
    out = c.attend(q.cuda(), shared=shared)
    k, v = c.read(C.ints([0, 3]), C.ints([0, 90, 180]), C.ints([0, 1]), total=180)
    for t in pool[2:]:
        for p in (*table[0][:3], *table[1][-3:-1]):
            t[:, p] = 2.0 ** -64
    want, tol = _want(q, pool, table, lens, dtype)
    R.check_attention(R.to64(out), want, tol)
    for got, codes, scale in ((k, pool[0], pool[2]), (v, pool[1], pool[3])):
        x = torch.from_numpy(C.values(codes, scale))[0, :, 0].to(got.dtype)  # [pages, page, dh]
        rows0, rows1 = x[table[0]].reshape(-1, dh)[:90], x[table[1]].reshape(-1, dh)[3:93]
        assert torch.equal(got[0, :, 0].cpu(), torch.cat((rows0, rows1)))
    assert not c.check()


# ------------------------------------------------------------------ a long prefix of many rows, through bf16 rows
def _wide(c, q, shared):
    """A workspace whose size says that the prefix goes through bf16 rows."""
    ws = c.attend_workspace(q, shared)
    assert ws.numel() > 4 * shared * c.k.shape[2] * c.k.shape[4]
    ws.fill_(255)
    return ws


@pytest.mark.parametrize("hkv,dh,page,shared,odd_page", [(2, 128, 32, 8192, False), (3, 64, 64, 8192, True), (8, 128, 16, 2048, True)])
def test_wide_prefix(hf, hkv, dh, page, shared, odd_page):
    """Entries without tokens of their own (their first rows see part of the prefix), an empty one, one that names
    no request, NaN codes at the prefix's end, an empty first entry."""
    pool, table, lens, refs = _shared_cache(hkv, dh, page, shared, [5, 0, 200, None, 1, 40] + [3] * 10, 51)
    if odd_page:
        last = table[0][shared // page - 1]
        pool[0].view(torch.uint8)[0, last, 0, page - 2] = 0x7f
        pool[1].view(torch.uint8)[0, last, 1, page - 3, 5] = 0xff
    c = _on_gpu(hf, pool, table, lens, refs, "bf16")
    q = _randn((16, 8, 8 * hkv, dh), "bf16", 52)
    ws = _wide(c, q, shared)
    want, tol = _want(q, pool, table, lens, "bf16")
    R.check_attention(R.to64(c.attend(q.cuda(), shared=shared, workspace=ws)), want, tol)
    assert not c.check()
    if odd_page:
        assert np.isnan(want).any() and np.isfinite(want[1, 0]).all()
    o = R.to64(c.attend(q.cuda(), C.ints([0, 1, 2, 3, -7, 5] + list(range(6, 16))), shared=shared, workspace=ws))
    assert (o[4] == 0).all() and c.check() == hf.CallStatus.BAD
    o[4] = want[4]
    R.check_attention(o, want, tol)
    c = _on_gpu(hf, pool, table, [0] + lens[1:], refs, "bf16")
    assert (c.attend(q.cuda(), shared=shared, workspace=ws) == 0).all() and c.check() == hf.CallStatus.BAD


def test_wide_prefix_with_pages_out_of_range_and_without_a_scale(hf):
    shared, page, n = 8192, 32, 16
    pool, table, lens, refs = _shared_cache(2, 128, page, shared, [5, 200] + [3] * (n - 2), 53)
    for x in pool[2:]:
        x[:, table[0][7]], x[:, table[0][8]] = float("nan"), 2.0 ** 64
    t = [list(r) for r in table]
    for r in t:
        r[3], r[40] = len(refs), -5
    c = _on_gpu(hf, pool, t, lens, refs, "bf16")
    q = _randn((n, 8, 16, 128), "bf16", 54)
    out = c.attend(q.cuda(), shared=shared, workspace=_wide(c, q, shared))
    assert c.check() == hf.CallStatus.BAD
    for x in pool[:2]:
        x.view(torch.uint8)[:, [table[0][3], table[0][40]]] = 0
    for x in pool[2:]:
        x[:, table[0][7:9]] = 2.0 ** -64
    want, tol = _want(q, pool, table, lens, "bf16")
    R.check_attention(R.to64(out), want, tol)


def test_wide_prefix_of_many_entries(hf):
    """More entries than a CTA plans for by itself."""
    pool, table, lens, refs = _shared_cache(2, 64, 128, 8192, [3, 17, 90, None, 64, 1], 55)
    c = _on_gpu(hf, pool, table, lens, refs, "bf16")
    rng = random.Random(6)
    req = [0] + [rng.randrange(6) for _ in range(499)]
    q = _randn((500, 2, 4, 64), "bf16", 56)
    want, tol = _want(q, pool, table, lens, "bf16", req=req)
    R.check_attention(R.to64(c.attend(q.cuda(), C.ints(req), shared=8192, workspace=_wide(c, q, 8192))), want, tol)
    assert not c.check()


def test_wide_prefix_replayed_and_two_at_once(hf):
    """The launches run into each other (the entries' own keys beside the prefix): with rows that change just before,
    in a graph, and on two streams at once."""
    shared = 16384
    pool, table, lens, refs = _shared_cache(4, 128, 32, shared, [700, 3, 90, 1] * 12, 57)
    c = _on_gpu(hf, pool, table, lens, refs, "bf16")
    qs = [_randn((48, 2, 16, 128), "bf16", 58 + i).cuda() for i in range(3)]
    ws = _wide(c, qs[0], shared)
    firsts = []
    for q in qs:
        first = c.attend(q, shared=shared)
        torch.cuda.synchronize()
        firsts.append(first.clone())
    few = [0, 1, 2, 45]
    want, tol = _want(qs[0][few], pool, table, lens, "bf16", req=few)
    R.check_attention(R.to64(firsts[0][few]), want, tol)
    q, out = torch.empty_like(qs[0]), torch.empty_like(qs[0])
    for i in (0, 1, 2, 1, 0, 2):  # no wait between the calls; the rows are written by the kernel just before
        q.copy_(qs[i])
        c.attend(q, shared=shared, out=out, workspace=ws)
        got = out.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, firsts[i])
    graph = torch.cuda.CUDAGraph()
    kept = [torch.empty_like(out) for _ in range(3)]
    with torch.cuda.graph(graph):
        for i in range(3):
            q.copy_(qs[i])
            c.attend(q, shared=shared, out=out, workspace=ws)
            kept[i].copy_(out)
    for _ in range(3):
        for k in kept:
            k.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(k, f) for k, f in zip(kept, firsts))
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(i, c.attend(qs[i], shared=shared, stream=streams[i % 2])) for _ in range(6) for i in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, firsts[i]) for i, o in outs) and not c.check()


def test_wide_prefix_whose_waits_run_out(hf):
    from speculative_decoding_drafter_hf_gb300 import _binding as B
    pool, table, lens, refs = _shared_cache(2, 128, 64, 8192, [5] * 16, 61)
    c = _on_gpu(hf, pool, table, lens, refs, "bf16")
    q = _randn((16, 8, 16, 128), "bf16", 62)
    want, tol = _want(q, pool, table, lens, "bf16")
    ws = _wide(c, q, 8192)
    try:
        B.hf_debug_set_wait_limit(None, 0)
        c.attend(q.cuda(), shared=8192, workspace=ws)
        assert c.check() == hf.CallStatus.TIMEOUT
    finally:
        B.hf_debug_set_wait_limit(None, -1)
    R.check_attention(R.to64(c.attend(q.cuda(), shared=8192, workspace=ws)), want, tol)
    assert not c.check()
