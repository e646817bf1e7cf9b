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
