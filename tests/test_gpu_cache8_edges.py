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
