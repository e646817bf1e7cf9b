"""What the 8-bit cache and the calls beside it must answer without a GPU."""
import ctypes
import re

import numpy as np
import pytest

from test_cache8_cpu import B, _cache  # noqa: F401
from test_target_edges_cpu import _code


def _plain_cache(B, **change):
    d = dict(k=16, v=16, table=16, lens=16, refs=16, work=16, status=16, dtype=1, n_layers=1, n_pages=20, n_kv_heads=2, page=16,
             head_dim=64, n_requests=4, table_ld=5)
    return B.HfPages(**{**d, **change})


@pytest.mark.parametrize("dtype,dh", [(0, 64), (0, 80), (1, 80), (1, 64)])
def test_workspaces_where_nothing_is_shared_or_all_is(B, dtype, dh):
    """No keys of a kind are no pieces, and no division by them."""
    p = ctypes.byref(_plain_cache(B, dtype=dtype, head_dim=dh))
    sizes = [B.hf_attention_pages_workspace(p, 4, 1, 4, shared) for shared in (0, 16, 80)]
    assert min(sizes) > 0
    p8 = ctypes.byref(_cache(B, rows=dtype, head_dim=dh))
    assert min(B.hf_attention_pages8_workspace(p8, 4, 1, 4, shared) for shared in (0, 16, 80)) > 0


@pytest.mark.parametrize("dtype", [0, 1])
def test_the_bf16_and_fp32_cache_take_as_many_entries_as_before(B, dtype):
    """An 8-bit cache counts more places for an entry; that must not narrow the other one."""
    def workspace(heads):
        p = _plain_cache(B, dtype=dtype, n_kv_heads=heads, table_ld=1)
        return B.hf_attention_pages_workspace(ctypes.byref(p), 1 << 20, 1, heads, 0)

    # (1 + 1) 2^20 (heads / 128 + heads) <= 2^30 - 1
    assert workspace(300) > 0 and workspace(508) > 0 and workspace(509) == 0


def test_what_runs_beside_a_prefix_comes_behind_its_wait():
    """The entries' own keys are read before that launch's wait: the launch directly before it triggers behind its own."""
    prefix, own, calls = _code("attn_tc.cu"), _code("attn_tc8.cu"), _code("attn_rows.cu")
    kernel = prefix[prefix.index("tc_kernel("):]
    assert re.search(r"const bool beside = MODE == PAGED && a\.dense;\s*if \(!beside\) pdl_trigger\(\);", kernel)
    assert re.search(r"pdl_wait\(\);\s*if \(beside\) pdl_trigger\(\);", kernel)
    assert "if (c.busy == 0) pdl_wait();" in own and own.rindex("if (c.busy) pdl_wait();") > own.rindex("tmem_dealloc(tmem, 512)")
    assert "const int busy = a.n <= kSmall &&" in calls and "if (!c.small) e = launch_attn_plan(" in own
    assert re.search(r"launch_attn_tc_pages\(b, w\.pre_items, st\);\s*if \(e == cudaSuccess\) e = launch_attn_tc8_pages\(a, 0, busy", calls)


def test_codes_of_weights_add_up():
    """Every 16-bit float from 0 to 2^15 as three e5m2 codes, w = a + b / 8 + c / 64 to 2^-9 of it, or 2^-23: the steps of
    split_weights (attn_tc8.cu)."""
    bits = np.arange(0, 0x7801, dtype=np.uint16)
    w, eight = bits.view(np.float16), np.float16(8)

    def upper(x):
        return (x.view(np.uint16) & np.uint16(0xff00)).view(np.float16)

    a = upper(w)
    rest = (w - a) * eight
    b = upper(rest)
    c = upper((((rest - b) * eight).view(np.uint16) + np.uint16(0x80)).view(np.float16))
    total = a.astype(np.float64) + b.astype(np.float64) / 8 + c.astype(np.float64) / 64
    assert np.isfinite(total).all()
    assert (np.abs(total - w.astype(np.float64)) <= np.maximum(2.0 ** -9 * w.astype(np.float64), 2.0 ** -23)).all()
