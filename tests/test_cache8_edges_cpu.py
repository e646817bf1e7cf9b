"""What the 8-bit cache and the calls beside it must answer without a GPU."""
import ctypes

import pytest

from test_cache8_cpu import B, _cache  # noqa: F401


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
