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
