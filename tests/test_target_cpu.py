"""Refusals of the target-side calls: every check below answers on the host,
before any CUDA call, so the pointers are never dereferenced."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def B():
    from speculative_decoding_drafter_hf_gb300 import build
    build.build()
    from speculative_decoding_drafter_hf_gb300 import _binding
    return _binding


def _refused(B, status, msg):
    assert status == B.Status.EINVAL
    assert msg in B.hf_last_error(None).decode()


PROMPT = dict(dtype=1, n_seq=2, total=10, hq=4, hkv=2, dh=64, q=16, q_ld=256, k=16, k_ld=128, v=16, v_ld=128, off=16,
              scale=0.0, out=16, out_ld=256, status=None, stream=None)


@pytest.mark.parametrize("change,msg", [
    (dict(dtype=2), "dtype"), (dict(n_seq=-1), "n_seq"), (dict(total=-1), "total"), (dict(hkv=3), "divide"),
    (dict(hkv=0), "n_kv_heads"), (dict(hq=260, hkv=2, q_ld=65 * 256, out_ld=65 * 256), "<= 64"),
    (dict(dh=12), "multiple of 8"), (dict(dh=264), "<= 256"), (dict(scale=-1.0), "scale"),
    (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"), (dict(q=None), "NULL"),
    (dict(off=None), "NULL"), (dict(out=None), "NULL"), (dict(q=8), "16-byte"), (dict(out=24), "16-byte"),
    (dict(q_ld=252), "stride"), (dict(k_ld=120), "stride"), (dict(v_ld=132), "16-byte"), (dict(out_ld=260), "16-byte"),
    (dict(off=18), "4-byte"), (dict(status=2), "4-byte"),
    (dict(total=1 << 30), "too large"), (dict(n_seq=1 << 24, hq=256, hkv=256, q_ld=1 << 14, k_ld=1 << 14, v_ld=1 << 14,
                                              out_ld=1 << 14), "too large"),
    (dict(scale=2e38), "scale"), (dict(q_ld=1 << 37), "stride"),
])
def test_prompt_refusals(B, change, msg):
    _refused(B, B.hf_attention_prompt(*{**PROMPT, **change}.values()), msg)


@pytest.mark.parametrize("change", [dict(n_seq=0, off=None), dict(total=0, q=None, k=None, v=None, out=None)])
def test_prompt_without_rows_needs_no_buffers(B, change):
    assert B.hf_attention_prompt(*{**PROMPT, **change}.values()) == B.Status.OK


CACHE = dict(k=16, v=16, table=16, lens=16, refs=16, work=16, status=16, dtype=1, n_layers=2, n_pages=20, n_kv_heads=2,
             page=16, head_dim=64, n_requests=4, table_ld=5)


def _cache(B, **change):
    return B.HfPages(**{**CACHE, **change})


@pytest.mark.parametrize("change,msg", [
    (dict(dtype=3), "dtype"), (dict(n_layers=0), "positive"), (dict(n_pages=0), "positive"),
    (dict(n_kv_heads=0), "positive"), (dict(table_ld=0), "positive"), (dict(page=12), "page"), (dict(page=4), "page"),
    (dict(page=256), "page"), (dict(head_dim=60), "head_dim"), (dict(head_dim=320), "head_dim"),
    (dict(n_kv_heads=2000), "1024"), (dict(n_requests=0), "4096"), (dict(n_requests=4097), "4096"),
    (dict(n_pages=1 << 27), "2^31"), (dict(table_ld=1 << 28), "2^31"), (dict(k=None), "NULL"), (dict(refs=None), "NULL"),
    (dict(work=None), "NULL"), (dict(k=24), "16-byte"), (dict(table=18), "4-byte"), (dict(status=17), "4-byte"),
])
def test_every_cache_call_refuses_a_bad_descriptor(B, change, msg):
    p = ctypes.byref(_cache(B, **change))
    _refused(B, B.hf_pages_extend(p, 16, 16, 2, None), msg)
    _refused(B, B.hf_pages_truncate(p, 16, 16, 2, None), msg)
    _refused(B, B.hf_pages_fork(p, 16, 16, 2, None), msg)
    _refused(B, B.hf_pages_compact(p, None, None), msg)
    _refused(B, B.hf_pages_write(p, 0, 1, 16, 16, 128, 0, 16, 16, 2, 8, None), msg)
    _refused(B, B.hf_attention_pages(p, 0, 2, 1, 4, 16, 256, 16, 0, 0.0, 16, 256, 16, 1 << 30, None), msg)
    if "NULL" not in msg and "byte" not in msg:  # sizes alone
        assert B.hf_pages_work_ints(p) == 0
        assert B.hf_attention_pages_workspace(p, 2, 1, 4, 0) == 0


def test_cache_lists_and_work(B):
    c = _cache(B)
    p = ctypes.byref(c)
    assert B.hf_pages_work_ints(p) == 16 + 2 * 20
    assert B.hf_pages_work_ints(ctypes.byref(_cache(B, n_requests=500))) == 16 + 2 * 500
    assert B.hf_pages_work_ints(None) == 0
    for n in (-1, 5):
        _refused(B, B.hf_pages_extend(p, 16, 16, n, None), "n_requests")
        _refused(B, B.hf_pages_truncate(p, 16, 16, n, None), "n_requests")
        _refused(B, B.hf_pages_fork(p, 16, 16, n, None), "n_requests")
        _refused(B, B.hf_pages_write(p, 0, 1, 16, 16, 128, 0, 16, 16, n, 8, None), "n_requests")
    _refused(B, B.hf_pages_extend(p, None, None, 1, None), "NULL")
    _refused(B, B.hf_pages_truncate(p, None, None, 1, None), "NULL")
    _refused(B, B.hf_pages_fork(p, None, 16, 1, None), "NULL")
    _refused(B, B.hf_pages_fork(p, 16, 18, 1, None), "4-byte")
    _refused(B, B.hf_pages_compact(p, 2, None), "4-byte")
    assert B.hf_pages_extend(p, None, None, 0, None) == B.Status.OK
    assert B.hf_pages_truncate(p, None, None, 0, None) == B.Status.OK
    assert B.hf_pages_fork(p, None, None, 0, None) == B.Status.OK


WRITE = dict(layer=0, layers=2, k=16, v=16, ld=128, step=1280, req=16, off=16, n=2, total=10)


@pytest.mark.parametrize("change,msg", [
    (dict(layer=-1), "layer"), (dict(layer=1), "layer"), (dict(layers=3), "layer"), (dict(layers=-1), "layer"),
    (dict(total=-1), "total"), (dict(k=None), "NULL"), (dict(off=None), "NULL"), (dict(ld=120), "ld"),
    (dict(step=-8), "layer_stride"), (dict(ld=132), "16 bytes"), (dict(step=1284), "16 bytes"), (dict(v=24), "16-byte"),
    (dict(off=18), "4-byte"), (dict(req=18), "4-byte"),
])
def test_write_refusals(B, change, msg):
    p = ctypes.byref(_cache(B))
    _refused(B, B.hf_pages_write(p, *{**WRITE, **change}.values(), None), msg)


ATTEND = dict(layer=0, n=2, rows=8, hq=4, q=16, q_ld=256, req=16, shared=32, scale=0.0, out=16, out_ld=256, ws=16,
              bytes=1 << 30)


@pytest.mark.parametrize("change,msg", [
    (dict(layer=2), "layer"), (dict(layer=-1), "layer"), (dict(n=-1), "n must"), (dict(rows=0), "rows"),
    (dict(rows=65), "rows"), (dict(hq=3), "divide"), (dict(shared=8), "multiple of page"),
    (dict(shared=-16), "multiple of page"), (dict(shared=96), "table_ld"), (dict(scale=-2.0), "scale"),
    (dict(req=None, n=5), "without a list"), (dict(q=None), "NULL"), (dict(out=None), "NULL"), (dict(ws=None), "NULL"),
    (dict(q_ld=248), "stride"), (dict(q=8), "16-byte"), (dict(out_ld=260), "16-byte"), (dict(req=18), "4-byte"),
    (dict(ws=24), "workspace"), (dict(bytes=0), "workspace"), (dict(n=1 << 20, rows=64, hq=128), "too large"),
])
def test_attend_refusals(B, change, msg):
    p = ctypes.byref(_cache(B))
    _refused(B, B.hf_attention_pages(p, *{**ATTEND, **change}.values(), None), msg)


def test_attend_workspace(B):
    p = ctypes.byref(_cache(B))
    assert B.hf_attention_pages_workspace(p, 2, 8, 4, 32) > 0
    assert B.hf_attention_pages_workspace(p, 2, 8, 3, 32) == 0
    assert B.hf_attention_pages(p, *{**ATTEND, "n": 0, "q": None, "out": None, "ws": None}.values(), None) == B.Status.OK


VERIFY = dict(t_dtype=1, x=16, x_ld=1000, d_dtype=0, y=16, y_ld=1000, tok=16, nd=None, u=16, noise=16, e_ld=1000,
              temp=None, batch=2, block=7, vocab=1000, n_acc=16, out=16, ws=16, bytes=1 << 30, status=None)


@pytest.mark.parametrize("change,msg", [
    (dict(t_dtype=2), "target_dtype"), (dict(d_dtype=-1), "draft_dtype"), (dict(batch=-1), "batch"),
    (dict(block=0), "block"), (dict(block=17), "block"), (dict(vocab=0), "vocab"), (dict(x_ld=999), "target_ld"),
    (dict(y_ld=999), "draft_ld"), (dict(e_ld=999), "noise_ld"), (dict(x=None), "NULL"), (dict(tok=None), "NULL"),
    (dict(u=None), "NULL"), (dict(noise=None), "NULL"), (dict(n_acc=None), "NULL"), (dict(out=None), "NULL"),
    (dict(ws=None), "NULL"), (dict(x=17), "aligned"), (dict(y=18), "aligned"), (dict(temp=2), "aligned"),
    (dict(nd=2), "aligned"), (dict(status=6), "aligned"), (dict(ws=20), "16-byte"), (dict(bytes=16), "workspace"),
    (dict(batch=1 << 20, vocab=1 << 28, x_ld=1 << 28, y_ld=1 << 28, e_ld=1 << 28), "too large"),
])
def test_verify_refusals(B, change, msg):
    _refused(B, B.hf_verify_tokens(*{**VERIFY, **change}.values(), None), msg)


def test_verify_workspace_and_empty_batch(B):
    assert B.hf_verify_workspace(2, 7, 1000) > 0
    assert B.hf_verify_workspace(2, 0, 1000) == 0
    a = {**VERIFY, "batch": 0, "x": None, "tok": None, "u": None, "noise": None, "n_acc": None, "out": None, "ws": None}
    assert B.hf_verify_tokens(*a.values(), None) == B.Status.OK


def test_descriptor_layout(B):
    assert ctypes.sizeof(B.HfPages) == 7 * 8 + 8 * 4
    assert B.HfPages.dtype.offset == 56 and B.HfPages.table_ld.offset == 84


def test_python_calls_refuse_cpu_tensors(B):
    import torch

    import speculative_decoding_drafter_hf_gb300 as hf
    q = torch.zeros(4, 2, 64)
    with pytest.raises(TypeError):
        hf.attention_prompt(q, q, q, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        hf.verify_tokens(torch.zeros(1, 8, 10), torch.zeros(1, 7, dtype=torch.int32), torch.zeros(1, 7), torch.zeros(1, 10))
    with pytest.raises(TypeError):
        k = torch.zeros(1, 4, 2, 16, 64)
        hf.Pages(k, k, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))
