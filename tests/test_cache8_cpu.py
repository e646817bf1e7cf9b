"""Refusals of the 8-bit cache's and the rotary calls: every check below answers on the host, before
any CUDA call, so the pointers are never dereferenced. And the rotary table, which the host makes."""
import ctypes

import numpy as np
import pytest

import _cache8_ref as C


@pytest.fixture(scope="module")
def B():
    from speculative_decoding_drafter_hf_gb300 import build
    build.build()
    from speculative_decoding_drafter_hf_gb300 import _binding
    return _binding


def _refused(B, status, msg):
    assert status == B.Status.EINVAL
    assert msg in B.hf_last_error(None).decode()


CACHE = dict(k=16, v=16, table=16, lens=16, refs=16, work=16, status=16, dtype=2, n_layers=2, n_pages=20, n_kv_heads=2,
             page=16, head_dim=64, n_requests=4, table_ld=5)
OUTER = dict(k_scale=16, v_scale=16, rows=1, reserved=0)


def _cache(B, **change):
    inner = {k: change.get(k, v) for k, v in CACHE.items()}
    outer = {k: change.get(k, v) for k, v in OUTER.items()}
    return B.HfPages8(pages=B.HfPages(**inner), **outer)


@pytest.mark.parametrize("change,msg", [
    (dict(dtype=1), "HF_E4M3"), (dict(dtype=0), "HF_E4M3"), (dict(n_layers=0), "positive"), (dict(page=12), "page"),
    (dict(head_dim=24), "multiple of 16"), (dict(head_dim=272), "<= 256"), (dict(n_requests=4097), "4096"),
    (dict(rows=2), "rows"), (dict(rows=-1), "rows"), (dict(reserved=1), "reserved"), (dict(k=None), "NULL"),
    (dict(k_scale=None), "NULL"), (dict(v_scale=None), "NULL"), (dict(k_scale=18), "4-byte"), (dict(v_scale=17), "4-byte"),
    (dict(k=24), "16-byte"), (dict(n_pages=1 << 27), "2^31"),
])
def test_every_call_refuses_a_bad_descriptor(B, change, msg):
    p = ctypes.byref(_cache(B, **change))
    _refused(B, B.hf_pages8_extend(p, 16, 16, 2, None), msg)
    _refused(B, B.hf_pages8_truncate(p, 16, 16, 2, None), msg)
    _refused(B, B.hf_pages8_fork(p, 16, 16, 2, None), msg)
    _refused(B, B.hf_pages8_compact(p, None, None), msg)
    _refused(B, B.hf_pages8_write(p, 0, 1, 16, 16, 128, 0, 16, 16, 2, 8, None), msg)
    _refused(B, B.hf_pages8_read(p, 0, 1, 16, 16, 128, 0, 16, 16, 16, 2, 8, None), msg)
    _refused(B, B.hf_attention_pages8(p, 0, 2, 1, 4, 16, 256, 16, 0, 0.0, 16, 256, 16, 1 << 30, None), msg)
    if "NULL" not in msg and "byte" not in msg:  # sizes alone
        assert B.hf_pages8_work_ints(p) == 0
        assert B.hf_attention_pages8_workspace(p, 2, 1, 4, 0) == 0


def test_null_descriptors_and_the_other_kind_of_cache(B):
    _refused(B, B.hf_pages8_compact(None, None, None), "NULL")
    _refused(B, B.hf_attention_pages8(None, 0, 2, 1, 4, 16, 256, 16, 0, 0.0, 16, 256, 16, 1 << 30, None), "NULL")
    assert B.hf_pages8_work_ints(None) == 0 and B.hf_attention_pages8_workspace(None, 2, 1, 4, 0) == 0
    c = _cache(B)
    _refused(B, B.hf_pages_compact(ctypes.byref(c.pages), None, None), "HF_F32 or HF_BF16")


WRITE = dict(layer=0, layers=2, k=16, v=16, ld=128, step=1280, req=16, off=16, n=2, total=10)


@pytest.mark.parametrize("change,msg", [
    (dict(layer=-1), "layer"), (dict(layer=1), "layer"), (dict(layers=3), "layer"), (dict(layers=-1), "layer"),
    (dict(total=-1), "total"), (dict(k=None), "NULL"), (dict(off=None), "NULL"), (dict(ld=120), "ld"),
    (dict(step=-8), "layer_stride"), (dict(ld=132), "16 bytes"), (dict(step=1284), "16 bytes"), (dict(v=24), "16-byte"),
    (dict(off=18), "4-byte"), (dict(req=18), "4-byte"), (dict(n=-1), "n must"), (dict(n=1 << 21), "n must"),
])
def test_write_and_read_refusals(B, change, msg):
    p = ctypes.byref(_cache(B))
    a = {**WRITE, **change}
    _refused(B, B.hf_pages8_write(p, *a.values(), None), msg)
    r = list(a.values())
    _refused(B, B.hf_pages8_read(p, *r[:7], 16, *r[7:], None), msg)


def test_lists_and_empty_calls(B):
    p = ctypes.byref(_cache(B))
    assert B.hf_pages8_work_ints(p) == 16 + 2 * 20
    _refused(B, B.hf_pages8_write(p, 0, 1, 16, 16, 128, 0, 16, 16, 5, 8, None), "n_requests")
    _refused(B, B.hf_pages8_read(p, 0, 1, 16, 16, 128, 0, None, 16, 16, 5, 8, None), "without a list")
    _refused(B, B.hf_pages8_read(p, 0, 1, 16, 16, 128, 0, 16, None, 16, 2, 8, None), "NULL")
    _refused(B, B.hf_pages8_read(p, 0, 1, 16, 16, 128, 0, 16, 18, 16, 2, 8, None), "4-byte")
    _refused(B, B.hf_pages8_extend(p, None, None, 1, None), "NULL")
    _refused(B, B.hf_pages8_fork(p, 16, 18, 1, None), "4-byte")
    assert B.hf_pages8_extend(p, None, None, 0, None) == B.Status.OK
    assert B.hf_pages8_write(p, 0, 0, None, None, 0, 0, None, None, 2, 8, None) == B.Status.OK
    assert B.hf_pages8_read(p, 0, 1, None, None, 0, 0, None, None, None, 2, 0, None) == B.Status.OK


ATTEND = dict(layer=0, n=2, rows=8, hq=4, q=16, q_ld=256, req=16, shared=32, scale=0.0, out=16, out_ld=256, ws=16,
              bytes=1 << 30)


@pytest.mark.parametrize("rows_type", [0, 1])
@pytest.mark.parametrize("change,msg", [
    (dict(layer=2), "layer"), (dict(n=-1), "n must"), (dict(rows=0), "rows"), (dict(rows=65), "rows"), (dict(hq=3), "divide"),
    (dict(shared=8), "multiple of page"), (dict(shared=96), "table_ld"), (dict(scale=float("nan")), "scale"),
    (dict(req=None, n=5), "without a list"), (dict(q=None), "NULL"), (dict(ws=None), "NULL"), (dict(q_ld=248), "stride"),
    (dict(q=8), "16-byte"), (dict(out_ld=258), "16-byte"), (dict(req=18), "4-byte"), (dict(ws=24), "workspace"),
    (dict(bytes=0), "hf_attention_pages8_workspace"), (dict(n=1 << 20, rows=64, hq=128), "too large"),
])
def test_attend_refusals(B, rows_type, change, msg):
    p = ctypes.byref(_cache(B, rows=rows_type))
    _refused(B, B.hf_attention_pages8(p, *{**ATTEND, **change}.values(), None), msg)
    assert B.hf_attention_pages8_workspace(p, 2, 8, 4, 32) > 0
    assert B.hf_attention_pages8(p, *{**ATTEND, "n": 0, "q": None, "out": None, "ws": None}.values(), None) == B.Status.OK


ROTARY = dict(dtype=1, inter=0, rows=3, hq=4, hkv=2, dh=64, dim=64, turns=16, f=1.0, pos=16, q=16, q_ld=256, k=16, k_ld=128,
              qo=16, qo_ld=256, ko=16, ko_ld=128)


@pytest.mark.parametrize("change,msg", [
    (dict(dtype=2), "dtype"), (dict(inter=2), "interleaved"), (dict(rows=-1), "rows"), (dict(hq=-1), "heads"),
    (dict(hkv=1 << 17), "heads"), (dict(dh=1), "head_dim"), (dict(dh=257), "head_dim"), (dict(dim=0), "dim"),
    (dict(dim=63), "even"), (dict(dim=66), "dim"), (dict(f=float("nan")), "attention"), (dict(f=float("inf")), "attention"),
    (dict(turns=None), "NULL"), (dict(pos=None), "NULL"), (dict(q=None), "NULL"), (dict(ko=None), "NULL"),
    (dict(turns=20), "8-byte"), (dict(pos=18), "4-byte"), (dict(q=17), "aligned"), (dict(ko=19), "aligned"),
    (dict(q_ld=255), "stride"), (dict(ko_ld=100), "stride"), (dict(k_ld=1 << 37), "stride"),
])
def test_rotary_refusals(B, change, msg):
    _refused(B, B.hf_rotary(*{**ROTARY, **change}.values(), None), msg)


def test_rotary_without_rows_or_heads_needs_no_buffers(B):
    none = dict(turns=None, pos=None, q=None, k=None, qo=None, ko=None)
    assert B.hf_rotary(*{**ROTARY, **none, "rows": 0}.values(), None) == B.Status.OK
    assert B.hf_rotary(*{**ROTARY, **none, "hq": 0, "hkv": 0}.values(), None) == B.Status.OK


def _table(B, dim, base, **s):
    out, f = np.zeros(max(dim // 2, 1), dtype=np.uint64), ctypes.c_float()
    scaling = ctypes.byref(B.HfRotaryScaling(**s)) if s else None
    return B.hf_rotary_table(dim, base, scaling, out.ctypes.data, ctypes.byref(f)), out, f.value


@pytest.mark.parametrize("args,msg", [
    (dict(dim=0), "dim"), (dict(dim=7), "dim"), (dict(dim=258), "dim"), (dict(base=1.0), "base"), (dict(base=float("nan")), "base"),
    (dict(base=float("inf")), "base"), (dict(kind=5), "kind"), (dict(kind=-1), "kind"), (dict(kind=1, factor=0.5), "factor"),
    (dict(kind=1, factor=float("nan")), "factor"), (dict(kind=2, factor=float("inf")), "factor"),
    (dict(kind=2, factor=2.0, dim=2), "dim > 2"), (dict(kind=2, factor=1e200, base=1e200), "too large"),
    (dict(kind=3, factor=2.0), "original"), (dict(kind=4, factor=2.0, original=-3), "original"),
    (dict(kind=3, factor=2.0, original=64, fast=1.0, slow=2.0), "fast"), (dict(kind=4, factor=2.0, original=64, slow=-1.0), "fast"),
    (dict(kind=4, factor=2.0, original=64, fast=float("inf")), "fast"), (dict(kind=1, factor=2.0, attention=-1.0), "attention"),
    (dict(kind=1, factor=2.0, attention=float("nan")), "attention"),
])
def test_table_refusals(B, args, msg):
    a = {"dim": 64, "base": 1e4, **args}
    status, _, _ = _table(B, a.pop("dim"), a.pop("base"), **a)
    _refused(B, status, msg)


@pytest.mark.parametrize("kind,args", [("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=2.5)),
                                       ("yarn", dict(factor=8.0, original=4096)), ("yarn", dict(factor=1.0, original=1)),
                                       ("yarn", dict(factor=3.0, original=32768, fast=16.0, slow=2.0, attention=0.7)),
                                       ("bands", dict(factor=8.0, original=8192)), ("bands", dict(factor=2.0, original=7, attention=2.0))])
@pytest.mark.parametrize("dim,base", [(128, 1e6), (30, 1e4), (4, 1.5), (256, 1e9)])
def test_table(B, kind, args, dim, base):
    status, turns, f = _table(B, dim, base, kind=B.ROTARY_SCALING[kind], **args)
    assert status == B.Status.OK
    w, want = C.frequencies(dim, base, kind, **args)
    assert abs(f - want) <= 2.0 ** -24 * want
    got = turns.astype(np.float64) * 2.0 ** -64
    # pow, the few operations after it, and the rounding to 2^-64 turns
    assert (np.abs(got - w / (2 * np.pi)) <= 2.0 ** -48 * w + 2.0 ** -64).all()
    assert _table(B, dim, base)[2] == 1.0


def test_layouts(B):
    assert ctypes.sizeof(B.HfPages8) == ctypes.sizeof(B.HfPages) + 24 and B.HfPages8.k_scale.offset == 88
    assert ctypes.sizeof(B.HfRotaryScaling) == 40


def test_python_calls_refuse_wrong_arguments(B):
    import torch

    import speculative_decoding_drafter_hf_gb300 as hf
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    k = torch.zeros(1, 4, 2, 16, 64)
    with pytest.raises(TypeError, match="float8"):
        hf.Pages8(k, k, k, k, i(2, 2), i(2), i(4))
    k8 = k.to(torch.float8_e4m3fn)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        hf.Pages8(k8, k8, k, k, i(2, 2), i(2), i(4), dtype=torch.float16)
    with pytest.raises(TypeError, match="CUDA"):
        hf.Pages8(k8, k8, k, k, i(2, 2), i(2), i(4))
    for bad in (dict(scaling="other"), dict(dim=66), dict(dim=63), dict(base=0.5), dict(scaling="yarn", factor=2.0)):
        with pytest.raises((ValueError, hf.HyflashError)):
            hf.Rotary(64, device="cpu", **bad)
    with pytest.raises(TypeError):
        hf.Rotary(64, device="cpu")(torch.zeros(1, 2, 64), None, i(1))
