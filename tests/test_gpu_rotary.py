"""hf_rotary on the GPU against the formulas in 64 bits (_cache8_ref.py, which also derives the tolerances)."""
import numpy as np
import pytest
import torch

import _cache8_ref as C
import _target_ref as R

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
KINDS = [("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=2.5)), ("yarn", dict(factor=8.0, original=4096)),
         ("yarn", dict(factor=3.0, original=32768, fast=16.0, slow=2.0, attention=0.7)),
         ("bands", dict(factor=8.0, original=8192)), ("none", dict(attention=1.5))]


@pytest.fixture(scope="module")
def hf():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from speculative_decoding_drafter_hf_gb300 import build
    build.build()
    import speculative_decoding_drafter_hf_gb300 as m
    return m


def _randn(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DT[dtype])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,T,hq,hkv,dh,dim", [
    ("bf16", 1, 32, 8, 128, 128), ("bf16", 37, 5, 1, 128, 64), ("f32", 13, 4, 2, 64, 48), ("f32", 3, 1, 1, 6, 2),
    ("bf16", 2, 3, 3, 80, 50), ("bf16", 700, 2, 1, 256, 256), ("f32", 9, 7, 2, 33, 20), ("bf16", 5, 2, 2, 72, 8),
    ("bf16", 11, 4, 1, 128, 24), ("bf16", 3, 2, 2, 64, 60), ("bf16", 6, 1, 3, 64, 40), ("f32", 4, 2, 1, 64, 12), ("f32", 4, 2, 1, 64, 10),
    ("bf16", 4, 2, 1, 36, 16), ("bf16", 4, 2, 1, 34, 32), ("f32", 3, 1, 2, 258 // 2 + 1, 4), ("bf16", 3, 5, 1, 127, 126),
])
def test_layouts_and_sizes(hf, dtype, T, hq, hkv, dh, dim, interleaved):
    x = _randn((T, hq + hkv + 1, dh), dtype, T)
    pos = [(i * 7919) % 100003 for i in range(T)]
    rot = hf.Rotary(dh, dim=dim, interleaved=interleaved)
    w, f = C.frequencies(dim, 1e6, "none")
    g = x.cuda()
    q, k = rot(g[:, :hq], g[:, hq:hq + hkv], C.ints(pos))
    for got, src in ((q, x[:, :hq]), (k, x[:, hq:hq + hkv])):
        want, tol = C.rotary(src, pos, w, f, interleaved, dtype == "bf16")
        R.check_attention(R.to64(got), want, tol)
        assert torch.equal(got[..., dim:].cpu(), src[..., dim:])  # (columns behind dim: the same bits)
    assert torch.equal(g.cpu(), x)
    # in place, inside the projection's output: the same bits, the rest of it left as it was
    rot(g[:, :hq], g[:, hq:hq + hkv], C.ints(pos), q_out=g[:, :hq], k_out=g[:, hq:hq + hkv])
    assert torch.equal(g[:, :hq], q) and torch.equal(g[:, hq:hq + hkv], k) and torch.equal(g[:, hq + hkv:].cpu(), x[:, hq + hkv:])
    # queries alone, other strides (16 bytes do not divide them)
    y = torch.zeros((T, hq * dh + 1), dtype=DT[dtype], device="cuda")
    y[:, :hq * dh] = x[:, :hq].reshape(T, -1).cuda()
    z = torch.full((T, hq * dh + 3), 9.0, dtype=DT[dtype], device="cuda")
    v = lambda t: t[:, :hq * dh].unflatten(1, (hq, dh))
    out, none = rot(v(y), None, C.ints(pos), q_out=v(z))
    assert none is None and (z[:, hq * dh:] == 9).all()
    want, tol = C.rotary(x[:, :hq], pos, w, f, interleaved, dtype == "bf16")
    R.check_attention(R.to64(out), want, tol)


@pytest.mark.parametrize("kind,args", KINDS)
@pytest.mark.parametrize("dim", [128, 30])
def test_scalings_at_far_positions(hf, kind, args, dim):
    pos = [0, 1, -1, 5, 4095, 32768, 131071, 1 << 20, 12345677, (1 << 31) - 1, -(1 << 31)]
    x = _randn((len(pos), 2, 128), "f32", 3)
    rot = hf.Rotary(128, dim=dim, base=1e4, scaling=kind, **args)
    w, f = C.frequencies(dim, 1e4, kind, **args)
    assert abs(rot.attention - f) <= 2.0 ** -23 * f
    q, _ = rot(x.cuda(), None, C.ints(pos))
    want, tol = C.rotary(x, pos, w, f, False, False)
    R.check_attention(R.to64(q), want, tol)
    # a rotation back: the negative positions, of the first rows (f = 1)
    if f == 1.0:
        back, _ = rot(q[:9], None, C.ints([-p for p in pos[:9]]))
        assert ((back.cpu() - x[:9]).abs() <= 2.0 ** -18 * x.abs().max()).all()


def test_no_rows_streams_and_graphs(hf):
    rot = hf.Rotary(64, interleaved=True)
    q, k = rot(torch.empty(0, 4, 64, device="cuda"), torch.empty(0, 2, 64, device="cuda"), C.ints([]))
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    x = _randn((50, 6, 64), "bf16", 4).cuda()
    pos = C.ints(list(range(50)))
    first, _ = rot(x, None, pos)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [rot(x, None, pos, stream=s)[0] for s in streams for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    out, graph = torch.zeros_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rot(x, None, pos, q_out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    pos.add_(3)  # the replay reads the positions of its own time
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, rot(x, None, pos)[0])


def test_wrong_arguments(hf):
    rot, x = hf.Rotary(64), torch.zeros(3, 4, 64, device="cuda")
    pos = C.ints([0, 1, 2])
    for bad, error in ((dict(positions=pos.cpu()), ValueError), (dict(positions=pos.long()), ValueError), (dict(positions=pos[:2]), ValueError),
                       (dict(q=x.half()), TypeError), (dict(q=x.cpu()), TypeError), (dict(q=x[..., :32]), ValueError),
                       (dict(q=x[0]), ValueError), (dict(k=x[:2]), ValueError), (dict(k=x.bfloat16()), TypeError),
                       (dict(q_out=x[:, :2]), ValueError), (dict(q_out=x.bfloat16()), TypeError),
                       (dict(q=x.transpose(0, 1).contiguous().transpose(0, 1)), ValueError)):
        a = {"q": x, "k": None, "positions": pos, "q_out": None, **bad}
        with pytest.raises(error):
            rot(a["q"], a["k"], a["positions"], q_out=a["q_out"])


def test_rows_and_strides_beyond_32_bits(hf):
    """Rows 2^31 elements apart and more."""
    rot = hf.Rotary(64)
    buf = torch.empty((5, 1 << 30), dtype=torch.bfloat16, device="cuda")
    x = _randn((5, 2, 64), "bf16", 6)
    q = buf[:, :128].unflatten(1, (2, 64))
    q.copy_(x)
    pos = [3, 1, 4, 1, 5]
    got, _ = rot(q, None, C.ints(pos))
    want, tol = C.rotary(x, pos, *C.frequencies(64, 1e6, "none"), False, True)
    R.check_attention(R.to64(got), want, tol)


def test_many_rows(hf):
    """As many rows as a prefill batch has: against the same rows in small calls, bit by bit."""
    rot = hf.Rotary(128, scaling="bands", factor=8.0, original=8192)
    x = _randn((20011, 6, 128), "bf16", 7).cuda()
    pos = C.ints([(31 * i) % 40000 for i in range(20011)])
    q, k = rot(x[:, :4], x[:, 4:], pos)
    for a in (0, 9999, 20000):
        qq, kk = rot(x[a:a + 11, :4], x[a:a + 11, 4:], pos[a:a + 11])
        assert torch.equal(q[a:a + 11], qq) and torch.equal(k[a:a + 11], kk)
