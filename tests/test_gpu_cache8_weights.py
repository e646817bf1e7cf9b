"""Attention over the 8-bit cache where one key holds most of a row's weight and the others share the rest: as an
attention sink does, its value is zero, so the output is what the small weights bring.

The bound is the one of _target_ref.attention for bf16 rows (weights to 2^-8, the result to 2^-8), with the
rows' part of a score that _cache8_ref.attention derives, and nothing for weights that are small: those of the cases lie
around 2^-11 to 2^-20 of the largest."""
import math

import pytest
import torch

import _cache8_ref as C
import _target_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hf():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from speculative_decoding_drafter_hf_gb300 import build
    build.build()
    import speculative_decoding_drafter_hf_gb300 as m
    return m


def _codes(x):
    """[pages, heads, page, dh] as codes and scales."""
    top = x.abs().amax((-1, -2))
    scale = torch.tensor([C.scale_for(float(t)) for t in top.flatten()], dtype=torch.float64).view(top.shape)
    return (x / scale[..., None, None]).float().to(torch.float8_e4m3fn), scale.float()


def _case(hf, dh, keys, rows, n, place, share, page=64, hkv=2, group=2, seed=1, floor=0.0):
    """floor: how far off a weight times its page's scale may be, of the largest. n requests that hold the same pages. Scores are normal draws; key `place` scores as much more as gives it
    `share` of a row's sum, its value is zero, the others' values are around 0.3."""
    g = torch.Generator().manual_seed(seed)
    pages = -(-keys // page)
    k = torch.randn((pages, hkv, page, dh), generator=g, dtype=torch.float64)
    v = 0.3 + 0.3 * torch.randn((pages, hkv, page, dh), generator=g, dtype=torch.float64)
    k[..., 0] = 0
    k[place // page, :, place % page] = 0
    k[place // page, :, place % page, 0] = 1
    v[place // page, :, place % page] = 0
    (k, ks), (v, vs) = _codes(k), _codes(v)
    order = torch.randperm(pages, generator=g)
    q = torch.randn((rows, hkv * group, dh), generator=g)
    q[..., 0] = math.log(share / (1 - share) * keys * math.exp(0.5)) * dh ** 0.5
    q = q.to(torch.bfloat16)
    put = lambda t: torch.empty_like(t).index_copy_(0, order, t)[None].cuda()
    c = hf.Pages8(put(k.view(torch.uint8)).view(torch.float8_e4m3fn), put(v.view(torch.uint8)).view(torch.float8_e4m3fn), put(ks),
                  put(vs), order.to(torch.int32)[None].repeat(n, 1).cuda(), C.ints([keys] * n), C.ints([n] * pages))
    # plain form, in 64 bits
    val = lambda t, s: (t.double() * s.double()[..., None, None]).transpose(0, 1).reshape(hkv, pages * page, dh)[:, :keys].cuda()
    kk, vv = val(k, ks), val(v, vs)
    qq = q.cuda().double().view(rows, hkv, group, dh)
    s = torch.einsum("rhgd,hkd->rhgk", qq, kk) * dh ** -0.5
    seen = torch.arange(keys, device="cuda") < keys - rows + 1 + torch.arange(rows, device="cuda")[:, None]
    p = torch.softmax(s.masked_fill(~seen[:, None, None], -math.inf), -1)
    o, mag = (torch.einsum("rhgk,hkd->rhgd", p, x).reshape(rows, -1, dh) for x in (vv, vv.abs()))
    top = qq.abs().amax(-1).view(rows, -1, 1)
    ds = (dh + 4) * R.U * torch.einsum("rhgd,hkd->rhgk", qq.abs(), kk.abs()).amax() * dh ** -0.5
    ds = ds + 2.0 ** -14 * top / 224 * kk.abs().sum(-1).max() * dh ** -0.5
    tol = (4 * ds + (keys + 16) * R.U + 2.0 ** -8) * mag + 2.0 ** -8 * o.abs()
    if floor:
        sv = vs.double().repeat_interleave(page, 0).T[:, :keys].cuda()  # [hkv, keys]
        top = (p * sv[None, :, None]).amax(-1).view(rows, -1, 1)
        tol = tol + floor * top * (vv.abs() / sv[..., None]).sum(1).repeat_interleave(group, 0)
    assert 0.6 * share < float(p[..., place].min()) and float(p[..., place].max()) < 1.4 * share
    return c, q.cuda().expand(n, *q.shape).contiguous(), R.to64(o), R.to64(tol)


@pytest.mark.parametrize("share", [0.3, 0.75, 0.96])
@pytest.mark.parametrize("place", ["first", "middle", "last"])
@pytest.mark.parametrize("dh,keys,rows", [(128, 4096, 1), (128, 32768, 1), (128, 4096, 8), (64, 4096, 1), (64, 32768, 8)])
def test_a_key_that_holds_most_of_the_weight(hf, dh, keys, rows, place, share):
    at = {"first": 3, "middle": keys // 2 + 5, "last": keys - rows - 3}[place]
    for n in (1, 64):
        c, q, want, tol = _case(hf, dh, keys, rows, n, at, share)
        out = R.to64(c.attend(q))
        for i in range(n):
            R.check_attention(out[i], want, tol, f"{n} requests, entry {i}")
        assert not c.check()


@pytest.mark.parametrize("share", [0.999, 0.9999])
@pytest.mark.parametrize("n", [1, 64])
def test_a_key_that_holds_nearly_all_of_the_weight(hf, n, share):
    """Where the weights of 32768 others end is derived: codes to half a step of 2^-22 (and 16-bit floats to half of
    2^-24), the largest at 2^10."""
    for place in (3, 20000):
        c, q, want, tol = _case(hf, 128, 32768, 2, n, place, share, floor=1.25 * 2.0 ** -33)
        out = R.to64(c.attend(q))
        for i in range(n):
            R.check_attention(out[i], want, tol, f"key {place}, entry {i}")


@pytest.mark.parametrize("place", [3, 2000, 4096 - 300, 4096 - 20])
@pytest.mark.parametrize("n,rows,group", [(24, 1, 2), (24, 5, 2), (64, 8, 2), (64, 8, 4)])
def test_beside_a_shared_prefix(hf, n, rows, group, place):
    """48, 240 and 1024 rows of a head: the prefix as codes; 2048: through bf16 rows."""
    c, q, want, tol = _case(hf, 128, 4096, rows, n, place, 0.96, group=group)
    out = R.to64(c.attend(q, shared=4096 - 256))
    for i in range(n):
        R.check_attention(out[i], want, tol, f"entry {i}")
    assert not c.check()


@pytest.mark.parametrize("group,rows", [(3, 5), (6, 5), (9, 5), (12, 4), (12, 5), (60, 1), (64, 3)])
def test_row_tiles_of_every_width(hf, group, rows):
    """15, 30, 45 and 48 rows of a head in a row tile, two tiles of a head, tiles of 60 and 64 rows."""
    for place in (7, 2050):
        c, q, want, tol = _case(hf, 128, 4096, rows, 3, place, 0.96, group=group)
        out = R.to64(c.attend(q))
        for i in range(3):
            R.check_attention(out[i], want, tol, f"entry {i}")
        for shared in (2048, 3584):
            R.check_attention(R.to64(c.attend(q, shared=shared))[2], want, tol, f"{shared} shared")
        assert not c.check()
