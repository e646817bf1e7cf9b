"""The target-side calls on the GPU against plain forms in 64 bits
(_target_ref.py, which also derives the tolerances)."""
import random

import numpy as np
import pytest
import torch

import _target_ref as R

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def hf():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from speculative_decoding_drafter_hf_gb300 import build
    build.build()
    import speculative_decoding_drafter_hf_gb300 as m
    return m


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=_gen(seed)) * scale).to(DT[dtype])


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ prompts
PROMPTS = [  # dtype, Hq, Hkv, dh, lengths
    ("f32", 4, 2, 64, [1, 0, 17, 64, 65, 130]),
    ("f32", 3, 1, 40, [33, 100]),
    ("f32", 2, 2, 256, [70]),
    ("f32", 5, 1, 8, [1]),
    ("f32", 2, 1, 64, [(7 * i) % 19 for i in range(40)]),            # more sequences than a warp has lanes
    ("bf16", 8, 2, 128, [1, 0, 17, 64, 65, 130]),
    ("bf16", 4, 2, 64, [200, 3, 1, 129]),
    ("bf16", 2, 2, 128, [257]),
    ("bf16", 3, 1, 128, [90, 45]),
    ("bf16", 5, 1, 64, [77, 52, 128]),
    ("bf16", 14, 2, 128, [40, 19]),
    ("bf16", 4, 4, 32, [90, 1]),
    ("bf16", 2, 1, 256, [70, 5]),
    ("bf16", 64, 1, 128, [9, 3]),
    ("bf16", 1, 1, 128, [0, 0, 300, 0]),
    ("bf16", 2, 1, 64, [(7 * i) % 23 for i in range(60)] + [300]),   # more sequences than a warp has lanes
    ("bf16", 2, 1, 64, [(5 * i) % 13 for i in range(200)] + [150]),  # more than are sorted by their work
]


@pytest.mark.parametrize("dtype,hq,hkv,dh,lens", PROMPTS)
def test_prompt(hf, dtype, hq, hkv, dh, lens):
    T = sum(lens)
    ends = [sum(lens[:i]) for i in range(len(lens) + 1)]
    x = _randn((T + 5, hq + 2 * hkv, dh), dtype, 1)  # one projection's output, rows behind the last sequence
    x[:, :hq] *= 2  # scores spread over several units
    d = x.cuda()
    q, k, v = d[:, :hq], d[:, hq:hq + hkv], d[:, hq + hkv:]
    out = torch.full((T + 5, hq, dh), 7.0, dtype=DT[dtype], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = hf.attention_prompt(q, k, v, _i32(ends), out=out, status=status)
    assert got is out
    want, tol = R.prompt(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], ends, dh ** -0.5, dtype == "bf16")
    o = R.to64(out)
    assert (o[T:] == 7.0).all()  # not written
    R.check_attention(o[:T], want[:T], tol[:T], "prompt")
    assert int(status) == 0


def test_prompt_starts_inside_the_buffer_and_takes_a_scale(hf):
    q, k, v = (_randn((60, h, 64), "bf16", 5 + h) for h in (4, 2, 2))
    out = torch.full((60, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    hf.attention_prompt(q.cuda(), k.cuda(), v.cuda(), _i32([7, 30, 51]), scale=0.3, out=out)
    want, tol = R.prompt(q, k, v, [7, 30, 51], 0.3, True)
    o = R.to64(out)
    assert (o[:7] == 3.0).all() and (o[51:] == 3.0).all()
    R.check_attention(o[7:51], want[7:51], tol[7:51])


@pytest.mark.parametrize("dtype,dh", [("f32", 64), ("bf16", 128), ("bf16", 64), ("bf16", 32)])
def test_prompt_odd_values_stay_with_the_rows_that_see_them(hf, dtype, dh):
    """NaN and infinities in one sequence's K and V reach neither another sequence nor an
    earlier row of their own."""
    lens = [50, 90, 40]
    ends = [0, 50, 140, 180]
    q, k, v = (_randn((180, h, dh), dtype, 11 + h) for h in (4, 2, 2))
    k[120:140] = float("nan")
    v[110, 1, 3] = float("inf")
    v[115:140] = float("nan")
    v[130, 0, 0] = -float("inf")
    o = R.to64(hf.attention_prompt(q.cuda(), k.cuda(), v.cuda(), _i32(ends)))
    k2, v2 = k.clone(), v.clone()
    k2[120:140] = 0
    v2[~torch.isfinite(v2)] = 0
    want, tol = R.prompt(q, k2, v2, ends, dh ** -0.5, dtype == "bf16")
    R.check_attention(o[:110], want[:110], tol[:110], "rows before")
    R.check_attention(o[140:], want[140:], tol[140:], "the next sequence")
    assert np.isnan(o[115:140]).all()
    assert np.isposinf(o[110:115, 2:, 3]).all()
    rest = o[110:115].copy()
    rest[:, 2:, 3] = 0
    assert np.isfinite(rest).all()


def test_prompt_large_scores_and_masked_infinity(hf):
    """Scores far apart: the running maximum moves by more than any fixed margin, up and down."""
    q, k, v = (_randn((300, h, 128), "bf16", 21 + h) for h in (2, 1, 1))
    k *= torch.linspace(0.01, 40, 300)[torch.randperm(300, generator=_gen(3))][:, None, None].to(torch.bfloat16)
    want, tol = R.prompt(q, k, v, [0, 300], 128 ** -0.5, True)
    o = R.to64(hf.attention_prompt(q.cuda(), k.cuda(), v.cuda(), _i32([0, 300])))
    R.check_attention(o, want, tol)


def test_prompt_bad_bounds_set_the_status(hf):
    q = _randn((20, 2, 64), "bf16", 1).cuda()
    for bad in ([0, 30], [0, 12, 5, 20], [-3, 10]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        hf.attention_prompt(q, q, q, _i32(bad), status=status)
        assert hf.CallStatus(int(status)) == hf.CallStatus.BAD


def test_prompt_long(hf):
    """A long sequence at a full model's heads, checked at a few rows."""
    T, hq, hkv, dh = 5001, 8, 2, 128
    q, k, v = (_randn((T, h, dh), "bf16", 31 + h) for h in (hq, hkv, hkv))
    o = R.to64(hf.attention_prompt(q.cuda(), k.cuda(), v.cuda(), _i32([0, 2, T])))
    q, k, v = R.to64(q), R.to64(k), R.to64(v)
    for i in (0, 1, 2, 127, 128, 129, 255, 256, 257, 1000, 2048, 3333, 4095, 4998, 4999, 5000):
        a = 0 if i < 2 else 2
        for h in range(hq):
            want, tol = R.attention(q[i, h], k[a:i + 1, h // 4], v[a:i + 1, h // 4], dh ** -0.5, True)
            R.check_attention(o[i, h], want, tol, f"row {i} head {h}")


# ------------------------------------------------------- attention over pages
ATTEND = [  # dtype, Hq, Hkv, dh, page, rows, shared, own lengths (None: an empty request)
    ("f32", 4, 2, 64, 16, 1, 0, [1, 15, 16, 17, 200, None]),
    ("f32", 4, 2, 64, 16, 8, 64, [0, 1, 8, 30, 300, None]),
    ("f32", 2, 1, 40, 8, 3, 8, [2, 50]),
    ("f32", 6, 1, 256, 32, 5, 0, [70, 3]),
    ("bf16", 8, 2, 128, 16, 1, 0, [1, 15, 16, 17, 200, None, 129]),
    ("bf16", 8, 2, 128, 16, 8, 0, [3, 8, 9, 1000, None]),
    ("bf16", 8, 2, 128, 32, 8, 128, [0, 1, 8, 30, 700, None]),
    ("bf16", 4, 2, 64, 64, 5, 640, [5, 64, 1]),
    ("bf16", 5, 1, 128, 8, 7, 8, [2, 50, 77]),
    ("bf16", 10, 2, 64, 128, 2, 256, [300, 5]),
    ("bf16", 16, 1, 128, 16, 16, 2048, [40, 100]),
    ("bf16", 64, 1, 64, 16, 3, 32, [33, 4]),
    ("bf16", 4, 4, 32, 16, 4, 32, [20, 3]),
    ("bf16", 2, 1, 256, 16, 64, 16, [64, 100]),
    ("bf16", 4, 4, 128, 64, 1, 4096, [1] * 9),
    ("bf16", 32, 8, 128, 32, 1, 4096, [1, 700, 33]),
]


def _shared_cache(dtype, hkv, dh, page, shared, own, seed, layers=1):
    """A cache whose requests share `shared` tokens, pages in shuffled places; unused rows hold NaN."""
    rng = random.Random(seed)
    n_shared = shared // page
    counts = [0 if x is None else -(-x // page) for x in own]
    total = n_shared + sum(counts) + 3
    ids = list(range(total))
    rng.shuffle(ids)
    k, v = (_randn((layers, total, hkv, page, dh), dtype, seed + s) for s in (1, 2))
    columns = n_shared + max(counts) + 1
    rows, lens, refs, at = [], [], [0] * total, n_shared
    used = torch.zeros((total, page), dtype=torch.bool)
    for x, c in zip(own, counts):
        row = [] if x is None else ids[:n_shared] + ids[at:at + c]
        at += c
        lens.append(0 if x is None else shared + x)
        for j, p in enumerate(row):
            refs[p] += 1
            used[p, :max(0, min(page, lens[-1] - j * page))] = True
        rows.append(row)
    k.permute(1, 3, 0, 2, 4)[~used] = float("nan")
    v.permute(1, 3, 0, 2, 4)[~used] = float("nan")
    table = [row + [-1] * (columns - len(row)) for row in rows]
    return k, v, table, lens, refs


def _on_gpu(hf, k, v, table, lens, refs):
    return hf.Pages(k.cuda(), v.cuda(), _i32(table), _i32(lens), _i32(refs))


@pytest.mark.parametrize("dtype,hq,hkv,dh,page,rows,shared,own", ATTEND)
def test_attend(hf, dtype, hq, hkv, dh, page, rows, shared, own):
    k, v, table, lens, refs = _shared_cache(dtype, hkv, dh, page, shared, own, 7, layers=2)
    c = _on_gpu(hf, k, v, table, lens, refs)
    n = len(own)
    x = _randn((n, rows, hq + 3, dh), dtype, 9, 2.0)
    q = x[:, :, :hq]
    out = torch.full((n, rows, hq, dh), 7.0, dtype=DT[dtype], device="cuda")
    ws = c.attend_workspace(q, shared)
    ws.fill_(255)  # NaN everywhere: the workspace needs no values
    got = c.attend(x.cuda()[:, :, :hq], layer=1, shared=shared, out=out, workspace=ws)
    assert got is out
    want, tol = R.pages(q, k[1], v[1], table, lens, dh ** -0.5, dtype == "bf16")
    R.check_attention(R.to64(out), want, tol, "attend")
    assert not c.check()
    # the same without the prefix in common: the keys are the same ones
    again = c.attend(x.cuda()[:, :, :hq], layer=1)
    R.check_attention(R.to64(again), want, tol, "attend, nothing shared")
    assert not c.check()


@pytest.mark.parametrize("shared", [0, 32])
def test_attend_many_entries(hf, shared):
    """More entries than requests: a list that repeats them, some of them empty, some long."""
    own = [3, 17, 200, None, 64, 1, 33, 700, 16]
    k, v, table, lens, refs = _shared_cache("bf16", 2, 64, 16, shared, own, 8)
    c = _on_gpu(hf, k, v, table, lens, refs)
    rng = random.Random(5)
    req = [0] + [rng.randrange(len(own)) for _ in range(339)]
    q = _randn((340, 2, 4, 64), "bf16", 5)
    o = R.to64(c.attend(q.cuda(), _i32(req), shared=shared))
    want, tol = R.pages(q, k[0], v[0], table, lens, 64 ** -0.5, True, req)
    R.check_attention(o, want, tol)
    assert not c.check()


def test_attend_lists_repeats_and_strange_entries(hf):
    k, v, table, lens, refs = _shared_cache("bf16", 2, 128, 16, 32, [5, 60, 33, 9], 3)
    c = _on_gpu(hf, k, v, table, lens, refs)
    q = _randn((5, 4, 8, 128), "bf16", 5)
    req = [2, 0, 2, 3, 1]
    want, tol = R.pages(q, k[0], v[0], table, lens, 0.11, True, req)
    for shared in (0, 32):
        R.check_attention(R.to64(c.attend(q.cuda(), _i32(req), shared=shared, scale=0.11)), want, tol)
        assert not c.check()
    # entries that name no request are zero and reported; the others are as before
    o = R.to64(c.attend(q.cuda(), _i32([2, -1, 2, 4, 1]), scale=0.11))
    assert (o[1] == 0).all() and (o[3] == 0).all()
    for i in (0, 2, 4):
        R.check_attention(o[i], want[i], tol[i])
    assert c.check() == hf.CallStatus.BAD
    # a length past the table, and a negative one
    c.lens.copy_(_i32([lens[0], 10 ** 6, -5, lens[3]]))
    o = R.to64(c.attend(q.cuda()[:4].contiguous()))
    w4, t4 = R.pages(q[:4], k[0], v[0], table, [lens[0], 0, 0, lens[3]], 128 ** -0.5, True)
    R.check_attention(o, w4, t4)
    assert c.check() == hf.CallStatus.BAD


@pytest.mark.parametrize("dtype,dh", [("f32", 64), ("bf16", 32)])
def test_attend_on_cuda_cores_strange_entries_and_prefixes(hf, dtype, dh):
    """The same rules where the CTAs look the lengths up for themselves."""
    k, v, table, lens, refs = _shared_cache(dtype, 2, dh, 16, 64, [5, 60, 33, 9], 6)
    c = _on_gpu(hf, k, v, table, lens, refs)
    req = [2, -1, 0, 4, 2] + [3, 1] * 200  # (more entries than CTAs that compare prefixes)
    n = len(req)
    q = _randn((n, 3, 4, dh), dtype, 5)
    good = [i for i in range(n) if 0 <= req[i] < 4]
    want, tol = R.pages(q[good], k[0], v[0], table, lens, dh ** -0.5, dtype == "bf16", [req[i] for i in good])
    for shared in (0, 64):
        o = R.to64(c.attend(q.cuda(), _i32(req), shared=shared))
        R.check_attention(o[good], want, tol)
        assert (o[[1, 3]] == 0).all() and c.check() == hf.CallStatus.BAD
        o = R.to64(c.attend(q[good].cuda(), _i32([req[i] for i in good]), shared=shared))
        R.check_attention(o, want, tol)
        assert not c.check()
    # one entry whose prefix is another (the last of 203): reported, the others as before
    t = [list(r) for r in table]
    t[0][2], t[0][4] = t[0][4], t[0][2]
    c = _on_gpu(hf, k, v, t, lens, refs)
    o = R.to64(c.attend(q[:203].cuda(), _i32([2, 2] + [1] * 200 + [0]), shared=64))
    want, tol = R.pages(q[:202], k[0], v[0], table, lens, dh ** -0.5, dtype == "bf16", [2, 2] + [1] * 200)
    R.check_attention(o[:202], want, tol)
    assert c.check() == hf.CallStatus.BAD
    # an empty first entry: nothing is shared, so the others' lengths break the rule
    c = _on_gpu(hf, k, v, table, [0] + lens[1:], refs)
    assert (c.attend(q[:4].cuda(), shared=64) == 0).all()
    assert c.check() == hf.CallStatus.BAD
    # lengths of an entry that fit neither the table nor the prefix
    for bad in (10 ** 6, -5, 40):
        c = _on_gpu(hf, k, v, table, [lens[0], bad, lens[2], lens[3]], refs)
        o = R.to64(c.attend(q[:4].cuda(), shared=64))
        want, tol = R.pages(q[:4], k[0], v[0], table, [lens[0], 0, lens[2], lens[3]], dh ** -0.5, dtype == "bf16")
        R.check_attention(o, want, tol)
        assert c.check() == hf.CallStatus.BAD


def test_attend_bad_pages_and_unequal_prefixes_are_reported(hf):
    k, v, table, lens, refs = _shared_cache("bf16", 2, 128, 16, 64, [5, 60, 33], 4)
    q = _randn((3, 2, 8, 128), "bf16", 5)
    want, tol = R.pages(q, k[0], v[0], table, lens, 128 ** -0.5, True)
    for bad in (-1, len(refs), 1 << 30):
        t = [list(r) for r in table]
        t[1][5] = bad
        c = _on_gpu(hf, k, v, t, lens, refs)
        for shared in (0, 64):
            o = R.to64(c.attend(q.cuda(), shared=shared))
            for i in (0, 2):
                R.check_attention(o[i], want[i], tol[i])
            assert c.check() == hf.CallStatus.BAD
    t = [list(r) for r in table]
    t[2][3], t[2][4] = t[2][4], t[2][3]
    c = _on_gpu(hf, k, v, t, lens, refs)
    o = R.to64(c.attend(q.cuda(), shared=64))
    for i in (0, 1):
        R.check_attention(o[i], want[i], tol[i])
    assert c.check() == hf.CallStatus.BAD
    # fewer tokens than the prefix; an empty first entry
    c = _on_gpu(hf, k, v, table, [lens[0], 40, lens[2]], refs)
    o = R.to64(c.attend(q.cuda(), shared=64))
    assert (o[1] == 0).all()
    R.check_attention(o[2], want[2], tol[2])
    assert c.check() == hf.CallStatus.BAD
    c = _on_gpu(hf, k, v, table, [0, lens[1], lens[2]], refs)
    assert (R.to64(c.attend(q.cuda(), shared=64)) == 0).all()
    assert c.check() == hf.CallStatus.BAD
    c = _on_gpu(hf, k, v, table, [0, 0, 0], refs)
    assert (R.to64(c.attend(q.cuda(), shared=64)) == 0).all()
    assert not c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attend_odd_values_stay_with_the_rows_that_see_them(hf, dtype):
    k, v, table, lens, refs = _shared_cache(dtype, 2, 128, 16, 32, [90, 60], 6)
    p = table[0][-2]  # the last page of request 0 (tokens 112 .. 121)
    k[0, p, :, 8] = float("nan")   # token 120
    v[0, p, 1, 6, 5] = float("inf")  # token 118
    q = _randn((2, 8, 4, 128), dtype, 5)  # rows at tokens 114 .. 121
    k2, v2 = k.clone(), v.clone()
    k2[0, p, :, 8] = 0
    v2[0, p, 1, 6, 5] = 0
    want, tol = R.pages(q, k2[0], v2[0], table, lens, 128 ** -0.5, dtype == "bf16")
    c = _on_gpu(hf, k, v, table, lens, refs)
    for shared in (0, 32):
        o = R.to64(c.attend(q.cuda(), shared=shared))
        R.check_attention(o[1], want[1], tol[1], "the other request")
        R.check_attention(o[0, :4], want[0, :4], tol[0, :4], "earlier rows")
        R.check_attention(o[0, :6, :2], want[0, :6, :2], tol[0, :6, :2], "the other head")
        assert np.isposinf(o[0, 4:6, 2:, 5]).all() and np.isfinite(np.delete(o[0, 4:6], 5, -1)).all()
        assert np.isnan(o[0, 6:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_pool_past_32_bits(hf, dtype):
    """Pages whose elements lie behind the first 2^32: extended, written, copied, attended, compacted."""
    hkv, page, dh = (16, 64, 128) if dtype == "bf16" else (16, 64, 64)
    n_pages = (1 << 32) // (hkv * page * dh) + 70
    c = hf.Pages.empty(1, n_pages, hkv, page, dh, 3, 6, dtype=DT[dtype])
    c.refs.fill_(1)
    c.refs[-40:] = 0  # only the last ones are free
    c.extend(_i32([100]), _i32([1]))
    k, v = (_randn((1, 100, hkv, dh), dtype, s) for s in (1, 2))
    c.write(k.cuda(), v.cuda(), _i32([0, 100]), _i32([1]))
    c.fork(_i32([1]), _i32([2]))
    c.extend(_i32([4, 4]), _i32([1, 2]))  # both take a copy of the half-filled page
    more = [_randn((1, 8, hkv, dh), dtype, s) for s in (3, 4)]
    c.write(more[0].cuda(), more[1].cuda(), _i32([0, 4, 8]), _i32([1, 2]))
    assert not c.check() and c.lens.tolist() == [0, 104, 104]
    q = _randn((2, 4, 2 * hkv, dh), dtype, 5)

    def expect(o):
        for i in range(2):
            kk = torch.cat([k[0], more[0][0, 4 * i:4 * i + 4]])
            vv = torch.cat([v[0], more[1][0, 4 * i:4 * i + 4]])
            for r in range(4):
                for h in range(0, 2 * hkv, 5):
                    want, tol = R.attention(R.to64(q[i, r, h]), R.to64(kk[:101 + r, h // 2]), R.to64(vv[:101 + r, h // 2]),
                                            dh ** -0.5, dtype == "bf16")
                    R.check_attention(o[i, r, h], want, tol, f"request {i} row {r} head {h}")

    for shared in (0, 64):
        expect(R.to64(c.attend(q.cuda(), _i32([1, 2]), shared=shared)))
    assert int(c.table[1, 0]) >= n_pages - 40 and not c.check()
    c.refs[5:20] = 0  # holes far before them
    c.compact()
    assert not c.check() and int(c.table[:, :2].max()) < n_pages - 40
    expect(R.to64(c.attend(q.cuda(), _i32([1, 2]))))
    assert not c.check()


# ----------------------------------------------------------------- page tables
def _same(c, ref, what):
    assert c.lens.tolist() == ref.lens, what
    assert c.refs.tolist() == ref.refs, what
    t = c.table.tolist()
    for r, row in enumerate(ref.rows):
        assert t[r][:len(row)] == row, f"{what}: request {r}"
    assert np.array_equal(R.to64(c.k), ref.k) and np.array_equal(R.to64(c.v), ref.v), f"{what}: pool"


@pytest.mark.parametrize("dtype,hkv,page,dh,layers,requests,pages_", [
    ("bf16", 2, 16, 64, 2, 9, 60), ("f32", 1, 8, 8, 1, 40, 300), ("bf16", 3, 32, 128, 3, 5, 25),
    ("f32", 2, 64, 40, 1, 7, 12), ("bf16", 1, 128, 16, 2, 3, 9000)])
def test_cache_random_calls(hf, dtype, hkv, page, dh, layers, requests, pages_):
    """A random sequence of calls against the rules kept in lists: tables, counts and data equal after each."""
    rng = random.Random(requests)
    columns = 11
    c = hf.Pages.empty(layers, pages_, hkv, page, dh, requests, columns, dtype=DT[dtype])
    c.k.zero_()
    c.v.zero_()
    ref = R.Cache(layers, pages_, hkv, page, dh, requests, columns)
    for step in range(40):
        rs = rng.sample(range(requests), rng.randint(1, requests))
        kind = rng.choice(["extend", "extend", "truncate", "fork", "compact"])
        if kind == "extend":
            counts = [rng.choice([0, 1, 3, page, rng.randint(0, 3 * page)]) for _ in rs]
            c.extend(_i32(counts), _i32(rs))
            said = ref.extend(rs, counts)
            assert c.check() == (hf.CallStatus[said] if said else 0), (step, kind)
            if not said and sum(counts):
                ends = [sum(counts[:i]) for i in range(len(rs) + 1)]
                k, v = (_randn((layers, ends[-1], hkv, dh), dtype, step * 2 + s) for s in (0, 1))
                c.write(k.cuda(), v.cuda(), _i32(ends), _i32(rs))
                ref.write(rs, ends, R.to64(k), R.to64(v))
        elif kind == "truncate":
            keep = [rng.choice([0, ref.lens[r], rng.randint(0, ref.lens[r])]) for r in rs]
            c.truncate(_i32(keep), _i32(rs))
            assert ref.truncate(rs, keep) == ""
        elif kind == "fork":
            into = [r for r in rs if ref.lens[r] == 0]
            rest = [r for r in range(requests) if r not in into]
            if not into or not rest:
                continue
            source = [rng.choice(rest) for _ in into]
            c.fork(_i32(source), _i32(into))
            assert ref.fork(source, into) == ""
        else:
            used = torch.zeros(1, dtype=torch.int32, device="cuda")
            c.compact(used)
            assert int(used) == ref.compact()
        assert not c.check()
        _same(c, ref, f"step {step}: {kind}")


def _small(hf):
    c = hf.Pages.empty(2, 6, 2, 8, 16, 4, 3)
    c.k.zero_()
    c.v.zero_()
    ref = R.Cache(2, 6, 2, 8, 16, 4, 3)
    c.extend(_i32([10, 3]), _i32([2, 0]))
    ref.extend([2, 0], [10, 3])
    return c, ref


def test_cache_calls_that_change_nothing(hf):
    c, ref = _small(hf)
    bad, full = hf.CallStatus.BAD, hf.CallStatus.FULL
    for f, args, said in [
            (c.extend, ([1, 1], [2, 2]), bad), (c.extend, ([1], [4]), bad), (c.extend, ([1], [-1]), bad),
            (c.extend, ([1, -1], [2, 0]), bad), (c.extend, ([15], [2]), full), (c.extend, ([16, 16], [1, 3]), full),
            (c.extend, ([2 ** 31 - 1], [2]), full),
            (c.truncate, ([3, 3], [2, 2]), bad), (c.truncate, ([11], [2]), bad), (c.truncate, ([-1], [2]), bad),
            (c.truncate, ([0], [9]), bad),
            (c.fork, ([2, 0], [1, 1]), bad), (c.fork, ([2], [0]), bad), (c.fork, ([4], [1]), bad), (c.fork, ([2], [-1]), bad),
            (c.fork, ([1], [1]), bad), (c.fork, ([2, 1], [1, 3]), bad)]:
        f(_i32(args[0]), _i32(args[1]))
        assert c.check() == said, (f.__name__, args)
        _same(c, ref, f"{f.__name__} {args}")


def test_cache_write_skips_bad_entries(hf):
    c, ref = _small(hf)
    k, v = (_randn((2, 8, 2, 16), "bf16", s) for s in (1, 2))
    for ends, rs in [([0, 4, 8], [2, 2]), ([0, 3, 3], [4, 0]), ([0, 5], [0]), ([0, 9], [2]), ([0, 3], [-1]), ([0, 3], [1])]:
        c.write(k.cuda(), v.cuda(), _i32(ends), _i32(rs))
        assert c.check() == hf.CallStatus.BAD, (ends, rs)
        _same(c, ref, f"write {ends} {rs}")
    # one layer, part of the rows, a good entry beside a bad one
    c.write(k[1].cuda(), v[1].cuda(), _i32([2, 4, 7]), _i32([0, 3]), layer=1)
    assert c.check() == hf.CallStatus.BAD
    ref.write([0], [2, 4], R.to64(k[1:]), R.to64(v[1:]), layer=1)
    _same(c, ref, "write one layer")


# ---------------------------------------------------------------- verification
VERIFY = [  # target, draft, B, S, V, row padding
    ("f32", "f32", 5, 7, 1000, 0), ("bf16", "f32", 4, 7, 5003, 0), ("bf16", "bf16", 3, 4, 257, 3),
    ("f32", "bf16", 2, 16, 33, 1), ("bf16", None, 6, 7, 4099, 0), ("f32", None, 3, 1, 1, 0),
    ("bf16", "f32", 1, 7, 70001, 5), ("f32", "f32", 9, 2, 7, 0),
]


def _verify_inputs(xt, yt, B, S, V, pad, seed):
    g = _gen(seed)
    base = torch.randn((B, S + 1, V + pad), generator=g) * 2.5
    x = base.to(DT[xt])
    y = None if yt is None else (base[:, :S] + 0.5 * torch.randn((B, S, V + pad), generator=g)).to(DT[yt])
    temp = torch.tensor([[1.0, 0.0, 0.7, 1.6][b % 4] for b in range(B)])
    pick = base[:, :S, :V] if y is None else y[..., :V].float()
    gumbel = -torch.log(torch.empty((B, S, V)).exponential_(generator=g))
    hot = torch.where(temp > 0, temp, torch.ones_like(temp))[:, None, None]
    tok = torch.where((temp > 0)[:, None] & (y is not None), (pick / hot + gumbel).argmax(-1), pick.argmax(-1)).int()
    u = torch.rand((B, S), generator=g)
    noise = torch.empty((B, V)).exponential_(generator=g)
    return x, y, tok, u, noise, temp


@pytest.mark.parametrize("xt,yt,B,S,V,pad", VERIFY)
def test_verify(hf, xt, yt, B, S, V, pad):
    seen = set()
    for seed in range(6):
        x, y, tok, u, noise, temp = _verify_inputs(xt, yt, B, S, V, pad, seed)
        nd = torch.tensor([(S, 0, S // 2)[(b + seed) % 3] for b in range(B)], dtype=torch.int32)
        for n_draft in (None, nd):
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            n, tokens = hf.verify_tokens(
                x.cuda()[..., :V], tok.cuda(), u.cuda(), noise.cuda(), draft_logits=None if y is None else y.cuda()[..., :V],
                temperature=temp.cuda(), n_draft=None if n_draft is None else n_draft.cuda(), status=status)
            n, tokens = n.tolist(), tokens.tolist()
            assert int(status) == 0
            for b in range(B):
                a, want, near = R.verify(R.to64(x[b, :, :V]), None if y is None else R.to64(y[b, :, :V]), tok[b].tolist(),
                                         S if n_draft is None else int(nd[b]), u[b].numpy(), R.to64(noise[b]),
                                         float(temp[b].double()))
                assert n[b] == a, (seed, b)
                assert tokens[b] == want or (tokens[b][:a - 1] == want[:a - 1] and tokens[b][a - 1] in near
                                             and tokens[b][a:] == want[a:]), (seed, b)
                seen.add(a)
    assert len(seen) > 1 or V == 1


def test_verify_ties_go_to_the_lowest_token(hf):
    V = 9000
    x = torch.zeros((2, 2, V))
    x[:, :, 5000] = x[:, :, 77] = x[:, :, 8999] = 3.0
    tok = torch.tensor([[77], [5000]], dtype=torch.int32)
    n, t = hf.verify_tokens(x.cuda(), tok.cuda(), torch.zeros(2, 1).cuda(), torch.ones(2, V).cuda(),
                            temperature=torch.zeros(2).cuda())
    assert n.tolist() == [2, 1] and t.tolist() == [[77, 77], [77, -1]]
    # equal scores in the race: equal logits under equal noise
    n, t = hf.verify_tokens(x.cuda(), tok.cuda(), torch.full((2, 1), 0.99).cuda(), torch.ones(2, V).cuda())
    assert n.tolist() == [1, 1] and t.tolist() == [[5000, -1], [77, -1]]


def test_verify_masked_logits_and_bad_requests(hf):
    B, S, V = 9, 3, 3001
    x, y, tok, u, noise, _ = _verify_inputs("f32", "f32", B, S, V, 0, 3)
    temp = torch.ones(B)
    tok[:] = x[:, :S].argmax(-1).int()
    y[:] = x[:, :S]  # p = q: every draft passes, and p - q is nowhere positive
    x[0, :, 1::2] = -float("inf")   # half of the vocabulary masked on the target's side
    x[1, 3] = -float("inf")         # the last row has nothing
    x[2, 1, 9] = float("nan")
    x[3, 0, 9] = float("inf")
    tok[4, 2] = V
    tok[5, 0] = -1
    temp[6] = -0.5
    y[7, 0, 5] = float("nan")
    x[8, 3, 5] = float("nan")       # a row behind the first rejected draft: never read
    u[8, 0] = 0.999
    y[8, 0, int(tok[8, 0])] += 9.0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    n, t = hf.verify_tokens(x.cuda(), tok.cuda(), u.cuda(), noise.cuda(), draft_logits=y.cuda(), temperature=temp.cuda(),
                            status=status)
    n, t = n.tolist(), t.tolist()
    for b in (0, 8):
        a, want, near = R.verify(R.to64(x[b]), R.to64(y[b]), tok[b].tolist(), S, u[b].numpy(), R.to64(noise[b]), 1.0)
        assert n[b] == a and t[b][:a - 1] == want[:a - 1] and t[b][a - 1] in near, b
    for b in range(1, 8):
        assert n[b] == 0 and t[b] == [-1] * (S + 1), b
    assert hf.CallStatus(int(status)) == hf.CallStatus.BAD
    nd = torch.tensor([0, 0, 0, 4, -1, 0, 0, 0, 0], dtype=torch.int32)
    n, t = hf.verify_tokens(x.cuda(), tok.cuda(), u.cuda(), noise.cuda(), n_draft=nd.cuda())
    assert [v > 0 for v in n.tolist()] == [True, True, True, False, False, True, True, True, True]


def test_verify_refuses_rows_that_overlap(hf):
    x = torch.zeros(1, 1, 50, device="cuda")
    tok, u, noise = torch.zeros(3, 1, dtype=torch.int32, device="cuda"), torch.zeros(3, 1, device="cuda"), torch.ones(3, 50, device="cuda")
    with pytest.raises(ValueError):
        hf.verify_tokens(x.expand(3, 2, 50), tok, u, noise)
    with pytest.raises(ValueError):
        hf.verify_tokens(torch.zeros(3, 2, 50, device="cuda"), tok, u, noise, draft_logits=x.expand(3, 1, 50))
    with pytest.raises(hf.HyflashError):
        q = torch.zeros(1, 2, 64, device="cuda").expand(5, 2, 64)
        hf.attention_prompt(q, q, q, _i32([0, 5]))


def test_verify_temperatures_at_the_edges(hf):
    """The smallest T picks the largest logit, the largest one is nearly uniform; a T that is no number is refused."""
    V = 40
    x = torch.randn((5, 2, V), generator=_gen(1))
    tok = x[:, :1].argmax(-1).int()
    temp = torch.tensor([1.2e-38, 3e38, float("inf"), float("nan"), 1e-39])
    noise = torch.ones(5, V)
    noise[1, 7] = 0.5
    n, t = hf.verify_tokens(x.cuda(), tok.cuda(), torch.full((5, 1), 0.5).cuda(), noise.cuda(), temperature=temp.cuda())
    assert n.tolist() == [2, 1, 0, 0, 0]
    assert t[0].tolist() == [int(tok[0]), int(x[0, 1].argmax())]
    assert t[1].tolist() == [7, -1] and (t[2:] == -1).all()


def test_verify_draws_from_the_residual(hf):
    """The next token's frequencies over many requests against w / sum(w), within five deviations."""
    B, V = 20000, 6
    p = torch.tensor([0.05, 0.4, 0.1, 0.2, 0.15, 0.1])
    q = torch.tensor([0.5, 0.1, 0.1, 0.1, 0.1, 0.1])
    g = _gen(2)
    tok = torch.multinomial(q, B, replacement=True, generator=g).int()[:, None]
    n, t = hf.verify_tokens(p.log().expand(B, 2, V).contiguous().cuda(), tok.cuda(), torch.rand((B, 1), generator=g).cuda(),
                            torch.empty((B, V)).exponential_(generator=g).cuda(),
                            draft_logits=q.log().expand(B, 1, V).contiguous().cuda())
    first = np.bincount(t[:, 0].cpu().numpy(), minlength=V) / B
    sd = np.sqrt(p.numpy() * (1 - p.numpy()) / B)
    assert (np.abs(first - p.numpy()) < 5 * sd).all(), first


# ------------------------------------------------------------- all of it together

def test_calls_on_another_stream_and_in_a_graph(hf):
    k, v, table, lens, refs = _shared_cache("bf16", 2, 128, 16, 64, [5, 60, 33], 4)
    q = _randn((3, 8, 8, 128), "bf16", 5).cuda()
    x, y, tok, u, noise, temp = (None if t is None else t.cuda() for t in _verify_inputs("bf16", "f32", 3, 7, 3000, 0, 1))
    pq, pk, pv = (_randn((150, h, 128), "bf16", h).cuda() for h in (8, 2, 2))
    off = _i32([0, 70, 150])
    c = _on_gpu(hf, k, v, table, lens, refs)
    want = (c.attend(q, shared=64), *hf.verify_tokens(x, tok, u, noise, draft_logits=y, temperature=temp),
            hf.attention_prompt(pq, pk, pv, off))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = (c.attend(q, shared=64, stream=s), *hf.verify_tokens(x, tok, u, noise, draft_logits=y, temperature=temp, stream=s),
           hf.attention_prompt(pq, pk, pv, off, stream=s))
    s.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    # captured, replayed twice with other inputs in the same places
    g = torch.cuda.CUDAGraph()
    keep, counts, ends = _i32([lens[0] - 1, lens[1], lens[2] - 3]), _i32([2, 2, 2]), _i32([0, 2, 4, 6])
    new = _randn((1, 6, 2, 128), "bf16", 77).cuda()
    with torch.cuda.graph(g):
        c.truncate(keep)
        c.extend(counts)
        c.write(new, new, ends)
        o = c.attend(q, shared=64)
        n, t = hf.verify_tokens(x, tok, u, noise, draft_logits=y, temperature=temp)
        po = hf.attention_prompt(pq, pk, pv, off)
    for seed in (91, 92):
        q.copy_(_randn((3, 8, 8, 128), "bf16", seed))
        x.copy_(_randn((3, 8, 3000), "bf16", seed, 2.5))
        pq.copy_(_randn((150, 8, 128), "bf16", seed))
        new.copy_(_randn((1, 6, 2, 128), "bf16", seed + 7))
        c.lens.copy_(_i32(lens))
        before = (c.table.clone(), c.refs.clone())
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(n, hf.verify_tokens(x, tok, u, noise, draft_logits=y, temperature=temp)[0])
        assert torch.equal(po, hf.attention_prompt(pq, pk, pv, off))
        assert c.lens.tolist() == [lens[0] + 1, lens[1] + 2, lens[2] - 1]
        w, tol = R.pages(q, c.k[0], c.v[0], c.table.tolist(), c.lens.tolist(), 128 ** -0.5, True)
        R.check_attention(R.to64(o), w, tol)
        c.table.copy_(before[0])
        c.refs.copy_(before[1])
    assert not c.check()


def test_results_repeat_bit_for_bit(hf):
    k, v, table, lens, refs = _shared_cache("bf16", 4, 128, 32, 1024, [500, 60, 33, 1000], 4)
    c = _on_gpu(hf, k, v, table, lens, refs)
    q = _randn((4, 8, 16, 128), "bf16", 5).cuda()
    first = c.attend(q, shared=1024)
    pq, pk, pv = (_randn((900, h, 128), "bf16", h).cuda() for h in (8, 2, 2))
    off = _i32([0, 333, 900])
    pfirst = hf.attention_prompt(pq, pk, pv, off)
    for _ in range(5):
        assert torch.equal(first, c.attend(q, shared=1024))
        assert torch.equal(pfirst, hf.attention_prompt(pq, pk, pv, off))


def test_a_round_of_a_serving_loop(hf):
    """Prompt, cache, fork, draft, verification pass, acceptance, commit: the calls in the order a loop makes
    them, each step against its plain form, the drafter taking n_accepted as it comes."""
    from workload import CONFIGS, make_layer_weights, make_prefix_feats, make_round_inputs
    cfg = CONFIGS["qwen3_4b_bf16"].replace(batch=3, n_q_heads=8, n_kv_heads=2)
    B, S, hq, hkv, dh, page, V = 3, cfg.block, 8, 2, 128, 16, 500
    P = 50  # the common prompt, in request B of the cache
    d = hf.Drafter(cfg, B)
    for l in range(cfg.n_layers):
        d.set_weights(l, make_layer_weights(cfg, l))
    d.prefill(make_prefix_feats(cfg, [P] * B).cuda(), [P] * B)
    c = hf.Pages.empty(1, 40, hkv, page, dh, B + 1, 8)
    ref = R.Cache(1, 40, hkv, page, dh, B + 1, 8)
    c.k.zero_()
    c.v.zero_()
    q, k, v = (_randn((P, h, dh), "bf16", 40 + h) for h in (hq, hkv, hkv))
    o = hf.attention_prompt(q.cuda(), k.cuda(), v.cuda(), _i32([0, P]))
    R.check_attention(R.to64(o), *R.prompt(q, k, v, [0, P], dh ** -0.5, True), "prompt")
    c.extend(_i32([P]), _i32([B]))
    c.write(k[None].cuda(), v[None].cuda(), _i32([0, P]), _i32([B]))
    ref.extend([B], [P])
    ref.write([B], [0, P], R.to64(k[None]), R.to64(v[None]))
    c.fork(_i32([B] * B), _i32(list(range(B))))
    ref.fork([B] * B, list(range(B)))
    shared = P // page * page
    pos = [P] * B
    for rnd in range(3):
        slot, feats = make_round_inputs(cfg, rnd, B)
        d.draft(slot.cuda())
        rows = S + 1
        c.extend(_i32([rows] * B))
        assert ref.extend(list(range(B)), [rows] * B) == ""
        q = _randn((B, rows, hq, dh), "bf16", 60 + rnd)
        k, v = (_randn((1, B * rows, hkv, dh), "bf16", 70 + 2 * rnd + s) for s in (0, 1))
        off = [rows * i for i in range(B + 1)]
        c.write(k.cuda(), v.cuda(), _i32(off))
        ref.write(list(range(B)), off, R.to64(k), R.to64(v))
        _same(c, ref, f"round {rnd}")
        o = c.attend(q.cuda(), shared=shared)
        w, tol = R.pages(q, c.k[0], c.v[0], c.table.tolist(), c.lens.tolist()[:B], dh ** -0.5, True)
        R.check_attention(R.to64(o), w, tol, f"round {rnd}")
        x, y, tok, u, noise, temp = _verify_inputs("bf16", "f32", B, S, V, 0, rnd)
        n, tokens = hf.verify_tokens(x.cuda(), tok.cuda(), u.cuda(), noise.cuda(), draft_logits=y.cuda(), temperature=temp.cuda())
        d.commit(feats.cuda(), n)
        keep = (c.lens[:B] - rows + n).to(torch.int32)
        c.truncate(keep)
        n = n.tolist()
        ref.truncate(list(range(B)), [x - rows + a for x, a in zip(ref.lens, n)])
        pos = [x + a for x, a in zip(pos, n)]
        assert all(1 <= a <= rows for a in n)
        assert c.lens.tolist()[:B] == pos
        d.sync()
        assert d.read(hf.Tensor.POS).tolist() == pos
    used = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.compact(used)
    assert int(used) == ref.compact()
    _same(c, ref, "compacted")
    assert not c.check()
    d.close()
