"""Rules of the target-side calls at their edges, on the GPU."""
import random

import numpy as np
import pytest
import torch

import _target_ref as R
import test_gpu_target as T
from test_gpu_target import DT, _gen, _i32, _on_gpu, _randn, _same, _shared_cache, _small, hf  # noqa: F401 (hf is a fixture)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- verification
@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("V,pad", [(9, 0), (3001, 0), (70001, 5)])
def test_greedy_rows_without_a_largest_logit_are_refused(hf, xt, V, pad):
    """T = 0: NaN, +infinity or nothing above -infinity in a row that is read refuses the request, wherever
    in the row it stands; in a row that is not read it does not matter."""
    B, S, nan, inf = 11, 3, float("nan"), float("inf")
    x = (torch.randn((B, S + 1, V + pad), generator=_gen(V)) * 2.5).to(DT[xt])
    x[9, :, ::2] = -inf  # masked tokens are no fault
    tok = x[:, :S, :V].float().argmax(-1).int()
    x[1, 0, 0] = nan
    x[2, 1, V - 1] = nan
    x[3, 3, V // 2] = nan  # the row of the next token
    x[4, 0, V // 3] = inf
    x[5, 2, V - 2] = inf
    x[6, 1] = -inf
    tok[7, 0] = (tok[7, 0] + 1) % V  # not the largest: the rows behind are not read
    x[7, 1, 0], x[7, 2], x[7, 3, 1] = nan, -inf, inf
    tok[8, 1] = (tok[8, 1] + 1) % V
    x[8, 1, 5] = nan
    x[10, 3, 0] = nan  # behind the drafts: n_draft is 2
    nd = torch.full((B,), S, dtype=torch.int32)
    nd[10] = 2
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    n, t = hf.verify_tokens(x.cuda()[..., :V], tok.cuda(), torch.zeros(B, S).cuda(), torch.ones(B, V).cuda(),
                            temperature=torch.zeros(B).cuda(), n_draft=nd.cuda(), status=status)
    n, t = n.tolist(), t.tolist()
    assert hf.CallStatus(int(status)) == hf.CallStatus.BAD
    for b in range(B):
        if b in (0, 7, 9, 10):
            a, want, _ = R.verify(R.to64(x[b, :, :V]), None, tok[b].tolist(), int(nd[b]), [0.0] * S, np.ones(V), 0.0)
            assert (n[b], t[b]) == (a, want), b
        else:
            assert (n[b], t[b]) == (0, [-1] * (S + 1)), b


def test_drafts_whose_probabilities_are_below_the_smallest_float(hf):
    """u q < p by the formula, not by numbers that have become zero."""
    V, inf = 50, float("inf")
    rows = [  # x(d), y(d), T, u, accepted
        (-300.0, -300.0, 1.0, 0.0, True), (-300.0, -310.0, 1.0, 0.5, True), (-300.0, -290.0, 1.0, 0.5, False),
        (-300.0, -inf, 1.0, 0.5, True), (-inf, -300.0, 1.0, 0.0, False), (-1.0, -1.0, 0.002, 0.0, True),
        (-1.0, -1.1, 0.002, 0.99, True), (-1.0, -0.9, 0.002, 0.01, False), (-300.0, -300.5, 1.0, 0.999, True),
        (-300.0, -299.5, 1.0, 0.7, False), (-300.0, -299.5, 1.0, 0.5, True), (-90.0, -inf, 1.0, 0.0, True),
        (-inf, -inf, 1.0, 0.0, False), (-1.0, -2.0, 1.0, 0.9, True), (-3.0, -1.0, 1.0, 0.9, False)]
    B = len(rows)
    x, y = torch.full((B, 2, V), -1000.0), torch.full((B, 1, V), -1000.0)
    x[:, :, 0] = y[:, :, 0] = 0.0
    for b, (xd, yd, *_) in enumerate(rows):
        x[b, 0, 1], y[b, 0, 1] = xd, yd
    tok = torch.ones((B, 1), dtype=torch.int32)
    u, temp = torch.tensor([[r[3]] for r in rows]), torch.tensor([r[2] for r in rows])
    n, _ = hf.verify_tokens(x.cuda(), tok.cuda(), u.cuda(), torch.ones(B, V).cuda(), draft_logits=y.cuda(), temperature=temp.cuda())
    assert [v == 2 for v in n.tolist()] == [r[4] for r in rows]
    # drafts chosen greedily: q = 1
    n, _ = hf.verify_tokens(x.cuda(), tok.cuda(), torch.zeros(B, 1).cuda(), torch.ones(B, V).cuda(), temperature=temp.cuda())
    assert [v == 2 for v in n.tolist()] == [r[0] > -inf for r in rows]


# ----------------------------------------------------------------- page tables
def test_write_bounds(hf):
    """Bounds that decrease: nothing is written. Bounds out of range: the rows of their entries are skipped."""
    c, ref = _small(hf)
    bad = hf.CallStatus.BAD
    k, v = (_randn((2, 8, 2, 16), "bf16", s) for s in (1, 2))
    for ends, rs in [([0, 8, 4], [2, 0]), ([0, 4, 2, 5], [2, 0, 1]), ([3, 0], [2]), ([5, 3, 4], [2, 0]), ([-2, 3], [2]),
                     ([0, 9], [2])]:
        c.write(k.cuda(), v.cuda(), _i32(ends), _i32(rs))
        assert c.check() == bad, ends
        _same(c, ref, f"write {ends}")
    for ends, rs, first in [([0, 4, 9], [2, 0], 4), ([2, 8, 9], [2, 0], 8)]:
        c.write(k.cuda(), v.cuda(), _i32(ends), _i32(rs))
        assert c.check() == bad, ends
        ref.write([2], [ends[0], first], R.to64(k), R.to64(v))
        _same(c, ref, f"write {ends}")
    c.write(k.cuda(), v.cuda(), _i32([1, 3]), _i32([0]))  # rows before and behind the entries are nobody's
    assert not c.check()
    ref.write([0], [1, 3], R.to64(k), R.to64(v))
    _same(c, ref, "write some rows")


def test_write_takes_the_strides_that_it_says(hf):
    """Rows and layers with strides of their own; K that is the same in every layer, beside V that is not."""
    c, ref = _small(hf)
    x = _randn((2, 8, 7, 16), "bf16", 3)  # one projection's output: K and V are heads of its rows
    d = x.cuda()
    c.write(d[:, 1:5, 3:5], d[:, 1:5, 5:7], _i32([0, 4]), _i32([2]))
    ref.write([2], [0, 4], R.to64(x[:, 1:5, 3:5]), R.to64(x[:, 1:5, 5:7]))
    _same(c, ref, "parts of a projection")
    both = d[:1, :6, :2].expand(2, 6, 2, 16)
    c.write(both, both, _i32([0, 6]), _i32([2]))
    ref.write([2], [0, 6], R.to64(both), R.to64(both))
    _same(c, ref, "the same rows in every layer")
    with pytest.raises(ValueError):
        c.write(both, d[:, :6, :2], _i32([0, 6]), _i32([2]))
    _same(c, ref, "refused")
    assert not c.check()


def test_a_new_cache_is_ready_on_every_stream(hf):
    """The cache's own buffers are set up when the constructor returns, whatever the current stream still has to do."""
    _small(hf)[0].truncate(_i32([3]))  # (a kernel's first launch may wait for the whole device)
    parts = [torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((1, 6, 1, 8, 8),) * 2]
    table, lens, refs = _i32([[0, 1], [2, -1]]), _i32([9, 3]), _i32([1, 1, 1, 0, 0, 0])
    keep = _i32([2, 3])
    used = [torch.full((64,), 77, dtype=torch.int32, device="cuda") for _ in range(20000)]
    torch.cuda.synchronize()
    del used  # (what the cache's scratch finds in its memory)
    s = torch.cuda.Stream()
    torch.cuda._sleep(200_000_000)
    c = hf.Pages(*parts, table, lens, refs)
    c.truncate(keep, stream=s)
    s.synchronize()
    with torch.cuda.stream(s):
        got = lens.tolist(), table.tolist(), refs.tolist()
    torch.cuda.synchronize()
    assert got == ([2, 3], [[0, -1], [2, -1]], [1, 0, 1, 0, 0, 0])
    assert not c.check()


def test_check_waits_for_every_stream(hf):
    c, _ = _small(hf)
    c.truncate(_i32([3]))  # (its first launch may wait for the whole device)
    s = torch.cuda.Stream()
    keep = _i32([11])
    req = _i32([2])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    c.truncate(keep, req, stream=s)
    assert c.check() == hf.CallStatus.BAD
    torch.cuda.synchronize()
    assert not c.check()


def test_a_cache_of_4096_requests(hf):
    """Lists at their longest: more free pages taken at once than a CTA holds near, copies for all, every request cut."""
    n, n_pages, page = 4096, 21000, 8
    rng = random.Random(1)
    c = hf.Pages.empty(1, n_pages, 1, page, 8, n, 4)
    c.k.zero_()
    c.v.zero_()
    ref = R.Cache(1, n_pages, 1, page, 8, n, 4)

    def extend_and_write(rs, counts, seed):
        c.extend(_i32(counts), _i32(rs))
        assert ref.extend(rs, counts) == "" and not c.check()
        ends = np.concatenate([[0], np.cumsum(counts)]).tolist()
        k, v = (_randn((1, ends[-1], 1, 8), "bf16", seed + s) for s in (0, 1))
        c.write(k.cuda(), v.cuda(), _i32(ends), _i32(rs))
        assert not c.check()
        ref.write(rs, ends, R.to64(k), R.to64(v))

    rs = rng.sample(range(n), 3000)
    extend_and_write(rs, [rng.randint(0, 17) for _ in rs], 1)
    _same(c, ref, "extended")
    into = [r for r in range(n) if ref.lens[r] == 0]
    source = [rng.choice(sorted(set(range(n)) - set(into))) for _ in into]
    c.fork(_i32(source), _i32(into))
    assert ref.fork(source, into) == "" and not c.check()
    _same(c, ref, "forked")
    rs = rng.sample(range(n), n)
    extend_and_write(rs, [rng.randint(0, 9) for _ in rs], 3)
    _same(c, ref, "all extended")
    keep = [rng.randint(0, x) for x in ref.lens]
    c.truncate(_i32(keep))
    assert ref.truncate(list(range(n)), keep) == "" and not c.check()
    _same(c, ref, "all cut")
    used = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.compact(used)
    assert int(used) == ref.compact() and not c.check()
    _same(c, ref, "compacted")
    c.truncate(_i32([0] * n))
    ref.truncate(list(range(n)), [0] * n)
    _same(c, ref, "empty")


# ------------------------------------------------------------------- attention
@pytest.mark.parametrize("n,shared", [(3, 64), (3, 0), (300, 64)])
def test_waits_that_run_out_are_reported(hf, n, shared):
    """With a limit of 0 every wait gives up: the status says so, nothing is read outside the buffers whatever the
    workspace held, and the next call is right."""
    from speculative_decoding_drafter_hf_gb300 import _binding as B
    k, v, table, lens, refs = _shared_cache("bf16", 2, 128, 16, 64, [5, 60, 33], 4)
    c = _on_gpu(hf, k, v, table, lens, refs)
    req = [i % 3 for i in range(n)]
    q = _randn((n, 2, 8, 128), "bf16", 5)
    d, list_ = q.cuda(), _i32(req)
    ws = c.attend_workspace(d, shared)
    p = [_randn((90, h, 128), "bf16", h) for h in (8, 2, 2)]
    dp, off = [t.cuda() for t in p], _i32([0, 40, 90])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for fill in (0, 0x7f, 0xff):
        ws.fill_(fill)
        try:
            assert B.hf_debug_set_wait_limit(None, 0) == 0
            o = c.attend(d, list_, shared=shared, workspace=ws)
            hf.attention_prompt(*dp, off, status=status)
            torch.cuda.synchronize()
        finally:
            B.hf_debug_set_wait_limit(None, -1)
        assert c.check() == hf.CallStatus.TIMEOUT and int(status) == hf.CallStatus.TIMEOUT
        assert n > 256 or (o == 0).all()
        status.zero_()
    want, tol = R.pages(q, k[0], v[0], table, lens, 128 ** -0.5, True, req)
    R.check_attention(R.to64(c.attend(d, list_, shared=shared, workspace=ws)), want, tol)
    want, tol = R.prompt(*p, [0, 40, 90], 128 ** -0.5, True)
    R.check_attention(R.to64(hf.attention_prompt(*dp, off, status=status)), want, tol)
    assert not c.check() and int(status) == 0


@pytest.mark.parametrize("dtype,hq,hkv,dh,page,rows,shared,own", [
    ("f32", 16, 2, 64, 16, 8, 64, [0, 1, 8, 30, 300, None]), ("f32", 8, 1, 64, 16, 5, 0, [3, 200]),
    ("bf16", 8, 1, 32, 32, 8, 32, [40, 7])])
def test_attend_more_than_32_rows_of_a_kv_head_on_cuda_cores(hf, dtype, hq, hkv, dh, page, rows, shared, own):
    T.test_attend(hf, dtype, hq, hkv, dh, page, rows, shared, own)


@pytest.mark.parametrize("dtype,hq,hkv,dh,lens", [
    ("f32", 4, 2, 80, [1, 70, 33]), ("f32", 3, 1, 120, [65, 2]), ("f32", 4, 1, 128, [130, 1]), ("f32", 2, 2, 200, [40]),
    ("bf16", 4, 2, 96, [90, 3]), ("bf16", 5, 1, 112, [33, 70]), ("bf16", 2, 1, 72, [0, 129]), ("bf16", 2, 2, 136, [66])])
def test_prompt_head_dims_between(hf, dtype, hq, hkv, dh, lens):
    T.test_prompt(hf, dtype, hq, hkv, dh, lens)


@pytest.mark.parametrize("dtype,hq,hkv,dh,page,rows,shared,own", [
    ("f32", 4, 2, 80, 16, 8, 64, [0, 30, 300, None]), ("f32", 3, 1, 120, 8, 1, 0, [1, 77]),
    ("f32", 4, 2, 128, 32, 16, 32, [20, 100]), ("bf16", 4, 2, 96, 16, 8, 64, [5, 200, None]),
    ("bf16", 6, 2, 112, 64, 3, 0, [64, 130]), ("bf16", 2, 1, 72, 16, 1, 32, [1, 90])])
def test_attend_head_dims_between(hf, dtype, hq, hkv, dh, page, rows, shared, own):
    T.test_attend(hf, dtype, hq, hkv, dh, page, rows, shared, own)


def _in_rows(x, pad, fill=0.0):
    """x [rows, heads, dh] on the GPU as part of rows that are `pad` elements longer, 16 bytes into them."""
    rows, heads, dh = x.shape
    first = 16 // x.element_size()
    buf = torch.full((rows, heads * dh + pad), fill, dtype=x.dtype, device="cuda")
    part = buf[:, first:first + heads * dh].unflatten(1, (heads, dh))
    part.copy_(x)
    return buf, part


@pytest.mark.parametrize("dtype,dh", [("bf16", 128), ("bf16", 64), ("bf16", 96), ("f32", 64)])
def test_rows_that_start_on_16_bytes_only(hf, dtype, dh):
    """Row strides that are a multiple of 16 bytes and of nothing more, out's too; what lies beside stays."""
    pad = 24 if dtype == "bf16" else 12
    x = [_randn((150, h, dh), dtype, h) for h in (8, 2, 2)]
    q, k, v = (_in_rows(t, pad)[1] for t in x)
    buf, out = _in_rows(torch.zeros(150, 8, dh, dtype=DT[dtype]), pad, 7.0)
    assert out.data_ptr() % 32 == 16 and out.stride(0) * out.element_size() % 32 == 16
    hf.attention_prompt(q, k, v, _i32([0, 20, 150]), out=out)
    want, tol = R.prompt(*x, [0, 20, 150], dh ** -0.5, dtype == "bf16")
    R.check_attention(R.to64(out), want, tol)
    out.fill_(7.0)
    assert (buf == 7.0).all()
    pk, pv, table, lens, refs = _shared_cache(dtype, 2, dh, 16, 32, [5, 60, 33], 4)
    c = _on_gpu(hf, pk, pv, table, lens, refs)
    y = _randn((3, 4, 8, dh), dtype, 9)
    q = _in_rows(y.flatten(0, 1), pad)[1].unflatten(0, (3, 4))
    want, tol = R.pages(y, pk[0], pv[0], table, lens, dh ** -0.5, dtype == "bf16")
    for shared in (0, 32):
        c.attend(q, shared=shared, out=out[:12].unflatten(0, (3, 4)))
        R.check_attention(R.to64(out[:12].unflatten(0, (3, 4))), want, tol)
        out.fill_(7.0)
        assert (buf == 7.0).all()
    assert not c.check()


@pytest.mark.parametrize("hq,hkv,dh", [(33, 1, 64), (86, 2, 128), (63, 3, 64)])
def test_groups_that_do_not_divide_a_tile(hf, hq, hkv, dh):
    T.test_prompt(hf, "bf16", hq, hkv, dh, [1, 9, 20])
    T.test_attend(hf, "bf16", hq, hkv, dh, 16, 5, 32, [0, 3, 140, None])


def test_calls_without_anything_to_do(hf):
    c = hf.Pages.empty(1, 4, 2, 16, 64, 2, 2)
    q = torch.zeros(0, 3, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert c.attend(q, _i32([])).shape == q.shape
    c.extend(_i32([]), _i32([]))
    c.write(torch.zeros(1, 0, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 0, 2, 64, dtype=torch.bfloat16, device="cuda"),
            _i32([0, 0]), _i32([1]))
    p = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert hf.attention_prompt(p, p, p, _i32([0])).shape == p.shape
    assert hf.attention_prompt(p, p, p, _i32([0, 0])).shape == p.shape
    n, t = hf.verify_tokens(torch.zeros(0, 4, 9, device="cuda"), torch.zeros(0, 3, dtype=torch.int32, device="cuda"),
                            torch.zeros(0, 3, device="cuda"), torch.zeros(0, 9, device="cuda"))
    assert n.shape == (0,) and t.shape == (0, 4)
    assert not c.check()


def test_two_streams_at_once_and_graphs_that_share_a_workspace(hf):
    """Calls on two streams, each with its own workspace, and two graphs replayed one after the other with one."""
    k, v, table, lens, refs = _shared_cache("bf16", 4, 128, 16, 512, [500, 60, 33, 1000], 4)
    c = _on_gpu(hf, k, v, table, lens, refs)
    qs = [_randn((4, r, 16, 128), "bf16", r).cuda() for r in (8, 3)]
    p = [_randn((900, h, 128), "bf16", h).cuda() for h in (8, 2, 2)]
    off = _i32([0, 333, 900])
    x = (torch.randn((3, 8, 9000), generator=_gen(1)) * 2.5).cuda()
    tok, u, noise = x[:, :7].argmax(-1).int(), torch.full((3, 7), 0.5, device="cuda"), torch.ones(3, 9000, device="cuda")

    def calls(i, stream=None):
        return (c.attend(qs[i], shared=512 * i, stream=stream), hf.attention_prompt(*p, off, stream=stream),
                *hf.verify_tokens(x, tok, u, noise, stream=stream))

    want = [calls(0), calls(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        got = [calls(i, s) for i, s in enumerate(streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
    ws = torch.empty(max(c.attend_workspace(q, 0).numel() + c.attend_workspace(q, 512).numel() for q in qs),
                     dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.attend(qs[i], shared=512 * i, workspace=ws))
        graphs.append(g)
    for i in (0, 1, 1, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        graphs[1 - i].replay()
        assert torch.equal(outs[i], want[i][0]) and torch.equal(outs[1 - i], want[1 - i][0])
    assert not c.check()


def test_calls_one_behind_the_other_without_a_wait(hf):
    """Every call of a round in one stream, many rounds, no synchronisation between: each sees what the one before
    left (lengths, tables, rows, drafts), as its copy made between synchronised calls does."""
    rng = random.Random(3)
    n, rows, page = 6, 4, 16

    def rounds(wait):
        c = hf.Pages.empty(1, 120, 2, page, 128, n, 20)
        c.k.zero_()
        c.v.zero_()
        got = []
        for r in range(12):
            c.extend(counts[r])
            wait()
            c.write(*new[r], ends)
            wait()
            got.append(c.attend(q[r]))
            wait()
            got += hf.verify_tokens(x[r], tok[r], u, noise)
            wait()
            c.truncate((c.lens - rows + got[-2]).to(torch.int32))
            wait()
            if r % 4 == 3:
                c.compact()
                wait()
        assert not c.check()
        return got + [c.lens, c.table, c.refs]

    counts = [_i32([rows] * n) for _ in range(12)]
    ends = _i32([rows * i for i in range(n + 1)])
    new = [[_randn((1, n * rows, 2, 128), "bf16", 10 * r + s).cuda() for s in (1, 2)] for r in range(12)]
    q = [_randn((n, rows, 8, 128), "bf16", 50 + r).cuda() for r in range(12)]
    x = [(torch.randn((n, rows, 500), generator=_gen(r)) * 2).cuda() for r in range(12)]
    tok = [t[:, :rows - 1].argmax(-1).int() for t in x]
    u = torch.tensor([[rng.random() for _ in range(rows - 1)] for _ in range(n)]).cuda()
    noise = torch.empty((n, 500)).exponential_(generator=_gen(9)).cuda()
    want = rounds(torch.cuda.synchronize)
    for _ in range(5):
        got = rounds(lambda: None)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
