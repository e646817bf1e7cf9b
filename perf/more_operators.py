"""Rotary positions and the 8-bit cache of the target: cases, plain forms and calls.

Between the target's projections and its attention a serving loop turns queries and keys
by their positions, writes keys and values into the cache, reads back what another kernel
wants as plain rows, and attends over the cache. Here the cache holds e4m3 values with a
scale for each page and KV head. ``run`` computes each step either with elementary torch
operations or, with ``own``, with the library.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
TOP = 448.0  # the largest e4m3 value
LOW, HIGH = -64, 63  # exponents of the scales


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # rotary: one request decodes one token: latency
        {"name": "rotary_step", "op": "rotary", "dtype": "bf16", "hq": 32, "hkv": 8, "dh": 128, "dim": 128,
         "interleaved": False, "scaling": "none", "n": 1, "lo": 1, "hi": 1, "reach": 8192, "shape": 21},
        # rotary: the serving batch verifies 8 rows each, half of the head turned, far positions
        {"name": "rotary_verify", "op": "rotary", "dtype": "bf16", "hq": 40, "hkv": 10, "dh": 128, "dim": 64,
         "interleaved": False, "scaling": "yarn", "n": 64, "lo": 8, "hi": 8, "reach": 131072, "shape": 22},
        # rotary: a prefill batch of mixed lengths, pairs of neighbours
        {"name": "rotary_prompt", "op": "rotary", "dtype": "bf16", "hq": 32, "hkv": 8, "dh": 128, "dim": 128,
         "interleaved": True, "scaling": "bands", "n": 16, "lo": 100, "hi": 8192, "reach": 1, "shape": 23},
        # rotary: the fp32 configuration's heads, prompts of odd lengths
        {"name": "rotary_fp32", "op": "rotary", "dtype": "f32", "hq": 4, "hkv": 2, "dh": 64, "dim": 48,
         "interleaved": True, "scaling": "linear", "n": 3, "lo": 33, "hi": 700, "reach": 32768, "shape": 24},
        # cache: a serving round's rows into three layers, and the pages that they went to read back
        {"name": "store_round", "op": "store", "dtype": "bf16", "hkv": 8, "dh": 128, "layers": 3,
         "n": 64, "rows": 8, "lo": 8, "hi": 4096, "page": 16, "shape": 25},
        # cache: the prompts of a prefill batch into one layer, and read back
        {"name": "store_prompt", "op": "store", "dtype": "bf16", "hkv": 10, "dh": 128, "layers": 1,
         "n": 16, "rows": 0, "lo": 1, "hi": 4096, "page": 64, "shape": 26},
        # cache: a short request of the fp32 configuration read back
        {"name": "load_short", "op": "load", "dtype": "f32", "hkv": 2, "dh": 64, "layers": 1,
         "n": 1, "rows": 0, "lo": 333, "hi": 333, "page": 16, "shape": 27},
        # cache: the prefixes of requests that move to another machine
        {"name": "load_prefixes", "op": "load", "dtype": "bf16", "hkv": 8, "dh": 128, "layers": 3,
         "n": 24, "rows": 0, "lo": 500, "hi": 8192, "page": 32, "shape": 28},
        # attention: one request, one token at a time, nothing shared: latency
        {"name": "attend_single", "op": "attend", "dtype": "bf16", "hq": 32, "hkv": 8, "dh": 128,
         "n": 1, "rows": 1, "shared": 0, "lo": 2048, "hi": 2048, "page": 16, "shape": 29},
        # attention: the serving batch verifying 8 rows each, a system prompt shared by all
        {"name": "attend_serving", "op": "attend", "dtype": "bf16", "hq": 32, "hkv": 8, "dh": 128,
         "n": 64, "rows": 8, "shared": 8192, "lo": 8, "hi": 4096, "page": 32, "shape": 30},
        # attention: the serving batch's prefixes, plain decoding, nothing shared
        {"name": "attend_long", "op": "attend", "dtype": "bf16", "hq": 40, "hkv": 10, "dh": 128,
         "n": 64, "rows": 1, "shared": 0, "lo": 2048, "hi": 32768, "page": 64, "shape": 31},
        # attention: the fp32 configuration's heads, 8 verified rows
        {"name": "attend_fp32", "op": "attend", "dtype": "f32", "hq": 4, "hkv": 2, "dh": 64,
         "n": 8, "rows": 8, "shared": 1024, "lo": 8, "hi": 700, "page": 16, "shape": 32},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "store", "load", "attend", "attend"])
    f32 = rng.random() < 0.25
    hkv, group = (rng.choice([1, 2]), rng.randint(1, 4)) if f32 else (rng.choice([1, 2, 4, 8, 10]), rng.randint(1, 8))
    case = {"op": op, "dtype": "f32" if f32 else "bf16", "hq": hkv * group, "hkv": hkv,
            "dh": 64 if f32 else rng.choice([64, 128]), "shape": rng.randrange(1 << 30)}
    if op == "rotary":
        hi = _log(rng, 1, 2048)
        return {**case, "dim": 2 * rng.randint(4, case["dh"] // 2), "interleaved": rng.random() < 0.5,
                "scaling": rng.choice(["none", "linear", "ntk", "yarn", "bands"]), "n": max(1, min(16, _log(rng, 1, max(2, 8192 // hi)))),
                "lo": rng.choice([1, hi]), "hi": hi, "reach": _log(rng, 1, 1 << 20)}
    if op == "attend":
        return {**case, "n": _log(rng, 1, 8 if f32 else 48), "rows": rng.choice([1, 1, 2, 5, 8]),
                "page": rng.choice([16, 32, 64]), "shared": 64 * rng.randint(0, 16 if f32 else 128),
                "lo": 1, "hi": _log(rng, 8, 700 if f32 else 4096)}
    del case["hq"]
    n = _log(rng, 1, 48)
    return {**case, "layers": rng.randint(1, 3), "n": n, "rows": rng.randint(0, 8) if op == "store" else 0,
            "page": rng.choice([8, 16, 32, 64, 128]), "lo": 1, "hi": _log(rng, 16, 32768 // n)}


def _lengths(case):
    """The case's own lengths, spread over their logarithm: they belong to the case and not to the seed."""
    rng = random.Random(case["shape"])
    return [_log(rng, case["lo"], case["hi"]) for _ in range(case["n"])]


def _layout(case):
    """Lengths and page lists of the requests, the shared pages first, in the order that a pool in use for a
    while has (shuffled), and the pool's size."""
    rng = random.Random(case["shape"] + 1)
    page, shared = case["page"], case.get("shared", 0)
    lens, whole = [shared + r for r in _lengths(case)], shared // page
    counts = [-(-x // page) - whole for x in lens]
    n_pages = whole + sum(counts)
    ids = list(range(n_pages))
    rng.shuffle(ids)
    lists, at = [], whole
    for x in counts:
        lists.append(ids[:whole] + ids[at:at + x])
        at += x
    return lens, lists, n_pages


def _written(case):
    """store: rows of each request that the pass writes, its newest; 0 rows stands for all of a new request."""
    return [min(case["rows"], x) if case["rows"] else x for x in _lengths(case)]


def _read(case):
    """First token of each request that is read back: of the page where its first written row lies, or its first."""
    if case["op"] == "load":
        return [0] * case["n"]
    return [(x - w) // case["page"] * case["page"] for x, w in zip(_lengths(case), _written(case))]


def _ends(counts):
    return [sum(counts[:i]) for i in range(len(counts) + 1)]


SCALING = {  # arguments of each kind, for positions up to 131072 from a target of 32768 (bands: 8192)
    "none": {}, "linear": {"factor": 4.0}, "ntk": {"factor": 4.0},
    "yarn": {"factor": 4.0, "original": 32768}, "bands": {"factor": 8.0, "original": 8192},
}


# ------------------------------------------------------------------- what a program has in hand
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(DTYPES[dtype])


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pool(case, g, n_pages):
    """Values and scales of one of the cache's two pools: heads of different sizes, as layers have them."""
    shape = (case.get("layers", 1), n_pages, case["hkv"], case["page"], case["dh"])
    codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(shape[:3], device="cuda")
    size = torch.exp(0.7 * torch.randn(shape[:1] + (1,) + shape[2:3], generator=g, device="cuda"))
    for i in range(shape[0]):
        x = torch.randn(shape[1:], generator=g, device="cuda") * size[i, :, :, None, None]
        scale[i] = _scale_for(x.abs().amax((-1, -2)))
        codes[i] = (x / scale[i][..., None, None]).to(torch.float8_e4m3fn)
    return codes, scale


def prepare(case, seed):
    g, n, op = _gen(seed), case["n"], case["op"]
    state = {"case": case}
    if op == "rotary":
        lens = _lengths(case)
        rng = random.Random(case["shape"] + 2)
        start = [rng.randrange(case["reach"]) for _ in lens]
        T, hq, hkv, dh = sum(lens), case["hq"], case["hkv"], case["dh"]
        qkv = _normal(g, (T, hq + 2 * hkv, dh), case["dtype"])  # one projection's output: Q | K | V
        state.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], positions=_ints([s + i for s, x in zip(start, lens) for i in range(x)]),
                     q_out=torch.empty((T, hq, dh), dtype=DTYPES[case["dtype"]], device="cuda"),
                     k_out=torch.empty((T, hkv, dh), dtype=DTYPES[case["dtype"]], device="cuda"))
        if own:
            import speculative_decoding_drafter_hf_gb300 as hf
            state["rotary"] = hf.Rotary(dh, dim=case["dim"], interleaved=case["interleaved"], scaling=case["scaling"],
                                        **SCALING[case["scaling"]])
        return state
    lens, lists, n_pages = _layout(case)
    table = torch.full((n, max(map(len, lists))), -1, dtype=torch.int32)
    refs = [0] * n_pages
    for i, pages in enumerate(lists):
        table[i, :len(pages)] = torch.tensor(pages, dtype=torch.int32)
        for x in pages:
            refs[x] += 1
    k, k_scale = _pool(case, g, n_pages)
    v, v_scale = _pool(case, g, n_pages)
    state.update(k=k, v=v, k_scale=k_scale, v_scale=v_scale, table=table.cuda(), lens=_ints(lens), refs=_ints(refs))
    if op == "attend":
        shape = (n, case["rows"], case["hq"], case["dh"])
        state.update(q=_normal(g, shape, case["dtype"]), out=torch.empty(shape, dtype=DTYPES[case["dtype"]], device="cuda"))
    else:
        first = _read(case)
        ends = _ends([x - a for x, a in zip(lens, first)])
        shape = (case["layers"], ends[-1], case["hkv"], case["dh"])
        state.update(first=_ints(first), ends=_ints(ends), k_rows=torch.empty(shape, dtype=DTYPES[case["dtype"]], device="cuda"),
                     v_rows=torch.empty(shape, dtype=DTYPES[case["dtype"]], device="cuda"))
    if op == "store":
        ends = _ends(_written(case))
        shape = (case["layers"], ends[-1], case["hkv"], case["dh"])
        size = torch.exp(0.7 * torch.randn((shape[0], 1, shape[2], 1), generator=g, device="cuda"))
        state.update(offsets=_ints(ends), new_k=_normal(g, shape, "f32", size).to(DTYPES[case["dtype"]]),
                     new_v=_normal(g, shape, "f32", size).to(DTYPES[case["dtype"]]))
    if own:  # what a program keeps between calls: the cache's handle and the attention's workspace
        import speculative_decoding_drafter_hf_gb300 as hf
        state["cache"] = hf.Pages8(k, v, k_scale, v_scale, state["table"], state["lens"], state["refs"],
                                   dtype=DTYPES[case["dtype"]])
        if op == "attend":
            state["workspace"] = state["cache"].attend_workspace(state["q"], case["shared"])
    return state


# ------------------------------------------------------------------- plain forms
def _scale_for(top):
    """The least power of two, of exponent -64 .. 63, that brings the largest value to 448 at most."""
    m, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(top > 0, e, torch.full_like(e, LOW)).clamp(LOW, HIGH)
    return torch.exp2(e.to(top.dtype))


def _frequencies(case):
    """Radians per position of every pair, in 64 bits, and the factor on cosines and sines."""
    d, base, kind, a = case["dim"], 1e6, case["scaling"], SCALING[case["scaling"]]
    if kind == "ntk":
        base *= a["factor"] ** (d / (d - 2))
    i = torch.arange(d // 2, dtype=torch.float64, device="cuda")
    w = base ** (-2 * i / d)
    if kind == "linear":
        w = w / a["factor"]
    if kind == "yarn":  # pairs that turn 32 times and more over the original length stay, below once they slow down
        lo, hi = (d * math.log(a["original"] / (2 * math.pi * b)) / (2 * math.log(base)) for b in (32.0, 1.0))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), d - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        w = w * (1 - ramp) + w / a["factor"] * ramp
    if kind == "bands":  # the same by turns over the original length, between 1 and 4
        t = ((a["original"] * w / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        w = w * t + w / a["factor"] * (1 - t)
    return w, 0.1 * math.log(a["factor"]) + 1 if kind == "yarn" else 1.0


def _turn(x, c, s, case):
    d, y = case["dim"], x.float()
    if case["interleaved"]:
        a, b = y[..., 0:d:2], y[..., 1:d:2]
    else:
        a, b = y[..., :d // 2], y[..., d // 2:d]
    a, b = a * c - b * s, b * c + a * s
    turned = torch.stack((a, b), -1).flatten(-2) if case["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((turned, y[..., d:]), -1).to(x.dtype)


def _plain_rotary(s):
    w, factor = _frequencies(s["case"])
    angle = s["positions"].double()[:, None, None] * w
    c, sn = (torch.cos(angle) * factor).float(), (torch.sin(angle) * factor).float()
    return {"q": _turn(s["q"], c, sn, s["case"]), "k": _turn(s["k"], c, sn, s["case"])}


def _to_codes(x, scale):
    return (x / scale).clamp(-TOP, TOP).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_write(s):
    page, lens, ends = s["k"].shape[3], s["lens"].long(), s["offsets"].long()
    t = torch.arange(s["new_k"].shape[1], device=lens.device)
    i = torch.bucketize(t, ends[1:], right=True)
    at = lens[i] - ends[i + 1] + t
    where, row = s["table"][i, at // page].long(), at % page
    ids, block = torch.unique(where, return_inverse=True)
    first = torch.full((len(ids),), page, device=t.device).scatter_reduce(0, block, row, "amin")
    kept = torch.arange(page, device=t.device)[None, :] < first[:, None]
    for codes, scale, new in ((s["k"], s["k_scale"], s["new_k"]), (s["v"], s["v_scale"], s["new_v"])):
        new = new.float()
        top = torch.zeros((new.shape[0], len(ids), new.shape[2]), device=t.device)
        top.index_reduce_(1, block, new.abs().amax(-1), "amax")
        old = scale[:, ids]
        now = torch.maximum(_scale_for(top), torch.where(first[:, None] > 0, old, torch.zeros_like(old)))
        scale[:, ids] = now
        raw = codes.view(torch.uint8)
        was = raw[:, ids]
        again = _to_codes(was.view(torch.float8_e4m3fn).float() * old[..., None, None], now[..., None, None])
        raw[:, ids] = torch.where(kept[None, :, None, :, None], again, was)
        raw[:, where, :, row] = _to_codes(new, now[:, block][..., None]).transpose(0, 1)


def _plain_read(s):
    page, ends = s["k"].shape[3], s["ends"].long()
    t = torch.arange(s["k_rows"].shape[1], device=ends.device)
    i = torch.bucketize(t, ends[1:], right=True)
    at = s["first"].long()[i] + t - ends[i]
    where, row = s["table"][i, at // page].long(), at % page
    out = []
    for codes, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
        x = codes.view(torch.uint8)[:, where, :, row].transpose(0, 1).contiguous().view(torch.float8_e4m3fn)
        out.append((x.float() * scale[:, where][..., None]).to(s["k_rows"].dtype))
    return out


def _plain_attend(s):
    q, table, lens = s["q"], s["table"].long().clamp(min=0), s["lens"].long()
    n, rows, hq, dh = q.shape
    hkv, page = s["k"].shape[2], s["k"].shape[3]
    L = table.shape[1] * page

    def pool(codes, scale):
        x = codes.view(torch.uint8)[0][table].view(torch.float8_e4m3fn).float()
        return x.mul_(scale[0][table][..., None, None]).permute(0, 2, 1, 3, 4).reshape(n, hkv, L, dh)

    x = q.float().view(n, rows, hkv, hq // hkv, dh).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, dh)
    p = torch.matmul(x * dh ** -0.5, pool(s["k"], s["k_scale"]).transpose(2, 3)).view(n, hkv, hq // hkv, rows, L)
    last = lens[:, None] - rows + torch.arange(rows, device=q.device)
    seen = (torch.arange(L, device=q.device) <= last[:, :, None])[:, None, None]
    p.masked_fill_(~seen, -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total > 0, total, torch.ones_like(total)))
    o = torch.matmul(p.view(n, hkv, -1, L), pool(s["v"], s["v_scale"])).view(n, hkv, hq // hkv, rows, dh)
    return o.permute(0, 3, 1, 2, 4).reshape(n, rows, hq, dh).to(q.dtype)


# ------------------------------------------------------------------- one pass
def run(state):
    s, op = state, state["case"]["op"]
    if op == "rotary":
        if not own:
            return _plain_rotary(s)
        q, k = s["rotary"](s["q"], s["k"], s["positions"], q_out=s["q_out"], k_out=s["k_out"])
        return {"q": q, "k": k}
    if op == "attend":
        if not own:
            return _plain_attend(s)
        return s["cache"].attend(s["q"], shared=s["case"]["shared"], out=s["out"], workspace=s["workspace"])
    if op == "store":
        if not own:
            _plain_write(s)
        else:
            s["cache"].write(s["new_k"], s["new_v"], s["offsets"])
    if not own:
        k, v = _plain_read(s)
    else:
        k, v = s["cache"].read(s["first"], s["ends"], k=s["k_rows"], v=s["v_rows"])
    if op == "load":
        return {"k": k, "v": v}
    return {"k": k, "v": v, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


# ------------------------------------------------------------------- what a pass cannot do without
def work(case):
    size, n = DTYPES[case["dtype"]].itemsize, case["n"]
    if case["op"] == "rotary":
        rows = sum(_lengths(case))
        return {"bytes": 2 * rows * (case["hq"] + case["hkv"]) * case["dh"] * size + 4 * rows,
                "flops": 3 * rows * (case["hq"] + case["hkv"]) * case["dim"]}
    lens = _layout(case)[0]
    row = 2 * case["hkv"] * case["dh"]  # values of one token, and bytes of them in the cache
    page_scales = 8 * case["hkv"]
    if case["op"] == "attend":
        pages = case["shared"] // case["page"] + sum(-(-x // case["page"]) - case["shared"] // case["page"] for x in lens)
        seen = sum(max(0, x - case["rows"] + r + 1) for x in lens for r in range(case["rows"]))
        return {"bytes": 2 * n * case["rows"] * case["hq"] * case["dh"] * size + page_scales * pages
                + row * (case["shared"] + sum(x - case["shared"] for x in lens)),
                "flops": 4 * case["hq"] * case["dh"] * seen}
    read = sum(x - a for x, a in zip(lens, _read(case)))
    moved = read * row * (1 + size) + page_scales * read // case["page"]
    if case["op"] == "store":
        moved += sum(_written(case)) * row * (1 + size) + page_scales * read // case["page"]
    return {"bytes": moved * case["layers"], "flops": read * row * case["layers"]}


# ------------------------------------------------------------------- from the definitions, in 64 bits
def _held(x, scale):
    """The e4m3 value nearest to x / scale, ties to the even one, times scale."""
    y = x.double() / scale
    size = y.abs().clamp(max=TOP)
    step = torch.exp2(torch.floor(torch.log2(size.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign(torch.round(size / step) * step, y) * scale


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        d, a, kind = case["dim"], SCALING[case["scaling"]], case["scaling"]
        base = 1e6 * (a["factor"] ** (d / (d - 2)) if kind == "ntk" else 1.0)
        out = {"q": s["q"].double(), "k": s["k"].double()}
        pos = s["positions"].double()[:, None]
        src = {x: out[x].clone() for x in out}
        for i in range(d // 2):
            w, size = base ** (-2.0 * i / d), 1.0
            if kind == "linear":
                w /= a["factor"]
            elif kind == "yarn":
                edge = [d * math.log(a["original"] / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (32, 1)]
                lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), d - 1)
                slow = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
                w, size = w * (1.0 - slow + slow / a["factor"]), 1.0 + 0.1 * math.log(a["factor"])
            elif kind == "bands":
                fast = min(max((a["original"] * w / (2 * math.pi) - 1) / 3, 0.0), 1.0)
                w *= fast + (1.0 - fast) / a["factor"]
            j0, j1 = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + d // 2)
            cos, sin = torch.cos(pos * w) * size, torch.sin(pos * w) * size
            for x in out:
                out[x][..., j0] = src[x][..., j0] * cos - src[x][..., j1] * sin
                out[x][..., j1] = src[x][..., j1] * cos + src[x][..., j0] * sin
        return out
    page, lens, table = case["page"], s["lens"].tolist(), s["table"].long()
    if case["op"] == "attend":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b, length in enumerate(lens):
            ids = table[b, :-(-length // page)]
            k, v = ((s[x][0].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * s[x + "_scale"][0][ids].double()[..., None, None])
                    .transpose(0, 1).flatten(1, 2)[:, :length] for x in ("k", "v"))
            for r in range(case["rows"]):
                m = length - case["rows"] + r + 1
                if m > 0:
                    q = s["q"][b, r].double().view(case["hkv"], -1, case["dh"])
                    z = torch.exp((q @ k[:, :m].transpose(1, 2)) / math.sqrt(case["dh"]))
                    out[b, r] = ((z @ v[:, :m]) / z.sum(-1, keepdim=True)).flatten(0, 1)
        return out
    got = {x + "_scale": s[x + "_scale"].double() for x in ("k", "v")} if case["op"] == "store" else {}
    for x in ("k", "v"):
        values = s[x].float().double() * s[x + "_scale"].double()[..., None, None]
        if case["op"] == "store":
            ends, t = s["offsets"].tolist(), 0
            for b, length in enumerate(lens):
                at = length - (ends[b + 1] - ends[b])
                while at < length:  # page by page
                    r0, count = at % page, min(page - at % page, length - at)
                    i = int(table[b, at // page])
                    new = s["new_" + x][:, t:t + count].double().transpose(1, 2)
                    top = new.abs().amax((2, 3))
                    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / TOP))
                    e = torch.where(top <= TOP * torch.exp2(e - 1), e - 1, e)  # (a logarithm rounded up)
                    scale = torch.exp2(e.clamp(LOW, HIGH))
                    if r0:
                        scale = torch.maximum(scale, got[x + "_scale"][:, i])
                        values[:, i, :, :r0] = _held(values[:, i, :, :r0], scale[..., None, None])
                    values[:, i, :, r0:r0 + count] = _held(new, scale[..., None, None])
                    got[x + "_scale"][:, i] = scale
                    at, t = at + count, t + count
        rows = []
        for b, first in enumerate(_read(case)):
            at = torch.arange(first, lens[b], device="cuda")
            rows.append(values[:, table[b, at // page], :, at % page].transpose(0, 1))
        got[x] = torch.cat(rows, 1)
    return got
