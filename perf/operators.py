"""The target model's half of a speculative round: cases, plain forms and calls.

Between hf_draft and hf_commit a serving loop runs the target over the drafted
tokens: attention over the prompts when a request arrives, attention of the
verified rows over a paged cache whose requests share a prefix, acceptance of
the drafted tokens, and the cache's page tables. ``run`` computes each of them
either with elementary torch operations or, with ``own``, with the library.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # prompts: the first tokens of a chat, three short requests at once
        {"name": "prompt_short", "op": "prompt", "dtype": "bf16", "hq": 32, "hkv": 8, "dh": 128,
         "n": 3, "lo": 1, "hi": 64, "shape": 1},
        # prompts: a prefill batch of mixed lengths, odd sizes, one-token prompts among them
        {"name": "prompt_ragged", "op": "prompt", "dtype": "bf16", "hq": 40, "hkv": 10, "dh": 128,
         "n": 16, "lo": 1, "hi": 2048, "shape": 2},
        # prompts: one long document, the repository's single-request prefix
        {"name": "prompt_long", "op": "prompt", "dtype": "bf16", "hq": 32, "hkv": 8, "dh": 128,
         "n": 1, "lo": 8192, "hi": 8192, "shape": 3},
        # prompts: the fp32 configuration's heads, for comparisons against another framework
        {"name": "prompt_fp32", "op": "prompt", "dtype": "f32", "hq": 4, "hkv": 2, "dh": 64,
         "n": 8, "lo": 100, "hi": 1500, "shape": 4},
        # cache: one request, one token at a time, nothing shared: latency
        {"name": "pages_single", "op": "attend", "dtype": "bf16", "hq": 32, "hkv": 8, "dh": 128,
         "n": 1, "rows": 1, "shared": 0, "lo": 2048, "hi": 2048, "page": 16, "shape": 5},
        # cache: the serving batch verifying 8 rows each, a system prompt shared by all
        {"name": "pages_serving", "op": "attend", "dtype": "bf16", "hq": 32, "hkv": 8, "dh": 128,
         "n": 64, "rows": 8, "shared": 8192, "lo": 8, "hi": 4096, "page": 32, "shape": 6},
        # cache: 24 readers of one long document, plain decoding
        {"name": "pages_document", "op": "attend", "dtype": "bf16", "hq": 40, "hkv": 10, "dh": 128,
         "n": 24, "rows": 1, "shared": 32768, "lo": 1, "hi": 1000, "page": 64, "shape": 7},
        # cache: the fp32 configuration's heads, 8 verified rows
        {"name": "pages_fp32", "op": "attend", "dtype": "f32", "hq": 4, "hkv": 2, "dh": 64,
         "n": 8, "rows": 8, "shared": 1024, "lo": 8, "hi": 700, "page": 16, "shape": 8},
        # verification: one request, fp32 logits on both sides: latency
        {"name": "verify_single", "op": "verify", "dtype": "f32", "n": 1, "slots": 7, "vocab": 151936,
         "drafts": True, "shape": 9},
        # verification: the serving batch, bf16 target logits, sampled drafts
        {"name": "verify_serving", "op": "verify", "dtype": "bf16", "n": 64, "slots": 7, "vocab": 100352,
         "drafts": True, "shape": 10},
        # page tables: a serving round (new requests forked from the prefix, the rejected rows freed, all
        # extended with copies on write, the new rows written into every layer)
        {"name": "cache_round", "op": "round", "dtype": "bf16", "hkv": 8, "dh": 128, "layers": 3,
         "n": 64, "rows": 8, "shared": 2040, "lo": 1, "hi": 2048, "page": 16, "shape": 11},
        # page tables: every third request leaves a full pool, which is then compacted
        {"name": "cache_compact", "op": "compact", "dtype": "bf16", "hkv": 8, "dh": 128, "layers": 3,
         "n": 64, "rows": 0, "shared": 0, "lo": 64, "hi": 4096, "page": 32, "shape": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "attend", "attend", "verify", "round", "compact"])
    shape = rng.randrange(1 << 30)
    if op == "verify":
        return {"op": op, "dtype": rng.choice(["f32", "bf16"]), "n": _log(rng, 1, 48), "slots": rng.randint(1, 8),
                "vocab": _log(rng, 1000, 100352), "drafts": rng.random() < 0.7, "shape": shape}
    f32 = rng.random() < 0.25
    hkv, group = (rng.choice([1, 2]), rng.randint(1, 4)) if f32 else (rng.choice([2, 4, 8, 10]), rng.randint(1, 8))
    case = {"op": op, "dtype": "f32" if f32 else "bf16", "hq": hkv * group, "hkv": hkv,
            "dh": 64 if f32 else rng.choice([64, 128]), "shape": shape}
    if op == "prompt":
        if not f32:
            while case["hq"] > 40:
                case["hq"] -= hkv
        hi = _log(rng, 16, 1500 if f32 else 7000)
        return {**case, "n": max(1, min(16, _log(rng, 1, max(2, 8192 // hi)))), "lo": rng.choice([1, hi // 2]), "hi": hi}
    if op == "attend":
        return {**case, "n": _log(rng, 1, 8 if f32 else 48), "rows": rng.choice([1, 1, 2, 5, 8]),
                "page": rng.choice([16, 32, 64]), "shared": 64 * rng.randint(0, 16 if f32 else 128),
                "lo": 1, "hi": _log(rng, 8, 700 if f32 else 2048)}
    del case["hq"]
    return {**case, "layers": rng.randint(1, 3), "n": _log(rng, 2, 64), "rows": rng.randint(1, 8) if op == "round" else 0,
            "page": rng.choice([16, 32, 64]), "shared": rng.randint(1, 2000) if op == "round" else 0,
            "lo": 1, "hi": _log(rng, 64, 2048)}


def _lengths(case):
    """The case's own lengths, spread over their logarithm: they belong to the case and not to the seed."""
    rng = random.Random(case["shape"])
    return [_log(rng, case["lo"], case["hi"]) for _ in range(case["n"])]


def _rejected(case):
    """Rows of the last round that each request takes back (cache round); a request that only joins has none."""
    rng = random.Random(case["shape"] + 1)
    return [rng.randint(0, case["rows"] - 1) if i % 2 and r > case["rows"] else 0 for i, r in enumerate(_lengths(case))]


def _layout(case):
    """Lengths and page lists of a pool's requests, the shared pages first, in an order that a pool in use for
    a while has (shuffled), and the pool's size. Cache round: every second request is new and still empty, to
    be forked from one more, the last, which holds the shared prefix."""
    rng = random.Random(case["shape"] + 2)
    page, shared = case["page"], case["shared"]
    whole = shared // page
    lens = [shared + r for r in _lengths(case)]
    spare = 0
    if case["op"] == "round":
        lens = [x if i % 2 else 0 for i, x in enumerate(lens)] + [shared]
        spare = case["n"] * (-(-case["rows"] // page) + 2)
    own_pages = [max(0, -(-x // page) - whole) for x in lens]
    n_pages = whole + sum(own_pages) + spare
    ids = list(range(n_pages))
    rng.shuffle(ids)
    lists, at = [], whole
    for length, x in zip(lens, own_pages):
        lists.append(ids[:whole] + ids[at:at + x] if length else [])
        at += x
    return lens, lists, n_pages


# ------------------------------------------------------------------- what a program has in hand
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(DTYPES[dtype])


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pool(case, g):
    lens, lists, n_pages = _layout(case)
    need = max(-(-(x + case["rows"]) // case["page"]) for x in lens)
    table = torch.full((len(lens), need), -1, dtype=torch.int32)
    refs = [0] * n_pages
    for i, pages in enumerate(lists):
        table[i, :len(pages)] = torch.tensor(pages, dtype=torch.int32)
        for x in pages:
            refs[x] += 1
    shape = (case.get("layers", 1), n_pages, case["hkv"], case["page"], case["dh"])
    return {"k": _normal(g, shape, case["dtype"]), "v": _normal(g, shape, case["dtype"]), "table": table.cuda(),
            "lens": _ints(lens), "refs": _ints(refs)}


def prepare(case, seed):
    g, n = _gen(seed), case["n"]
    state = {"case": case}
    if case["op"] == "prompt":
        lens = _lengths(case)
        ends = [sum(lens[:i]) for i in range(n + 1)]
        T, hq, hkv, dh = ends[-1], case["hq"], case["hkv"], case["dh"]
        qkv = _normal(g, (T, hq + 2 * hkv, dh), case["dtype"])  # one projection's output: Q | K | V
        state.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], offsets=_ints(ends), longest=max(lens),
                     out=torch.empty((T, hq, dh), dtype=DTYPES[case["dtype"]], device="cuda"))
    elif case["op"] == "verify":
        S, V = case["slots"], case["vocab"]
        base = torch.randn((n, S + 1, V), generator=g, device="cuda") * 2.5
        state["target"] = base.to(DTYPES[case["dtype"]])
        draft = base[:, :S] + torch.randn((n, S, V), generator=g, device="cuda") * 0.5
        warm = torch.tensor([0.0 if i % 8 == 3 else 0.7 if i % 2 else 1.0 for i in range(n)], device="cuda")
        race = torch.empty((n, S, V), device="cuda").exponential_(generator=g)
        heat = torch.where(warm > 0, warm, torch.ones_like(warm))[:, None, None]
        soft = torch.softmax(draft / heat, -1)
        pick = torch.where(warm[:, None] > 0, (soft / race).argmax(-1), draft.argmax(-1))
        state.update(tokens=(pick if case["drafts"] else draft.argmax(-1)).to(torch.int32),
                     draft=draft if case["drafts"] else None, temperature=warm,
                     u=torch.rand((n, S), generator=g, device="cuda"),
                     noise=torch.empty((n, V), device="cuda").exponential_(generator=g))
    else:
        state.update(_pool(case, g))
        if case["op"] == "attend":
            shape = (n, case["rows"], case["hq"], case["dh"])
            state.update(q=_normal(g, shape, case["dtype"]), out=torch.empty(shape, dtype=DTYPES[case["dtype"]], device="cuda"))
        else:
            state.update({x + "0": state[x].clone() for x in ("table", "lens", "refs")}, requests=_ints(list(range(n))))
        if case["op"] == "round":
            rows, L = case["rows"], case["layers"]
            fork = list(range(0, n, 2))
            keep = [x - r if i % 2 else case["shared"] for i, (x, r) in enumerate(zip(_layout(case)[0], _rejected(case)))]
            shape = (L, n * rows, case["hkv"], case["dh"])
            state.update(source=_ints([n] * len(fork)), joined=_ints(fork), keep=_ints(keep), counts=_ints([rows] * n), offsets=_ints([rows * i for i in range(n + 1)]),
                         new_k=_normal(g, shape, case["dtype"]), new_v=_normal(g, shape, case["dtype"]))
        if case["op"] == "compact":
            state["gone"] = _ints(list(range(0, n, 3)))
            state["zero"] = torch.zeros_like(state["gone"])
    if own:  # what a program keeps between calls: the cache's handle and the calls' workspaces
        import speculative_decoding_drafter_hf_gb300 as hf
        if "table" in state:
            state["cache"] = hf.Pages(state["k"], state["v"], state["table"], state["lens"], state["refs"])
        if case["op"] == "attend":
            state["workspace"] = state["cache"].attend_workspace(state["q"], case["shared"])
        if case["op"] == "verify":
            state["workspace"] = hf.verify_workspace(state["target"], state["draft"])
    return state


# ------------------------------------------------------------------- plain forms
def _softmax_rows(scores, seen):
    """Softmax of the scores that are seen, zero where a row sees nothing; works in place."""
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = scores.sum(-1, keepdim=True)
    return scores.div_(torch.where(total > 0, total, torch.ones_like(total)))


def _plain_prompt(s):
    q, k, v, ends, L = s["q"], s["k"], s["v"], s["offsets"].long(), s["longest"]
    n, (T, hq, dh), hkv = len(ends) - 1, q.shape, k.shape[1]
    at = torch.arange(L, device=q.device)
    inside = at[None] < (ends[1:] - ends[:-1])[:, None]
    token = torch.where(inside, ends[:-1, None] + at[None], 0)
    qp = q[token].float().view(n, L, hkv, hq // hkv, dh).permute(0, 2, 3, 1, 4).reshape(n, hkv, hq // hkv * L, dh)
    kp = k[token].float().permute(0, 2, 3, 1)
    vp = v[token].float().permute(0, 2, 1, 3)
    p = torch.matmul(qp * dh ** -0.5, kp).view(n, hkv, hq // hkv, L, L)
    p = _softmax_rows(p, at[None, :] <= at[:, None])
    o = torch.matmul(p.view(n, hkv, hq // hkv * L, L), vp).view(n, hkv, hq // hkv, L, dh)
    return o.permute(0, 3, 1, 2, 4).reshape(n, L, hq, dh)[inside].to(q.dtype)


def _plain_attend(s):
    q, table, lens = s["q"], s["table"].long(), s["lens"].long()
    n, rows, hq, dh = q.shape
    hkv, page = s["k"].shape[2], s["k"].shape[3]
    L = table.shape[1] * page
    take = table.clamp(min=0)
    k = s["k"][0][take].float().permute(0, 2, 1, 3, 4).reshape(n, hkv, L, dh)
    v = s["v"][0][take].float().permute(0, 2, 1, 3, 4).reshape(n, hkv, L, dh)
    x = q.float().view(n, rows, hkv, hq // hkv, dh).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, dh)
    p = torch.matmul(x * dh ** -0.5, k.transpose(2, 3)).view(n, hkv, hq // hkv, rows, L)
    last = lens[:, None] - rows + torch.arange(rows, device=q.device)
    seen = torch.arange(L, device=q.device) <= last[:, :, None]
    p = _softmax_rows(p, seen[:, None, None])
    o = torch.matmul(p.view(n, hkv, -1, L), v).view(n, hkv, hq // hkv, rows, dh)
    return o.permute(0, 3, 1, 2, 4).reshape(n, rows, hq, dh).to(q.dtype)


def _soft64(x, heat):
    x = x.double() / heat
    x = (x - x.amax(-1, keepdim=True)).exp_()
    return x.div_(x.sum(-1, keepdim=True))


def _plain_verify(s):
    x, tok, T = s["target"], s["tokens"].long(), s["temperature"].double()
    n, S = tok.shape
    cold = T == 0
    heat = torch.where(cold, torch.ones_like(T), T)[:, None, None]
    p = _soft64(x, heat)
    best = x.float().argmax(-1)
    hot = torch.zeros_like(p[:, :S]).scatter_(2, tok[:, :, None], 1.0) if s["draft"] is None else _soft64(s["draft"], heat)
    pd = p[:, :S].gather(2, tok[:, :, None])[..., 0]
    qd = hot.gather(2, tok[:, :, None])[..., 0]
    ok = torch.where(cold[:, None], best[:, :S] == tok, s["u"].double() * qd < pd)
    a = ok.long().cumprod(1).sum(1)
    b = torch.arange(n, device=x.device)
    pa, qa = p[b, a], hot[b, a.clamp(max=S - 1)] * (a < S)[:, None]
    w = (pa - qa).clamp(min=0)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, pa)
    new = torch.where(cold, best[b, a], (w / s["noise"].double()).argmax(1))
    slot = torch.arange(S + 1, device=x.device)[None]
    tokens = torch.where(slot < a[:, None], torch.cat([tok, tok[:, :1]], 1), torch.where(slot == a[:, None], new[:, None], -1))
    return {"n_accepted": (a + 1).to(torch.int32), "tokens": tokens.to(torch.int32)}


def _plain_fork(s, source, joined):
    page = s["k"].shape[3]
    rows = s["table"][source.long()]
    j = torch.arange(rows.shape[1], device=rows.device)[None]
    mine = j < -(-s["lens"][source.long()].long() // page)[:, None]
    s["refs"].index_add_(0, rows[mine].long(), torch.ones_like(rows[mine]))
    s["table"][joined.long()] = torch.where(mine, rows, -1)
    s["lens"][joined.long()] = s["lens"][source.long()]


def _plain_truncate(s, requests, keep):
    page, r = s["k"].shape[3], requests.long()
    j = torch.arange(s["table"].shape[1], device=r.device)[None]
    old, new = -(-s["lens"][r].long() // page), -(-keep.long() // page)
    drop = (j >= new[:, None]) & (j < old[:, None])
    rows = s["table"][r]
    s["refs"].index_add_(0, rows[drop].long(), torch.full_like(rows[drop], -1))
    s["table"][r] = torch.where(drop, -1, rows)
    s["lens"][r] = keep


def _plain_extend(s, requests, counts):
    page, r = s["k"].shape[3], requests.long()
    old = s["lens"][r].long()
    new = old + counts
    have, want = -(-old // page), -(-new // page)
    j = torch.arange(s["table"].shape[1], device=r.device)[None]
    rows = s["table"][r].long()
    last = rows.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0]
    copied = (old % page > 0) & (counts > 0) & (s["refs"][last.clamp(min=0)] > 1)
    fresh = ((j >= have[:, None]) & (j < want[:, None])) | ((j == have[:, None] - 1) & copied[:, None])
    free = (s["refs"] == 0).nonzero()[:, 0]
    pick = free[:int(fresh.sum())]
    s["refs"][pick] = 1
    s["refs"].index_add_(0, last[copied], torch.full_like(last[copied], -1, dtype=torch.int32))
    rows[fresh] = pick
    into = rows.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0]
    s["k"][:, into[copied]] = s["k"][:, last[copied]]
    s["v"][:, into[copied]] = s["v"][:, last[copied]]
    s["table"][r] = rows.to(torch.int32)
    s["lens"][r] = new.to(torch.int32)


def _plain_write(s, requests, offsets, k, v):
    page, r = s["k"].shape[3], requests.long()
    t = torch.arange(k.shape[1], device=r.device)
    i = torch.bucketize(t, offsets[1:].long(), right=True)
    at = s["lens"][r[i]].long() - offsets[i + 1] + t
    where = s["table"][r[i], at // page].long()
    s["k"][:, where, :, at % page] = k.transpose(0, 1)
    s["v"][:, where, :, at % page] = v.transpose(0, 1)


def _plain_compact(s):
    live = s["refs"] > 0
    n = int(live.sum())
    ids = torch.arange(len(live), device=live.device)
    high, hole = ids[live & (ids >= n)], ids[~live & (ids < n)]
    to = ids.clone()
    to[high] = hole
    s["k"][:, hole] = s["k"][:, high]
    s["v"][:, hole] = s["v"][:, high]
    s["refs"][hole] = s["refs"][high]
    s["refs"][high] = 0
    s["table"].copy_(torch.where(s["table"] >= 0, to[s["table"].clamp(min=0).long()], -1))


# ------------------------------------------------------------------- one pass
def run(state):
    s, op = state, state["case"]["op"]
    if op == "prompt":
        if not own:
            return _plain_prompt(s)
        import speculative_decoding_drafter_hf_gb300 as hf
        return hf.attention_prompt(s["q"], s["k"], s["v"], s["offsets"], out=s["out"])
    if op == "attend":
        if not own:
            return _plain_attend(s)
        return s["cache"].attend(s["q"], shared=s["case"]["shared"], out=s["out"], workspace=s["workspace"])
    if op == "verify":
        if not own:
            return _plain_verify(s)
        import speculative_decoding_drafter_hf_gb300 as hf
        n, tokens = hf.verify_tokens(s["target"], s["tokens"], s["u"], s["noise"], draft_logits=s["draft"],
                                     temperature=s["temperature"], workspace=s["workspace"])
        return {"n_accepted": n, "tokens": tokens}
    # the cache as the round finds it: its data moves the same way again
    s["table"].copy_(s["table0"])
    s["lens"].copy_(s["lens0"])
    s["refs"].copy_(s["refs0"])
    if op == "round":
        if not own:
            _plain_fork(s, s["source"], s["joined"])
            _plain_truncate(s, s["requests"], s["keep"])
            _plain_extend(s, s["requests"], s["counts"])
            _plain_write(s, s["requests"], s["offsets"], s["new_k"], s["new_v"])
        else:
            s["cache"].fork(s["source"], s["joined"])
            s["cache"].truncate(s["keep"], s["requests"])
            s["cache"].extend(s["counts"], s["requests"])
            s["cache"].write(s["new_k"], s["new_v"], s["offsets"], s["requests"])
    elif not own:
        _plain_truncate(s, s["gone"], s["zero"])
        _plain_compact(s)
    else:
        s["cache"].truncate(s["zero"], s["gone"])
        s["cache"].compact()
    return {x: s[x] for x in ("k", "v", "table", "lens", "refs")}


# ------------------------------------------------------------------- what a pass cannot do without
def work(case):
    size, n = DTYPES[case["dtype"]].itemsize, case["n"]
    if case["op"] == "prompt":
        lens = _lengths(case)
        return {"bytes": sum(lens) * (2 * case["hq"] + 2 * case["hkv"]) * case["dh"] * size,
                "flops": 4 * case["hq"] * case["dh"] * sum(x * (x + 1) // 2 for x in lens)}
    if case["op"] == "verify":
        S, V = case["slots"], case["vocab"]
        rows = n * (S + 1) * size + (n * S * 4 if case["drafts"] else 0) + n * 4
        return {"bytes": rows * V, "flops": 3 * V * n * (2 * S + 1 if case["drafts"] else S + 1)}
    lens, lists, n_pages = _layout(case)
    row = 2 * case["hkv"] * case["dh"] * size  # K and V of one token
    if case["op"] == "attend":
        seen = sum(max(0, x - case["rows"] + r + 1) for x in lens for r in range(case["rows"]))
        return {"bytes": 2 * n * case["rows"] * case["hq"] * case["dh"] * size
                + row * (case["shared"] + sum(x - case["shared"] for x in lens)),
                "flops": 4 * case["hq"] * case["dh"] * seen}
    row *= case["layers"]
    if case["op"] == "round":  # every joining request copies the prefix's last page if it is partly filled, and so do
        # the others where their last page is still a shared one
        kept = [case["shared"] if i % 2 == 0 else x - r for i, (x, r) in enumerate(zip(lens, _rejected(case)))]
        copies = sum(x % case["page"] > 0 and (i % 2 == 0 or x < case["shared"] // case["page"] * case["page"])
                     for i, x in enumerate(kept))
        return {"bytes": 2 * row * (n * case["rows"] + copies * case["page"]) + 4 * n_pages, "flops": 0}
    live = [x for i, pages in enumerate(lists) if i % 3 for x in pages]
    return {"bytes": 2 * row * case["page"] * sum(x >= len(live) for x in live) + 8 * n_pages, "flops": 0}


# ------------------------------------------------------------------- from the definitions, in 64 bits
def exact(case, seed):
    if case["op"] in ("round", "compact"):
        return None  # nothing is computed: bytes are moved
    s = prepare(case, seed)
    if case["op"] == "prompt":
        ends, group = s["offsets"].tolist(), case["hq"] // case["hkv"]
        out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        for i0, i1 in zip(ends, ends[1:]):
            for h in range(case["hq"]):
                q, k, v = s["q"][i0:i1, h].double(), s["k"][i0:i1, h // group].double(), s["v"][i0:i1, h // group].double()
                z = torch.tril(torch.exp((q @ k.T) / math.sqrt(case["dh"])))
                out[i0:i1, h] = (z @ v) / z.sum(1)[:, None]
        return out
    if case["op"] == "attend":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        group, lens = case["hq"] // case["hkv"], s["lens"].tolist()
        for b, length in enumerate(lens):
            pages = s["table"][b, :-(-length // case["page"])].long()
            k = s["k"][0][pages].double().transpose(0, 1).flatten(1, 2)[:, :length]
            v = s["v"][0][pages].double().transpose(0, 1).flatten(1, 2)[:, :length]
            for r in range(case["rows"]):
                n = length - case["rows"] + r + 1
                if n > 0:
                    q = s["q"][b, r].double().view(case["hkv"], group, -1)
                    z = torch.exp(torch.einsum("hgd,hjd->hgj", q, k[:, :n]) / math.sqrt(case["dh"]))
                    o = torch.einsum("hgj,hjd->hgd", z, v[:, :n]) / z.sum(-1)[..., None]
                    out[b, r] = o.flatten(0, 1)
        return out
    count, tokens = [], []
    S = case["slots"]
    for b in range(case["n"]):
        T, a, row = float(s["temperature"][b]), 0, s["tokens"][b].tolist()
        x = s["target"][b].double()
        if T == 0:
            best = [int((y == y.max()).nonzero()[0]) for y in x]
            while a < S and best[a] == row[a]:
                a += 1
            new = best[a]
        else:
            p = torch.exp(x / T - torch.logsumexp(x / T, 1)[:, None])
            q = torch.zeros((S + 1, case["vocab"]), dtype=torch.float64, device="cuda")
            if case["drafts"]:
                y = s["draft"][b].double() / T
                q[:S] = torch.exp(y - torch.logsumexp(y, 1)[:, None])
            else:
                q[torch.arange(S), row] = 1.0
            while a < S and float(s["u"][b, a]) * float(q[a, row[a]]) < float(p[a, row[a]]):
                a += 1
            w = torch.clamp(p[a] - q[a], min=0)
            new = int(torch.argmax((w if float(w.sum()) > 0 else p[a]) / s["noise"][b].double()))
        count.append(a + 1)
        tokens.append(row[:a] + [new] + [-1] * (S - a))
    return {"n_accepted": _ints(count), "tokens": _ints(tokens)}
