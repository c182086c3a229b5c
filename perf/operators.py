"""The cache side of a speculative-decode verify step: what is measured, and its plain form.

Three operators, each the next one's input:

  plan    block tables, slot maps, positions and tree visibility masks from request lengths
  append  the new tokens' K and V rows into the paged cache (bf16, or e4m3 with a scale a head)
  attn    attention of a tree of drafted tokens (or one token, or a prompt) over the paged cache

`own` false: elementary torch operations in 32 bits.  `own` true: the library's entry points.
Lengths and trees follow from a case alone (its "mix"), values and page orders from the seed.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _plan_case(B, n, ctx, page, tree, mix):
    return {"op": "plan", "B": B, "n": n, "ctx": ctx, "page": page, "tree": tree, "mix": mix}


def _append_case(T, Hkv, D, page, kv, mix):
    return {"op": "append", "T": T, "Hkv": Hkv, "D": D, "page": page, "kv": kv, "mix": mix}


def _attn_case(B, n, ctx, Hq, Hkv, D, page, kv, tree, mix):
    return {"op": "attn", "B": B, "n": n, "ctx": ctx, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "kv": kv,
            "tree": tree, "mix": mix}


def listed():
    return [
        # the verify step's own batch: eight requests, a tree of eight drafted tokens each
        {"name": "plan_verify_8", **_plan_case(8, 8, 4096, 64, True, 1)},
        # a full serving batch with large trees of uneven size and small pages
        {"name": "plan_trees_512", **_plan_case(512, 64, 32768, 16, True, 2)},
        # a batch of prompts: long chains, most pages new
        {"name": "plan_prompts_64", **_plan_case(64, 4096, 2048, 32, False, 3)},
        # eight drafted tokens of one layer (latency)
        {"name": "append_verify_8", **_append_case(8, 8, 128, 64, "bf16", 4)},
        # prompts into an 8-bit cache (bandwidth, rounding)
        {"name": "append_prompts_e4m3", **_append_case(16411, 8, 128, 32, "e4m3", 5)},
        # one token of one request, a short cache: latency
        {"name": "attn_token_1", **_attn_case(1, 1, 1000, 32, 8, 128, 64, "bf16", False, 6)},
        # one request's verify step: a tree of eight over some thousand cached tokens
        {"name": "attn_verify_8", **_attn_case(1, 8, 4096, 32, 8, 128, 64, "bf16", True, 7)},
        # the 128-row verify step: 16 requests of 8 drafted tokens, 7 query heads a K/V head
        {"name": "attn_verify_128", **_attn_case(16, 8, 8192, 56, 8, 128, 32, "bf16", True, 8)},
        # a large batch of single tokens over an 8-bit cache: the cache's bandwidth
        {"name": "attn_token_128_e4m3", **_attn_case(128, 1, 16384, 56, 8, 128, 64, "e4m3", False, 9)},
        # wide trees over long contexts: compute
        {"name": "attn_tree_61_long", **_attn_case(4, 61, 32768, 64, 8, 128, 64, "bf16", True, 10)},
        # the smaller head width, small pages, 8-bit cache, trees past one mask word
        {"name": "attn_tree_33_e4m3", **_attn_case(16, 33, 16384, 32, 4, 64, 16, "e4m3", True, 11)},
        # prompts behind cached prefixes: the chain form, compute
        {"name": "attn_prompt_2000", **_attn_case(4, 2000, 4096, 32, 8, 128, 64, "bf16", False, 12)},
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "attn"])
    mix = rng.randrange(1 << 20)
    if op == "plan":
        tree = rng.random() < 0.6
        B = _log_int(rng, 1, 512)
        n = _log_int(rng, 1, 64) if tree else _log_int(rng, 1, min(4096, 262144 // B))
        return _plan_case(B, n, _log_int(rng, 16, 32768), rng.choice([16, 32, 48, 64]), tree, mix)
    if op == "append":
        return _append_case(_log_int(rng, 1, 16411), rng.choice([1, 4, 8]), rng.choice([64, 128]),
                            rng.choice([16, 32, 64]), rng.choice(["bf16", "e4m3"]), mix)
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 4, 7, 8])
    D, page, kv = rng.choice([64, 128, 128]), rng.choice([16, 32, 64]), rng.choice(["bf16", "e4m3"])
    kind = rng.choice(["token", "tree", "prompt"])
    if kind == "token":
        B, n, ctx = _log_int(rng, 1, 128), 1, _log_int(rng, 64, 16384)
    elif kind == "tree":
        n = _log_int(rng, 2, 64)
        B, ctx = _log_int(rng, 1, min(32, 256 // n)), _log_int(rng, 64, 32768)
    else:
        n = _log_int(rng, 65, 2000)
        B, ctx = _log_int(rng, 1, 4), _log_int(rng, 16, 4096)
    most = [max(work(c)[k] for c in listed()) for k in ("bytes", "flops")]
    while True:
        case = _attn_case(B, n, ctx, Hq, Hkv, D, page, kv, kind == "tree", mix)
        w = work(case)
        if w["bytes"] <= most[0] and w["flops"] <= most[1]:
            return case
        ctx //= 2


def _lengths(case):
    """(cached lengths, new tokens) of the case's requests: uneven, some at their largest, some new."""
    r = random.Random(case["mix"])
    B, n, ctx = case["B"], case["n"], case["ctx"]
    cs = [ctx if b == 0 else r.choice([ctx, r.randint(ctx // 4, ctx), r.randint(ctx // 4, ctx), r.randint(0, ctx)])
          for b in range(B)]
    ns = [n if b == 0 else r.choice([n, n, r.randint((n + 1) // 2, n), r.randint(1, n)]) for b in range(B)]
    return cs, ns


def _parents(case, ns):
    """Each row's parent inside its request's tree (-1: the last cached token): always an earlier row."""
    r = random.Random(case["mix"] + 1)
    return [p for n in ns for p in [-1 if i == 0 else r.randint(max(-1, i - 6), i - 1) for i in range(n)]]


def _depths(ns, parents):
    d, at = [], 0
    for n in ns:
        for i in range(n):
            p = parents[at + i]
            d.append(0 if p < 0 else d[at + p] + 1)
        at += n
    return d


def work(case):
    if case["op"] == "append":
        row = case["T"] * case["Hkv"] * case["D"] * 2
        return {"bytes": row * (2 + (2 if case["kv"] == "bf16" else 1)) + 8 * case["T"], "flops": 0}
    cs, ns = _lengths(case)
    B, T, page = len(cs), sum(ns), case["page"]
    W = (case["n"] + 31) // 32 if case["tree"] else 0
    if case["op"] == "plan":
        new = sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(cs, ns))
        seen = sum(c % page != 0 for c in cs)                         # partly filled pages: read, not taken
        return {"bytes": 8 * B + 4 * (B + 1) + T * ((4 if W else 0) + 12 + 4 * W) + 8 * new + 4 * seen, "flops": 0}
    if case["tree"]:
        seen = sum(c * n for c, n in zip(cs, ns)) + sum(d + 1 for d in _depths(ns, _parents(case, ns)))
    else:
        seen = sum(c * n + n * (n + 1) // 2 for c, n in zip(cs, ns))
    keys = sum(c + n for c, n in zip(cs, ns))
    elem = 2 if case["kv"] == "bf16" else 1
    pages = sum(-(-(c + n) // page) for c, n in zip(cs, ns))
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    return {"bytes": 2 * keys * Hkv * D * elem + T * Hq * (D * 4 + 4) + 4 * (T * W + pages + 2 * B),
            "flops": 4 * Hq * D * seen}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _cache(g, n_pages, Hkv, page, D, scale):
    """A cache of normal values, [n_pages, Hkv, page, D]: bf16, or e4m3 codes of value / scale."""
    x = torch.randn(n_pages, Hkv, page, D, generator=g, device=DEV, dtype=torch.bfloat16)
    if scale is None:
        return x
    return (x / scale.to(torch.bfloat16)[None, :, None, None]).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _scales(g, Hkv):
    return 0.01 + 0.01 * torch.rand(Hkv, generator=g, device=DEV, dtype=torch.float32)


def _mask_words(ns, parents, W):
    """[T, W] int32: bit j of a row's words = row j of its request is the row itself or an ancestor."""
    rows, at = [], 0
    for n in ns:
        for i in range(n):
            p = parents[at + i]
            rows.append((rows[at + p] if p >= 0 else 0) | (1 << i))
        at += n
    words = [[(m >> (32 * w)) & 0xFFFFFFFF for w in range(W)] for m in rows]
    return torch.tensor(words, dtype=torch.int64, device=DEV).to(torch.int32)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _prepare_plan(case, g):
    cs, ns = _lengths(case)
    B, T, page = len(cs), sum(ns), case["page"]
    W = (case["n"] + 31) // 32 if case["tree"] else 0
    old = [-(-c // page) for c in cs]
    new = [-(-(c + n) // page) for c, n in zip(cs, ns)]
    taken = sum(new) - sum(old)
    n_pages, max_pages = sum(new) + 64, max(new) + 3
    ids = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32)
    host, at = ids.cpu(), taken + 64
    for b in range(B):
        table[b, :old[b]] = host[at:at + old[b]]
        at += old[b]
    s = {"case": case, "B": B, "T": T, "W": W, "n_pages": n_pages, "max_pages": max_pages, "most": case["n"],
         "ctx_len": _i32(cs), "n_new": _i32(ns), "parents": _i32(_parents(case, ns)) if W else None,
         "free_pages": ids[:taken + 64].contiguous(), "block_table": table.to(DEV),
         "row_start": torch.empty(B + 1, dtype=torch.int32, device=DEV),
         "slots": torch.empty(T, dtype=torch.int64, device=DEV),
         "positions": torch.empty(T, dtype=torch.int32, device=DEV),
         "mask": torch.empty(T, W, dtype=torch.int32, device=DEV) if W else None,
         "used": torch.empty(2, dtype=torch.int32, device=DEV)}
    return s, dict(B=B, T=T, Hq=8, Hkv=8, D=128, page=page, n_pages=n_pages, max_pages=max_pages, mask_words=W)


def _prepare_append(case, g):
    T, Hkv, D, page = case["T"], case["Hkv"], case["D"], case["page"]
    e4m3 = case["kv"] == "e4m3"
    n_pages = -(-T // page) + 128
    ks, vs = (_scales(g, Hkv), _scales(g, Hkv)) if e4m3 else (None, None)
    # rows as a fused projection leaves them: K and V next to each other, row by row
    kv = (_randn(g, T, 2, Hkv, D) * 1.2).to(torch.bfloat16)
    page_of = torch.randperm(n_pages, generator=g, device=DEV)
    at = torch.arange(T, device=DEV) + random.Random(case["mix"]).randrange(page)
    s = {"case": case, "k_new": kv[:, 0], "v_new": kv[:, 1], "slots": page_of[at // page] * page + at % page,
         "k_scale": ks, "v_scale": vs, "k_cache": _cache(g, n_pages, Hkv, page, D, ks),
         "v_cache": _cache(g, n_pages, Hkv, page, D, vs)}
    return s, dict(B=1, T=T, Hq=Hkv, Hkv=Hkv, D=D, page=page, n_pages=n_pages, max_pages=n_pages, e4m3=e4m3,
                   kv_stride=2 * Hkv * D)


def _prepare_attn(case, g):
    cs, ns = _lengths(case)
    B, T, page, Hq, Hkv, D = len(cs), sum(ns), case["page"], case["Hq"], case["Hkv"], case["D"]
    e4m3 = case["kv"] == "e4m3"
    W = (case["n"] + 31) // 32 if case["tree"] else 0
    pages = [-(-(c + n) // page) for c, n in zip(cs, ns)]
    n_pages, max_pages = sum(pages) + 8, max(pages) + 2
    ks, vs = (_scales(g, Hkv), _scales(g, Hkv)) if e4m3 else (None, None)
    k, v = _cache(g, n_pages, Hkv, page, D, ks), _cache(g, n_pages, Hkv, page, D, vs)
    ids = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32)
    host, at, tails = ids.cpu(), 0, []
    for b in range(B):
        table[b, :pages[b]] = host[at:at + pages[b]]
        at += pages[b]
        last = int(host[at - 1])
        tails += [last * page + o for o in range((cs[b] + ns[b] - 1) % page + 1, page)]
    # what was never written holds anything: NaN here
    nan = torch.tensor(tails, dtype=torch.int64, device=DEV)
    for c in (k, v):
        raw = c.view(torch.uint8) if e4m3 else c
        raw[nan // page, :, nan % page] = 0x7F if e4m3 else float("nan")
        raw[ids[at:].long()] = 0x7F if e4m3 else float("nan")
    gain = 0.5 + 2.5 * torch.rand(Hq, generator=g, device=DEV)   # flat heads and sharp ones
    q = (_randn(g, T, Hq, D) * gain[None, :, None]).to(torch.bfloat16)
    row_start = [0]
    for n in ns:
        row_start.append(row_start[-1] + n)
    s = {"case": case, "B": B, "T": T, "W": W, "q": q, "k_cache": k, "v_cache": v, "block_table": table.to(DEV),
         "ctx_len": _i32(cs), "row_start": _i32(row_start),
         "mask": _mask_words(ns, _parents(case, ns), W) if W else None, "k_scale": ks, "v_scale": vs,
         "scale": D ** -0.5, "pages": max(pages), "most": max(ns),
         "out": torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV),
         "lse": torch.empty(T, Hq, dtype=torch.float32, device=DEV)}
    return s, dict(B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, page=page, n_pages=n_pages, max_pages=max_pages, mask_words=W,
                   e4m3=e4m3, scale=D ** -0.5)


def prepare(case, seed):
    make = {"plan": _prepare_plan, "append": _prepare_append, "attn": _prepare_attn}[case["op"]]
    s, shape = make(case, _gen(seed))
    if own:   # the shape descriptor and workspace that a program keeps
        import mxfp4_mixture_experts_route_gb300 as moe
        s["shape"] = moe.KVShape.of(**shape)
        s["ws"] = moe.new_kv_workspace(s["shape"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _plain_plan(s):
    page, B, T, W = s["case"]["page"], s["B"], s["T"], s["W"]
    c, n, table, free = s["ctx_len"].long(), s["n_new"].long(), s["block_table"], s["free_pages"]
    row_start = torch.cat([n.new_zeros(1), n.cumsum(0)])
    old, new = (c + page - 1) // page, (c + n + page - 1) // page
    first = (new - old).cumsum(0) - (new - old)                       # pages taken by earlier requests
    j = torch.arange(s["max_pages"], device=DEV)[None]
    fresh = (j >= old[:, None]) & (j < new[:, None])
    table.copy_(torch.where(fresh, free[(first[:, None] + j - old[:, None]).clamp(0, len(free) - 1)], table))
    r = torch.arange(T, device=DEV)
    b = torch.searchsorted(row_start, r, right=True) - 1
    i = r - row_start[b]
    at = c[b] + i
    slots = table[b, at // page].long() * page + at % page
    out = {"row_start": row_start.int(), "block_table": table, "slots": slots,
           "used": torch.stack([row_start[-1], (new - old).sum()]).int()}
    if not W:
        return {**out, "positions": at.int()}
    up = s["parents"].long()
    seen = torch.arange(32 * W, device=DEV)[None] == i[:, None]       # [T, 32 W]: the row itself
    jump = torch.where(up >= 0, row_start[b] + up, r)                 # a root stays where it is
    for _ in range(max(1, (s["most"] - 1).bit_length())):             # ancestors within 2^k steps
        seen = seen | seen[jump]
        jump = jump[jump]
    words = (seen.view(T, W, 32).long() << torch.arange(32, device=DEV)).sum(2).int()
    return {**out, "positions": (c[b] + seen.sum(1) - 1).int(), "mask": words}


def _plain_append(s):
    page = s["case"]["page"]
    p, o = s["slots"] // page, s["slots"] % page
    if s["k_scale"] is None:
        s["k_cache"][p, :, o] = s["k_new"]
        s["v_cache"][p, :, o] = s["v_new"]
    else:
        k = (s["k_new"].float() / s["k_scale"][None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        v = (s["v_new"].float() / s["v_scale"][None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s["k_cache"].view(torch.uint8)[p, :, o] = k.view(torch.uint8)
        s["v_cache"].view(torch.uint8)[p, :, o] = v.view(torch.uint8)
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _gathered(cache, table, scale):
    """Every request's rows of a cache in order, fp32: [B, Hkv, keys, D]."""
    pages = (cache if scale is None else cache.view(torch.uint8))[table]       # [B, pages, Hkv, page, D]
    x = pages.float() if scale is None else pages.view(torch.float8_e4m3fn).float() * scale[None, None, :, None, None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_attn(s):
    c = s["case"]
    B, N, Hkv, G, D = s["B"], s["most"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    table = s["block_table"][:, :s["pages"]].long().clamp(min=0)
    k, v = _gathered(s["k_cache"], table, s["k_scale"]), _gathered(s["v_cache"], table, s["v_scale"])
    start, ctx = s["row_start"].long(), s["ctx_len"].long()
    r = torch.arange(s["T"], device=DEV)
    b = torch.searchsorted(start, r, right=True) - 1
    i = r - start[b]
    n = start[1:] - start[:-1]
    q = torch.zeros(B, N, c["Hq"], D, device=DEV)
    q[b, i] = s["q"].float()
    q = q.view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    key = torch.arange(k.shape[2], device=DEV)
    j = key[None, :] - ctx[:, None]                                            # [B, keys]: index among the new rows
    real = j < n[:, None]
    if s["mask"] is None:
        see = j[:, None] <= torch.arange(N, device=DEV)[None, :, None]
    else:
        bits = torch.zeros(B, N, s["W"], dtype=torch.int64, device=DEV)
        bits[b, i] = s["mask"].long() & 0xFFFFFFFF
        jc = j.clamp(0, 32 * s["W"] - 1)[:, None].expand(B, N, -1)
        see = (j[:, None] < 0) | ((bits.gather(2, jc // 32) >> (jc % 32)) & 1).bool()
    see = (see & real[:, None])[:, None, :, None, :].expand(B, Hkv, N, G, -1).reshape(B, Hkv, N * G, -1)
    x = torch.where(see, q @ k.transpose(2, 3) * s["scale"], float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    v = torch.where(real[:, None, :, None], v, 0.0)
    o = p @ v / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).view(B, Hkv, N, G).permute(0, 2, 1, 3).reshape(B, N, Hkv * G)
    o = o.view(B, Hkv, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, Hkv * G, D)
    return {"out": o[b, i].to(torch.bfloat16), "lse": lse[b, i]}


def _own(s):
    import mxfp4_mixture_experts_route_gb300 as moe
    op = s["case"]["op"]
    if op == "plan":
        moe.kv_plan(s["shape"], s["ctx_len"], s["n_new"], s["parents"], s["free_pages"], s["block_table"],
                    s["row_start"], s["slots"], s["positions"], s["mask"], s["used"], s["ws"])
        names = ["row_start", "block_table", "slots", "used", "positions"] + (["mask"] if s["W"] else [])
    elif op == "append":
        moe.kv_append(s["shape"], s["k_new"], s["v_new"], s["slots"], s["k_scale"], s["v_scale"], s["k_cache"],
                      s["v_cache"], s["ws"])
        names = ["k_cache", "v_cache"]
    else:
        moe.tree_attention(s["shape"], s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["ctx_len"],
                           s["row_start"], s["mask"], s["k_scale"], s["v_scale"], s["out"], s["lse"], s["ws"])
        names = ["out", "lse"]
    return {k: s[k] for k in names}


def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "append": _plain_append, "attn": _plain_attn}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    page = case["page"]
    if case["op"] == "append":
        out = {}
        for x in ("k", "v"):
            cache = s[x + "_cache"].to(torch.float64)
            new = s[x + "_new"].to(torch.float64)
            if s[x + "_scale"] is not None:
                new = (new / s[x + "_scale"].to(torch.float64)[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
            flat = cache.transpose(1, 2).reshape(-1, case["Hkv"], case["D"])
            flat[s["slots"]] = new
            out[x + "_cache"] = flat.view(-1, page, case["Hkv"], case["D"]).transpose(1, 2).contiguous()
        return out
    cs, ns = _lengths(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if 4 * Hq * D * sum(n * (c + n) for c, n in zip(cs, ns)) > 4e12:
        return None
    out = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["T"], Hq, dtype=torch.float64, device=DEV)
    up = _parents(case, ns)
    at = 0
    for b, (c, n) in enumerate(zip(cs, ns)):
        keys = torch.arange(c + n, device=DEV)
        page_of = s["block_table"][b].long()[keys // page]
        kv = []
        for x in ("k", "v"):
            t = s[x + "_cache"]
            t = t.view(torch.uint8)[page_of, :, keys % page].view(torch.float8_e4m3fn) if case["kv"] == "e4m3" \
                else t[page_of, :, keys % page]
            t = t.to(torch.float64)                                   # [keys, Hkv, D]
            if s[x + "_scale"] is not None:
                t = t * s[x + "_scale"].to(torch.float64)[:, None]
            kv.append(t)
        see = torch.zeros(n, n, dtype=torch.bool)
        for i in range(n):
            if case["tree"]:
                if up[at + i] >= 0:
                    see[i] = see[up[at + i]]
                see[i, i] = True
            else:
                see[i, :i + 1] = True
        see = torch.cat([torch.ones(n, c, dtype=torch.bool), see], 1).to(DEV)
        for h in range(Hq):
            k, v = (t[:, h // (Hq // Hkv)] for t in kv)
            x = s["q"][at:at + n, h].to(torch.float64) @ k.T * s["scale"]
            x = x.masked_fill(~see, float("-inf"))
            lse[at:at + n, h] = torch.logsumexp(x, 1)
            out[at:at + n, h] = torch.softmax(x, 1) @ v
        at += n
    return {"out": out, "lse": lse}
