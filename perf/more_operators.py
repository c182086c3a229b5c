"""The dense projections around a layer's attention, in MXFP4: what is measured, and its plain form.

Four operators, as a layer uses them one after the other:

  quant   rows to MXFP4 (e2m1 codes, one e8m0 scale a 32 elements) and back: a checkpoint's weights, a step's rows
  dequant MXFP4 rows to bf16 or fp32
  linear  out = x . w^T with MXFP4 weights, x bf16 or MXFP4
  qkv     the norms and rotation of query and key heads, with the append of K and V to the paged cache

`own` false: elementary torch operations in 32 bits.  `own` true: the library's entry points.
Lengths follow from a case alone (its "mix"), values and page orders from the seed.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
MAX_POS = 32768


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _quant_case(rows, K, dtype):
    return {"op": "quant", "rows": rows, "K": K, "dtype": dtype}


def _dequant_case(rows, K, dtype):
    return {"op": "dequant", "rows": rows, "K": K, "dtype": dtype}


def _linear_case(T, N, K, x):
    return {"op": "linear", "T": T, "N": N, "K": K, "x": x}


def _qkv_case(T, Hq, Hkv, D, R, page, kv, norm, interleaved, mix):
    return {"op": "qkv", "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "R": R, "page": page, "kv": kv, "norm": norm,
            "interleaved": interleaved, "mix": mix}


def listed():
    return [
        # a verify step's eight rows before a product of two MXFP4 operands (latency)
        {"name": "quant_rows_8", **_quant_case(8, 4096, "bf16")},
        # a checkpoint's gate and up rows of 16 experts (bandwidth)
        {"name": "quant_w13", **_quant_case(16 * 2048, 4096, "bf16")},
        # a few rows of a projection read back, as an odd number of them (latency)
        {"name": "dequant_rows_65", **_dequant_case(65, 4096, "f32")},
        # the down rows of 16 experts, for a program that wants bf16 weights (bandwidth)
        {"name": "dequant_w2", **_dequant_case(16 * 7168, 2048, "bf16")},
        # one token's query, key and value projection: 32 and 8 heads (latency)
        {"name": "linear_bf16_1", **_linear_case(1, 6144, 4096, "bf16")},
        # the 128-row verify step's, 56 and 8 heads on 7168 (the weights' bandwidth)
        {"name": "linear_bf16_128", **_linear_case(128, 9216, 7168, "bf16")},
        # prompts behind weights kept at 4 bits (compute)
        {"name": "linear_bf16_4096", **_linear_case(4096, 6144, 4096, "bf16")},
        # the verify step's output projection with its rows quantised (latency, the weights' bandwidth)
        {"name": "linear_mx_8", **_linear_case(8, 7168, 4096, "mxfp4")},
        # ragged: an odd number of tokens, a part of a weight tile, half a K stage
        {"name": "linear_mx_333", **_linear_case(333, 1000, 4224, "mxfp4")},
        # prompts with both operands at 4 bits (compute)
        {"name": "linear_mx_8192", **_linear_case(8192, 14336, 7168, "mxfp4")},
        # eight drafted tokens of one layer (latency)
        {"name": "qkv_verify_8", **_qkv_case(8, 32, 8, 128, 128, 64, "bf16", True, False, 1)},
        # prompts into an 8-bit cache (bandwidth)
        {"name": "qkv_prompts_e4m3", **_qkv_case(16411, 56, 8, 128, 128, 32, "e4m3", True, False, 2)},
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["quant", "dequant", "linear", "linear", "linear", "qkv"])
    if op in ("quant", "dequant"):
        K = 32 * _log_int(rng, 1, 256)
        rows = _log_int(rng, 1, min(1 << 18, (1 << 27) // K))
        dtype = rng.choice(["bf16", "f16", "f32"])
        return (_quant_case if op == "quant" else _dequant_case)(rows, K, dtype)
    if op == "qkv":
        D = rng.choice([64, 128, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        return _qkv_case(_log_int(rng, 1, 16411), Hkv * rng.choice([1, 4, 7, 8]), Hkv, D,
                         rng.choice([D, D, D // 2, 16, 0]), rng.choice([16, 32, 64]), rng.choice(["bf16", "e4m3"]),
                         rng.random() < 0.7, rng.random() < 0.3, rng.randrange(1 << 20))
    x, T, K = rng.choice(["bf16", "mxfp4"]), _log_int(rng, 1, 8192), 128 * _log_int(rng, 1, 64)
    N = 8 * _log_int(rng, 1, 2048)
    most = {c["x"]: work(c)["flops"] for c in listed() if c["op"] == "linear"}
    while work(_linear_case(T, N, K, x))["flops"] > most[x]:
        T = -(-T // 2)
    return _linear_case(T, N, K, x)


def _positions(case):
    """(positions, cache rows) of the case's rows: requests of uneven lengths behind uneven contexts, -1 in the last
    rows, which no request owns."""
    r = random.Random(case["mix"])
    T, pos, req = case["T"], [], []
    tail = min(T // 4, 3)
    while len(pos) < T - tail:
        n = min(T - tail - len(pos), r.choice([1, 8, r.randint(1, 64), r.randint(1, 4096)]))
        c = r.randint(0, MAX_POS - n)
        pos += range(c, c + n)
        req += [n]
    return pos + [-1] * tail, req


def work(case):
    if case["op"] in ("quant", "dequant"):
        n = case["rows"] * case["K"]
        size = 4 if case["dtype"] == "f32" else 2
        code = n // 2 + n // 32
        # quant: rows in, codes and scales out, and the values read back from them
        return {"bytes": 2 * n * size + 2 * code if case["op"] == "quant" else n * size + code, "flops": 0}
    if case["op"] == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        x = T * K * 2 if case["x"] == "bf16" else T * K // 2 + T * K // 32
        return {"bytes": N * K // 2 + N * K // 32 + x + T * N * 2, "flops": 2 * T * N * K}
    T, Hq, Hkv, D, R = case["T"], case["Hq"], case["Hkv"], case["D"], case["R"]
    pos, _ = _positions(case)
    live = sum(p >= 0 for p in pos)
    elem = 2 if case["kv"] == "bf16" else 1
    return {"bytes": live * D * (4 * Hq + 2 * Hkv * (2 + elem)) + 12 * T + len(set(pos) - {-1}) * R * 4, "flops": 0}


# ---------------------------------------------------------------------------
# MXFP4 in elementary operations
# ---------------------------------------------------------------------------
def _grid(device):
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device)


def _scale_of(byte):
    """2^(byte - 127) in fp32; NaN for 255."""
    b = byte.to(torch.int32)
    bits = torch.where(b == 0, 0x00400000, torch.where(b == 255, 0x7FC00000, b << 23))
    return bits.view(torch.float32)


def _to_mx(x):
    """Rows of fp32 to packed codes and scale bytes: the scale is the block maximum's power of two over 4, a code the
    nearest of the grid, ties to the even code, beyond 6 the code of 6."""
    blocks = x.view(x.shape[0], -1, 32)
    top = (blocks.abs().amax(-1).contiguous().view(torch.int32) >> 23) & 255
    byte = torch.where(top == 255, 255, (top - 2).clamp(min=0))
    inv = torch.where(byte == 255, 0, (254 - byte) << 23).view(torch.float32)
    v = blocks * inv[..., None]
    a = v.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for limit, strict in ((0.25, True), (0.75, False), (1.25, True), (1.75, False), (2.5, True), (3.5, False), (5.0, True)):
        code += a > limit if strict else a >= limit
    code |= torch.signbit(v).to(torch.uint8) << 3
    code = torch.where(byte[..., None] == 255, 0, code).view(x.shape[0], -1, 2)
    return (code[..., 0] | code[..., 1] << 4).contiguous(), byte.to(torch.uint8)


def _from_mx(codes, scales):
    c = torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1, 32)
    value = _grid(codes.device)[(c & 7).long()]
    value = torch.where(c > 7, -value, value)
    return (value * _scale_of(scales)[..., None]).view(codes.shape[0], -1)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _rows(g, rows, K):
    """Activations: normal values, each row and a few channels of a size of their own."""
    x = _randn(g, rows, K) * torch.exp(0.3 * _randn(g, rows, 1))
    return x * torch.where(torch.rand(K, generator=g, device=DEV) < 0.01, 8.0, 1.0)


def _mx_weights(g, N, K):
    """A projection's weights, quantised: normal values of variance 1 / K, rows of sizes of their own."""
    codes = torch.empty(N, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(N, K // 32, dtype=torch.uint8, device=DEV)
    for at in range(0, N, 4096):
        n = min(4096, N - at)
        codes[at:at + n], scales[at:at + n] = _to_mx(_randn(g, n, K) * torch.exp(0.3 * _randn(g, n, 1)) * K ** -0.5)
    return codes, scales


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _rope_table(R):
    """cos and sin of position * 10000^(-2 i / R), i = 0 .. R/2 - 1: [MAX_POS, R] fp32, angles in 64 bits."""
    i = torch.arange(R // 2, device=DEV, dtype=torch.float64)
    angle = torch.arange(MAX_POS, device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (-2 * i / max(R, 1))
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _prepare_qkv(case, g):
    T, Hq, Hkv, D, R, page = case["T"], case["Hq"], case["Hkv"], case["D"], case["R"], case["page"]
    e4m3 = case["kv"] == "e4m3"
    pos, req = _positions(case)
    n_pages = sum(-(-n // page) + 1 for n in req) + 8
    page_of, slots, at, p = torch.randperm(n_pages, generator=g, device=DEV).tolist(), [], 0, 0
    for n in req:
        first = pos[at] % page
        slots += [page_of[p + (first + i) // page] * page + (first + i) % page for i in range(n)]
        at, p = at + n, p + -(-(first + n) // page)
    slots += [-1] * (T - len(slots))
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    # the rows as the fused projection leaves them: Q, K and V heads next to each other
    qkv = _randn(g, T, Hq + 2 * Hkv, D).mul_(1.2).to(torch.bfloat16)

    def cache():
        return _randn(g, n_pages, Hkv, page, D).to(dt)

    def weight():
        return 0.5 + torch.rand(D, generator=g, device=DEV, dtype=torch.float32) if case["norm"] else None

    def scale():
        return 0.02 + 0.01 * torch.rand(Hkv, generator=g, device=DEV, dtype=torch.float32) if e4m3 else None

    return {"case": case, "q_in": qkv[:, :Hq], "k_new": qkv[:, Hq:Hq + Hkv], "v_new": qkv[:, Hq + Hkv:],
            "positions": _i32(pos), "slots": torch.tensor(slots, dtype=torch.int64, device=DEV), "q_norm": weight(),
            "k_norm": weight(), "table": _rope_table(R) if R else None, "k_scale": scale(), "v_scale": scale(),
            "q": torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=DEV), "k_cache": cache(), "v_cache": cache(),
            "n_pages": n_pages, "eps": 1e-6}


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op in ("quant", "dequant"):
        rows, K, dt = case["rows"], case["K"], TYPES[case["dtype"]]
        if op == "quant":
            s = {"case": case, "x": _rows(g, rows, K).to(dt),
                 "codes": torch.empty(rows, K // 2, dtype=torch.uint8, device=DEV),
                 "scales": torch.empty(rows, K // 32, dtype=torch.uint8, device=DEV)}
        else:
            codes, scales = _mx_weights(g, rows, K)
            s = {"case": case, "codes": codes, "scales": scales}
        s["y"] = torch.empty(rows, K, dtype=dt, device=DEV)
    elif op == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        w, ws = _mx_weights(g, N, K)
        x, xs = _rows(g, T, K), None
        if case["x"] == "mxfp4":
            x, xs = _to_mx(x)
        else:
            x = x.to(torch.bfloat16)
        s = {"case": case, "x": x, "xs": xs, "w": w, "ws": ws,
             "out": torch.empty(T, N, dtype=torch.bfloat16, device=DEV)}
    else:
        s = _prepare_qkv(case, g)
    if own:   # the shape descriptors and workspaces that a program keeps
        import mxfp4_mixture_experts_route_gb300 as moe
        if op == "linear":
            s["shape"] = moe.MXShape.of(case["T"], case["N"], case["K"], x_mxfp4=case["x"] == "mxfp4")
            s["work"] = moe.new_mx_workspace(s["shape"])
        elif op == "qkv":
            T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
            width = (Hq + 2 * Hkv) * D
            s["shape"] = moe.KVShape.of(1, T, Hq, Hkv, D, case["page"], s["n_pages"], s["n_pages"],
                                        e4m3=case["kv"] == "e4m3", kv_stride=width)
            s["rope"] = moe.Rope.of(case["R"], MAX_POS if case["R"] else 0, eps=s["eps"],
                                    interleaved=case["interleaved"], q_in_stride=width)
            s["work"] = moe.new_kv_workspace(s["shape"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _rotate(x, table, pos, interleaved):
    """The first R of the last dimension by the angles of the rows' positions; x [rows, heads, D] fp32."""
    if table is None:
        return x
    R = table.shape[1]
    cos, sin = table[pos, :R // 2][:, None], table[pos, R // 2:][:, None]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([c, d], -1).flatten(-2) if interleaved else torch.cat([c, d], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _plain_qkv(s):
    c = s["case"]
    live = s["positions"] >= 0
    rows = live.nonzero()[:, 0]
    pos, slots = s["positions"][rows].long(), s["slots"][rows]

    def head(x, w):
        x = x[rows].float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w
        return _rotate(x, s["table"], pos, c["interleaved"])

    s["q"][rows] = head(s["q_in"], s["q_norm"]).to(torch.bfloat16)
    p, o = slots // c["page"], slots % c["page"]
    for x, cache, scale in ((head(s["k_new"], s["k_norm"]), s["k_cache"], s["k_scale"]),
                            (s["v_new"][rows].float(), s["v_cache"], s["v_scale"])):
        if scale is None:
            cache[p, :, o] = x.to(torch.bfloat16)
        else:
            code = (x / scale[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            cache.view(torch.uint8)[p, :, o] = code.view(torch.uint8)
    return {"q": s["q"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain(s):
    op = s["case"]["op"]
    if op == "qkv":
        return _plain_qkv(s)
    if op == "linear":
        x = s["x"].float() if s["xs"] is None else _from_mx(s["x"], s["xs"])
        return (x @ _from_mx(s["w"], s["ws"]).t()).to(torch.bfloat16)
    codes, scales = _to_mx(s["x"].float()) if op == "quant" else (s["codes"], s["scales"])
    return _from_mx(codes, scales).to(TYPES[s["case"]["dtype"]])


def _own(s):
    import mxfp4_mixture_experts_route_gb300 as moe
    op = s["case"]["op"]
    if op == "linear":
        moe.mx_linear(s["shape"], s["x"], s["xs"], s["w"], s["ws"], s["out"], s["work"])
        return s["out"]
    if op == "qkv":
        moe.qkv_append(s["shape"], s["rope"], s["q_in"], s["k_new"], s["v_new"], s["positions"], s["slots"],
                       s["q_norm"], s["k_norm"], s["table"], s["k_scale"], s["v_scale"], s["q"], s["k_cache"],
                       s["v_cache"], s["work"])
        return {"q": s["q"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "quant":
        moe.mx_quantize(s["x"], s["codes"], s["scales"])
    moe.mx_dequantize(s["codes"], s["scales"], s["y"])
    return s["y"]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_values(codes, scales):
    """sign * (mantissa / 2) * 2^max(exponent, 1) / 2 * 2^(byte - 127), by the format's fields."""
    c = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.int64, device=DEV)
    c[:, 0::2], c[:, 1::2] = codes % 16, codes // 16
    sign, e, m = 1 - 2 * (c // 8), c // 2 % 4, c % 2
    v = sign * (torch.where(e > 0, 1.0, 0.0).double() + 0.5 * m) * torch.exp2((e.clamp(min=1) - 1).double())
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "dequant":
        return _exact_values(s["codes"], s["scales"])
    if case["op"] == "quant":
        out = torch.empty(case["rows"], case["K"], dtype=torch.float64, device=DEV)
        for at in range(0, case["rows"], 4096):
            x = s["x"][at:at + 4096].double().unflatten(1, (-1, 32))
            exponent = torch.frexp(x.abs().amax(-1, keepdim=True))[1] - 3   # floor(log2(top)) - 2
            scale = torch.exp2(exponent.clamp(min=-127).double())
            v = x / scale
            step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).double()
            out[at:at + 4096] = ((v / step).round() * step).clamp(-6, 6).mul(scale).flatten(1)
        return out
    if case["op"] == "linear":
        x = s["x"].double() if s["xs"] is None else _exact_values(s["x"], s["xs"])
        return x @ _exact_values(s["w"], s["ws"]).T
    D, R, page = case["D"], case["R"], case["page"]
    q = s["q"].double()
    caches = {"k": s["k_cache"].double(), "v": s["v_cache"].double()}
    i = torch.arange(R // 2, device=DEV)
    lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + R // 2)
    rows = torch.tensor([t for t, p in enumerate(_positions(case)[0]) if p >= 0], device=DEV)
    if R:   # the table's own entries: they are an input
        cos, sin = s["table"].double()[s["positions"][rows].long()].split(R // 2, 1)

    def head(x, w):
        x = x.double()[rows]
        if w is not None:
            x = x / (x.square().sum(-1, keepdim=True) / D + s["eps"]).sqrt() * w.double()
        if R:
            z = torch.complex(x[..., lo], x[..., hi]) * torch.complex(cos, sin)[:, None]
            x[..., lo], x[..., hi] = z.real, z.imag
        return x

    q[rows] = head(s["q_in"], s["q_norm"])
    for n, x in (("k", head(s["k_new"], s["k_norm"])), ("v", s["v_new"].double()[rows])):
        if s[n + "_scale"] is not None:
            x = (x / s[n + "_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        flat = caches[n].transpose(1, 2).reshape(-1, case["Hkv"], D)
        flat[s["slots"][rows]] = x
        caches[n] = flat.view(-1, page, case["Hkv"], D).transpose(1, 2).contiguous()
    return {"q": q, "k_cache": caches["k"], "v_cache": caches["v"]}
