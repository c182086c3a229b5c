"""The cache calls on the GPU against plain forms in 64 bits: page plan, append, tree attention.

Tolerances of the attention follow from its number formats (per output element,
p the softmax weights, A = sum_j p_j |v_j|):
  - scores: fp32 sums of D products that are exact in fp32, in any order, and
    fp32 products with the scale: an error of at most
    e_s = D 2^-22 scale sum|q k| + 2^-21 |x| in the exponent, so p is off by 2 e_s p;
    with an e4m3 cache q enters as two e4m3 terms under one power of two a row,
    exact within 2^9 of the row's largest magnitude and within 2^-17 of that
    magnitude below: scale 2^-17 max|q| sum|k| more;
  - the weights enter the second product in bf16 (2^-9 each), or as two e4m3
    terms: 2^-8 each, or 2^-15 of the row's largest weight for small ones;
    their sum does not: 2^-8 A together;
  - the output is rounded to bf16: 2^-9 |o|, doubled for the fp32 sums' order.
"""
import random

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import mxfp4_mixture_experts_route_gb300 as moe  # noqa: E402
from libmoe_util import ensure_built  # noqa: E402

DEV = "cuda"
E4M3_MAX = 448.0


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def cdiv(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------
# page plan
# ---------------------------------------------------------------------------
def plan_reference(ctx, new, parents, free, table, page, T, W):
    rows, slots, pos, masks, at = [0], [-1] * T, [-1] * T, [0] * T, 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        old, tot = cdiv(c, page), cdiv(c + n, page)
        for j in range(old, tot):
            table[b][j] = free[at]
            at += 1
        for i in range(n):
            r = rows[-1] + i
            slots[r] = table[b][(c + i) // page] * page + (c + i) % page
            if parents is None:
                pos[r] = c + i
            else:
                up, depth, bits = i, -1, 0
                while up >= 0:
                    bits |= 1 << up
                    depth += 1
                    up = parents[rows[-1] + up]
                pos[r], masks[r] = c + depth, bits
        rows.append(rows[-1] + n)
    return rows, slots, pos, [[(m >> 32 * w) & 0xFFFFFFFF for w in range(W)] for m in masks], at


def run_plan(ctx, new, parents, free, table, page, T, W, n_pages, n_free=None, Hkv=1):
    B = len(ctx)
    shape = moe.KVShape.of(B, T, Hkv, Hkv, 64, page, n_pages, len(table[0]), mask_words=W)
    ws = moe.new_kv_workspace(shape)
    out = dict(table=i32(table), row_start=torch.full((B + 1,), -7, dtype=torch.int32, device=DEV),
               slots=torch.full((T,), -7, dtype=torch.int64, device=DEV),
               pos=torch.full((T,), -7, dtype=torch.int32, device=DEV),
               mask=torch.full((T, W), -7, dtype=torch.int32, device=DEV) if W else None,
               used=i32([-7, -7]))
    f = i32(free) if free else None
    moe.kv_plan(shape, i32(ctx), i32(new), i32(parents) if W else None, f, out["table"], out["row_start"],
                out["slots"], out["pos"], out["mask"], out["used"], ws)
    return out, ws


def random_plan(seed, B, most_ctx, most_new, page, W):
    r = random.Random(seed)
    ctx = [r.choice([0, 1, page - 1, page, r.randint(0, most_ctx)]) for _ in range(B)]
    new = [r.choice([0, 1, r.randint(0, most_new), most_new]) for _ in range(B)]
    parents = [r.randint(-1, i - 1) for n in new for i in range(n)]
    need = sum(cdiv(c + n, page) for c, n in zip(ctx, new))
    n_pages, width = need + 5, max(cdiv(c + n, page) for c, n in zip(ctx, new)) + 2
    ids = list(range(n_pages))
    r.shuffle(ids)
    table, at = [], 0
    for c in ctx:
        k = cdiv(c, page)
        table.append(ids[at:at + k] + [-1] * (width - k))
        at += k
    return ctx, new, parents, ids[at:], table, n_pages


@pytest.mark.parametrize("B,most_ctx,most_new,page,W,extra", [
    (1, 100, 8, 16, 1, 0), (3, 100, 1, 8, 0, 0), (7, 300, 33, 48, 2, 5), (5, 50, 700, 64, 0, 3),
    (257, 90, 32, 16, 1, 1), (1024, 40, 3, 8, 0, 0), (4, 10, 1024, 32, 32, 0)])
def test_plan(B, most_ctx, most_new, page, W, extra):
    ctx, new, parents, free, table, n_pages = random_plan(B, B, most_ctx, most_new, page, W)
    T = max(1, sum(new) + extra)
    want_table = [list(t) for t in table]
    rows, slots, pos, masks, taken = plan_reference(ctx, new, parents if W else None, free, want_table, page, T, W)
    got, ws = run_plan(ctx, new, parents, free, table, page, T, W, n_pages)
    moe.check_device_status(ws, "kv_plan")
    assert got["row_start"].tolist() == rows
    assert got["table"].tolist() == want_table
    assert got["slots"].tolist() == slots
    assert got["pos"].tolist() == pos
    assert got["used"].tolist() == [rows[-1], taken]
    if W:
        assert [[x & 0xFFFFFFFF for x in m] for m in got["mask"].tolist()] == masks


def test_plan_refuses_lengths():
    # request 1 is negative, request 2 longer than the table: they get no rows; the others stay right
    got, ws = run_plan([3, -1, 60, 0], [2, 2, 10, 3], None, [9, 8, 7], [[1, -1, -1, -1]] * 4, 16, 8, 0, 10)
    rc, det = moe.device_status(ws)
    assert rc == moe.MOE_ERR_BAD_LENGTHS and det in (1, 2)
    assert got["row_start"].tolist() == [0, 2, 2, 2, 5]
    assert got["slots"].tolist() == [16 + 3, 16 + 4, 9 * 16, 9 * 16 + 1, 9 * 16 + 2, -1, -1, -1]
    # more rows than the arrays hold: cut off
    got, ws = run_plan([0, 0], [5, 5], None, [4, 2], [[-1], [-1]], 16, 7, 0, 8)
    assert moe.device_status(ws) == (moe.MOE_ERR_BAD_LENGTHS, 2)
    assert got["row_start"].tolist() == [0, 5, 7] and got["slots"].tolist()[5:] == [32, 33]
    # a tree larger than its mask
    got, ws = run_plan([0], [33], [-1] * 33, [4, 2, 3], [[-1] * 3], 16, 33, 1, 8)
    assert moe.device_status(ws) == (moe.MOE_ERR_BAD_LENGTHS, 0) and got["row_start"].tolist() == [0, 0]


def test_plan_refuses_pages_and_parents():
    got, ws = run_plan([0, 0], [20, 4], None, [5, 6], [[-1, -1], [-1, -1]], 16, 24, 0, 8)
    assert moe.device_status(ws) == (moe.MOE_ERR_NO_PAGES, 1)
    assert got["table"].tolist() == [[5, 6], [-1, -1]] and got["slots"].tolist()[20:] == [-1] * 4
    assert got["used"].tolist() == [24, 2]
    got, ws = run_plan([0], [2], None, [8], [[-1]], 16, 2, 0, 8)         # page id 8 of 8
    assert moe.device_status(ws) == (moe.MOE_ERR_BAD_PAGE, 8) and got["slots"].tolist() == [-1, -1]
    got, ws = run_plan([0], [3], [-1, 1, 0], [1], [[-1]], 16, 3, 1, 8)   # row 1 its own parent
    assert moe.device_status(ws) == (moe.MOE_ERR_BAD_PARENT, 1)
    assert got["mask"].tolist() == [[1], [2], [5]]


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def make_cache(n_pages, Hkv, page, D, e4m3, layout, fill):
    """(cache indexable as [page, head, offset], its strides): packed, token-major, or K and V page by page in one buffer."""
    dt = torch.uint8 if e4m3 else torch.bfloat16
    if layout == "packed":
        c = torch.empty(n_pages, Hkv, page, D, dtype=dt, device=DEV)
        st = {}
    elif layout == "tokens":
        c = torch.empty(n_pages, page, Hkv, D, dtype=dt, device=DEV).transpose(1, 2)
        st = dict(page_stride=page * Hkv * D, head_stride=D, token_stride=Hkv * D)
    else:
        c = torch.empty(n_pages, 2, Hkv, page, D + 16, dtype=dt, device=DEV)[:, 0, :, :, :D]
        st = dict(page_stride=2 * Hkv * page * (D + 16), head_stride=page * (D + 16), token_stride=D + 16)
    c.fill_(fill)
    return c, st


@pytest.mark.parametrize("T,Hkv,D,page,e4m3,layout", [
    (1, 1, 64, 8, False, "packed"), (7, 8, 128, 16, False, "tokens"), (33, 3, 64, 48, True, "packed"),
    (130, 8, 128, 64, True, "mixed"), (2011, 5, 128, 32, False, "mixed"), (1, 1, 64, 8, True, "tokens")])
def test_append(T, Hkv, D, page, e4m3, layout):
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    n_pages = cdiv(T, page) + 3
    k, st = make_cache(n_pages, Hkv, page, D, e4m3, layout, 1)
    v, _ = make_cache(n_pages, Hkv, page, D, e4m3, layout, 2)
    pad = 8 if T % 2 else 0
    x = torch.randn(2, T, Hkv * D + pad, generator=g, device=DEV).mul_(3).bfloat16()
    x[0, 0, :4] = torch.tensor([0.0, float("inf"), -1e30, float("nan")], device=DEV)
    slots = torch.randperm(n_pages * page, generator=g, device=DEV)[:T].contiguous()
    if T > 5:
        slots[3] = -1
    sc = [0.01 + torch.rand(Hkv, generator=g, device=DEV) for _ in range(2)] if e4m3 else [None, None]
    want = [c.clone() for c in (k, v)]
    for w, xx, s in zip(want, x, sc):
        rows = xx[:, :Hkv * D].view(T, Hkv, D)
        if e4m3:
            rows = (rows.float() / s[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        ok = slots >= 0
        w[slots[ok] // page, :, slots[ok] % page] = rows[ok]
    shape = moe.KVShape.of(1, T, Hkv, Hkv, D, page, n_pages, n_pages, e4m3=e4m3, kv_stride=Hkv * D + pad, **st)
    ws = moe.new_kv_workspace(shape)
    moe.kv_append(shape, x[0], x[1], slots, sc[0], sc[1], k, v, ws)
    moe.check_device_status(ws, "kv_append")
    for got, w in zip((k, v), want):
        if e4m3:
            nan = (w & 0x7F) == 0x7F
            assert torch.equal(nan, (got & 0x7F) == 0x7F)
            assert torch.equal(got[~nan], w[~nan])
        else:
            assert torch.equal(got.contiguous().view(torch.int16), w.contiguous().view(torch.int16))


def test_append_codes_of_every_bf16():
    """Every bf16 value under ordinary, exact, tiny and huge scales: the codes of the rounded quotient, ties among them."""
    x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    scales = torch.tensor([0.0137, 1.0, 0.75, 3.0, 1e-3, 1e-38, 1e-41, 1e30, 2.0 ** -8, 0.3333, 7.7, 100.0])
    Hkv, D = len(scales), 64
    T = (1 << 16) // D
    rows = x.view(T, 1, D).expand(T, Hkv, D).contiguous()
    want = (rows.float() / scales[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    shape = moe.KVShape.of(1, T, Hkv, Hkv, D, 16, T // 16, T // 16, e4m3=True)
    ws = moe.new_kv_workspace(shape)
    k, v = (torch.zeros(T // 16, Hkv, 16, D, dtype=torch.uint8, device=DEV) for _ in range(2))
    sc = scales.to(DEV)
    moe.kv_append(shape, rows.to(DEV), rows.to(DEV), torch.arange(T, device=DEV), sc, sc, k, v, ws)
    moe.check_device_status(ws, "kv_append")
    got = k.transpose(1, 2).reshape(T, Hkv, D).cpu()
    nan = (want & 0x7F) == 0x7F
    assert torch.equal(nan, (got & 0x7F) == 0x7F) and torch.equal(got[~nan], want[~nan]) and torch.equal(k, v)


def test_append_refuses_slots():
    shape = moe.KVShape.of(1, 2, 1, 1, 64, 8, 4, 4)
    ws = moe.new_kv_workspace(shape)
    k, _ = make_cache(4, 1, 8, 64, False, "packed", 0)
    v, _ = make_cache(4, 1, 8, 64, False, "packed", 0)
    x = torch.ones(2, 2, 64, device=DEV).bfloat16()
    moe.kv_append(shape, x[0], x[1], torch.tensor([32, 31], device=DEV), None, None, k, v, ws)
    assert moe.device_status(ws) == (moe.MOE_ERR_BAD_PAGE, 4)
    assert k.float().sum().item() == 64 and k[3, 0, 7].float().sum().item() == 64


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
class Batch:
    """A batch over a paged cache whose unwritten slots hold NaN."""

    def __init__(self, ctx, new, Hq, Hkv, D, page, e4m3=False, tree=None, layout="packed", seed=0, extra_rows=0,
                 extra_pages=2, gain=2.0, q_pad=0, mask=None):
        r, g = random.Random(seed), torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.ctx, self.new, self.Hq, self.Hkv, self.D, self.page, self.e4m3 = ctx, new, Hq, Hkv, D, page, e4m3
        B, total = len(ctx), sum(new)
        self.T = T = max(1, total + extra_rows)
        pages = [cdiv(c + n, page) for c, n in zip(ctx, new)]
        n_pages, width = sum(pages) + extra_pages, max(pages) + 1
        ids = list(range(n_pages))
        r.shuffle(ids)
        self.table, at = [], 0
        for p in pages:
            self.table.append(ids[at:at + p] + [-5] * (width - p))
            at += p
        nan = 0x7F if e4m3 else float("nan")
        self.k, st = make_cache(n_pages, Hkv, page, D, e4m3, layout, nan)
        self.v, _ = make_cache(n_pages, Hkv, page, D, e4m3, layout, nan)
        self.ks, self.vs = ((0.01 + 0.02 * torch.rand(Hkv, generator=g, device=DEV) for _ in range(2)) if e4m3
                            else (None, None))
        for b in range(B):
            n = ctx[b] + new[b]
            if n == 0:
                continue
            a = torch.arange(n, device=DEV)
            pg = torch.tensor(self.table[b], device=DEV)[a // page]
            for c, s in ((self.k, self.ks), (self.v, self.vs)):
                x = torch.randn(n, Hkv, D, generator=g, device=DEV)
                if e4m3:
                    x = (x / s[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
                c[pg, :, a % page] = x.to(c.dtype)
        row = Hq * D + q_pad
        q = torch.randn(T, row, generator=g, device=DEV).mul_(gain).bfloat16()
        self.q_rows, self.q = q, q[:, :Hq * D].view(T, Hq, D)
        self.see = []           # per request: [n, n] truth values among the new rows
        for b, n in enumerate(new):
            m = torch.zeros(n, n, dtype=torch.bool)
            for i in range(n):
                if mask is not None:
                    m[i] = torch.tensor([bool(mask(b, i, j)) for j in range(n)], dtype=torch.bool)
                elif tree:
                    up = r.randint(max(-1, i - 5), i - 1)
                    if up >= 0:
                        m[i] = m[up]
                    m[i, i] = True
                else:
                    m[i, :i + 1] = True
            self.see.append(m)
        self.W = W = cdiv(max(new + [1]), 32) if tree or mask is not None else 0
        self.mask = None
        if W:
            # bits past a request's rows are set: nothing may look at them
            words = [[0xFFFFFFFF] * W for _ in range(T)]
            t = 0
            for m in self.see:
                for i in range(len(m)):
                    bits = sum(1 << j for j in range(len(m)) if m[i, j]) | ~((1 << len(m)) - 1)
                    words[t] = [(bits >> 32 * w) & 0xFFFFFFFF for w in range(W)]
                    t += 1
            self.mask = torch.tensor(words, dtype=torch.int64, device=DEV).to(torch.int32)
        self.row_start = [0]
        for n in new:
            self.row_start.append(self.row_start[-1] + n)
        self.shape = moe.KVShape.of(B, T, Hq, Hkv, D, page, n_pages, width, mask_words=W, e4m3=e4m3, q_stride=row, **st)
        self.out = torch.full((T, Hq, D), 77.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((T, Hq), 77.0, dtype=torch.float32, device=DEV)
        self.ws = moe.new_kv_workspace(self.shape)

    def run(self, stream=None, lse=True, ctx=None, row_start=None, table=None):
        self.args = (i32(self.table if table is None else table), i32(self.ctx if ctx is None else ctx),
                     i32(self.row_start if row_start is None else row_start))
        self.again(stream, lse)

    def again(self, stream=None, lse=True):
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        moe.tree_attention(self.shape, self.q_rows, self.k, self.v, *self.args, self.mask, self.ks, self.vs, self.out,
                           self.lse if lse else None, self.ws, stream)

    def rows(self, cache, scale, b):
        n = self.ctx[b] + self.new[b]
        a = torch.arange(n, device=DEV)
        x = cache[torch.tensor(self.table[b], device=DEV)[a // self.page], :, a % self.page]
        x = x.contiguous().view(torch.float8_e4m3fn).double() if self.e4m3 else x.double()
        return x if scale is None else x * scale.double()[:, None]

    def reference(self, b):
        """(out, lse, tolerance of out, of lse) of request b's rows, [n, Hq, ...]."""
        c, n, G, scale = self.ctx[b], self.new[b], self.Hq // self.Hkv, self.D ** -0.5
        k, v = (x.repeat_interleave(G, 1) for x in (self.rows(self.k, self.ks, b), self.rows(self.v, self.vs, b)))
        q = self.q[self.row_start[b]:self.row_start[b] + n].double()
        see = torch.cat([torch.ones(n, c, dtype=torch.bool), self.see[b]], 1).to(DEV)[:, None]
        x = torch.einsum("ihd,jhd->ihj", q, k) * scale
        x = torch.where(see, x, float("-inf"))
        lse = torch.logsumexp(x, 2)
        empty = ~see.any(2)
        p = torch.exp(x - torch.where(empty, 0.0, lse)[..., None])
        v0 = torch.where(see.any(0).T[:, :, None], v, 0.0) if c + n else v
        out = torch.einsum("ihj,jhd->ihd", p, v0)
        kk = torch.where(k.isfinite(), k, 0.0).abs()
        e_s = self.D * 2.0 ** -22 * scale * torch.einsum("ihd,jhd->ihj", q.abs(), kk) + 2.0 ** -21 * x.abs()
        if self.e4m3:
            e_s = e_s + scale * 2.0 ** -17 * q.abs().amax(2)[..., None] * kk.sum(2).T[None]
        e_s = torch.where(see, e_s, 0.0).amax(2, keepdim=True) if c + n else torch.zeros_like(lse)[..., None]
        A = torch.einsum("ihj,jhd->ihd", p, v0.abs())
        tol = 2.0 ** -8 * (A + out.abs()) + 2 * e_s * A + 1e-30
        if self.e4m3:
            small = torch.where(see, torch.clamp(2.0 ** -15 * p.amax(2, keepdim=True) - 2.0 ** -8 * p, min=0), 0.0)
            tol = tol + torch.einsum("ihj,jhd->ihd", small, v0.abs())
        tol_l = e_s[..., 0] + (c + n) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * torch.where(empty, 0.0, lse).abs()
        return out, lse, tol, tol_l

    def check(self, lse=True):
        moe.check_device_status(self.ws, "tree_attention")
        for b, n in enumerate(self.new):
            if n == 0:
                continue
            o, l, tol, tol_l = self.reference(b)
            r = slice(self.row_start[b], self.row_start[b] + n)
            assert torch.isfinite(self.out[r]).all(), b
            worst = ((self.out[r].double() - o).abs() / tol).max().item()
            assert worst <= 1.0, (b, worst)
            if lse:
                got = self.lse[r].double()
                none = torch.isinf(l)
                assert torch.equal(none, got == float("-inf")), b
                assert ((got - l).abs()[~none] <= tol_l[~none]).all(), b
        past = slice(self.row_start[-1], self.T)
        assert (self.out[past] == 77.0).all() and (not lse or (self.lse[past] == 77.0).all())


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,new,Hq,Hkv,page,tree,layout", [
    ([0], [1], 1, 1, 8, False, "packed"),                       # one key
    ([127], [1], 8, 8, 16, False, "packed"),                    # a tile exactly
    ([128], [1], 8, 1, 16, False, "tokens"),                    # one key past it
    ([1000], [8], 32, 8, 64, True, "packed"),
    ([5, 0, 300, 129], [3, 7, 0, 1], 14, 2, 48, True, "mixed"),     # 7 heads a group; a request without rows
    ([63, 255, 1], [33, 64, 2], 16, 4, 32, True, "tokens"),     # two mask words
    ([700], [300], 8, 2, 64, False, "packed"),                  # several query tiles, chains
    ([90, 40], [130, 513], 4, 4, 16, False, "packed"),          # one head a group
    ([33], [20], 128, 1, 8, True, "packed"),                    # 128 heads on one K/V head
    ([50], [9], 66, 2, 1024, True, "packed"),                   # 33 heads a group
])
def test_attention(ctx, new, Hq, Hkv, page, tree, layout, D, e4m3):
    t = Batch(ctx, new, Hq, Hkv, D, page, e4m3, tree, layout, seed=sum(ctx) + D, extra_rows=3, q_pad=16)
    t.run()
    t.check()


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("ctx,new,Hq,Hkv,D", [
    ([40000], [1], 8, 8, 128),            # one row a head over a long cache: split over the GPU and joined
    ([3001] * 40, [1] * 40, 8, 2, 64),    # many single tokens
    ([9000, 100, 4000], [61, 5, 64], 32, 2, 128),   # large trees: two query tiles side by side
    (list(range(0, 2100, 7)), [1 + b % 5 for b in range(300)], 4, 2, 64),   # a request for every few tiles
    ([55, 300, 0], [302, 151, 513], 32, 8, 128),    # short segments of many rows: cuts move to their ends
    ([512], [512], 32, 8, 64),
    ([9000, 8000, 8191, 7777, 1000], [33, 17, 40, 33, 9], 32, 4, 64),   # segments of two, one and a part of a tile
])
def test_attention_long(ctx, new, Hq, Hkv, D, e4m3):
    t = Batch(ctx, new, Hq, Hkv, D, 16, e4m3, tree=max(new) > 1, seed=1)
    t.run()
    t.check()
    first = t.out.clone(), t.lse.clone()
    for _ in range(3):                    # bitwise repeatable
        t.run()
    assert torch.equal(first[0], t.out) and torch.equal(first[1], t.lse)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_rows_that_see_nothing_or_little(e4m3):
    # an empty row with and without cached tokens before it, rows that see only a later or only one row
    see = {0: lambda i, j: i == 2 and j == 4, 1: lambda i, j: j == 0 and i > 0, 2: lambda i, j: False}
    t = Batch([0, 130, 0], [5, 40, 1], 8, 2, 128, 16, e4m3, mask=lambda b, i, j: see[b](i, j), seed=3)
    t.run()
    t.check()
    assert (t.out[0] == 0).all() and torch.isinf(t.lse[0]).all() and (t.out[45] == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("e4m3,tree", [(False, True), (False, False), (True, True)])
def test_what_a_row_does_not_see_does_not_reach_it(e4m3, tree, bad):
    if e4m3 and bad != bad or not e4m3:
        t = Batch([100, 300], [6, 150], 8, 2, 128, 16, e4m3, mask=(lambda b, i, j: j <= i) if tree else None, seed=4)
        t.run()
        clean = t.out.clone(), t.lse.clone()
        # request 1, new row 77: K and V hold NaN or infinities; only the rows from 77 on see it
        a = t.ctx[1] + 77
        pg, o = t.table[1][a // 16], a % 16
        t.k[pg, :, o] = 0x7F if e4m3 else bad
        t.v[pg, 0, o, 5] = 0x7F if e4m3 else bad
        t.run()
        r = t.row_start[1] + 77
        for got, want in zip((t.out, t.lse), clean):
            assert torch.equal(got[:r], want[:r])
        assert not torch.isfinite(t.out[r:, :4]).all()


def test_a_seen_infinity_in_v_reaches_its_column_only():
    t = Batch([20], [40], 4, 1, 64, 16, mask=lambda b, i, j: j <= i, seed=5)
    t.run()
    clean = t.out.clone()
    a = 20 + 30
    t.v[t.table[0][a // 16], 0, a % 16, 9] = float("-inf")
    t.run()
    assert torch.equal(t.out[:30], clean[:30])
    assert (t.out[30:, :, 9] == float("-inf")).all()
    rest = [d for d in range(64) if d != 9]
    assert torch.isfinite(t.out[30:][:, :, rest]).all()


@pytest.mark.parametrize("new,Hq", [(1, 4), (9, 4), (20, 4), (60, 8)])
def test_a_seen_infinity_among_the_cached_tokens(new, Hq):
    # every row sees it, few rows or many: its column is infinite, the others are what they were
    t = Batch([700], [new], Hq, 1, 128, 16, tree=True, seed=11)
    t.run()
    clean = t.out.clone()
    t.v[t.table[0][333 // 16], 0, 333 % 16, 100] = float("inf")
    t.run()
    moe.check_device_status(t.ws)
    assert (t.out[:, :, 100] == float("inf")).all()
    rest = [d for d in range(128) if d != 100]
    assert torch.equal(t.out[:, :, rest], clean[:, :, rest])


def test_scores_far_apart():
    # one key per row takes all the weight; the running maximum moves by hundreds between tiles
    t = Batch([900], [3], 4, 2, 64, 16, gain=40.0, seed=6)
    t.run()
    t.check()


def test_rising_scores():
    # keys of growing length along a fixed direction: the maximum rises in every tile
    for e4m3 in (False, True):
        t = Batch([2000], [2], 4, 1, 128, 16, e4m3, seed=7)
        u = torch.randn(128, device=DEV)
        u /= u.norm()
        a = torch.arange(2002, device=DEV)
        pg = torch.tensor(t.table[0], device=DEV)[a // 16]
        x = torch.linspace(0, 60, 2002, device=DEV)[:, None, None] * u
        if e4m3:
            x = (x / t.ks[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        t.k[pg, :, a % 16] = x.to(t.k.dtype)
        t.q_rows[:] = (u * 11.3 * 3).bfloat16().repeat(4)[None, :t.q_rows.shape[1]]
        t.run()
        t.check()


def test_offsets_past_32_bits():
    # a cache of over 2^32 elements, used at its far end
    t = Batch([200], [8], 8, 8, 128, 64, tree=True, extra_pages=70000, seed=8)
    assert t.k.numel() > 1 << 32
    far = list(range(t.shape.n_pages - 4, t.shape.n_pages))
    moved = []
    for new_pg, old in zip(far, t.table[0]):
        moved.append(new_pg)
        if new_pg != old:
            t.k[new_pg], t.v[new_pg] = t.k[old], t.v[old]
    t.table[0][:4] = moved
    t.run()
    t.check()
    x = torch.randn(2, 8, 8, 128, device=DEV).bfloat16()
    slots = torch.tensor([far[3] * 64 + 56 + i for i in range(8)], device=DEV)
    moe.kv_append(t.shape, x[0], x[1], slots, None, None, t.k, t.v, t.ws)
    moe.check_device_status(t.ws)
    assert torch.equal(t.k[far[3], :, 56:64], x[0].transpose(0, 1)) and torch.equal(t.v[far[3], :, 56:64], x[1].transpose(0, 1))


def test_refused_lengths_and_pages():
    t = Batch([100, 50, 30], [4, 4, 4], 8, 2, 64, 16, seed=9)
    t.run()
    t.check()
    want = t.out.clone()
    t.out.fill_(77.0)
    t.run(ctx=[100, -1, 30])
    assert moe.device_status(t.ws) == (moe.MOE_ERR_BAD_LENGTHS, 1)
    assert (t.out[4:8] == 77.0).all() and torch.equal(t.out[:4], want[:4]) and torch.equal(t.out[8:], want[8:])
    t.run(row_start=[0, 4, 8, 99])
    assert moe.device_status(t.ws) == (moe.MOE_ERR_BAD_LENGTHS, 2)
    bad = [list(r) for r in t.table]
    bad[1][2] = t.shape.n_pages
    t.out.fill_(77.0)
    t.run(table=bad)
    assert moe.device_status(t.ws) == (moe.MOE_ERR_BAD_PAGE, t.shape.n_pages)
    assert torch.equal(t.out[:4], want[:4]) and torch.equal(t.out[8:], want[8:])


def test_other_stream_and_no_lse():
    t = Batch([500, 70], [8, 3], 16, 4, 128, 32, tree=True, seed=10)
    s = torch.cuda.Stream()
    t.run(stream=s, lse=False)
    s.synchronize()
    t.check(lse=False)
    assert (t.lse == 77.0).all()


def test_two_streams_at_once():
    """Launches of two streams (one of high priority) compete for the SMs; the CTAs of each wait for one another's parts."""
    ts = [Batch([3000, 70, 900], [8, 3, 1], 16, 4, 128, 32, tree=True, seed=11),
          Batch([7000], [2], 8, 2, 64, 16, tree=True, seed=12)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream(priority=-1)]
    for t, s in zip(ts, streams):
        t.run(stream=s)
    for _ in range(50):
        for t, s in zip(ts, streams):
            t.again(stream=s)
    for t, s in zip(ts, streams):
        s.synchronize()
        t.check()


def test_captured_calls_follow_the_lengths():
    """plan, append and attention in one captured graph, replayed with other lengths, pages and values."""
    B, n, Hq, Hkv, D, page, width = 3, 4, 8, 2, 64, 16, 12
    T = B * n
    shape = moe.KVShape.of(B, T, Hq, Hkv, D, page, 40, width, mask_words=1)
    ws = moe.new_kv_workspace(shape)
    k = torch.randn(40, Hkv, page, D, device=DEV).bfloat16()
    v = torch.randn(40, Hkv, page, D, device=DEV).bfloat16()
    q, kn, vn = (torch.randn(T, h, D, device=DEV).bfloat16() for h in (Hq, Hkv, Hkv))
    ctx, new, parents = i32([3, 40, 0]), i32([4, 2, 3]), i32([-1, 0, 0, 2] + [-1, 0] + [-1, 0, 1] + [0] * 3)
    table, free = i32([[b * 10 + j for j in range(10)] + [-1, -1] for b in range(B)]), i32([39, 38, 37, 36, 35, 34])
    rs, sl = torch.empty(B + 1, dtype=torch.int32, device=DEV), torch.empty(T, dtype=torch.int64, device=DEV)
    pos, mask = torch.empty(T, dtype=torch.int32, device=DEV), torch.empty(T, 1, dtype=torch.int32, device=DEV)
    used, out = i32([0, 0]), torch.zeros(T, Hq, D, device=DEV).bfloat16()

    def step():
        moe.kv_plan(shape, ctx, new, parents, free, table, rs, sl, pos, mask, used, ws)
        moe.kv_append(shape, kn, vn, sl, None, None, k, v, ws)
        moe.tree_attention(shape, q, k, v, table, ctx, rs, mask, None, None, out, None, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens, news in (([3, 40, 0], [4, 2, 3]), ([100, 0, 17], [1, 4, 4])):
        ctx.copy_(i32(lens))
        new.copy_(i32(news))
        parents.copy_(i32(([-1, 0, 0, 2] * B)[:T]))
        ps = [([-1, 0, 0, 2])[:m] for m in news]
        parents[:sum(news)].copy_(i32([p for x in ps for p in x]))
        q.copy_(torch.randn_like(q.float()))
        out.zero_()
        graph.replay()
        moe.check_device_status(ws, "graph")
        got = out.clone()
        step()
        moe.check_device_status(ws, "calls")
        assert torch.equal(got, out) and (got[:sum(news)].float().abs().sum((1, 2)) > 0).all()
        assert (got[sum(news):] == 0).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_verify_steps(e4m3):
    """The example's steps: what is accepted stays, in order, and every layer's attention and block see it."""
    from mxfp4_mixture_experts_route_gb300.verify_step import VerifyStep
    s = VerifyStep(B=3, n=6, layers=2, page=8, most_ctx=200, e4m3=e4m3)
    kept = [[[[], []] for _ in range(s.B)] for _ in range(s.layers)]      # layer, request: rows of K, of V
    scale = s.shape.scale

    def stored(x):
        if not e4m3:
            return x.double()
        return (x.float() / s.k_scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).double() * s.k_scale[:, None].double()

    for _ in range(9):
        trees, paths = s.draft()
        s.step(trees)
        assert s.used.tolist()[0] == sum(map(len, trees))
        starts = s.row_start.tolist()
        for layer in range(s.layers):
            new = [stored(x) for x in s.kv_new[layer]]
            for b, (tree, path) in enumerate(zip(trees, paths)):
                q = s.q[layer][starts[b]:starts[b] + len(tree)].double()
                rows = [kept[layer][b][x] + list(new[x][starts[b]:starts[b] + len(tree)]) for x in (0, 1)]
                k, v = (torch.stack(x).repeat_interleave(4, 1) for x in rows)
                c = len(kept[layer][b][0])
                assert c == s.lens[b]
                see = torch.ones(len(tree), c + len(tree), dtype=torch.bool, device=DEV)
                for i, p in enumerate(tree):
                    see[i, c:] = False
                    while True:
                        see[i, c + i] = True
                        if p < 0:
                            break
                        see[i, c + p] = True
                        p = tree[p]
                x = torch.where(see[:, None], torch.einsum("ihd,jhd->ihj", q, k) * scale, float("-inf"))
                p = torch.softmax(x, 2)
                want, mass = torch.einsum("ihj,jhd->ihd", p, v), torch.einsum("ihj,jhd->ihd", p, v.abs())
                got = s.attn[layer][starts[b]:starts[b] + len(tree)].double()
                # bf16 weights (relative 2^-9 a weight, and of their sum) and a bf16 result; scores' errors lie below
                assert ((got - want).abs() <= 2.0 ** -7 * mass + 2.0 ** -8 * want.abs() + 1e-6).all()
                for y in (0, 1):
                    kept[layer][b][y] += [new[y][starts[b] + t] for t in path]
            block = s.blocks[layer]
            out = block.out.clone()
            assert torch.equal(out, block.forward(s.attn[layer].view(s.T, -1))[2]) and out.isfinite().all()
        s.accept(paths)
        held = sorted(p for x in s.pages for p in x)
        assert sorted(held + s.free_pages) == list(range(s.shape.n_pages))
