"""Norms, rotation and append of a projection's rows on the GPU against a plain form in 64 bits.

Tolerances, z the exact result, y_i and y_j the pair's normalised elements: the norm's factor
is an fp32 sum of D squares and a reciprocal square root (relative 2^-18 for D <= 128, counting
D 2^-24 / 2 and the root's few units), every product and sum after it 2^-24 relative:
2^-17 (|y_i| + |y_j|) together.  Then one rounding: bf16 2^-8 of z; e4m3 2^-4 of z / scale, or
half of its smallest step, 2^-10.
"""
import random

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import mxfp4_mixture_experts_route_gb300 as moe  # noqa: E402
from libmoe_util import ensure_built  # noqa: E402

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


class Case:
    def __init__(self, T, Hq, Hkv, D, R, page=16, e4m3=False, norm="qk", inter=False, max_pos=4096, seed=0, fused=True,
                 in_place=False, odd_cache=False):
        g = torch.Generator(device=DEV).manual_seed(seed)
        r = random.Random(seed)
        self.T, self.Hq, self.Hkv, self.D, self.R, self.page, self.e4m3, self.inter = T, Hq, Hkv, D, R, page, e4m3, inter
        self.n_pages = -(-T // page) + 3
        width = (Hq + 2 * Hkv) * D
        rows = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV).mul_(1.5).bfloat16()
        if not fused:
            self.q_in, self.k, self.v = rows[:, :Hq].clone(), rows[:, Hq:Hq + Hkv].clone(), rows[:, Hq + Hkv:].clone()
        else:
            self.q_in, self.k, self.v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        self.q = self.q_in if in_place else torch.full((T, Hq, D), -77.0, dtype=torch.bfloat16, device=DEV)
        qs = width if fused else 0
        dt = torch.uint8 if e4m3 else torch.bfloat16
        fill = 0x55 if e4m3 else -77.0
        # [page][token][head] instead of the packed [page][head][token], the rows of a token 16 elements apart
        pad = 16 if odd_cache else 0
        self.caches = [torch.full((self.n_pages, Hkv, page, D), fill, dtype=dt, device=DEV) if not odd_cache else
                       torch.full((self.n_pages, page, Hkv, D + pad), fill, dtype=dt, device=DEV) for _ in "kv"]
        strides = {} if not odd_cache else dict(token_stride=Hkv * (D + pad), head_stride=D + pad, page_stride=page * Hkv * (D + pad))
        self.shape = moe.KVShape.of(1, T, Hq, Hkv, D, page, self.n_pages, self.n_pages, e4m3=e4m3,
                                    kv_stride=width if fused else 0, q_stride=qs if in_place else 0, **strides)
        self.rope = moe.Rope.of(R, max_pos if R else 0, interleaved=inter, q_in_stride=qs)
        self.table = moe.rope_table(max_pos, R) if R else None
        self.pos = torch.tensor([r.choice([0, 1, max_pos - 1, r.randrange(max_pos)]) for _ in range(T)], dtype=torch.int32, device=DEV)
        self.slots = torch.tensor(r.sample(range(self.n_pages * page), T), dtype=torch.int64, device=DEV)
        self.qn, self.kn = (0.5 + torch.rand(D, generator=g, device=DEV) if c in norm else None for c in "qk")
        self.scales = [0.01 + 0.02 * torch.rand(Hkv, generator=g, device=DEV) for _ in "kv"] if e4m3 else [None, None]
        self.ws = moe.new_kv_workspace(self.shape)
        self.before = [self.q.clone()] + [c.clone() for c in self.caches]
        self.q64, self.k64, self.v64 = self.q_in.double().clone(), self.k.double(), self.v.double()

    def run(self, stream=None):
        moe.qkv_append(self.shape, self.rope, self.q_in, self.k, self.v, self.pos, self.slots, self.qn, self.kn, self.table,
                       *self.scales, self.q, *self.caches, self.ws, stream)

    def head(self, x, w):
        """(z, |y_i| + |y_j|) in 64 bits."""
        y = x
        if w is not None:
            y = x * (x.square().mean(-1, keepdim=True) + float(torch.tensor(1e-6))).rsqrt() * w.double()
        z, size, R = y.clone(), y.abs(), self.R
        if R:
            i = torch.arange(R // 2, device=DEV)
            a, b = (2 * i, 2 * i + 1) if self.inter else (i, i + R // 2)
            row = self.table[self.pos.long().clamp(0, len(self.table) - 1)].double()[:, None]
            cos, sin = row[..., :R // 2], row[..., R // 2:]
            z[..., a], z[..., b] = y[..., a] * cos - y[..., b] * sin, y[..., b] * cos + y[..., a] * sin
            size[..., a] = size[..., b] = y[..., a].abs() + y[..., b].abs()
        return z, size

    def check(self):
        pos, slots = self.pos.long(), self.slots
        fine = (pos >= 0) & ((pos < len(self.table)) if self.R else True)
        z, size = self.head(self.q64, self.qn)
        want, got = z[fine], self.q[fine].double()
        assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -17 * size[fine]).all()
        assert torch.equal(self.q[~fine], self.before[0][~fine])
        kept = fine & (slots >= 0) & (slots < self.n_pages * self.page)
        at = slots[kept]
        for cache, old, s, (z, size) in zip(self.caches, self.before[1:], self.scales,
                                            (self.head(self.k64, self.kn), (self.v64, torch.zeros_like(self.v64)))):
            if cache.shape[1] != self.Hkv or cache.shape[3] != self.D:      # the odd layout
                assert torch.equal(cache[..., self.D:], old[..., self.D:])
                cache, old = (c[..., :self.D].transpose(1, 2) for c in (cache, old))
            flat, was = (c.transpose(1, 2).reshape(-1, self.Hkv, self.D) for c in (cache, old))
            got, want, size = flat[at], z[kept], size[kept]
            if s is None:
                assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -17 * size).all()
            else:
                want, size = (want / s.double()[:, None]).clamp(-448, 448), size / s.double()[:, None]
                got = got.view(torch.float8_e4m3fn).double()
                assert ((got - want).abs() <= (2.0 ** -4 * want.abs()).clamp(min=2.0 ** -10) + 2.0 ** -16 * size).all()
            rest = torch.ones(len(flat), dtype=torch.bool, device=DEV)
            rest[at] = False
            assert torch.equal(flat[rest], was[rest])


CASES = [
    dict(T=1, Hq=32, Hkv=8, D=128, R=128), dict(T=8, Hq=32, Hkv=8, D=128, R=128), dict(T=3, Hq=1, Hkv=1, D=64, R=64),
    dict(T=5, Hq=7, Hkv=1, D=128, R=64), dict(T=17, Hq=6, Hkv=3, D=128, R=96), dict(T=40, Hq=5, Hkv=5, D=64, R=16),
    dict(T=9, Hq=4, Hkv=2, D=64, R=48), dict(T=33, Hq=56, Hkv=8, D=128, R=0), dict(T=2000, Hq=14, Hkv=2, D=128, R=128),
    dict(T=3001, Hq=9, Hkv=3, D=64, R=32), dict(T=700, Hq=56, Hkv=8, D=128, R=16)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("kw", CASES, ids=str)
def test_qkv_append(kw, inter, e4m3):
    c = Case(**kw, inter=inter, e4m3=e4m3, seed=kw["T"])
    c.run()
    moe.check_device_status(c.ws)
    c.check()


@pytest.mark.parametrize("kw", [
    dict(T=2000, Hq=56, Hkv=8, D=128, R=128), dict(T=2000, Hq=56, Hkv=8, D=128, R=128, e4m3=True),
    dict(T=1300, Hq=99, Hkv=3, D=128, R=64, inter=True, in_place=True), dict(T=4001, Hq=33, Hkv=3, D=64, R=64, e4m3=True, odd_cache=True),
    dict(T=1501, Hq=8, Hkv=8, D=128, R=0, norm=""), dict(T=12001, Hq=6, Hkv=2, D=64, R=48, inter=True, e4m3=True),
    dict(T=2100, Hq=40, Hkv=40, D=64, R=64, fused=False)], ids=str)
def test_many_heads(kw):
    c = Case(**kw, seed=9)
    c.pos[1] = c.pos[kw["T"] - 2] = -1
    c.slots[2] = -1
    c.run()
    moe.check_device_status(c.ws)
    c.check()


@pytest.mark.parametrize("kw", [dict(norm=""), dict(norm="q"), dict(norm="k"), dict(in_place=True), dict(fused=False),
                                dict(fused=False, in_place=True), dict(odd_cache=True), dict(odd_cache=True, e4m3=True),
                                dict(page=1024, e4m3=True), dict(R=0, norm="")], ids=str)
@pytest.mark.parametrize("T", [6, 1500])
def test_forms(kw, T):
    c = Case(**{**dict(T=T, Hq=12, Hkv=4, D=128, R=128, seed=3), **kw})
    c.run()
    moe.check_device_status(c.ws)
    c.check()


def test_without_norm_and_rotation_it_is_the_append():
    for e4m3 in (False, True):
        c = Case(T=50, Hq=8, Hkv=2, D=64, R=0, norm="", e4m3=e4m3)
        c.run()
        other = [b.clone() for b in c.before[1:]]
        moe.kv_append(c.shape, c.k, c.v, c.slots, *c.scales, *other, c.ws)
        assert torch.equal(c.q, c.q_in) and all(torch.equal(a, b) for a, b in zip(c.caches, other))


def test_rows_that_are_skipped_and_refused():
    c = Case(T=40, Hq=8, Hkv=2, D=128, R=64, max_pos=100)
    c.pos[3] = c.pos[39] = -1
    c.slots[5] = c.slots[39] = -1
    c.run()
    moe.check_device_status(c.ws)
    c.check()
    c.pos[7] = 100
    c.run()
    assert moe.device_status(c.ws) == (moe.MOE_ERR_BAD_LENGTHS, 7)
    c = Case(T=40, Hq=8, Hkv=2, D=128, R=64, max_pos=100)
    c.slots[9] = c.n_pages * 16 + 35
    c.run()
    assert moe.device_status(c.ws) == (moe.MOE_ERR_BAD_PAGE, c.n_pages + 2)
    c.check()


def test_a_row_that_is_not_finite_stays_its_own():
    c = Case(T=12, Hq=8, Hkv=2, D=128, R=64)
    c.q_in[4, 3, 70] = float("inf")        # behind the rotated part
    c.k[5, 1, 0] = float("nan")
    c.v[6, 0, 9] = float("nan")
    c.run()
    moe.check_device_status(c.ws)
    bad = ~c.q.isfinite()
    assert bad[4, 3].any() and not torch.cat([bad[:4], bad[5:]]).any() and not bad[4, :3].any() and not bad[4, 4:].any()
    flat = [x.transpose(1, 2).reshape(-1, 2, 128)[c.slots] for x in c.caches]
    assert flat[0][5, 1].isnan().all() and flat[0].isnan().sum() == 128
    assert flat[1][6, 0, 9].isnan() and flat[1].isnan().sum() == 1


def test_infinities_behind_the_rotation_without_a_norm():
    c = Case(T=4, Hq=2, Hkv=2, D=128, R=64, norm="")
    c.q_in[1, 1, 100] = float("inf")
    c.run()
    assert c.q[1, 1, 100] == float("inf") and (~c.q.isfinite()).sum() == 1


def test_captured_with_new_inputs_and_on_another_stream():
    c = Case(T=24, Hq=8, Hkv=2, D=128, R=128)
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    n = Case(T=24, Hq=8, Hkv=2, D=128, R=128, seed=5)
    for a, b in ((c.q_in, n.q_in), (c.k, n.k), (c.v, n.v), (c.pos, n.pos), (c.slots, n.slots)):
        a.copy_(b)
    for a, b in zip([c.q, *c.caches], c.before):
        a.copy_(b)
    c.q64, c.k64, c.v64 = c.q_in.double(), c.k.double(), c.v.double()
    graph.replay()
    torch.cuda.synchronize()
    c.check()
    n.qn, n.kn = c.qn, c.kn
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    n.run(side)
    side.synchronize()
    assert torch.equal(n.q, c.q) and all(torch.equal(a, b) for a, b in zip(n.caches, c.caches))


def test_rows_far_apart():
    # offsets of rows past 2^31 elements
    T, Hq, Hkv, D = 5, 4, 2, 64
    width = (1 << 29) + 64
    big = torch.zeros(T * width, dtype=torch.bfloat16, device=DEV)
    c = Case(T=T, Hq=Hq, Hkv=Hkv, D=D, R=64, fused=False)
    q, k, v = (big.as_strided((T, h, D), (width, D, 1), at) for h, at in ((Hq, 0), (Hkv, Hq * D), (Hkv, (Hq + Hkv) * D)))
    q.copy_(c.q_in), k.copy_(c.k), v.copy_(c.v)
    c.run()
    far = [c.q.clone()] + [x.clone() for x in c.caches]
    c.shape.kv_stride = c.rope.q_in_stride = width
    c.q_in, c.k, c.v = q, k, v
    for a, b in zip([c.q, *c.caches], c.before):
        a.copy_(b)
    c.run()
    moe.check_device_status(c.ws)
    assert all(torch.equal(a, b) for a, b in zip(far, [c.q, *c.caches]))
    c.check()
