"""Attention with a sink: one cached token takes most of each row's weight, and its V is next to nothing.

That is the usual shape of attention in language models.  The output is then
made of the many small weights beside the large one, so a number format of the
weights has to hold both.  The bound is that of weights in bf16, whatever the
cache's type (A = sum_j p_j |v_j|):
  - scores: e_s = D 2^-22 scale sum|q k| + 2^-21 |x| in the exponent (fp32 sums in any
    order, fp32 products with the scale), and with an e4m3 cache
    scale 2^-17 max|q| sum|k| for q as two e4m3 terms; p is off by 2 e_s p;
  - the weights' rounding 2^-9 each and their sum's none, the output's 2^-9 |o|,
    doubled for the fp32 sums' order: 2^-8 (A + |o|).
"""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import mxfp4_mixture_experts_route_gb300 as moe  # noqa: E402
from libmoe_util import ensure_built  # noqa: E402
from test_gpu_kv import Batch  # noqa: E402

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def encode(x, scale):
    return x.bfloat16() if scale is None else (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


class SinkBatch(Batch):
    """Every row's query has a part along one direction; the K of `at`, a cached token, lies along it."""

    def __init__(self, ctx, new, Hq, Hkv, D, e4m3, weight, at=0, seed=0):
        super().__init__(ctx, new, Hq, Hkv, D, 16, e4m3, tree=max(new) > 1, seed=seed, gain=0.3)
        g = torch.Generator(device=DEV)
        g.manual_seed(seed + 1)
        u = torch.randn(D, generator=g, device=DEV)
        u /= u.norm()
        along = 4.0
        self.q_rows += (along * u).bfloat16().repeat(Hq)
        scale = D ** -0.5
        var = (along * scale) ** 2 + 0.3 ** 2               # of the other keys' scores
        for b, c in enumerate(ctx):
            # ln of the others' sum, and the sink's share over theirs
            x = math.log(c + 1) + var / 2 + math.log(weight / (1 - weight))
            pg, o = self.table[b][at // 16], at % 16
            for h in range(Hkv):
                self.k[pg, h, o] = encode(u * (x / (along * scale)), self.ks[h] if e4m3 else None)
                self.v[pg, h, o] = encode(torch.full((D,), 1e-3, device=DEV), self.vs[h] if e4m3 else None)
        # V of mean 1: weights that are lost do not cancel
        if e4m3:
            for h in range(Hkv):
                v = self.v[:, h].view(torch.float8_e4m3fn).float() * self.vs[h]
                self.v[:, h] = torch.where(v.isnan() | (v.abs() < 2e-3), self.v[:, h], encode(v + 1, self.vs[h]))
        else:
            self.v.copy_(torch.where(self.v.isnan() | (self.v.abs() < 2e-3), self.v, self.v + 1))

    def tight(self, b):
        """(out, lse, tolerance of out, of lse, the sink's weights) of request b's rows."""
        c, n, G, scale = self.ctx[b], self.new[b], self.Hq // self.Hkv, self.D ** -0.5
        k, v = (x.repeat_interleave(G, 1) for x in (self.rows(self.k, self.ks, b), self.rows(self.v, self.vs, b)))
        q = self.q_rows[self.row_start[b]:self.row_start[b] + n].double().view(n, self.Hq, self.D)
        see = torch.cat([torch.ones(n, c, dtype=torch.bool), self.see[b]], 1).to(DEV)[:, None]
        x = torch.where(see, torch.einsum("ihd,jhd->ihj", q, k) * scale, float("-inf"))
        lse = torch.logsumexp(x, 2)
        p = torch.exp(x - lse[..., None])
        out, A = torch.einsum("ihj,jhd->ihd", p, v), torch.einsum("ihj,jhd->ihd", p, v.abs())
        e_s = self.D * 2.0 ** -22 * scale * torch.einsum("ihd,jhd->ihj", q.abs(), k.abs()) + 2.0 ** -21 * x.abs()
        if self.e4m3:
            e_s = e_s + scale * 2.0 ** -17 * q.abs().amax(2)[..., None] * k.abs().sum(2).T[None]
        e_s = torch.where(see, e_s, 0.0).amax(2, keepdim=True)
        tol_l = e_s[..., 0] + (c + n) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * lse.abs()
        return out, lse, 2.0 ** -8 * (A + out.abs()) + 2 * e_s * A, tol_l, p

    def check_tight(self, requests, at=0):
        moe.check_device_status(self.ws, "tree_attention")
        worst = 0.0
        for b in requests:
            o, l, tol, tol_l, p = self.tight(b)
            assert 0.5 < p[:, :, at].mean().item() < 0.98       # (it is a sink)
            r = slice(self.row_start[b], self.row_start[b] + self.new[b])
            worst = max(worst, ((self.out[r].double() - o).abs() / tol).max().item())
            assert ((self.lse[r].double() - l).abs() <= tol_l).all(), b
        assert worst <= 1.0, worst


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,Hq,Hkv", [(1, 4, 1), (1, 8, 1), (5, 8, 1), (8, 8, 1), (9, 8, 1), (16, 32, 2)])
@pytest.mark.parametrize("ctx,B,weight", [(4096, 320, 0.85), (16384, 160, 0.8), (16384, 160, 0.9)])
def test_sink_in_whole_segments(ctx, B, weight, n, Hq, Hkv, D, e4m3):
    # more segments than CTAs, so that most lie in one CTA's share; the sink in their first tile
    B //= Hkv
    t = SinkBatch([ctx] * B, [n] * B, Hq, Hkv, D, e4m3, weight, seed=ctx + n)
    t.run()
    t.check_tight([0, 1, B // 2, B - 1])


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,Hq,Hkv,at", [(1, 8, 2, 0), (8, 32, 4, 5), (7, 8, 1, 9000), (20, 32, 8, 700)])
def test_sink_in_divided_segments(n, Hq, Hkv, at, D, e4m3):
    t = SinkBatch([12000], [n], Hq, Hkv, D, e4m3, 0.85, at=at, seed=n)
    t.run()
    t.check_tight([0], at)
