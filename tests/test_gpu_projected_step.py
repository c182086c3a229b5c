"""Verify steps from the layers' input rows: projection, norms and append, attention, projection, block, in one graph.

Each call is checked on the inputs that it found, by its own tolerance:
  - a product: fp32 sums (K 2^-23 A, A = sum |x w|), a bf16 x as two e4m3 terms (2^-17 of its block's
    largest magnitude each), one rounding to bf16 (2^-8);
  - the norms and rotation: 2^-17 (|y_i| + |y_j|) and one rounding (bf16 2^-8; the cache's e4m3 2^-4, or
    half of its smallest step, 2^-10);
  - the attention: bf16 weights and a bf16 result, 2^-7 of sum p |v| and 2^-8 of itself.
"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import mxfp4_mixture_experts_route_gb300 as moe  # noqa: E402
from libmoe_util import ensure_built  # noqa: E402
from test_gpu_mx import check as check_product, quantize_reference, values  # noqa: E402

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def rotated(x, w, pos, table):
    """(z, |y_i| + |y_j|) of head rows x [rows, heads, D] in 64 bits."""
    y = x.double()
    y = y * (y.square().mean(-1, keepdim=True) + float(torch.tensor(1e-6))).rsqrt() * w.double()
    half = y.shape[-1] // 2
    cos, sin = table[pos.long()].double()[:, None].split(half, 2)
    a, b = y[..., :half], y[..., half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1), (a.abs() + b.abs()).repeat(1, 1, 2)


@pytest.mark.parametrize("e4m3", [False, True])
def test_projected_steps(e4m3):
    from mxfp4_mixture_experts_route_gb300.verify_step import VerifyStep
    s = VerifyStep(B=3, n=6, layers=2, page=8, most_ctx=200, e4m3=e4m3, projections=True, H=512, Hq=8, Hkv=2)
    Hq, Hkv = 8, 2
    kept = [[[[], []] for _ in range(s.B)] for _ in range(s.layers)]      # layer, request: rows of K, of V as cached
    for _ in range(6):
        trees, paths = s.draft()
        s.step(trees)
        rows, starts = sum(map(len, trees)), s.row_start.tolist()
        pos, slots = s.positions[:rows], s.slots[:rows]
        for layer in range(s.layers):
            # the fused projection
            x = s.x[layer].double()
            top = x.abs().unflatten(1, (-1, 32)).amax(-1).repeat_interleave(32, 1)
            check_product(s.qkv[layer].flatten(1), x, 2.0 ** -17 * top, values(*s.w_qkv[layer]))
            # heads to q and the cache
            qkv = s.qkv[layer][:rows]
            z, size = rotated(qkv[:, :Hq], s.norms[layer][0], pos, s.rope_table)
            assert ((s.q[layer][:rows].double() - z).abs() <= 2.0 ** -8 * z.abs() + 2.0 ** -17 * size).all()
            new = []
            for c, (want, size), scale in zip(s.caches[layer], (rotated(qkv[:, Hq:Hq + Hkv], s.norms[layer][1], pos, s.rope_table),
                                                                (qkv[:, Hq + Hkv:].double(), 0.0)), (s.k_scale, s.v_scale)):
                got = c.transpose(1, 2).reshape(-1, Hkv, 128)[slots]
                if e4m3:
                    f, got = scale.double()[:, None], got.view(torch.float8_e4m3fn).double()
                    w = (want / f).clamp(-448, 448)
                    assert ((got - w).abs() <= (2.0 ** -4 * w.abs()).clamp(min=2.0 ** -10) + 2.0 ** -16 * (size / f)).all()
                    new.append(got * f)
                else:
                    got = got.double()
                    assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -17 * size).all()
                    new.append(got)
            # the attention over what earlier steps kept and this step's rows
            for b, (tree, path) in enumerate(zip(trees, paths)):
                at = slice(starts[b], starts[b] + len(tree))
                k, v = (torch.stack(kept[layer][b][y] + list(new[y][at])).repeat_interleave(Hq // Hkv, 1) for y in (0, 1))
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
                score = torch.einsum("ihd,jhd->ihj", s.q[layer][at].double(), k) * s.shape.scale
                p = torch.softmax(torch.where(see[:, None], score, float("-inf")), 2)
                want, mass = torch.einsum("ihj,jhd->ihd", p, v), torch.einsum("ihj,jhd->ihd", p, v.abs())
                got = s.attn[layer][at].double()
                assert ((got - want).abs() <= 2.0 ** -7 * mass + 2.0 ** -8 * want.abs() + 1e-6).all()
                for y in (0, 1):
                    kept[layer][b][y] += [new[y][starts[b] + t] for t in path]
        # the last layer's rows, quantised, through the output projection (the buffers are shared by the layers)
        last = s.attn[-1].flatten(1)
        codes, scales = quantize_reference(last)
        assert torch.equal(codes, s.attn_codes) and torch.equal(scales, s.attn_scales)
        x = values(codes, scales)
        check_product(s.block_in[-1], x, torch.zeros_like(x), values(*s.w_o[-1]))
        block = s.blocks[-1]
        out = block.out.clone()
        assert torch.equal(out, block.forward(s.block_in[-1])[2]) and out.isfinite().all()
        s.accept(paths)
