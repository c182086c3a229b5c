"""Refusals of the dense MXFP4 calls and of qkv_append (no GPU): they return before anything is enqueued."""
import ctypes

import pytest

import mxfp4_mixture_experts_route_gb300 as moe
from libmoe_util import ensure_built

INVALID, SHAPE, ALIGN, WS = (moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED_SHAPE, moe.MOE_ERR_ALIGNMENT,
                             moe.MOE_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def L():
    return ensure_built()


@pytest.mark.parametrize("name", ["moe_mx_quantize", "moe_mx_dequantize"])
@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), INVALID), (dict(rows=-1), INVALID), (dict(K=0), INVALID), (dict(dtype=3), INVALID),
    (dict(dtype=-1), INVALID), (dict(stride=-8), INVALID), (dict(wide=None), INVALID), (dict(codes=None), INVALID),
    (dict(scales=None), INVALID), (dict(K=48), SHAPE), (dict(K=(1 << 20) + 32), SHAPE), (dict(rows=1 << 38), SHAPE),
    (dict(stride=64), SHAPE), (dict(stride=1 << 40), SHAPE), (dict(rows=1 << 30, stride=1 << 35), SHAPE),
    (dict(stride=132), ALIGN), (dict(stride=130, dtype=2), ALIGN), (dict(wide=0x1008), ALIGN),
    (dict(codes=0x2004), ALIGN), (dict(scales=0x3001), ALIGN)])
def test_rows(L, name, kw, code):
    a = dict(rows=4, K=128, dtype=0, wide=0x1000, stride=0, codes=0x2000, scales=0x3000)
    a.update(kw)
    wide = [a["wide"], a["stride"]]
    args = wide + [a["codes"], a["scales"]] if name == "moe_mx_quantize" else [a["codes"], a["scales"]] + wide
    assert getattr(L, name)(a["rows"], a["K"], a["dtype"], *args, None) == code


def nbytes(L, s):
    n = ctypes.c_size_t(0)
    return L.moe_mx_workspace_bytes(ctypes.byref(s) if s is not None else None, ctypes.byref(n)), n.value


BASE = dict(T=8, N=256, K=512)


@pytest.mark.parametrize("kw", [{}, dict(T=1 << 20, K=128), dict(N=8), dict(N=1 << 20), dict(K=128), dict(K=65536),
                                dict(x_stride=520), dict(out_stride=264), dict(x_mxfp4=True), dict(x_mxfp4=True, x_stride=512)])
def test_supported_shapes(L, kw):
    rc, n = nbytes(L, moe.MXShape.of(**{**BASE, **kw}))
    assert rc == moe.MOE_OK and n % 256 == 0 and n >= 256


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(x_stride=-8), INVALID),
    (dict(out_stride=-8), INVALID), (dict(T=(1 << 20) + 1), SHAPE), (dict(N=12), SHAPE), (dict(N=(1 << 20) + 8), SHAPE),
    (dict(K=192), SHAPE), (dict(K=65536 + 128), SHAPE), (dict(x_stride=504), SHAPE), (dict(out_stride=248), SHAPE),
    (dict(x_stride=1 << 38), SHAPE), (dict(x_mxfp4=True, x_stride=520), SHAPE), (dict(x_stride=516), ALIGN),
    (dict(out_stride=260), ALIGN)])
def test_refused_shapes(L, kw, code):
    assert nbytes(L, moe.MXShape.of(**{**BASE, **kw}))[0] == code


def linear(L, s, **kw):
    a = dict(x=0x1000, xs=None, w=0x2000, ws=0x3000, out=0x4000, work=0x10000, nbytes=None)
    a.update(kw)
    n = nbytes(L, s)[1] if a["nbytes"] is None else a["nbytes"]
    return L.moe_mx_linear(ctypes.byref(s), a["x"], a["xs"], a["w"], a["ws"], a["out"], a["work"], n, None)


def test_linear_arguments(L):
    s, m = moe.MXShape.of(**BASE), moe.MXShape.of(**BASE, x_mxfp4=True)
    for name in ("x", "w", "ws", "out", "work"):
        assert linear(L, s, **{name: None}) == INVALID
        assert linear(L, s, **{name: 0x9008}) == ALIGN
    assert linear(L, s, w=0x2010) == ALIGN                    # 32 bytes
    assert linear(L, s, work=0x10080) == ALIGN
    assert linear(L, s, nbytes=nbytes(L, s)[1] - 1) == WS
    assert linear(L, s, xs=0x5000) == INVALID and linear(L, m) == INVALID     # scales go with MXFP4 x
    assert linear(L, m, xs=0x5008) == ALIGN
    s.flags = 2
    assert nbytes(L, s)[0] == INVALID
    assert nbytes(L, None)[0] == INVALID
    assert L.moe_mx_workspace_bytes(ctypes.byref(m), None) == INVALID


def qkv(L, shape, rope, **kw):
    a = dict(q_in=0x1000, k=0x2000, v=0x3000, pos=0x4000, slots=0x5000, qn=0x6000, kn=0x7000, table=0x8000, ks=None,
             vs=None, q=0x9000, kc=0xA000, vc=0xB000, ws=0x10000, nbytes=None)
    a.update(kw)
    n = ctypes.c_size_t(0)
    L.moe_kv_workspace_bytes(ctypes.byref(shape), ctypes.byref(n))
    return L.moe_qkv_append(ctypes.byref(shape), ctypes.byref(rope) if rope is not None else None, a["q_in"], a["k"],
                            a["v"], a["pos"], a["slots"], a["qn"], a["kn"], a["table"], a["ks"], a["vs"], a["q"],
                            a["kc"], a["vc"], a["ws"], n.value if a["nbytes"] is None else a["nbytes"], None)


KV = dict(B=4, T=32, Hq=32, Hkv=8, D=128, page=64, n_pages=100, max_pages=20)


def test_qkv_arguments(L):
    s, r = moe.KVShape.of(**KV), moe.Rope.of(128, 4096)
    for name in ("q_in", "k", "v", "pos", "slots", "q", "kc", "vc", "ws"):
        assert qkv(L, s, r, **{name: None}) == INVALID
        assert qkv(L, s, r, **{name: 0xC008}) == ALIGN
    for name in ("qn", "kn", "table"):
        assert qkv(L, s, r, **{name: 0xC004}) == ALIGN
    assert qkv(L, s, None) == INVALID
    assert qkv(L, s, r, table=None) == INVALID and qkv(L, s, moe.Rope.of(0)) == INVALID
    assert qkv(L, s, r, nbytes=0) == WS
    assert qkv(L, s, r, ks=0xC000, vs=0xC100) == INVALID
    e = moe.KVShape.of(**KV, e4m3=True)
    assert qkv(L, e, r) == INVALID and qkv(L, e, r, ks=0xC000) == INVALID
    # in place with rows at different distances
    assert qkv(L, s, moe.Rope.of(128, 4096, q_in_stride=48 * 128), q=0x1000) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(R=-16), INVALID), (dict(R=128, max_pos=0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(q_in_stride=-8), INVALID), (dict(R=8), SHAPE), (dict(R=144), SHAPE),
    (dict(q_in_stride=4088), SHAPE), (dict(q_in_stride=1 << 38), SHAPE), (dict(q_in_stride=4100), ALIGN)])
def test_rope(L, kw, code):
    a = dict(R=64, max_pos=100)
    a.update(kw)
    assert qkv(L, moe.KVShape.of(**KV), moe.Rope.of(**a)) == code


def test_rope_flags(L):
    r = moe.Rope.of(64, 100, interleaved=True)
    r.flags |= 2
    assert qkv(L, moe.KVShape.of(**KV), r) == INVALID


def test_binding_refuses_rows_it_cannot_describe():
    torch = pytest.importorskip("torch")
    c, s = torch.empty(4, 32, dtype=torch.uint8), torch.empty(4, 2, dtype=torch.uint8)
    for x in (torch.empty(4, 64, dtype=torch.float64), torch.empty(64, 4).t(), torch.empty(1, 64).expand(4, 64)):
        with pytest.raises(moe.MoEError) as e:
            moe.mx_quantize(x, c, s)
        assert e.value.code == INVALID
    for codes, scales in ((c[:3], s), (c, s[:, :1]), (c.t(), s), (torch.empty(4, 32), s)):
        with pytest.raises(moe.MoEError) as e:
            moe.mx_dequantize(codes, scales, torch.empty(4, 64))
        assert e.value.code == INVALID


def test_binding_refuses_what_has_no_rows():
    torch = pytest.importorskip("torch")
    c, s = torch.empty(4, 32, dtype=torch.uint8), torch.empty(4, 2, dtype=torch.uint8)
    for x in (torch.tensor(1.0), torch.empty(0, 64)):
        with pytest.raises(moe.MoEError) as e:
            moe.mx_quantize(x, c, s)
        assert e.value.code == INVALID


@pytest.mark.parametrize("x_mxfp4", [False, True])
@pytest.mark.parametrize("N,K", [(6144, 2048), (6144, 4096), (512, 8192), (1024, 2560), (5120, 1536), (8, 128), (264, 640),
                                 (9216, 7168), (14336, 65536)])
def test_a_workspace_serves_fewer_rows(L, N, K, x_mxfp4):
    # whatever tiles a row count takes, and for every N and smaller K too
    sizes = [nbytes(L, moe.MXShape.of(T, N, K, x_mxfp4=x_mxfp4)) for T in [*range(1, 300), 511, 512, 1000, 4096, 1 << 20]]
    assert all(rc == moe.MOE_OK for rc, _ in sizes) and sizes == sorted(sizes)
    for T in (1, 8, 9, 24, 49, 300, 4096):
        n = nbytes(L, moe.MXShape.of(T, N, K, x_mxfp4=x_mxfp4))[1]
        assert all(nbytes(L, moe.MXShape.of(T, m, K, x_mxfp4=x_mxfp4))[1] == n for m in (8, 1000, 6144, 1 << 20))
        assert nbytes(L, moe.MXShape.of(T, N, max(128, K // 256 * 128), x_mxfp4=x_mxfp4))[1] <= n
        assert nbytes(L, moe.MXShape.of(T, N, K, x_mxfp4=True))[1] <= n


class Product:
    """Tensors of a product on the host: calls that the binding lets through end at the workspace, of one byte."""

    def __init__(self, T=5, N=72, K=256, x_mxfp4=False, **strides):
        import torch

        def u8(*size):
            return torch.zeros(size, dtype=torch.uint8)

        self.shape = moe.MXShape.of(T, N, K, x_mxfp4=x_mxfp4, **strides)
        self.x, self.xs = (u8(T, K // 2), u8(T, K // 32)) if x_mxfp4 else (torch.zeros(T, K, dtype=torch.bfloat16), None)
        self.w, self.w_scales, self.out = u8(N, K // 2), u8(N, K // 32), torch.zeros(T, N, dtype=torch.bfloat16)

    def code(self):
        import torch
        ws = torch.empty(512, dtype=torch.uint8)
        at = -ws.data_ptr() % 256
        with pytest.raises(moe.MoEError) as e:
            moe.mx_linear(self.shape, self.x, self.xs, self.w, self.w_scales, self.out, ws[at:at + 1], stream=NoStream)
        return e.value.code


class NoStream:
    cuda_stream = None


@pytest.mark.parametrize("x_mxfp4", [False, True])
def test_product_binding_refuses_tensors_too_small(L, x_mxfp4):
    assert Product(x_mxfp4=x_mxfp4).code() == WS
    for name in ("x", "xs", "w", "w_scales", "out"):
        p = Product(x_mxfp4=x_mxfp4)
        t = getattr(p, name)
        if t is None:
            continue
        setattr(p, name, t[:-1])                                # a row too few
        assert p.code() == INVALID, name
        setattr(p, name, t[:, :-8].contiguous())                # rows too short
        assert p.code() == INVALID, name
        setattr(p, name, t.t().contiguous().t())                # the other way round
        assert p.code() == INVALID, name
        setattr(p, name, t[:1].expand_as(t))                    # one row in the place of all
        assert p.code() == INVALID, name
        setattr(p, name, t.repeat(2, 1)[::2])                   # rows further apart than the descriptor says
        assert p.code() == INVALID, name
        setattr(p, name, t.repeat(2, 1))                        # more rows than are used
        assert p.code() == WS, name
        setattr(p, name, t.view(-1))                            # the same bytes
        assert p.code() == WS, name


def test_product_binding_takes_rows_apart(L):
    import torch
    p = Product(x_stride=264, out_stride=96)
    assert p.code() == INVALID                                  # packed rows
    wide, out = torch.zeros(5, 264, dtype=torch.bfloat16), torch.zeros(5, 96, dtype=torch.bfloat16)
    for x in (wide, wide[:, :256], wide.view(-1)[:4 * 264 + 256], wide.view(5, 33, 8)[:, :32]):
        for o in (out, out[:, :72], out.view(-1)[:4 * 96 + 72], out.view(5, 12, 8)[:, :9]):
            p.x, p.out = x, o
            assert p.code() == WS
    p.x, p.out = wide[:, :256], out[:, :64]                     # rows too short
    assert p.code() == INVALID
    p.out = out.view(-1)[:4 * 96 + 64]                          # the last one too short
    assert p.code() == INVALID
    p.out = out.float()[:, :72]                                 # of another size
    assert p.code() == INVALID
    p.out, p.x = out, wide.view(5, 33, 8)[:, ::2][:, :16]       # rows with gaps
    assert p.code() == INVALID
    p = Product(T=1)                                            # a single row, whatever stands between rows
    p.x, p.out = wide[:1, :256], out[:1, :72]
    assert p.code() == WS


def test_binding_refuses_rows_that_are_not_evenly_apart():
    torch = pytest.importorskip("torch")
    c, s = torch.empty(4, 2, 32, dtype=torch.uint8), torch.empty(4, 2, 2, dtype=torch.uint8)
    for x in (torch.empty(4, 3, 64)[:, :2], torch.empty(2, 4, 64).transpose(0, 1), torch.empty(4, 2, 64).expand(1, 4, 2, 64)[:, :, [1]]
              .expand(1, 4, 2, 64)):
        for call in (lambda: moe.mx_quantize(x, c, s), lambda: moe.mx_dequantize(c, s, x)):
            with pytest.raises(moe.MoEError) as e:
                call()
            assert e.value.code == INVALID


def test_product_binding_takes_rows_of_more_dimensions(L):
    import torch
    p = Product(T=6, x_stride=264, out_stride=96)
    wide, out = torch.zeros(2, 3, 264, dtype=torch.bfloat16), torch.zeros(2, 3, 96, dtype=torch.bfloat16)
    p.x, p.out = wide[:, :, :256], out[:, :, :72]               # evenly apart through both dimensions
    assert p.code() == WS
    p.x, p.out = wide.view(6, 1, 33, 8)[:, :, :32], out.view(2, 3, 1, 12, 8)[..., :9, :]
    assert p.code() == WS
    p.x = torch.zeros(2, 4, 264, dtype=torch.bfloat16)[:, :3, :256]     # a gap behind every third row
    assert p.code() == INVALID
    p.x = torch.zeros(2, 8, 264, dtype=torch.bfloat16)[:, :6, :256]     # as above, but six before the gap
    assert p.code() == WS
    p.x = torch.zeros(3, 2, 264, dtype=torch.bfloat16).transpose(0, 1)[..., :256]
    assert p.code() == INVALID
    p = Product(T=6)
    p.x = torch.zeros(2, 8, 256, dtype=torch.bfloat16)[:, :6]           # packed rows, six of them in one piece
    assert p.code() == WS
    p.x = torch.zeros(2, 8, 256, dtype=torch.bfloat16)[:, :5]
    assert p.code() == INVALID
