"""Dense MXFP4 on the GPU against plain forms in 64 bits: quantise, read back, product.

Quantise and read back are exact or rounded once, so they are compared for equality.
The product's tolerance, with A = sum_k |x_k w_k| (all in 64 bits):
  - the products are exact in fp32; an fp32 sum of K of them in any order, with an
    adder that may truncate, is off by at most K 2^-23 A;
  - a bf16 x enters as two e4m3 terms, off by at most 2^-17 of its block's
    largest magnitude: sum_k 2^-17 max|x block| |w_k| more;
  - the result is rounded to bf16: 2^-8 of it (and of what is above).
"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import mxfp4_mixture_experts_route_gb300 as moe  # noqa: E402
from libmoe_util import ensure_built  # noqa: E402

DEV = "cuda"
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def values(codes, scales):
    """What codes and scale bytes stand for, in 64 bits."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    v = torch.tensor(GRID + [-x for x in GRID], dtype=torch.float64, device=DEV)[c]
    s = torch.exp2(scales.double() - 127)
    s[scales == 255] = float("nan")
    return v * s.repeat_interleave(32, -1)


def quantize_reference(x):
    """Codes and scale bytes by search: the scale from the block maximum's exponent, each code the nearest of the
    grid, of two as near the even one."""
    x = x.double().unflatten(-1, (-1, 32))
    top = x.abs().amax(-1)
    bad = ~x.isfinite().all(-1)
    e = torch.frexp(torch.where(bad, 1.0, top))[1].long() - 1            # floor(log2 top)
    byte = torch.where(top == 0, 0, (e - 2 + 127).clamp(min=0))
    v = torch.where(bad[..., None], 0.0, x / torch.exp2(byte.double() - 127)[..., None])
    grid = torch.tensor(GRID, dtype=torch.float64, device=DEV)
    code = torch.zeros(v.shape, dtype=torch.uint8, device=DEV)
    best = (v.abs() - grid[0]).abs()
    for i in range(1, 8):
        d = (v.abs() - grid[i]).abs()
        take = (d < best) | ((d == best) & (i % 2 == 0))
        code = torch.where(take, i, code)
        best = torch.minimum(best, d)
    code = torch.where(bad[..., None], 0, code + 8 * torch.signbit(v)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, torch.where(bad, 255, byte).to(torch.uint8)


def guarded(n, fill=0xAB):
    """A byte buffer with 64 bytes before and behind its n that have to stay."""
    buf = torch.full((n + 128,), fill, dtype=torch.uint8, device=DEV)
    return buf, buf[64:64 + n]


def guards_ok(buf, n, fill=0xAB):
    return bool((buf[:64] == fill).all() and (buf[64 + n:] == fill).all())


def spread_rows(seed, rows, K, dtype):
    """Normal values of very different blocks: zeros, ties, tiny, large, subnormal and saturating ones."""
    g = gen(seed)
    x = torch.randn(rows, K, generator=g, device=DEV, dtype=torch.float64).unflatten(1, (-1, 32))
    kind = torch.randint(0, 6, x.shape[:2], generator=g, device=DEV)[..., None]
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.25, -0.75, -5.0, 0.0, -0.0, 6.0, 7.5, 4.0],
                        dtype=torch.float64, device=DEV).repeat(2)
    x = torch.where(kind == 1, ties, x)
    x = torch.where(kind == 2, 0.0, x)
    x = torch.where(kind == 3, x * 2.0 ** (-16 if dtype == torch.float16 else -128), x)
    x = torch.where(kind == 4, x * 2.0 ** (11 if dtype == torch.float16 else 120), x)
    return x.flatten(1).to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,K,pad", [(1, 32, 0), (3, 96, 8), (65, 4096, 0), (700, 1056, 24), (5000, 2048, 0), (1, 65536, 0)])
def test_quantize(rows, K, pad, dtype):
    x = spread_rows(rows + K, rows, K + pad, DTYPES[dtype]) if pad == 0 else \
        torch.cat([spread_rows(rows, rows, K, DTYPES[dtype]), torch.full((rows, pad), float("nan"), dtype=DTYPES[dtype], device=DEV)], 1)
    x = x[:, :K]
    cb, codes = guarded(rows * K // 2)
    sb, scales = guarded(rows * K // 32)
    moe.mx_quantize(x, codes, scales)
    want = quantize_reference(x)
    assert torch.equal(scales.view(rows, -1), want[1])
    assert torch.equal(codes.view(rows, -1), want[0])
    assert guards_ok(cb, codes.numel()) and guards_ok(sb, scales.numel())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantize_every_pattern(dtype):
    # each pattern next to others of its own exponent, and next to others of any
    bits = torch.arange(65536, device=DEV, dtype=torch.int32)
    for order in (bits, bits[torch.randperm(65536, generator=gen(1), device=DEV)]):
        x = order.to(torch.int16).view(DTYPES[dtype]).view(64, 1024)
        codes = torch.empty(64, 512, dtype=torch.uint8, device=DEV)
        scales = torch.empty(64, 32, dtype=torch.uint8, device=DEV)
        moe.mx_quantize(x, codes, scales)
        want = quantize_reference(x)
        assert torch.equal(scales, want[1]) and torch.equal(codes, want[0])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_block_that_is_not_finite_reads_back_as_nan(bad):
    x = torch.randn(4, 128, device=DEV)
    x[1, 40], x[3, 127] = bad, bad
    codes = torch.empty(4, 64, dtype=torch.uint8, device=DEV)
    scales = torch.empty(4, 4, dtype=torch.uint8, device=DEV)
    y = torch.empty(4, 128, dtype=torch.bfloat16, device=DEV)
    moe.mx_quantize(x, codes, scales)
    moe.mx_dequantize(codes, scales, y)
    nan = torch.zeros(4, 128, dtype=torch.bool, device=DEV)
    nan[1, 32:64] = nan[3, 96:] = True
    assert torch.equal(y.isnan(), nan) and (scales == 255).sum() == 2
    assert (codes[1, 16:32] == 0).all() and (codes[3, 48:] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_dequantize_every_code_and_scale(dtype):
    scales = torch.arange(256, device=DEV).to(torch.uint8).view(256, 1)
    codes = (torch.arange(16, device=DEV).to(torch.uint8) * 16 + torch.arange(15, -1, -1, device=DEV).to(torch.uint8)).repeat(256, 1)
    y = torch.empty(256, 32, dtype=DTYPES[dtype], device=DEV)
    moe.mx_dequantize(codes, scales, y)
    want = values(codes, scales).float().to(DTYPES[dtype])
    assert torch.equal(y.isnan(), want.isnan())
    assert torch.equal(y.nan_to_num(7.0, float("inf"), float("-inf")), want.nan_to_num(7.0, float("inf"), float("-inf")))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,K,pad", [(1, 32, 8), (33, 96, 0), (70, 4096, 16), (4000, 1024, 0)])
def test_dequantize(rows, K, pad, dtype):
    g = gen(rows)
    codes = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    scales = torch.randint(118, 135, (rows, K // 32), dtype=torch.uint8, device=DEV, generator=g)
    full = torch.full((rows, K + pad), -7.0, dtype=DTYPES[dtype], device=DEV)
    y = full[:, :K]
    moe.mx_dequantize(codes, scales, y)
    assert torch.equal(y, values(codes, scales).to(DTYPES[dtype])) and (full[:, K:] == -7.0).all()


def test_rows_past_32_bit_offsets():
    rows, K = (1 << 21) + 3, 1056                       # 2^31 elements and some
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
    x[-2:] = torch.randn(2, K, device=DEV)
    x[0] = 1.0
    codes = torch.full((rows, K // 2), 255, dtype=torch.uint8, device=DEV)
    scales = torch.full((rows, K // 32), 255, dtype=torch.uint8, device=DEV)
    moe.mx_quantize(x, codes, scales)
    want = quantize_reference(x[-2:])
    assert torch.equal(codes[-2:], want[0]) and torch.equal(scales[-2:], want[1])
    assert not codes[1:-2].any() and not scales[1:-2].any() and (codes[0] == 0x66).all()
    moe.mx_dequantize(codes, scales, x)
    assert torch.equal(x[-2:], values(*want).bfloat16()) and (x[0] == 1).all() and not x[1:-2].any()


def test_quantize_takes_rows_of_more_dimensions():
    x = torch.randn(3, 5, 64, device=DEV, dtype=torch.bfloat16)
    codes, scales = (torch.empty(3, 5, n, dtype=torch.uint8, device=DEV) for n in (32, 2))
    moe.mx_quantize(x, codes, scales)
    want = quantize_reference(x)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------
def weights(seed, N, K):
    g = gen(seed)
    return (torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV, generator=g),
            torch.randint(116, 124, (N, K // 32), dtype=torch.uint8, device=DEV, generator=g))


def tokens(seed, T, K, kind):
    """(x, xs, x in 64 bits, the largest error of an element as it enters)."""
    g = gen(seed + 1000)
    if kind == "mxfp4":
        x = torch.randint(0, 256, (T, K // 2), dtype=torch.uint8, device=DEV, generator=g)
        xs = torch.randint(122, 130, (T, K // 32), dtype=torch.uint8, device=DEV, generator=g)
        return x, xs, values(x, xs), torch.zeros(T, K, dtype=torch.float64, device=DEV)
    x = torch.randn(T, K, device=DEV, generator=g) * torch.exp2(torch.randint(-12, 3, (T, K), device=DEV, generator=g).float())
    x = x.bfloat16()
    top = x.double().abs().unflatten(1, (-1, 32)).amax(-1).repeat_interleave(32, 1)
    return x, None, x.double(), 2.0 ** -17 * top


def product(x, xs, w, ws, T, N, K, kind, work=None, out=None, x_stride=0, out_stride=0):
    shape = moe.MXShape.of(T, N, K, x_mxfp4=kind == "mxfp4", x_stride=x_stride, out_stride=out_stride)
    work = moe.new_mx_workspace(shape) if work is None else work
    out = torch.full((T, N), -77.0, dtype=torch.bfloat16, device=DEV) if out is None else out
    moe.mx_linear(shape, x, xs, w, ws, out, work)
    return out, work


def check(out, x64, off, w64):
    want, mass = x64 @ w64.T, x64.abs() @ w64.abs().T
    err = x64.shape[1] * 2.0 ** -23 * mass + off @ w64.abs().T
    tol = err + 2.0 ** -8 * (want.abs() + err)
    bad = (out.double() - want).abs() / tol.clamp(min=1e-300)
    assert bad.max() <= 1, (bad.max().item(), (bad > 1).sum().item(), (bad > 1).nonzero()[:4].tolist())


SHAPES = [(1, 8, 128), (1, 128, 256), (3, 136, 384), (8, 256, 1024), (5, 6144, 4096), (9, 1000, 640), (16, 512, 4224),
          (17, 264, 2048), (33, 1024, 1152), (64, 128, 7168), (65, 392, 512), (100, 2048, 1536), (128, 1280, 4096),
          (129, 160, 896), (255, 640, 2176), (257, 520, 1280), (300, 4096, 256), (1000, 1000, 1024), (2049, 768, 640),
          (700, 8, 65536), (5, 20000, 4096), (40, 9736, 5120), (3, 19464, 3968), (200, 6152, 16384)]


@pytest.mark.parametrize("kind", ["mxfp4", "bf16"])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_linear(T, N, K, kind):
    w, ws = weights(N + K, N, K)
    x, xs, x64, off = tokens(T + K, T, K, kind)
    out, work = product(x, xs, w, ws, T, N, K, kind)
    moe.check_device_status(work, "mx_linear")
    check(out, x64, off, values(w, ws))


@pytest.mark.parametrize("T,N,K,kind", [
    (1, 39680, 4096, "mxfp4"), (8, 40008, 3968, "mxfp4"), (30, 39680, 4096, "mxfp4"), (50, 39680, 4096, "mxfp4"),
    (100, 39688, 4096, "mxfp4"), (4, 39680, 4096, "bf16"), (8, 39688, 4096, "bf16"), (12, 40008, 3968, "bf16"),
    (30, 39680, 4096, "bf16"), (60, 39680, 4096, "bf16"), (40, 19848, 4224, "mxfp4")])
def test_linear_more_than_two_rounds_of_tiles(T, N, K, kind):
    w, ws = weights(N + K, N, K)
    x, xs, x64, off = tokens(T + K, T, K, kind)
    first, work = product(x, xs, w, ws, T, N, K, kind)
    again, _ = product(x, xs, w, ws, T, N, K, kind, work=work)
    moe.check_device_status(work, "mx_linear")
    assert torch.equal(first, again)
    check(first, x64, off, values(w, ws))


# the tilings and ways of sharing K that SHAPES does not reach, the pairs' in several rounds with ragged ends too
CUTS = [(1, 8, 1792, "bf16"), (1, 152, 2560, "bf16"), (1, 3040, 1536, "bf16"), (1, 3704, 1152, "bf16"),
        (1, 6128, 1408, "bf16"), (1, 9904, 512, "bf16"), (2, 8, 1920, "bf16"), (13, 3304, 2560, "bf16"),
        (16, 8, 1536, "bf16"), (16, 1032, 4096, "bf16"), (17, 1480, 5248, "bf16"), (17, 1480, 5248, "mxfp4"),
        (17, 6208, 1920, "bf16"), (29, 2056, 1024, "bf16"), (33, 1848, 3712, "bf16"), (33, 1912, 5248, "mxfp4"),
        (33, 2344, 2560, "bf16"), (33, 3240, 2816, "mxfp4"), (33, 3320, 2176, "mxfp4"), (33, 3416, 1920, "bf16"),
        (33, 6712, 1408, "bf16"), (33, 6712, 1408, "mxfp4"), (50, 4920, 1152, "mxfp4"), (50, 4952, 640, "bf16"),
        (61, 904, 4096, "bf16"), (100, 4976, 1152, "mxfp4"), (100, 10208, 640, "mxfp4"), (129, 1936, 5888, "mxfp4"),
        (129, 4032, 1920, "mxfp4"), (300, 8, 7936, "bf16"), (300, 8, 7936, "mxfp4"), (300, 280, 3456, "bf16"),
        (600, 8, 5248, "mxfp4"), (600, 16, 2432, "bf16"), (600, 16, 2432, "mxfp4"), (600, 5224, 384, "bf16"),
        (700, 9736, 1280, "bf16"), (700, 9736, 1280, "mxfp4"), (1000, 16, 3456, "bf16"), (1000, 16, 3456, "mxfp4"),
        (1000, 280, 3840, "mxfp4"), (1000, 1808, 640, "bf16"), (1000, 2640, 384, "mxfp4"),
        (1000, 3760, 128, "mxfp4"), (1000, 3904, 128, "mxfp4"), (1000, 4416, 128, "bf16"), (1000, 4912, 128, "bf16"),
        (1000, 4912, 128, "mxfp4"), (1000, 5568, 128, "bf16"), (1025, 6152, 384, "bf16"), (1025, 6152, 384, "mxfp4"),
        (1500, 4104, 640, "bf16"), (1500, 4104, 640, "mxfp4"), (2049, 2056, 1152, "bf16"),
        (2049, 2056, 1152, "mxfp4"), (4001, 1000, 2176, "bf16"), (4001, 1000, 2176, "mxfp4")]


@pytest.mark.parametrize("T,N,K,kind", CUTS)
def test_linear_every_cut(T, N, K, kind):
    w, ws = weights(N + K, N, K)
    x, xs, x64, off = tokens(T + K, T, K, kind)
    buf = torch.full((T + 2, N), -77.0, dtype=torch.bfloat16, device=DEV)
    out, work = product(x, xs, w, ws, T, N, K, kind, out=buf[1:-1])
    moe.check_device_status(work, "mx_linear")
    check(out, x64, off, values(w, ws))
    assert (buf[0] == -77.0).all() and (buf[-1] == -77.0).all()


@pytest.mark.parametrize("kind", ["mxfp4", "bf16"])
def test_linear_places_every_element(kind):
    # one element of x and of w at a time reaches the one place of out it belongs to
    T, N, K = 40, 200, 1152
    for t, n, k in [(0, 0, 0), (39, 199, 1151), (7, 127, 128), (8, 128, 129), (31, 130, 255), (32, 5, 1024), (15, 64, 1055)]:
        x = torch.zeros(T, K, device=DEV)
        x[t, k] = 3.0
        w = torch.zeros(N, K, device=DEV)
        w[n, k] = -0.5
        codes, scales = torch.empty(N, K // 2, dtype=torch.uint8, device=DEV), torch.empty(N, K // 32, dtype=torch.uint8, device=DEV)
        moe.mx_quantize(w, codes, scales)
        xc, xs = x.bfloat16(), None
        if kind == "mxfp4":
            xc, xs = torch.empty(T, K // 2, dtype=torch.uint8, device=DEV), torch.empty(T, K // 32, dtype=torch.uint8, device=DEV)
            moe.mx_quantize(x, xc, xs)
        out, _ = product(xc, xs, codes, scales, T, N, K, kind)
        want = torch.zeros(T, N, device=DEV)
        want[t, n] = -1.5
        assert torch.equal(out.float(), want)


@pytest.mark.parametrize("kind", ["mxfp4", "bf16"])
@pytest.mark.parametrize("T", [2, 70, 300])
def test_linear_strides_and_what_is_around(kind, T):
    N, K = 264, 1408
    w, ws = weights(4, N, K)
    x, xs, x64, off = tokens(5, T, K, kind)
    x_stride = 0
    if kind == "bf16":
        wide = torch.full((T, K + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
        wide[:, :K] = x
        x, x_stride = wide, K + 24
    full = torch.full((T + 4, N + 40), -77.0, dtype=torch.bfloat16, device=DEV)
    product(x, xs, w, ws, T, N, K, kind, out=full[2:], x_stride=x_stride, out_stride=N + 40)
    check(full[2:-2, :N], x64, off, values(w, ws))
    full[2:-2, :N] = -77.0
    assert (full == -77.0).all()


@pytest.mark.parametrize("kind", ["mxfp4", "bf16"])
def test_linear_repeats_bitwise_and_shares_a_workspace(kind):
    # shapes of different tilings through one workspace, back to back
    cases = [(T, N, K) for T, N, K in SHAPES if T <= 300]
    data = [(weights(i, N, K), tokens(i, T, K, kind)) for i, (T, N, K) in enumerate(cases)]
    most = max(moe.mx_workspace_bytes(moe.MXShape.of(*c, x_mxfp4=kind == "mxfp4")) for c in cases)
    big = max(cases, key=lambda c: moe.mx_workspace_bytes(moe.MXShape.of(*c, x_mxfp4=kind == "mxfp4")))
    work = moe.new_mx_workspace(moe.MXShape.of(*big, x_mxfp4=kind == "mxfp4"))
    assert work.numel() == most
    outs = [[product(x, xs, w, ws, *c, kind, work=work)[0] for c, ((w, ws), (x, xs, _, _)) in zip(cases, data)] for _ in range(3)]
    moe.check_device_status(work, "mx_linear")
    for c, a, b, e, ((w, ws), (_, _, x64, off)) in zip(cases, *outs, data):
        assert torch.equal(a, b) and torch.equal(a, e), c
        check(a, x64, off, values(w, ws))


def test_linear_captured_and_on_another_stream():
    T, N, K = 8, 768, 1024
    w, ws = weights(1, N, K)
    x, _, _, _ = tokens(2, T, K, "bf16")
    shape, qshape = moe.MXShape.of(T, N, K), moe.MXShape.of(T, 1024, N, x_mxfp4=True)
    w2, ws2 = weights(3, 1024, N)
    work, work2 = moe.new_mx_workspace(shape), moe.new_mx_workspace(qshape)
    y, z = torch.empty(T, N, dtype=torch.bfloat16, device=DEV), torch.empty(T, 1024, dtype=torch.bfloat16, device=DEV)
    yc, ys = torch.empty(T, N // 2, dtype=torch.uint8, device=DEV), torch.empty(T, N // 32, dtype=torch.uint8, device=DEV)

    def chain(stream=None):
        moe.mx_linear(shape, x, None, w, ws, y, work, stream)
        moe.mx_quantize(y, yc, ys, stream)
        moe.mx_linear(qshape, yc, ys, w2, ws2, z, work2, stream)

    chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    side = torch.cuda.Stream()
    for i in range(5):
        x.copy_(tokens(i + 9, T, K, "bf16")[0])
        graph.replay()
        torch.cuda.synchronize()
        got = z.clone()
        check(y, x.double(), tokens(i + 9, T, K, "bf16")[3], values(w, ws))
        assert [t.tolist() for t in quantize_reference(y)] == [yc.tolist(), ys.tolist()]
        check(z, values(yc, ys), torch.zeros(T, N, dtype=torch.float64, device=DEV), values(w2, ws2))
        z.zero_()
        torch.cuda.synchronize()
        chain(side)
        side.synchronize()
        assert torch.equal(z, got)
    moe.check_device_status(work)
    moe.check_device_status(work2)


@pytest.mark.parametrize("T", [4, 80, 400])
@pytest.mark.parametrize("kind", ["mxfp4", "bf16"])
def test_linear_rows_that_are_not_finite(kind, T):
    N, K = 136, 640
    w, ws = weights(8, N, K)
    w[0] = 0                                            # (zero weights too: NaN, as 0 * NaN)
    x, xs, x64, off = tokens(9, T, K, kind)
    if kind == "mxfp4":
        xs[1, 7] = xs[T - 1, 19] = 255
    else:
        x[1, 230], x[T - 1, 639] = float("inf"), float("nan")
    out, work = product(x, xs, w, ws, T, N, K, kind)
    moe.check_device_status(work)
    keep = [t for t in range(T) if t not in (1, T - 1)]
    assert out[[1, T - 1]].isnan().all()
    check(out[keep], x64[keep], off[keep], values(w, ws))


@pytest.mark.parametrize("kind", ["mxfp4", "bf16"])
def test_linear_weight_scale_of_255(kind):
    T, N, K = 20, 300 // 8 * 8, 512
    w, ws = weights(8, N, K)
    ws[5, 3] = ws[N - 1, 15] = 255
    x, xs, x64, off = tokens(9, T, K, kind)
    out, work = product(x, xs, w, ws, T, N, K, kind)
    assert moe.device_status(work) == (moe.MOE_ERR_BAD_SCALE, 255)
    assert out[:, [5, N - 1]].isnan().all()
    keep = [n for n in range(N) if n not in (5, N - 1)]
    check(out[:, keep], x64, off, values(w[keep], ws[keep]))
    moe.check_device_status(work)


@pytest.mark.parametrize("kind", ["mxfp4", "bf16"])
@pytest.mark.parametrize("low,high", [(0, 6), (240, 246)])
def test_linear_extreme_scales(kind, low, high):
    # weights of 2^-127 and up against large x, and of 2^113 and up against small x: the products are ordinary
    T, N, K = 24, 136, 384
    g = gen(3)
    w, ws = weights(8, N, K)
    ws = torch.randint(low, high, ws.shape, dtype=torch.uint8, device=DEV, generator=g)
    shift = 100 if low == 0 else -100
    x, xs, x64, off = tokens(9, T, K, kind)
    if kind == "mxfp4":
        xs = (xs.int() + shift).to(torch.uint8)
        x64, off = values(x, xs), off
    else:
        x = (x.double() * 2.0 ** shift).bfloat16()
        x64, off = x.double(), off * 2.0 ** shift
    out, work = product(x, xs, w, ws, T, N, K, kind)
    moe.check_device_status(work)
    check(out, x64, off, values(w, ws))


@pytest.mark.parametrize("T", [1, 3, 8])
def test_linear_few_tokens_place_every_element(T):
    N, K = 136, 1536
    g = gen(T)
    for _ in range(6):
        t, n, k = (int(torch.randint(0, m, (1,), device=DEV, generator=g)) for m in (T, N, K))
        x = torch.zeros(T, K, device=DEV, dtype=torch.bfloat16)
        x[t, k] = 3.0
        w = torch.zeros(N, K, device=DEV)
        w[n, k] = -0.5
        codes, scales = torch.empty(N, K // 2, dtype=torch.uint8, device=DEV), torch.empty(N, K // 32, dtype=torch.uint8, device=DEV)
        moe.mx_quantize(w, codes, scales)
        out, _ = product(x, None, codes, scales, T, N, K, "bf16")
        want = torch.zeros(T, N, device=DEV)
        want[t, n] = -1.5
        assert torch.equal(out.float(), want)


@pytest.mark.parametrize("T,bad", [(1, 0), (6, 2), (8, 7)])
def test_linear_few_tokens_that_are_not_finite(T, bad):
    N, K = 200, 2048
    w, ws = weights(8, N, K)
    w[0] = 0
    x, _, x64, off = tokens(9, T, K, "bf16")
    x[bad, 1000] = float("-inf")
    out, work = product(x, None, w, ws, T, N, K, "bf16")
    moe.check_device_status(work)
    keep = [t for t in range(T) if t != bad]
    assert out[bad].isnan().all()
    if keep:
        check(out[keep], x64[keep], off[keep], values(w, ws))


@pytest.mark.parametrize("T,N,K,kind", [(1 << 20, 8, 128, "bf16"), (1 << 20, 8, 128, "mxfp4"), (1, 1 << 20, 128, "bf16"),
                                        (2, 1 << 20, 128, "mxfp4")])
def test_linear_largest_sides(T, N, K, kind):
    w, ws = weights(1, N, K)
    x, xs, x64, off = tokens(2, T, K, kind)
    out, work = product(x, xs, w, ws, T, N, K, kind)
    moe.check_device_status(work)
    check(out, x64, off, values(w, ws))


def test_linear_out_rows_past_32_bit_offsets():
    T, N, K = 5, 136, 256
    stride = (1 << 29) + 8                              # the last row begins past 2^31 elements
    w, ws = weights(1, N, K)
    for kind in ("bf16", "mxfp4"):
        x, xs, x64, off = tokens(2, T, K, kind)
        big = torch.full((T * stride,), -77.0, dtype=torch.bfloat16, device=DEV)
        out = big.as_strided((T, N), (stride, 1))
        product(x, xs, w, ws, T, N, K, kind, out=out, out_stride=stride)
        check(out, x64, off, values(w, ws))
        out.fill_(-77.0)
        assert (big == -77.0).all()


def test_linear_on_two_streams_at_once():
    # every way of sharing the work out, beside another call on another stream
    cases = [(8, 7168, 4096, "mxfp4"), (5, 20000, 4096, "bf16"), (600, 2048, 1024, "bf16"), (300, 6144, 2048, "mxfp4"),
             (100, 1024, 4096, "bf16"), (1000, 1536, 512, "mxfp4")]
    data = []
    for i, (T, N, K, kind) in enumerate(cases):
        w, ws = weights(i, N, K)
        x, xs, _, _ = tokens(i, T, K, kind)
        shape = moe.MXShape.of(T, N, K, x_mxfp4=kind == "mxfp4")
        outs = [torch.empty(T, N, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
        data.append((shape, x, xs, w, ws, outs, [moe.new_mx_workspace(shape) for _ in range(3)]))
    for shape, x, xs, w, ws, outs, works in data:
        moe.mx_linear(shape, x, xs, w, ws, outs[2], works[2])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream(priority=-1)]
    for _ in range(10):
        for k, stream in enumerate(streams):
            for i in range(len(data)):
                shape, x, xs, w, ws, outs, works = data[(i + 3 * k) % len(data)]
                moe.mx_linear(shape, x, xs, w, ws, outs[k], works[k], stream)
        torch.cuda.synchronize()
        for shape, x, xs, w, ws, outs, works in data:
            assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[2])
    for d in data:
        for work in d[-1]:
            moe.check_device_status(work)


def test_two_graphs_share_a_workspace():
    T1, N1, K1, T2, N2, K2 = 5, 20000, 4096, 40, 1000, 2176
    a, b = moe.MXShape.of(T1, N1, K1), moe.MXShape.of(T2, N2, K2)
    work = moe.new_mx_workspace(max((a, b), key=moe.mx_workspace_bytes))
    (w1, s1), (w2, s2) = weights(1, N1, K1), weights(2, N2, K2)
    x1, x2 = tokens(1, T1, K1, "bf16")[0], tokens(2, T2, K2, "bf16")[0]
    o1, o2 = torch.empty(T1, N1, dtype=torch.bfloat16, device=DEV), torch.empty(T2, N2, dtype=torch.bfloat16, device=DEV)

    def first():
        moe.mx_linear(a, x1, None, w1, s1, o1, work)

    def second():
        moe.mx_linear(b, x2, None, w2, s2, o2, work)

    graphs = []
    for call in (first, second):
        call()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    want = o1.clone(), o2.clone()
    for i in (0, 1, 1, 0, 0, 1):
        (o1, o2)[i].zero_()
        graphs[i].replay()
        graphs[1 - i].replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, want[0]) and torch.equal(o2, want[1])
    moe.check_device_status(work)
