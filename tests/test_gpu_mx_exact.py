"""Products whose sums are exact, compared for equality, and the cuts that test_gpu_mx.py's shapes do not take.

Long sums of random values have a tolerance that hides a block of 32 elements left out.  Here every product
is +1, -1 or 0 (a block's weights are 2^-j and its one element of x 2^j), every partial sum in any order is a whole number
below 2^24, and so is exact in fp32, with an adder that truncates too.  A result of 256 or less is exact in bf16
and a block more or less shows in it; a larger one has to be the nearest bf16 all the same.
"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import mxfp4_mixture_experts_route_gb300 as moe  # noqa: E402
from libmoe_util import ensure_built  # noqa: E402
from test_gpu_mx import check, gen, product, tokens, values, weights  # noqa: E402

DEV = "cuda"

# (operands, CTAs of a tile, its tokens, CTAs that share its K): bf16 2, 64, 1; mxfp4 1, 128 and 1, 6, 7 and 8
CUTS = [(37, 205880, 384, "bf16"), (12345, 8, 896, "mxfp4"), (1187, 168, 10880, "mxfp4"), (580, 344, 12416, "mxfp4"),
        (369, 592, 14720, "mxfp4")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.mark.parametrize("T,N,K,kind", CUTS)
def test_cuts_of_their_own(T, N, K, kind):
    w, ws = weights(N + K, N, K)
    x, xs, x64, off = tokens(T + K, T, K, kind)
    buf = torch.full((T + 2, N), -77.0, dtype=torch.bfloat16, device=DEV)
    out, work = product(x, xs, w, ws, T, N, K, kind, out=buf[1:-1])
    moe.check_device_status(work, "mx_linear")
    for n in range(0, N, 16384):
        check(out[:, n:n + 16384], x64, off, values(w[n:n + 16384], ws[n:n + 16384]))
    assert (buf[0] == -77.0).all() and (buf[-1] == -77.0).all()


def signs(T, N, K, kind):
    """(x, xs, w, scales of w, the exact sums): one element of +-2^j in every block of a row of x, weights of +-2^-j."""
    g, blocks = gen(T + N + K), K // 32

    def bits(*shape):
        return torch.randint(0, 2, shape, generator=g, device=DEV)

    j = torch.randint(-20, 21, (blocks,), generator=g, device=DEV)
    at = torch.randint(0, 32, (T, blocks), generator=g, device=DEV)
    x = torch.zeros(T, blocks, 32, device=DEV).scatter_(2, at[..., None], 2.0 * bits(T, blocks)[..., None] - 1)
    # e2m1 codes: 2 is 1, 10 is -1
    w = bits(N, K)
    codes = 2 + 8 * w
    packed = (codes[:, 0::2] | codes[:, 1::2] << 4).to(torch.uint8)
    w_scales = (127 - j).to(torch.uint8).repeat(N, 1)
    want = x.flatten(1) @ (1.0 - 2.0 * w.float()).T
    if kind == "bf16":
        return (x * torch.exp2(j.float())[:, None]).flatten(1).bfloat16(), None, packed, w_scales, want
    c = torch.where(x > 0, 2, torch.where(x < 0, 10, 0)).flatten(1)
    return (c[:, 0::2] | c[:, 1::2] << 4).to(torch.uint8), (127 + j).to(torch.uint8).repeat(T, 1), packed, w_scales, want


# the longest K and one that ends in half a stage; few tokens to many, K whole and shared, single CTAs and pairs
@pytest.mark.parametrize("kind", ["mxfp4", "bf16"])
@pytest.mark.parametrize("K", [65536, 65408])
@pytest.mark.parametrize("T,N", [(1, 8), (3, 200), (33, 264), (250, 16), (740, 24), (1480, 8), (17, 9984), (40, 9768),
                                 (100, 9880), (225, 9864)])
def test_long_sums_leave_nothing_out(T, N, K, kind):
    x, xs, w, ws, want = signs(T, N, K, kind)
    assert want.abs().max() < 1 << 24 and (want.abs() <= 256).float().mean() > 0.99
    out, work = product(x, xs, w, ws, T, N, K, kind)
    moe.check_device_status(work, "mx_linear")
    assert torch.equal(out, want.bfloat16())


@pytest.mark.parametrize("kind", ["mxfp4", "bf16"])
@pytest.mark.parametrize("T,N,K", [(1, 6144, 4096), (8, 7168, 4096), (5, 1000, 2560), (16, 512, 16384), (50, 136, 12160),
                                   (100, 1000, 7040), (333, 1000, 4224), (600, 6152, 1152), (1187, 168, 10880), (580, 344, 12416),
                                   (369, 592, 14720)])
def test_sums_leave_nothing_out(T, N, K, kind):
    x, xs, w, ws, want = signs(T, N, K, kind)
    out, work = product(x, xs, w, ws, T, N, K, kind)
    moe.check_device_status(work, "mx_linear")
    assert torch.equal(out, want.bfloat16())


# K ends in half a stage: the scale bytes behind a row's are the next row's first, over codes that are zeros
@pytest.mark.parametrize("kind", ["mxfp4", "bf16"])
@pytest.mark.parametrize("T", [4, 20, 40, 100, 300])
@pytest.mark.parametrize("N,K", [(136, 640), (264, 384), (392, 1152), (4104, 128)])
def test_a_row_of_nan_leaves_the_row_before_it(T, N, K, kind):
    x, xs, w, ws, want = signs(T, N, K, kind)
    bad_t, bad_n = [2, T - 1], [1, 77, N - 1]
    for i, t in enumerate(bad_t):
        if kind == "mxfp4":
            xs[t, i:i + 2] = 255                    # among the row's first four scale bytes
        else:
            x[t, 32 * i + 5] = x[t, 32 * i + 90] = float("inf")
    for i, n in enumerate(bad_n):
        ws[n, i] = 255
    out, work = product(x, xs, w, ws, T, N, K, kind)
    assert moe.device_status(work) == (moe.MOE_ERR_BAD_SCALE, 255)
    nan = torch.zeros(T, N, dtype=torch.bool, device=DEV)
    nan[bad_t], nan[:, bad_n] = True, True
    assert torch.equal(out.isnan(), nan)
    assert torch.equal(out[~nan], want.bfloat16()[~nan])
