"""Products by the cuts that test_gpu_mx.py's shapes do not take, against 64 bits with its tolerance."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import mxfp4_mixture_experts_route_gb300 as moe  # noqa: E402
from libmoe_util import ensure_built  # noqa: E402
from test_gpu_mx import check, product, tokens, values, weights  # noqa: E402

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
