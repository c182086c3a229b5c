"""The cache calls at sizes whose counts pass 31 bits."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import mxfp4_mixture_experts_route_gb300 as moe  # noqa: E402
from libmoe_util import ensure_built  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def test_append_of_more_pieces_than_31_bits_count():
    # 2^20 rows of 256 heads x 128: 2^32 pieces of 16 bytes; all rows but a few have no slot
    T, Hkv, D, page = 1 << 20, 256, 128, 8
    torch.cuda.empty_cache()
    x = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, 77777, (1 << 19) - 1, 1 << 19, T - 2, T - 1]
    for r in rows:
        x[r] = torch.randn(Hkv, D, device="cuda").bfloat16()
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    slots[rows] = torch.arange(len(rows), device="cuda") + 3
    shape = moe.KVShape.of(1, T, Hkv, Hkv, D, page, 2, 2)
    ws = moe.new_kv_workspace(shape)
    k, v = (torch.zeros(2, Hkv, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.kv_append(shape, x, x, slots, None, None, k, v, ws)
    moe.check_device_status(ws, "kv_append")
    for c in (k, v):
        flat = c.transpose(1, 2).reshape(2 * page, Hkv, D)
        assert torch.equal(flat[3:3 + len(rows)], x[rows])
        assert not flat[:3].any() and not flat[3 + len(rows):].any()
    del x
    torch.cuda.empty_cache()
