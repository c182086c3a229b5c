"""Infinities and NaN among the cached tokens' V, with few rows: the right columns, in a bounded time.

Every row sees a cached token, so its column is what it holds.  Finding it out may look at a
column's keys once: 16,384 of them, at less than 0.5 us each, are 8 ms; a limit of 10 ms for the call.
"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import mxfp4_mixture_experts_route_gb300 as moe  # noqa: E402
from libmoe_util import ensure_built  # noqa: E402
from test_gpu_kv import Batch  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def put(t, b, key, column, value):
    t.v[t.table[b][key // t.page], :, key % t.page, column] = 0x7F if t.e4m3 else value


def timed(t):
    t.again()
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    t.again()
    b.record()
    moe.check_device_status(t.ws, "tree_attention")
    return a.elapsed_time(b)


@pytest.mark.parametrize("n,Hq", [(1, 7), (5, 8)])
@pytest.mark.parametrize("D,e4m3,value", [(64, False, float("inf")), (64, False, float("nan")), (64, True, float("nan")),
                                          (128, True, float("nan")), (128, False, float("inf"))])
def test_specials_of_cached_tokens(D, e4m3, value, n, Hq):
    B, ctx = 160, 16384                     # a request a CTA and more: whole segments
    t = Batch([ctx] * B, [n] * B, Hq, 1, D, 64, e4m3, tree=n > 1, seed=21)
    t.run()
    clean = t.out.clone(), t.lse.clone()
    for b in range(B):
        put(t, b, 1000 + 90 * b, 33, value)
        put(t, b, 16000, 34, value)         # (of the same four columns)
    ms = timed(t)
    special = (lambda x: x.isnan()) if value != value else (lambda x: x == value)
    assert special(t.out[:, :, 33:35]).all()
    rest = [x for x in range(D) if x not in (33, 34)]
    assert torch.equal(t.out[:, :, rest], clean[0][:, :, rest]) and torch.equal(t.lse, clean[1])
    assert ms < 10.0, ms


@pytest.mark.parametrize("D,e4m3", [(64, False), (64, True), (128, True)])
def test_both_infinities_or_a_nan_beside_one(D, e4m3):
    t = Batch([3000], [3], 8, 1, D, 16, e4m3, tree=True, seed=22)
    t.run()
    clean = t.out.clone()
    put(t, 0, 10, 5, float("inf"))
    put(t, 0, 2900, 5, float("-inf"))
    put(t, 0, 700, 9, float("inf"))
    put(t, 0, 701, 9, float("nan"))
    put(t, 0, 300, 60, float("-inf"))
    t.run()
    moe.check_device_status(t.ws, "tree_attention")
    assert t.out[:, :, [5, 9]].isnan().all()
    assert (t.out[:, :, 60].isnan() if e4m3 else t.out[:, :, 60] == float("-inf")).all()
    rest = [x for x in range(D) if x not in (5, 9, 60)]
    assert torch.equal(t.out[:, :, rest], clean[:, :, rest])


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_nothing_but_nan(e4m3):
    """Wide trees over a V of NaN: every row, its 4 columns at a time, 4 M pieces, 3,450 for each warp; below 50 us each 175 ms."""
    t = Batch([4096] * 4, [1024] * 4, 32, 8, 128, 64, e4m3, tree=True, seed=23)
    t.v.fill_(0x7F if e4m3 else float("nan"))
    t.run()
    ms = timed(t)
    assert t.out.isnan().all() and t.lse.isfinite().all()
    assert ms < 175.0, ms
