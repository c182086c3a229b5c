"""The free list's length on the device: a captured plan sees the list grow and shrink."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import mxfp4_mixture_experts_route_gb300 as moe  # noqa: E402
from libmoe_util import ensure_built  # noqa: E402
from test_gpu_kv import cdiv, i32, run_plan  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.mark.parametrize("B", [1, 3, 600])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("have", [0, 1, 2, 5])
def test_negative_entries_end_the_list(B, tree, have):
    # every request takes one page; the list has room for B + 4 and holds `have` fewer than are needed (at most B)
    have = max(0, B - have)
    parents = [-1, 0] * B if tree else None
    ids = list(range(have))
    got, ws = run_plan([0] * B, [2] * B, parents, ids + [-1] * (B + 4 - have), [[-7]] * B, 16, 2 * B, 1 if tree else 0,
                       B + 8)
    want = (moe.MOE_ERR_NO_PAGES, B - have) if have < B else (moe.MOE_OK, 0)
    rc, det = moe.device_status(ws)
    assert (rc, det if rc else 0) == want
    assert got["used"].tolist() == [2 * B, have]
    assert [r[0] for r in got["table"].tolist()] == ids + [-1] * (B - have)
    assert got["slots"].tolist() == [s for p in ids for s in (16 * p, 16 * p + 1)] + [-1] * (2 * (B - have))


def test_a_hole_in_the_list_is_reported():
    got, ws = run_plan([0] * 3, [1] * 3, None, [4, -1, 5, 6], [[-7]] * 3, 16, 3, 0, 8)
    assert moe.device_status(ws) == (moe.MOE_ERR_BAD_PAGE, -1)
    assert got["table"].tolist() == [[4], [-1], [5]] and got["slots"].tolist() == [64, -1, 80]


def test_captured_plan_sees_the_list_run_short():
    B, page, width = 4, 8, 3
    shape = moe.KVShape.of(B, 3 * B, 1, 1, 64, page, 16, width)
    ws = moe.new_kv_workspace(shape)
    ctx, new, free, used = i32([0] * B), i32([3] * B), i32(range(16)), i32([0, 0])
    table, rs, pos = i32([[-1] * width] * B), i32([0] * (B + 1)), i32([0] * (3 * B))
    slots = torch.zeros(3 * B, dtype=torch.int64, device="cuda")

    def plan():
        moe.kv_plan(shape, ctx, new, None, free, table, rs, slots, pos, None, used, ws)

    plan()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan()
    for held in (16, 4, 3, 0, 2, 5):
        free.copy_(i32([15 - i for i in range(held)] + [-1] * (16 - held)))
        graph.replay()
        rc, missing = moe.device_status(ws)
        assert (rc, missing) == ((moe.MOE_ERR_NO_PAGES, B - held) if held < B else (moe.MOE_OK, missing))
        taken = min(B, held)
        assert used.tolist() == [3 * B, taken]
        assert table[:, 0].tolist() == [15 - i for i in range(taken)] + [-1] * (B - taken)


def test_a_verify_step_without_pages_fails_and_shares_none():
    from mxfp4_mixture_experts_route_gb300.verify_step import VerifyStep
    s = VerifyStep(B=3, n=6, layers=1, page=8, most_ctx=200)
    for _ in range(4):
        trees, paths = s.draft()
        s.step(trees)
        s.accept(paths)
    s.free_pages = s.free_pages[:1]
    with pytest.raises(moe.MoEError) as e:
        for _ in range(20):
            trees, paths = s.draft()
            s.step(trees)
            s.accept(paths)
    assert e.value.code == moe.MOE_ERR_NO_PAGES
    held = [p for b, row in enumerate(s.table.tolist())
            for p in row[:cdiv(s.lens[b] + s.new[b].item(), s.page)] if p >= 0]
    assert len(held) == len(set(held))
