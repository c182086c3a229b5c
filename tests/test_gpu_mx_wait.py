"""The product's waits begin behind the kernels in front of the call, on a real GPU.

A kernel may let the next one start long before it ends, so the limit of a wait inside
the product's kernel must not count that time.  The library's wait-test variant, whose
waits give up after 1 ms, makes the call behind a kernel that lets its successor start at
once and ends 20 ms later: the product has to come out as the ordinary library's, without
MOE_ERR_TIMEOUT.
"""
import ctypes
import os

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import mxfp4_mixture_experts_route_gb300 as moe  # noqa: E402
from libmoe_util import ensure_built  # noqa: E402
from test_gpu_mx import product, tokens, weights  # noqa: E402


@pytest.fixture(scope="module")
def waitlib():
    ensure_built()
    from mxfp4_mixture_experts_route_gb300.build import WAIT_TEST_LIB, build_wait_test_library
    if not os.path.exists(WAIT_TEST_LIB):
        build_wait_test_library()
    L = moe.load_library(WAIT_TEST_LIB)
    L.moe_test_early_kernel.argtypes = [ctypes.c_int, ctypes.c_void_p]
    return L


# one CTA a tile and clusters that share K, the terms of x in the kernel or before it, pairs of CTAs
@pytest.mark.parametrize("T,N,K,kind", [(1, 6144, 4096, "bf16"), (8, 7168, 4096, "mxfp4"), (8, 39680, 512, "mxfp4"),
                                        (64, 1024, 2048, "bf16"),
                                        (128, 9216, 1024, "bf16"), (600, 2048, 1024, "mxfp4"), (600, 2048, 1024, "bf16")])
def test_a_slow_kernel_in_front_is_no_timeout(waitlib, T, N, K, kind):
    w, ws = weights(N + K, N, K)
    x, xs, _, _ = tokens(T + K, T, K, kind)
    want, work = product(x, xs, w, ws, T, N, K, kind)
    moe.check_device_status(work)
    out = torch.full_like(want, -77.0)
    shape = moe.MXShape.of(T, N, K, x_mxfp4=kind == "mxfp4")
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    for _ in range(3):
        assert waitlib.moe_test_early_kernel(20000, stream) == moe.MOE_OK
        assert waitlib.moe_mx_linear(ctypes.byref(shape), x.data_ptr(), None if xs is None else xs.data_ptr(), w.data_ptr(),
                                     ws.data_ptr(), out.data_ptr(), work.data_ptr(), work.numel(), stream) == moe.MOE_OK
        assert moe.device_status(work) == (moe.MOE_OK, 0)
        assert torch.equal(out, want)
        out.fill_(-77.0)
