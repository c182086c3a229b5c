"""Which cuts of a product the estimate takes, and that the GPU tests' shapes take all of them (no GPU).

A cut is (operands, CTAs of a tile, tokens of a tile, CTAs that share a tile's K).  Numbers fitted anew move shapes
from one to another: a cut that no tested shape takes any more fails here.
"""
import ctypes
import math
import random

import pytest

import mxfp4_mixture_experts_route_gb300 as moe
from libmoe_util import ensure_built

pytest.importorskip("torch")      # (the lists of shapes stand in the GPU tests)


@pytest.fixture(scope="module")
def L():
    return ensure_built()


def cut(T, N, K, kind):
    return (kind, *moe.mx_linear_cut(moe.MXShape.of(T, N, K, x_mxfp4=kind == "mxfp4")))


def shapes_of_the_tests():
    from test_gpu_mx import CUTS, SHAPES
    from test_gpu_mx_exact import CUTS as MORE
    return [(*s, kind) for s in SHAPES for kind in ("bf16", "mxfp4")] + CUTS + MORE


def drawn_shapes(rng, n):
    """Supported shapes, most of the sizes that models have and some of every size."""
    def log(lo, hi):
        return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))
    for _ in range(n):
        T = log(1, 3000) if rng.random() < 0.7 else log(1, 1 << 20)
        N = 8 * (log(1, 2500) if rng.random() < 0.7 else log(1, 1 << 17))
        yield T, N, 128 * log(1, 512), rng.choice(["bf16", "mxfp4"])


def test_every_cut_has_a_tested_shape(L):
    tested = {cut(*s) for s in shapes_of_the_tests()}
    out = [ctypes.c_int32(0) for _ in range(3)]
    at, untested = [ctypes.byref(o) for o in out], {}
    for T, N, K, kind in drawn_shapes(random.Random(5), 300000):
        assert L.moe_mx_linear_cut(moe.MXShape(T, N, K, kind == "mxfp4", 0, 0), *at) == moe.MOE_OK
        c = (kind, *(o.value for o in out))
        if c not in tested:
            untested.setdefault(c, (T, N, K))
    assert not untested


def test_cuts_are_ones_that_the_kernel_has(L):
    for T, N, K, kind in drawn_shapes(random.Random(6), 3000):
        _, ctas, tokens, parts = cut(T, N, K, kind)
        if ctas == 2:
            assert tokens in range(64, 257, 32) and parts == 1
        else:
            assert ctas == 1 and tokens in ((16, 32, 64, 128) if kind == "mxfp4" else (8, 16, 32, 64))
            assert 1 <= parts <= min(8, -(-K // 256))
            # a shared tile's clusters run at once
            tiles = -(-N // 128) * -(-T // tokens)
            assert parts == 1 or tiles * parts <= 152


def test_cut_arguments(L):
    out = ctypes.c_int32(-5)
    s = moe.MXShape.of(8, 256, 512)
    assert L.moe_mx_linear_cut(ctypes.byref(s), None, ctypes.byref(out), None) == moe.MOE_OK and out.value > 0
    assert L.moe_mx_linear_cut(ctypes.byref(s), None, None, None) == moe.MOE_OK
    assert L.moe_mx_linear_cut(None, None, None, None) == moe.MOE_ERR_INVALID_ARG
    s.K = 192
    out.value = -5
    assert L.moe_mx_linear_cut(ctypes.byref(s), ctypes.byref(out), None, None) == moe.MOE_ERR_UNSUPPORTED_SHAPE
    assert out.value == -5
    with pytest.raises(moe.MoEError):
        moe.mx_linear_cut(s)
