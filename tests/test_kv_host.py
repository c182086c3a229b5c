"""The cache calls' host-side refusals (no GPU): they return before anything is enqueued."""
import ctypes

import pytest

import mxfp4_mixture_experts_route_gb300 as moe
from libmoe_util import ensure_built

BASE = dict(B=4, T=32, Hq=32, Hkv=8, D=128, page=64, n_pages=100, max_pages=20)


@pytest.fixture(scope="module")
def L():
    return ensure_built()


def nbytes(L, s):
    n = ctypes.c_size_t(0)
    return L.moe_kv_workspace_bytes(ctypes.byref(s) if s is not None else None, ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw", [
    {}, dict(D=64), dict(e4m3=True), dict(mask_words=32), dict(Hq=1024, Hkv=8), dict(page=8), dict(page=48),
    dict(page=1024), dict(T=1 << 20, B=4096), dict(q_stride=48 * 128, kv_stride=48 * 128),
    dict(token_stride=8 * 128, head_stride=128, page_stride=64 * 8 * 128)])
def test_supported_shapes(L, kw):
    rc, n = nbytes(L, moe.KVShape.of(**{**BASE, **kw}))
    assert rc == moe.MOE_OK and n % 256 == 0 and n >= 256


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), moe.MOE_ERR_INVALID_ARG), (dict(T=0), moe.MOE_ERR_INVALID_ARG),
    (dict(mask_words=-1), moe.MOE_ERR_INVALID_ARG), (dict(scale=0.0), moe.MOE_ERR_INVALID_ARG),
    (dict(scale=float("nan")), moe.MOE_ERR_INVALID_ARG), (dict(scale=float("inf")), moe.MOE_ERR_INVALID_ARG),
    (dict(scale=-1.0), moe.MOE_ERR_INVALID_ARG), (dict(q_stride=-8), moe.MOE_ERR_INVALID_ARG),
    (dict(B=4097), moe.MOE_ERR_UNSUPPORTED_SHAPE), (dict(T=(1 << 20) + 1), moe.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(D=96), moe.MOE_ERR_UNSUPPORTED_SHAPE), (dict(Hq=33), moe.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(Hq=1032, Hkv=8), moe.MOE_ERR_UNSUPPORTED_SHAPE), (dict(page=12), moe.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(page=1032), moe.MOE_ERR_UNSUPPORTED_SHAPE), (dict(mask_words=33), moe.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(n_pages=1 << 25), moe.MOE_ERR_UNSUPPORTED_SHAPE), (dict(max_pages=1 << 25), moe.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(token_stride=64), moe.MOE_ERR_UNSUPPORTED_SHAPE), (dict(q_stride=1024), moe.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(kv_stride=512), moe.MOE_ERR_UNSUPPORTED_SHAPE), (dict(page_stride=1 << 40), moe.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(token_stride=132), moe.MOE_ERR_ALIGNMENT), (dict(token_stride=136, e4m3=True), moe.MOE_ERR_ALIGNMENT),
    (dict(q_stride=32 * 128 + 4), moe.MOE_ERR_ALIGNMENT), (dict(kv_stride=8 * 128 + 4), moe.MOE_ERR_ALIGNMENT)])
def test_refused_shapes(L, kw, code):
    assert nbytes(L, moe.KVShape.of(**{**BASE, **kw}))[0] == code


def test_bad_flags_and_null_shape(L):
    s = moe.KVShape.of(**BASE)
    s.flags = 2
    assert nbytes(L, s)[0] == moe.MOE_ERR_INVALID_ARG
    assert nbytes(L, None)[0] == moe.MOE_ERR_INVALID_ARG
    assert L.moe_kv_workspace_bytes(ctypes.byref(moe.KVShape.of(**BASE)), None) == moe.MOE_ERR_INVALID_ARG


def plan(L, s, **kw):
    a = dict(ctx=0x1000, n_new=0x2000, parents=None, free=0x3000, n_free=8, table=0x4000, row_start=0x5000,
             slots=0x6000, positions=0x7000, mask=None, used=0x8000, ws=0x10000, nbytes=None)
    a.update(kw)
    n = nbytes(L, s)[1] if a["nbytes"] is None else a["nbytes"]
    return L.moe_kv_plan(ctypes.byref(s), a["ctx"], a["n_new"], a["parents"], a["free"], a["n_free"], a["table"],
                         a["row_start"], a["slots"], a["positions"], a["mask"], a["used"], a["ws"], n, None)


def append(L, s, **kw):
    a = dict(k_new=0x1000, v_new=0x2000, slots=0x3000, ks=None, vs=None, k=0x4000, v=0x5000, ws=0x10000, nbytes=None)
    a.update(kw)
    n = nbytes(L, s)[1] if a["nbytes"] is None else a["nbytes"]
    return L.moe_kv_append(ctypes.byref(s), a["k_new"], a["v_new"], a["slots"], a["ks"], a["vs"], a["k"], a["v"],
                           a["ws"], n, None)


def attend(L, s, **kw):
    a = dict(q=0x1000, k=0x2000, v=0x3000, table=0x4000, ctx=0x5000, row_start=0x6000, mask=None, ks=None, vs=None,
             out=0x7000, lse=None, ws=0x10000, nbytes=None)
    a.update(kw)
    n = nbytes(L, s)[1] if a["nbytes"] is None else a["nbytes"]
    return L.moe_tree_attention(ctypes.byref(s), a["q"], a["k"], a["v"], a["table"], a["ctx"], a["row_start"],
                                a["mask"], a["ks"], a["vs"], a["out"], a["lse"], a["ws"], n, None)


@pytest.mark.parametrize("call", [plan, append, attend])
def test_workspace_refusals(L, call):
    s = moe.KVShape.of(**BASE)
    assert call(L, s, ws=None) == moe.MOE_ERR_INVALID_ARG
    assert call(L, s, ws=0x10080) == moe.MOE_ERR_ALIGNMENT
    assert call(L, s, nbytes=128) == moe.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("name", ["ctx", "n_new", "table", "row_start", "slots", "positions", "used"])
def test_plan_pointers(L, name):
    s = moe.KVShape.of(**BASE)
    assert plan(L, s, **{name: None}) == moe.MOE_ERR_INVALID_ARG
    assert plan(L, s, **{name: 0x9004}) == moe.MOE_ERR_ALIGNMENT


def test_plan_tree_arguments(L):
    s, t = moe.KVShape.of(**BASE), moe.KVShape.of(**BASE, mask_words=1)
    assert plan(L, s, parents=0x9000) == moe.MOE_ERR_INVALID_ARG      # a tree needs mask words
    assert plan(L, s, mask=0x9000) == moe.MOE_ERR_INVALID_ARG
    assert plan(L, t, parents=0x9000) == moe.MOE_ERR_INVALID_ARG
    assert plan(L, t, mask=0x9000) == moe.MOE_ERR_INVALID_ARG
    assert plan(L, t, parents=0x9004, mask=0xA000) == moe.MOE_ERR_ALIGNMENT
    assert plan(L, s, n_free=-1) == moe.MOE_ERR_INVALID_ARG
    assert plan(L, s, free=None) == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["k_new", "v_new", "slots", "k", "v"])
def test_append_pointers(L, name):
    s = moe.KVShape.of(**BASE)
    assert append(L, s, **{name: None}) == moe.MOE_ERR_INVALID_ARG
    assert append(L, s, **{name: 0x9008}) == moe.MOE_ERR_ALIGNMENT


@pytest.mark.parametrize("name", ["q", "k", "v", "table", "ctx", "row_start", "out"])
def test_attention_pointers(L, name):
    s = moe.KVShape.of(**BASE)
    assert attend(L, s, **{name: None}) == moe.MOE_ERR_INVALID_ARG
    assert attend(L, s, **{name: 0x9008}) == moe.MOE_ERR_ALIGNMENT


@pytest.mark.parametrize("call", [append, attend])
def test_scales_go_with_the_cache_type(L, call):
    s, e = moe.KVShape.of(**BASE), moe.KVShape.of(**BASE, e4m3=True)
    assert call(L, s, ks=0x9000, vs=0xA000) == moe.MOE_ERR_INVALID_ARG
    assert call(L, e) == moe.MOE_ERR_INVALID_ARG
    assert call(L, e, ks=0x9000) == moe.MOE_ERR_INVALID_ARG
    assert call(L, e, ks=0x9000, vs=0xA008) == moe.MOE_ERR_ALIGNMENT


def test_attention_mask_goes_with_the_words(L):
    assert attend(L, moe.KVShape.of(**BASE), mask=0x9000) == moe.MOE_ERR_INVALID_ARG
    assert attend(L, moe.KVShape.of(**BASE, mask_words=1)) == moe.MOE_ERR_INVALID_ARG
    assert attend(L, moe.KVShape.of(**BASE, mask_words=1), mask=0x9004) == moe.MOE_ERR_ALIGNMENT
    assert attend(L, moe.KVShape.of(**BASE), lse=0x9004) == moe.MOE_ERR_ALIGNMENT
