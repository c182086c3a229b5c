"""Python binding of libmoe, the routed MXFP4 mixture-of-experts block on GB300.

Argument marshalling only (and, for the dense MXFP4 calls, a check that the tensors
hold what the call says of them): every step of the block runs in the library's CUDA
kernels.  Tensors are PyTorch CUDA tensors (device memory and streams come from
PyTorch); the calls are the C entry points of include/moe.h under the same
names without the ``moe_`` prefix.  There is no CPU fallback: if libmoe.so is
missing, importing the binding's entry points raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "_lib", "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED_SHAPE = -2
MOE_ERR_ALIGNMENT = -3
MOE_ERR_WORKSPACE = -4
MOE_ERR_CUDA = -5
MOE_ERR_TIMEOUT = -6
MOE_ERR_BAD_IDS = -7
MOE_ERR_BAD_SCALE = -8
MOE_ERR_NO_DEVICE = -9
MOE_ERR_BAD_LENGTHS = -10
MOE_ERR_NO_PAGES = -11
MOE_ERR_BAD_PARENT = -12
MOE_ERR_BAD_PAGE = -13

MOE_POST_NORM = 1
MOE_LOGIT_OFFSET = 2
MOE_KV_E4M3 = 1
MOE_ROPE_INTERLEAVED = 1
MOE_MX_X_MXFP4 = 1
MOE_BF16, MOE_F16, MOE_F32 = 0, 1, 2

# every symbol include/moe.h declares
EXPORTS = ("moe_abi_version", "moe_strerror", "moe_workspace_bytes", "moe_workspace_init",
           "moe_route", "moe_experts", "moe_forward", "moe_forward_host", "moe_device_status",
           "moe_timing_enable", "moe_timing_collect", "moe_kernel_name", "moe_forward_noalloc",
           "moe_workspace_region", "moe_latent_workspace_bytes", "moe_latent_forward",
           "moe_kv_workspace_bytes", "moe_kv_plan", "moe_kv_append", "moe_tree_attention", "moe_qkv_append",
           "moe_mx_quantize", "moe_mx_dequantize", "moe_mx_workspace_bytes", "moe_mx_linear", "moe_mx_linear_cut")

# workspace regions (moe_workspace_region)
MOE_WS_STATUS, MOE_WS_POS, MOE_WS_TILES, MOE_WS_XQ, MOE_WS_XS, MOE_WS_HQ, MOE_WS_HS, MOE_WS_Y, MOE_WS_LOGITS = range(9)


class MoEShape(ctypes.Structure):
    _fields_ = [("S", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("I", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("norm_eps", ctypes.c_float)]

    @classmethod
    def of(cls, S, d, E, k, I, post_norm=False, logit_offset=False, norm_eps=1e-6):
        flags = (MOE_POST_NORM if post_norm else 0) | (MOE_LOGIT_OFFSET if logit_offset else 0)
        return cls(S, d, E, k, I, flags, norm_eps)


class LatentShape(ctypes.Structure):
    """moe_latent_shape: the latent-MoE layer around the routed block."""
    _fields_ = [("S", ctypes.c_int32), ("H", ctypes.c_int32), ("LAT", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("I", ctypes.c_int32),
                ("SI", ctypes.c_int32), ("flags", ctypes.c_uint32), ("norm_eps", ctypes.c_float)]

    @classmethod
    def of(cls, S, H, LAT, E, k, I, SI, logit_offset=False, norm_eps=1e-6):
        return cls(S, H, LAT, E, k, I, SI, MOE_LOGIT_OFFSET if logit_offset else 0, norm_eps)


class KVShape(ctypes.Structure):
    """moe_kv_shape: a batch of requests over a paged K/V cache.  Strides are in
    elements, 0 the packed layout (cache [n_pages, Hkv, page, D])."""
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("D", ctypes.c_int32), ("page", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("W", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("scale", ctypes.c_float), ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("q_stride", ctypes.c_int64), ("kv_stride", ctypes.c_int64)]

    @classmethod
    def of(cls, B, T, Hq, Hkv, D, page, n_pages, max_pages, mask_words=0, e4m3=False, scale=None, page_stride=0,
           head_stride=0, token_stride=0, q_stride=0, kv_stride=0):
        return cls(B, T, Hq, Hkv, D, page, n_pages, max_pages, mask_words, MOE_KV_E4M3 if e4m3 else 0,
                   D ** -0.5 if scale is None else scale, page_stride, head_stride, token_stride, q_stride, kv_stride)


class Rope(ctypes.Structure):
    """moe_rope: the heads' norms and the rotation of qkv_append."""
    _fields_ = [("R", ctypes.c_int32), ("max_pos", ctypes.c_int32), ("flags", ctypes.c_uint32), ("eps", ctypes.c_float),
                ("q_in_stride", ctypes.c_int64)]

    @classmethod
    def of(cls, R, max_pos=0, eps=1e-6, interleaved=False, q_in_stride=0):
        return cls(R, max_pos, MOE_ROPE_INTERLEAVED if interleaved else 0, eps, q_in_stride)


class MXShape(ctypes.Structure):
    """moe_mx_shape: a product of x [T, K] with MXFP4 weights [N, K]."""
    _fields_ = [("T", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("x_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64)]

    @classmethod
    def of(cls, T, N, K, x_mxfp4=False, x_stride=0, out_stride=0):
        return cls(T, N, K, MOE_MX_X_MXFP4 if x_mxfp4 else 0, x_stride, out_stride)


class MoEError(RuntimeError):
    def __init__(self, code: int, where: str, detail: int | None = None):
        self.code = code
        self.detail = detail
        msg = f"{where}: {strerror(code)} ({code})"
        if detail is not None:
            msg += f", detail {detail}"
        super().__init__(msg)


_lib = None
_raw_stream = None

_P = ctypes.c_void_p
_SP = ctypes.POINTER(MoEShape)


def lib() -> ctypes.CDLL:
    """The loaded libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libmoe.so not built ({LIB_PATH}); run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        _lib = load_library(LIB_PATH)
    return _lib


def load_library(path: str) -> ctypes.CDLL:
    """A build of the library at `path` with the entry points' C types set."""
    L = ctypes.CDLL(path)
    L.moe_abi_version.restype = ctypes.c_int
    L.moe_strerror.restype = ctypes.c_char_p
    L.moe_strerror.argtypes = [ctypes.c_int]
    L.moe_workspace_bytes.argtypes = [_SP, ctypes.POINTER(ctypes.c_size_t)]
    L.moe_workspace_init.argtypes = [_P, ctypes.c_size_t, _P]
    L.moe_route.argtypes = [_SP, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
    L.moe_experts.argtypes = [_SP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
    L.moe_forward.argtypes = [_SP] + [_P] * 13 + [ctypes.c_size_t, _P]
    L.moe_forward_host.argtypes = [_SP] + [_P] * 13 + [ctypes.c_size_t, _P]
    L.moe_device_status.argtypes = [_P, ctypes.POINTER(ctypes.c_int32), _P]
    L.moe_forward_noalloc.argtypes = [_SP] + [_P] * 14
    L.moe_workspace_region.argtypes = [_SP, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t),
                                       ctypes.POINTER(ctypes.c_size_t)]
    _LSP = ctypes.POINTER(LatentShape)
    L.moe_latent_workspace_bytes.argtypes = [_LSP, ctypes.POINTER(ctypes.c_size_t)]
    L.moe_latent_forward.argtypes = [_LSP] + [_P] * 17 + [ctypes.c_size_t, _P]
    _KSP = ctypes.POINTER(KVShape)
    L.moe_kv_workspace_bytes.argtypes = [_KSP, ctypes.POINTER(ctypes.c_size_t)]
    L.moe_kv_plan.argtypes = [_KSP] + [_P] * 4 + [ctypes.c_int32] + [_P] * 7 + [ctypes.c_size_t, _P]
    L.moe_kv_append.argtypes = [_KSP] + [_P] * 8 + [ctypes.c_size_t, _P]
    L.moe_tree_attention.argtypes = [_KSP] + [_P] * 12 + [ctypes.c_size_t, _P]
    L.moe_qkv_append.argtypes = [_KSP, ctypes.POINTER(Rope)] + [_P] * 14 + [ctypes.c_size_t, _P]
    L.moe_mx_quantize.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_int, _P, ctypes.c_int64, _P, _P, _P]
    L.moe_mx_dequantize.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_int, _P, _P, _P, ctypes.c_int64, _P]
    _MSP = ctypes.POINTER(MXShape)
    L.moe_mx_workspace_bytes.argtypes = [_MSP, ctypes.POINTER(ctypes.c_size_t)]
    L.moe_mx_linear.argtypes = [_MSP] + [_P] * 6 + [ctypes.c_size_t, _P]
    L.moe_mx_linear_cut.argtypes = [_MSP] + [ctypes.POINTER(ctypes.c_int32)] * 3
    L.moe_timing_enable.argtypes = [ctypes.c_int]
    L.moe_timing_collect.argtypes = [_P, _P, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    L.moe_kernel_name.argtypes = [ctypes.c_int]
    L.moe_kernel_name.restype = ctypes.c_char_p
    for name in EXPORTS:
        if name not in ("moe_strerror", "moe_kernel_name"):
            getattr(L, name).restype = ctypes.c_int
    return L


def strerror(code: int) -> str:
    try:
        return lib().moe_strerror(code).decode()
    except RuntimeError:
        return f"status {code}"


def _check(rc: int, where: str) -> None:
    if rc != MOE_OK:
        raise MoEError(rc, where)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is not None:
        return stream.cuda_stream
    global _raw_stream
    if _raw_stream is None:
        import torch
        # the current stream's handle without a Stream object around it (which costs 3 us a call)
        raw, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
        _raw_stream = (lambda: raw(dev())) if raw and dev and torch.cuda.is_initialized() else None
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream()


def abi_version() -> int:
    return lib().moe_abi_version()


def workspace_bytes(shape: MoEShape) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)), "moe_workspace_bytes")
    return n.value


def workspace_region(shape: MoEShape, region: int) -> tuple[int, int]:
    """(byte offset, bytes) of one workspace region (MOE_WS_*)."""
    off, n = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib().moe_workspace_region(ctypes.byref(shape), region, ctypes.byref(off), ctypes.byref(n)),
           "moe_workspace_region")
    return off.value, n.value


def read_region(shape: MoEShape, ws, region: int, dtype=None):
    """A CPU copy of one workspace region (after the stream has finished): a
    uint8 tensor, viewed as `dtype` when given."""
    off, n = workspace_region(shape, region)
    t = ws[off:off + n].cpu()
    return t if dtype is None else t.view(dtype)


def new_workspace(shape: MoEShape, device="cuda", stream=None):
    """A device workspace (uint8 tensor, 256-byte aligned) prepared by moe_workspace_init."""
    return _workspace(workspace_bytes(shape), device, stream)


def _workspace(nbytes, device, stream):
    import torch
    buf = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 256
    ws = buf[off:off + nbytes]
    _check(lib().moe_workspace_init(ws.data_ptr(), nbytes, _stream(stream)), "moe_workspace_init")
    return ws


def route(shape, x, w_gate, bias, logit_off, ids, weights, ws, stream=None) -> None:
    _check(lib().moe_route(ctypes.byref(shape), _ptr(x), _ptr(w_gate), _ptr(bias), _ptr(logit_off),
                           _ptr(ids), _ptr(weights), _ptr(ws), ws.numel(), _stream(stream)), "moe_route")


def experts(shape, x, ids, weights, w13, w13s, w2, w2s, norm_w, out, ws, stream=None) -> None:
    _check(lib().moe_experts(ctypes.byref(shape), _ptr(x), _ptr(ids), _ptr(weights), _ptr(w13),
                             _ptr(w13s), _ptr(w2), _ptr(w2s), _ptr(norm_w), _ptr(out), _ptr(ws),
                             ws.numel(), _stream(stream)), "moe_experts")


def forward(shape, x, w_gate, bias, logit_off, w13, w13s, w2, w2s, norm_w, ids, weights, out, ws,
            stream=None) -> None:
    _check(lib().moe_forward(ctypes.byref(shape), _ptr(x), _ptr(w_gate), _ptr(bias), _ptr(logit_off),
                             _ptr(w13), _ptr(w13s), _ptr(w2), _ptr(w2s), _ptr(norm_w), _ptr(ids),
                             _ptr(weights), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_forward")


def forward_host(shape, x_host, w_gate, bias, logit_off, w13, w13s, w2, w2s, norm_w, ids_host,
                 weights_host, out_host, ws, stream=None) -> None:
    """x_host / ids_host / weights_host / out_host are (pinned) CPU tensors."""
    _check(lib().moe_forward_host(ctypes.byref(shape), _ptr(x_host), _ptr(w_gate), _ptr(bias),
                                  _ptr(logit_off), _ptr(w13), _ptr(w13s), _ptr(w2), _ptr(w2s),
                                  _ptr(norm_w), _ptr(ids_host), _ptr(weights_host), _ptr(out_host),
                                  _ptr(ws), ws.numel(), _stream(stream)), "moe_forward_host")


def latent_workspace_bytes(shape: LatentShape) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_latent_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)), "moe_latent_workspace_bytes")
    return n.value


def latent_forward(shape, x, w_gate, bias, logit_off, w_ld, w13, w13s, w2, w2s, ln_w, w_up, w_sgu, w_sd,
                   ids, weights, out, ws, stream=None) -> None:
    _check(lib().moe_latent_forward(ctypes.byref(shape), _ptr(x), _ptr(w_gate), _ptr(bias), _ptr(logit_off),
                                    _ptr(w_ld), _ptr(w13), _ptr(w13s), _ptr(w2), _ptr(w2s), _ptr(ln_w),
                                    _ptr(w_up), _ptr(w_sgu), _ptr(w_sd), _ptr(ids), _ptr(weights), _ptr(out),
                                    _ptr(ws), ws.numel(), _stream(stream)), "moe_latent_forward")


def kv_workspace_bytes(shape: KVShape) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_kv_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)), "moe_kv_workspace_bytes")
    return n.value


def new_kv_workspace(shape: KVShape, device="cuda", stream=None):
    """A device workspace (uint8 tensor, 256-byte aligned) of the cache calls, prepared by moe_workspace_init."""
    return _workspace(kv_workspace_bytes(shape), device, stream)


# The cache calls run once a layer or a step on a few microseconds of GPU work, so
# their marshalling is kept short: tensors that are always there are not asked for None.
def kv_plan(shape, ctx_len, n_new, parents, free_pages, block_table, row_start, slots, positions, mask, used, ws,
            stream=None) -> None:
    """Block tables, slots, positions and masks.  A negative entry ends free_pages, whose length a captured graph keeps."""
    rc = (_lib or lib()).moe_kv_plan(
        ctypes.byref(shape), ctx_len.data_ptr(), n_new.data_ptr(), _ptr(parents), _ptr(free_pages),
        0 if free_pages is None else free_pages.numel(), block_table.data_ptr(), row_start.data_ptr(), slots.data_ptr(),
        positions.data_ptr(), _ptr(mask), used.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream))
    if rc:
        raise MoEError(rc, "moe_kv_plan")


def kv_append(shape, k_new, v_new, slots, k_scale, v_scale, k_cache, v_cache, ws, stream=None) -> None:
    rc = (_lib or lib()).moe_kv_append(
        ctypes.byref(shape), k_new.data_ptr(), v_new.data_ptr(), slots.data_ptr(), _ptr(k_scale), _ptr(v_scale),
        k_cache.data_ptr(), v_cache.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream))
    if rc:
        raise MoEError(rc, "moe_kv_append")


def tree_attention(shape, q, k_cache, v_cache, block_table, ctx_len, row_start, mask, k_scale, v_scale, out, lse, ws,
                   stream=None) -> None:
    """Attention of the new tokens over the cache; lse may be None."""
    rc = (_lib or lib()).moe_tree_attention(
        ctypes.byref(shape), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
        ctx_len.data_ptr(), row_start.data_ptr(), _ptr(mask), _ptr(k_scale), _ptr(v_scale), out.data_ptr(), _ptr(lse),
        ws.data_ptr(), ws.numel(), _stream(stream))
    if rc:
        raise MoEError(rc, "moe_tree_attention")


def rope_table(max_pos, R, base=10000.0, device="cuda"):
    """qkv_append's table: cos, then sin, of position * base^(-2 i / R), i = 0 .. R/2 - 1.  [max_pos, R] fp32, from
    angles in 64 bits."""
    import torch
    i = torch.arange(R // 2, dtype=torch.float64, device=device)
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * base ** (-2 * i / R)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def qkv_append(shape, rope, q_in, k_new, v_new, positions, slots, q_norm, k_norm, cos_sin, k_scale, v_scale, q, k_cache,
               v_cache, ws, stream=None) -> None:
    """Norms and rotation of query and key heads, and the append of K and V; q may be q_in, norms may be None."""
    rc = (_lib or lib()).moe_qkv_append(
        ctypes.byref(shape), ctypes.byref(rope), q_in.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
        positions.data_ptr(), slots.data_ptr(), _ptr(q_norm), _ptr(k_norm), _ptr(cos_sin), _ptr(k_scale), _ptr(v_scale),
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream))
    if rc:
        raise MoEError(rc, "moe_qkv_append")


_mx_types = {}


def _mx_rows(t, codes, scales):
    """(rows, K, MOE_* type, distance of rows or 0 where they are packed) of a tensor whose last dimension is K and whose
    others are rows, next to packed codes [rows, K/2] and scales [rows, K/32]."""
    if not _mx_types:
        import torch
        _mx_types.update({torch.bfloat16: MOE_BF16, torch.float16: MOE_F16, torch.float32: MOE_F32})
    dt = _mx_types.get(t.dtype)
    n = t.numel()
    if dt is None or not n or not t.dim():
        raise MoEError(MOE_ERR_INVALID_ARG, "mx rows (bf16, fp16 or fp32)")
    K = t.shape[-1]
    stride = 0
    if not t.is_contiguous():
        if t.dim() != 2:
            try:
                t = t.view(-1, K)
            except RuntimeError:
                raise MoEError(MOE_ERR_INVALID_ARG, "mx rows (evenly apart)") from None
        stride = t.stride(0)
        if (K > 1 and t.stride(1) != 1) or (n > K and stride < K):
            raise MoEError(MOE_ERR_INVALID_ARG, "mx rows (elements of a row side by side, rows apart)")
        if n == K:
            stride = 0
    if (codes.numel() * 2 != n or scales.numel() * 32 != n or codes.element_size() != 1 or scales.element_size() != 1
            or not codes.is_contiguous() or not scales.is_contiguous()):
        raise MoEError(MOE_ERR_INVALID_ARG, "mx codes [rows, K/2] and scales [rows, K/32] (packed bytes)")
    return n // K, K, dt, stride


def mx_quantize(x, codes, scales, stream=None) -> None:
    """Rows x [..., K] (bf16, fp16 or fp32) to MXFP4 codes [..., K/2] and scales [..., K/32] (uint8)."""
    rows, K, dt, stride = _mx_rows(x, codes, scales)
    rc = (_lib or lib()).moe_mx_quantize(rows, K, dt, x.data_ptr(), stride, codes.data_ptr(), scales.data_ptr(),
                                         _stream(stream))
    if rc:
        raise MoEError(rc, "moe_mx_quantize")


def mx_dequantize(codes, scales, y, stream=None) -> None:
    """MXFP4 rows read back into y [..., K] (bf16, fp16 or fp32)."""
    rows, K, dt, stride = _mx_rows(y, codes, scales)
    rc = (_lib or lib()).moe_mx_dequantize(rows, K, dt, codes.data_ptr(), scales.data_ptr(), y.data_ptr(), stride,
                                           _stream(stream))
    if rc:
        raise MoEError(rc, "moe_mx_dequantize")


def mx_workspace_bytes(shape: MXShape) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_mx_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)), "moe_mx_workspace_bytes")
    return n.value


def mx_linear_cut(shape: MXShape) -> tuple[int, int, int]:
    """(CTAs of a tile, tokens of a tile, CTAs of a cluster that share a tile's K) of mx_linear (diagnostics)."""
    cut = [ctypes.c_int32(0) for _ in range(3)]
    _check(lib().moe_mx_linear_cut(ctypes.byref(shape), *map(ctypes.byref, cut)), "moe_mx_linear_cut")
    return tuple(c.value for c in cut)


def new_mx_workspace(shape: MXShape, device="cuda", stream=None):
    """A device workspace (uint8 tensor, 256-byte aligned) of mx_linear, prepared by moe_workspace_init."""
    return _workspace(mx_workspace_bytes(shape), device, stream)


_mx_fields = struct.Struct("iiiIqq").unpack_from      # of an MXShape, in one step


def _rows_fit(t, rows, width, stride) -> bool:
    """Whether `rows` rows of `width` 16-bit elements, `stride` elements apart (0: packed), are t's, in its elements' order."""
    stride = stride or width
    if t.element_size() != 2:
        return False
    if t.is_contiguous():
        return t.numel() >= (rows - 1) * stride + width
    sizes, strides = t.shape, t.stride()
    i, piece = len(sizes), 1                             # the last dimensions that are in one piece
    while i and (sizes[i - 1] == 1 or strides[i - 1] == piece):
        i -= 1
        piece *= sizes[i]
    if piece >= (rows - 1) * stride + width:
        return True
    count = 1                                            # those before them: rows evenly apart
    while i and (sizes[i - 1] == 1 or strides[i - 1] == stride * count):
        i -= 1
        count *= sizes[i]
    return piece >= width and count >= rows


def mx_linear(shape, x, xs, w, w_scales, out, ws, stream=None) -> None:
    """out = x . w^T with MXFP4 w; x bf16 (xs None) or MXFP4 codes with scales xs; out bf16.  Tensors that do not hold
    what the descriptor says are refused."""
    # (a small product is as long as this call, so the checks of packed tensors are written out)
    T, N, K, codes, x_stride, out_stride = _mx_fields(shape)
    if not ((x.nbytes >= T * K // 2 and x.is_contiguous() if codes else _rows_fit(x, T, K, x_stride))
            and (xs is None or xs.nbytes >= T * K // 32 and xs.is_contiguous())
            and w.nbytes >= N * K // 2 and w.is_contiguous() and w_scales.nbytes >= N * K // 32 and w_scales.is_contiguous()
            and (not out_stride and out.nbytes == 2 * T * N and out.is_contiguous() or _rows_fit(out, T, N, out_stride))):
        raise MoEError(MOE_ERR_INVALID_ARG, "moe_mx_linear (tensors that the descriptor does not describe)")
    rc = (_lib or lib()).moe_mx_linear(shape, x.data_ptr(), None if xs is None else xs.data_ptr(), w.data_ptr(),
                                       w_scales.data_ptr(), out.data_ptr(), ws.data_ptr(), ws.numel(),
                                       _raw_stream() if stream is None and _raw_stream else _stream(stream))
    if rc:
        raise MoEError(rc, "moe_mx_linear")


def device_status(ws, stream=None) -> tuple[int, int]:
    """(status, detail) latched on the device since the last call; clears it."""
    det = ctypes.c_int32(0)
    rc = lib().moe_device_status(_ptr(ws), ctypes.byref(det), _stream(stream))
    return rc, det.value


def check_device_status(ws, where="device", stream=None) -> None:
    rc, det = device_status(ws, stream)
    if rc != MOE_OK:
        raise MoEError(rc, where, det)


def timing_enable(max_launches: int) -> None:
    _check(lib().moe_timing_enable(max_launches), "moe_timing_enable")


def timing_collect(cap: int = 4096) -> list[tuple[str, float]]:
    """(kernel name, ms) of the launches recorded since enable / the last collect."""
    ids = (ctypes.c_int32 * cap)()
    ms = (ctypes.c_float * cap)()
    n = ctypes.c_int(0)
    _check(lib().moe_timing_collect(ids, ms, cap, ctypes.byref(n)), "moe_timing_collect")
    return [(lib().moe_kernel_name(ids[i]).decode(), ms[i]) for i in range(n.value)]


def kernel_names() -> list[str]:
    out, i = [], 0
    while (nm := lib().moe_kernel_name(i)) is not None:
        out.append(nm.decode())
        i += 1
    return out


class DeviceWeights:
    """Device copies of one block's weights and the step input, from host arrays
    (numpy or torch CPU): x / w_gate as bf16 bit patterns (uint16), the packed
    e2m1 and e8m0 tensors as uint8, bias / logit_off / norm_w as fp32."""

    def __init__(self, shape: MoEShape, x, w_gate, bias, logit_off, w13, w13s, w2, w2s, norm_w,
                 device="cuda"):
        import torch

        def up(a, dtype=None):
            if a is None:
                return None
            t = torch.as_tensor(a)
            if dtype is not None:
                t = t.view(dtype)
            return t.contiguous().to(device)

        self.shape = shape
        self.x = up(x, torch.bfloat16) if x is not None else None
        self.w_gate = up(w_gate, torch.bfloat16)
        self.bias = up(bias)
        self.logit_off = up(logit_off)
        self.w13, self.w13s, self.w2, self.w2s = up(w13), up(w13s), up(w2), up(w2s)
        self.norm_w = up(norm_w)
        S, k, d = shape.S, shape.k, shape.d
        self.ids = torch.empty((S, k), dtype=torch.int32, device=device)
        self.weights = torch.empty((S, k), dtype=torch.float32, device=device)
        self.out = torch.empty((S, d), dtype=torch.float32, device=device)
        self.ws = new_workspace(shape, device)

    def forward(self, x=None, stream=None):
        forward(self.shape, self.x if x is None else x, self.w_gate, self.bias, self.logit_off,
                self.w13, self.w13s, self.w2, self.w2s, self.norm_w, self.ids, self.weights,
                self.out, self.ws, stream)
        return self.ids, self.weights, self.out


class DeviceLatentWeights:
    """Device copies of one latent-MoE layer's weights and step input (host
    arrays: bf16 bit patterns as uint16, packed e2m1 / e8m0 as uint8, fp32)."""

    def __init__(self, shape: LatentShape, x, w_gate, bias, logit_off, w_ld, w13, w13s, w2, w2s, ln_w,
                 w_up, w_sgu, w_sd, device="cuda"):
        import torch

        def up(a, dtype=None):
            if a is None:
                return None
            t = torch.as_tensor(a)
            if dtype is not None:
                t = t.view(dtype)
            return t.contiguous().to(device)

        bf = torch.bfloat16
        self.shape = shape
        self.x = up(x, bf)
        self.w_gate, self.bias, self.logit_off = up(w_gate, bf), up(bias), up(logit_off)
        self.w_ld, self.w_up, self.ln_w = up(w_ld, bf), up(w_up, bf), up(ln_w)
        self.w13, self.w13s, self.w2, self.w2s = up(w13), up(w13s), up(w2), up(w2s)
        self.w_sgu, self.w_sd = up(w_sgu, bf), up(w_sd, bf)
        S, k, H = shape.S, shape.k, shape.H
        self.ids = torch.empty((S, k), dtype=torch.int32, device=device)
        self.weights = torch.empty((S, k), dtype=torch.float32, device=device)
        self.out = torch.empty((S, H), dtype=torch.float32, device=device)
        nbytes = latent_workspace_bytes(shape)
        buf = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
        off = (-buf.data_ptr()) % 256
        self.ws = buf[off:off + nbytes]
        _check(lib().moe_workspace_init(self.ws.data_ptr(), nbytes, _stream(None)), "moe_workspace_init")

    def forward(self, x=None, stream=None):
        latent_forward(self.shape, self.x if x is None else x, self.w_gate, self.bias, self.logit_off, self.w_ld,
                       self.w13, self.w13s, self.w2, self.w2s, self.ln_w, self.w_up, self.w_sgu, self.w_sd,
                       self.ids, self.weights, self.out, self.ws, stream)
        return self.ids, self.weights, self.out
