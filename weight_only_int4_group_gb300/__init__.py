"""Python binding of libq4.so, the GB300 weight-only INT4 group-128 library.

Argument marshalling only: every step runs in the library's CUDA kernels.
PyTorch is used for device memory and the current CUDA stream.  Importing
this package fails loudly when libq4.so has not been built; there is no
fallback of any kind.

Names follow include/q4.h: quantize, quantize_sym, repack, unpack, xsum,
gemv, gemm, check, weight_bytes, gemv_workspace_bytes, gemm_workspace_bytes,
repack_compact, unpack_compact, gemv_noalloc and the two timeout
self-tests; the serving operators cache_plan, rope_append and attention over
a KVCache, or in 8 bits over a KVCache8 with cache_read (rope_frequencies makes
their angles).  A QWeight carries its layout (TILED or COMPACT), and every
product call passes that layout and the buffer's byte count to the library,
which refuses a mismatch.
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# Q4_LIBRARY selects another build of the same library (the bounds-checked
# libq4_debug.so); the named file must exist, there is no fallback.
LIB_PATH = os.environ.get("Q4_LIBRARY") or os.path.join(_HERE, "libq4.so")
GROUP = 128
TILE_ROWS = 16
TILE_BYTES = 1104
CMP_TILE_BYTES = 1072
GEMV_MAX_M = 16

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_MISALIGNED, ERR_CUDA, ERR_TIMEOUT, ERR_BOUNDS = range(7)
F32, BF16, F16 = 0, 1, 2
LAYOUT_TILED, LAYOUT_COMPACT = 1, 2
PATH_AUTO, PATH_FMA, PATH_MMA = 0, 1, 2

_DTYPE = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
I8, E4M3 = 0, 1
_CODE = {torch.int8: I8, torch.float8_e4m3fn: E4M3}


ROPE_HALF, ROPE_INTERLEAVED = 0, 1


class _KVCacheArg(ctypes.Structure):
    """q4_kv_cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("type", ctypes.c_int),
                ("blocks", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("block_size", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("block_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64)]


class _KVCache8Arg(ctypes.Structure):
    """q4_kv_cache8."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_exp", "v_exp")] + [
        ("code", ctypes.c_int), ("type", ctypes.c_int)] + [
        (n, ctypes.c_int64) for n in ("blocks", "heads", "block_size", "head_dim", "block_stride",
                                      "head_stride", "token_stride")]


class Q4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.q4_status_str(status).decode()
        if status == ERR_CUDA:
            msg += ": " + _lib.q4_last_cuda_error().decode()
        super().__init__(f"{where}: {msg} (status {status})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, Z, S = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    lib.q4_quantize.argtypes = [P, I, I, P, P, P, P]
    lib.q4_quantize_sym.argtypes = [P, I, I, P, P, P, P]
    lib.q4_weight_bytes.argtypes = [I, I, S]
    lib.q4_weight_bytes.restype = Z
    lib.q4_repack.argtypes = [P, P, P, I, I, P, P]
    lib.q4_unpack.argtypes = [P, I, I, P, P, P, P]
    lib.q4_repack_compact.argtypes = [P, P, P, I, I, P, P]
    lib.q4_unpack_compact.argtypes = [P, I, I, P, P, P, P]
    lib.q4_xsum.argtypes = [P, S, I, I, P, P]
    lib.q4_gemv_workspace_bytes.argtypes = [I, I, I]
    lib.q4_gemv_workspace_bytes.restype = Z
    lib.q4_gemm_workspace_bytes.argtypes = [I, I, I]
    lib.q4_gemm_workspace_bytes.restype = Z
    prod = [P, S, I, I, I, P, S, Z, P, S, P, Z, P]  # x, xt, M, N, K, qw, layout, bytes, y, yt, ws, wsb, stream
    lib.q4_gemv.argtypes = prod
    lib.q4_gemv_path.argtypes = prod[:-1] + [S, P]
    lib.q4_gemv_timeout_selftest.argtypes = prod
    lib.q4_gemm.argtypes = prod
    lib.q4_gemm_timeout_selftest.argtypes = prod
    lib.q4_gemv_noalloc.argtypes = [P, S, I, I, I, P, S, Z, P, S, P]
    F, C = ctypes.c_float, ctypes.POINTER(_KVCacheArg)
    lib.q4_cache_plan.argtypes = [P, P, I, I, P, I, I, P, P, I, I, P, P, P, P, P, P]
    lib.q4_rope_append.argtypes = [P, I, I, I, I, S, P, F, P, P, P, I, C, P]
    lib.q4_attention.argtypes = [P, I, I, I, C, P, I, I, P, P, I, I, F, I, P, S, I, P, P, Z, P]
    lib.q4_attention_timeout_selftest.argtypes = lib.q4_attention.argtypes
    lib.q4_attention_workspace_bytes.argtypes = [I, I, I, I]
    lib.q4_attention_workspace_bytes.restype = Z
    C8 = ctypes.POINTER(_KVCache8Arg)
    lib.q4_rope_append8.argtypes = [P, I, I, I, I, S, P, F, P, P, P, I, C8, P]
    lib.q4_cache_read8.argtypes = [C8, P, I, I, P, P, I, I, P, I, P, I, S, P]
    lib.q4_attention8.argtypes = [P, I, I, I, C8, P, I, I, P, P, I, I, F, I, P, S, I, P, P, Z, P]
    lib.q4_attention8_timeout_selftest.argtypes = lib.q4_attention8.argtypes
    lib.q4_attention8_workspace_bytes.argtypes = [I, I, I, I]
    lib.q4_attention8_workspace_bytes.restype = Z
    lib.q4_check.argtypes = [P]
    lib.q4_debug_bounds_selftest.argtypes = [P, P]
    lib.q4_status_str.argtypes = [S]
    lib.q4_status_str.restype = ctypes.c_char_p
    lib.q4_last_cuda_error.restype = ctypes.c_char_p
    for f in ("q4_quantize", "q4_quantize_sym", "q4_repack", "q4_unpack", "q4_repack_compact",
              "q4_unpack_compact", "q4_xsum", "q4_gemv", "q4_gemv_path", "q4_gemv_timeout_selftest",
              "q4_gemm", "q4_gemm_timeout_selftest", "q4_gemv_noalloc", "q4_check",
              "q4_cache_plan", "q4_rope_append", "q4_attention",
              "q4_attention_timeout_selftest", "q4_rope_append8", "q4_cache_read8", "q4_attention8",
              "q4_attention8_timeout_selftest",
              "q4_debug_bounds_selftest"):
        getattr(lib, f).restype = S
    return lib


_lib = _load()


def lib():
    """The loaded ctypes library (for callers that marshal their own pointers)."""
    return _lib


def _stream(stream=None) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ok(status: int, where: str):
    if status != OK:
        raise Q4Error(status, where)


# The library launches on the thread's current device, which addresses of
# another one must not reach: every tensor's device is compared with it.
_current_device = torch._C._cuda_getDevice


def _elsewhere(name: str, index: int, dev: int):
    """Refuses a tensor of device `index` (-1: the host), which is not `dev`."""
    raise ValueError(f"{name} must be a CUDA tensor" if index < 0 else
                     f"{name} is on CUDA device {index}, the current device is {dev}")


def _cuda(t: torch.Tensor, name: str):
    on = t.get_device()
    if on < 0 or on != _current_device():
        _elsewhere(name, on, -1 if on < 0 else _current_device())
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# ------------------------------------------------------------------ API
def weight_bytes(N: int, K: int, layout: int = LAYOUT_TILED) -> int:
    return int(_lib.q4_weight_bytes(N, K, layout))


def weight_bytes_compact(N: int, K: int) -> int:
    return weight_bytes(N, K, LAYOUT_COMPACT)


def gemv_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_lib.q4_gemv_workspace_bytes(M, N, K))


def gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_lib.q4_gemm_workspace_bytes(M, N, K))


def quantize(w: torch.Tensor, stream=None, symmetric: bool = False):
    """w f32 [N][K] (cuda) -> (packed u8 [N][K/2], scale f32 [N][K/128], zero u8 [N][K/128]).

    ``symmetric`` calls q4_quantize_sym (max|w|/7 scales, zero 8)."""
    _cuda(w, "w")
    if w.dtype != torch.float32 or w.dim() != 2:
        raise ValueError("w must be a 2-D float32 tensor")
    N, K = w.shape
    packed = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    scale = torch.empty((N, max(K // GROUP, 1)), dtype=torch.float32, device=w.device)
    zero = torch.empty((N, max(K // GROUP, 1)), dtype=torch.uint8, device=w.device)
    fn, name = (_lib.q4_quantize_sym, "q4_quantize_sym") if symmetric else \
        (_lib.q4_quantize, "q4_quantize")
    _ok(fn(w.data_ptr(), N, K, packed.data_ptr(), scale.data_ptr(), zero.data_ptr(),
           _stream(stream)), name)
    return packed, scale, zero


def quantize_sym(w: torch.Tensor, stream=None):
    """Symmetric group-128 quantization (q4_quantize_sym); same outputs as quantize."""
    return quantize(w, stream, symmetric=True)


def repack(packed: torch.Tensor, scale: torch.Tensor, zero: torch.Tensor, N: int, K: int,
           out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Canonical arrays -> tiled kernel layout (uint8 [weight_bytes(N, K)])."""
    for t, n in ((packed, "packed"), (scale, "scale"), (zero, "zero")):
        _cuda(t, n)
    nb = weight_bytes(N, K)
    if nb == 0:
        raise ValueError(f"invalid shape {N}x{K}")
    if out is None:
        out = torch.empty(nb, dtype=torch.uint8, device=packed.device)
    _cuda(out, "out")
    _ok(_lib.q4_repack(packed.data_ptr(), scale.data_ptr(), zero.data_ptr(), N, K,
                       out.data_ptr(), _stream(stream)), "q4_repack")
    return out


def unpack(qw: torch.Tensor, N: int, K: int, stream=None):
    _cuda(qw, "qw")
    packed = torch.empty((N, K // 2), dtype=torch.uint8, device=qw.device)
    scale = torch.empty((N, K // GROUP), dtype=torch.float32, device=qw.device)
    zero = torch.empty((N, K // GROUP), dtype=torch.uint8, device=qw.device)
    _ok(_lib.q4_unpack(qw.data_ptr(), N, K, packed.data_ptr(), scale.data_ptr(),
                       zero.data_ptr(), _stream(stream)), "q4_unpack")
    return packed, scale, zero


def repack_compact(packed: torch.Tensor, scale: torch.Tensor, zero: torch.Tensor, N: int, K: int,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Canonical arrays -> compact tiles (binary16 scales, 4-bit zeros)."""
    for t, n in ((packed, "packed"), (scale, "scale"), (zero, "zero")):
        _cuda(t, n)
    nb = weight_bytes(N, K, LAYOUT_COMPACT)
    if nb == 0:
        raise ValueError(f"invalid shape {N}x{K}")
    if out is None:
        out = torch.empty(nb, dtype=torch.uint8, device=packed.device)
    _cuda(out, "out")
    _ok(_lib.q4_repack_compact(packed.data_ptr(), scale.data_ptr(), zero.data_ptr(), N, K,
                               out.data_ptr(), _stream(stream)), "q4_repack_compact")
    return out


def unpack_compact(qw: torch.Tensor, N: int, K: int, stream=None):
    """Compact tiles -> (codes u8 [N][K/2], binary16 scale bits int16 [N][K/128], zeros u8 [N][K/128])."""
    _cuda(qw, "qw")
    packed = torch.empty((N, K // 2), dtype=torch.uint8, device=qw.device)
    scale16 = torch.empty((N, K // GROUP), dtype=torch.int16, device=qw.device)
    zero = torch.empty((N, K // GROUP), dtype=torch.uint8, device=qw.device)
    _ok(_lib.q4_unpack_compact(qw.data_ptr(), N, K, packed.data_ptr(), scale16.data_ptr(),
                               zero.data_ptr(), _stream(stream)), "q4_unpack_compact")
    return packed, scale16, zero


def xsum(x: torch.Tensor, stream=None) -> torch.Tensor:
    _cuda(x, "x")
    M, K = x.shape
    out = torch.empty((M, K // GROUP), dtype=torch.float32, device=x.device)
    _ok(_lib.q4_xsum(x.data_ptr(), _DTYPE[x.dtype], M, K, out.data_ptr(), _stream(stream)),
        "q4_xsum")
    return out


@dataclass
class QWeight:
    """A weight matrix in one of the tiled kernel layouts (compact: binary16
    scales and 4-bit zeros)."""
    data: torch.Tensor  # uint8 [weight_bytes(N, K, layout)]
    N: int
    K: int
    compact: bool = False

    @property
    def layout(self) -> int:
        return LAYOUT_COMPACT if self.compact else LAYOUT_TILED

    @property
    def nbytes(self) -> int:
        return self.data.numel() * self.data.element_size()

    @classmethod
    def from_float(cls, w: torch.Tensor, stream=None, symmetric: bool = False,
                   compact: bool = False) -> "QWeight":
        N, K = w.shape
        packed, scale, zero = quantize(w, stream, symmetric=symmetric)
        if compact:
            return cls(repack_compact(packed, scale, zero, N, K, stream=stream), N, K, True)
        return cls(repack(packed, scale, zero, N, K, stream=stream), N, K)


def _zeros(nb: int, device) -> torch.Tensor | None:
    if nb == 0:
        return None
    return torch.zeros(nb, dtype=torch.uint8, device=device or torch.cuda.current_device())


def workspace(M: int, N: int, K: int, device=None) -> torch.Tensor | None:
    """A zero-filled workspace for q4_gemv (None when none is needed)."""
    return _zeros(gemv_workspace_bytes(M, N, K), device)


def gemm_workspace(M: int, N: int, K: int, device=None) -> torch.Tensor | None:
    """A zero-filled workspace for q4_gemm (None when none is needed)."""
    return _zeros(gemm_workspace_bytes(M, N, K), device)


def _ws(ws):
    if ws is None:
        return 0, 0
    on = ws.get_device()
    if on < 0 or on != _current_device():
        _elsewhere("ws", on, -1 if on < 0 else _current_device())
    return ws.data_ptr(), ws.numel()


def _product_args(x: torch.Tensor, qw: QWeight, out_dtype, out):
    _cuda(x, "x")
    M, K = x.shape
    if K != qw.K:
        raise ValueError(f"x has K={K}, weight has K={qw.K}")
    dev = x.get_device()
    if qw.data.get_device() != dev:
        _elsewhere("qw", qw.data.get_device(), dev)
    if out is None:
        out = torch.empty((M, qw.N), dtype=out_dtype or x.dtype, device=x.device)
    elif out.get_device() != dev:
        _elsewhere("out", out.get_device(), dev)
    return M, K, out


def gemv(x: torch.Tensor, qw: QWeight, out_dtype=None, out: torch.Tensor | None = None,
         ws: torch.Tensor | None = None, path: int = PATH_AUTO, stream=None) -> torch.Tensor:
    """y [M][N] = x [M][K] * w_hat^T for 1 <= M <= 16."""
    M, K, out = _product_args(x, qw, out_dtype, out)
    if ws is None:
        ws = workspace(M, qw.N, K, x.device)
    wsp, wsb = _ws(ws)
    _ok(_lib.q4_gemv_path(x.data_ptr(), _DTYPE[x.dtype], M, qw.N, K, qw.data.data_ptr(),
                          qw.layout, qw.nbytes, out.data_ptr(), _DTYPE[out.dtype], wsp, wsb,
                          path, _stream(stream)), "q4_gemv")
    return out


def gemv_noalloc(x: torch.Tensor, qw: QWeight, out_dtype=None, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """q4_gemv_noalloc: q4_gemv with the library's static scratch array as
    its workspace (for callers that cannot allocate device memory)."""
    M, K, out = _product_args(x, qw, out_dtype, out)
    _ok(_lib.q4_gemv_noalloc(x.data_ptr(), _DTYPE[x.dtype], M, qw.N, K, qw.data.data_ptr(),
                             qw.layout, qw.nbytes, out.data_ptr(), _DTYPE[out.dtype],
                             _stream(stream)), "q4_gemv_noalloc")
    return out


def gemv_timeout_selftest(x: torch.Tensor, qw: QWeight, out: torch.Tensor,
                          ws: torch.Tensor | None = None, stream=None) -> None:
    M, K = x.shape
    wsp, wsb = _ws(ws)
    _ok(_lib.q4_gemv_timeout_selftest(x.data_ptr(), _DTYPE[x.dtype], M, qw.N, K,
                                      qw.data.data_ptr(), qw.layout, qw.nbytes, out.data_ptr(),
                                      _DTYPE[out.dtype], wsp, wsb, _stream(stream)),
        "q4_gemv_timeout_selftest")


def gemm(x: torch.Tensor, qw: QWeight, out_dtype=None, out: torch.Tensor | None = None,
         ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y [M][N] = X [M][K] * w_hat^T on the tcgen05 tensor cores (any M)."""
    M, K, out = _product_args(x, qw, out_dtype, out)
    if ws is None:
        ws = gemm_workspace(M, qw.N, K, x.device)
    wsp, wsb = _ws(ws)
    _ok(_lib.q4_gemm(x.data_ptr(), _DTYPE[x.dtype], M, qw.N, K, qw.data.data_ptr(), qw.layout,
                     qw.nbytes, out.data_ptr(), _DTYPE[out.dtype], wsp, wsb, _stream(stream)),
        "q4_gemm")
    return out


def gemm_timeout_selftest(x: torch.Tensor, qw: QWeight, out: torch.Tensor,
                          ws: torch.Tensor | None = None, stream=None) -> None:
    M, K = x.shape
    wsp, wsb = _ws(ws)
    _ok(_lib.q4_gemm_timeout_selftest(x.data_ptr(), _DTYPE[x.dtype], M, qw.N, K,
                                      qw.data.data_ptr(), qw.layout, qw.nbytes, out.data_ptr(),
                                      _DTYPE[out.dtype], wsp, wsb, _stream(stream)),
        "q4_gemm_timeout_selftest")


# -------------------------------------------------- serving operators
class KVCache:
    """A blocked KV cache: k and v, [blocks][heads][block_size][head_dim] in
    bf16 or f16, both with the same strides; the last dimension is contiguous
    (a [blocks][block_size][heads][head_dim] buffer is passed as
    ``t.transpose(1, 2)``).  The tensors are used where they lie."""

    _append, _append_name = _lib.q4_rope_append, "q4_rope_append"
    _attend, _attend_name, _eight_bit = _lib.q4_attention, "q4_attention", False
    _attend_selftest = _lib.q4_attention_timeout_selftest

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        for t, n in ((k, "k"), (v, "v")):
            if not t.is_cuda:
                raise ValueError(f"{n} must be a CUDA tensor")
            if t.dim() != 4 or t.dtype not in (torch.bfloat16, torch.float16):
                raise ValueError(f"{n} must be a 4-D bfloat16 or float16 tensor")
        if k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must have the same shape, strides, type and device")
        if k.shape[3] > 1 and k.stride(3) != 1:
            raise ValueError("the last dimension must be contiguous")
        self.k, self.v, self._on = k, v, k.get_device()
        self.dtype, (_, self.heads, self.block_size, self.head_dim) = k.dtype, k.shape
        self._arg = _KVCacheArg(k.data_ptr(), v.data_ptr(), _DTYPE[k.dtype], *k.shape, *k.stride()[:3])
        self._ref = ctypes.byref(self._arg)

    @classmethod
    def empty(cls, blocks: int, heads: int, block_size: int, head_dim: int, dtype=torch.bfloat16,
              device=None) -> "KVCache":
        shape = (blocks, heads, block_size, head_dim)
        device = device or torch.cuda.current_device()
        return cls(torch.empty(shape, dtype=dtype, device=device),
                   torch.empty(shape, dtype=dtype, device=device))


class KVCache8:
    """A blocked KV cache in 8 bits (q4_kv_cache8): codes k and v, int8 or
    float8_e4m3fn [blocks][heads][block_size][head_dim], with the layouts that
    KVCache takes, and the exponents of their scales, uint8 [blocks][heads]: a
    code c stands for c * 2 ** (exp - 127).  ``dtype``: of queries and of values
    read back, bfloat16 or float16.  rope_append quantises into it, attention
    reads it and cache_read gives its values."""

    _append, _append_name = _lib.q4_rope_append8, "q4_rope_append8"
    _attend, _attend_name, _eight_bit = _lib.q4_attention8, "q4_attention8", True
    _attend_selftest = _lib.q4_attention8_timeout_selftest

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_exp: torch.Tensor, v_exp: torch.Tensor,
                 dtype=torch.bfloat16):
        for t, n in ((k, "k"), (v, "v"), (k_exp, "k_exp"), (v_exp, "v_exp")):
            if not t.is_cuda:
                raise ValueError(f"{n} must be a CUDA tensor")
            if t.device != k.device:
                raise ValueError("all tensors of a cache must lie on one device")
        if k.dim() != 4 or k.dtype not in _CODE:
            raise ValueError("k must be a 4-D int8 or float8_e4m3fn tensor")
        if k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k and v must have the same shape, strides and type")
        if k.shape[3] > 1 and k.stride(3) != 1:
            raise ValueError("the last dimension must be contiguous")
        for t, n in ((k_exp, "k_exp"), (v_exp, "v_exp")):
            if t.shape != k.shape[:2] or t.dtype != torch.uint8 or not t.is_contiguous():
                raise ValueError(f"{n} must be a contiguous uint8 tensor [blocks][heads]")
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("dtype must be bfloat16 or float16")
        self.k, self.v, self.k_exp, self.v_exp, self._on = k, v, k_exp, v_exp, k.get_device()
        self.dtype, (_, self.heads, self.block_size, self.head_dim) = dtype, k.shape
        self._arg = _KVCache8Arg(k.data_ptr(), v.data_ptr(), k_exp.data_ptr(), v_exp.data_ptr(), _CODE[k.dtype],
                                 _DTYPE[dtype], *k.shape, *k.stride()[:3])
        self._ref = ctypes.byref(self._arg)

    @classmethod
    def empty(cls, blocks: int, heads: int, block_size: int, head_dim: int, code=torch.int8,
              dtype=torch.bfloat16, device=None) -> "KVCache8":
        shape = (blocks, heads, block_size, head_dim)
        device = device or torch.cuda.current_device()
        return cls(*(torch.empty(shape, dtype=code, device=device) for _ in "kv"),
                   *(torch.zeros(shape[:2], dtype=torch.uint8, device=device) for _ in "kv"), dtype)


@dataclass
class CachePlan:
    """What q4_cache_plan writes for one step."""
    q_start: torch.Tensor   # int32 [B + 1]
    kv_len: torch.Tensor    # int32 [B]; 0: not served, the request keeps the length it had
    position: torch.Tensor  # int32 [T]
    slot: torch.Tensor      # int64 [T]
    counts: torch.Tensor    # int32 [4]: rows used, tokens served, free blocks left, requests not served

    @classmethod
    def empty(cls, B: int, T: int, device=None) -> "CachePlan":
        device = device or torch.cuda.current_device()
        i32 = torch.int32
        return cls(torch.empty(B + 1, dtype=i32, device=device), torch.empty(B, dtype=i32, device=device),
                   torch.empty(T, dtype=i32, device=device), torch.empty(T, dtype=torch.int64, device=device),
                   torch.empty(4, dtype=i32, device=device))


# The checks below are a call's whole host cost beside the launch: a few tenths
# of a microsecond each, where a decode step's kernels take several.
def _raw_stream(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _on(stream):
    """What a call allocates itself (outputs, a workspace) belongs to the
    stream it runs on, so that filling, use and reuse stay in order."""
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(stream))


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _array(t: torch.Tensor, name: str, dtype, dev: int, n: int | None = None) -> int:
    """Address of a contiguous array of n elements on device dev."""
    if t.get_device() != dev:
        _elsewhere(name, t.get_device(), dev)
    if not (t.dtype == dtype and t.is_contiguous() and (n is None or t.numel() == n)):
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor" +
                         ("" if n is None else f" of {n} elements") + f", is {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _table(table: torch.Tensor, B: int, dev: int):
    """Address, row stride and width of a block table."""
    if table.get_device() != dev:
        _elsewhere("table", table.get_device(), dev)
    if not (table.dtype == torch.int32 and table.dim() == 2 and table.shape[0] == B):
        raise ValueError(f"table must be an int32 CUDA tensor of {B} rows")
    width = table.shape[1]
    stride, one = table.stride()
    if one != 1 and width > 1:
        raise ValueError("the table's rows must be contiguous")
    # the row stride of a single row is never used
    return table.data_ptr(), stride if B > 1 else max(stride, width), width


def _rows(t: torch.Tensor, name: str, dtype, dev: int):
    """Token rows, 2-D or 3-D, contiguous but for the stride between rows:
    their address, number, elements and stride."""
    if t.get_device() != dev:
        _elsewhere(name, t.get_device(), dev)
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        n = shape[1] * shape[2]
        dense = (stride[2] == 1 or shape[2] == 1) and (stride[1] == shape[2] or shape[1] == 1)
    else:
        n = shape[-1] if len(shape) == 2 else 0
        dense = len(shape) == 2 and (stride[1] == 1 or n == 1)
    if not (dense and t.dtype == dtype and shape[0] >= 1):
        raise ValueError(f"{name} must be {dtype} CUDA rows of contiguous elements, is {t.dtype} {tuple(shape)}")
    return t.data_ptr(), shape[0], n, stride[0] if shape[0] > 1 else max(stride[0], n)


def cache_plan(cached: torch.Tensor, fresh: torch.Tensor, table: torch.Tensor,
               free_blocks: torch.Tensor, free_count: torch.Tensor, block_size: int, T: int,
               out: CachePlan | None = None, stream=None) -> CachePlan:
    """The step's plan from request lengths (q4_cache_plan): int32 ``cached``
    and ``fresh`` [B]; ``table`` int32 [B][W] gets the blocks of the new tokens,
    taken from the end of ``free_blocks`` int32, of which the first
    ``free_count`` (int32 [1]) are free.  T token rows.  A step's loop keeps
    one ``out``: allocating its five arrays takes longer than the plan."""
    B, dev = cached.numel(), _current_device()
    tp, ts, width = _table(table, B, dev)
    if out is None:
        if stream is None:
            out = CachePlan.empty(B, T, cached.device)
        else:
            with _on(stream):
                out = CachePlan.empty(B, T, cached.device)
    i32 = torch.int32
    _ok(_lib.q4_cache_plan(_array(cached, "cached", i32, dev), _array(fresh, "fresh", i32, dev, B), B, block_size, tp, ts,
                           width, _array(free_blocks, "free_blocks", i32, dev), _array(free_count, "free_count", i32, dev, 1),
                           free_blocks.numel(), T, _array(out.q_start, "q_start", i32, dev, B + 1),
                           _array(out.kv_len, "kv_len", i32, dev, B), _array(out.position, "position", i32, dev, T),
                           _array(out.slot, "slot", torch.int64, dev, T), _array(out.counts, "counts", i32, dev, 4),
                           _raw_stream(stream, dev)), "q4_cache_plan")
    return out


def rope_frequencies(rot: int, base: float = 10000.0, stretch: float = 1.0, by_parts: bool = False,
                     length: int = 4096, slow: float = 1.0, fast: float = 32.0, device=None):
    """(freq f64 [rot / 2], factor) for rope_append: base ** (-2 i / rot), and
    for contexts ``stretch`` times longer than ``length`` either every
    frequency over ``stretch`` (position interpolation) or, ``by_parts``,
    only those of pairs that turn fewer than ``slow`` times over ``length``
    tokens; those that turn more than ``fast`` times are kept, with a linear
    ramp between, and cos and sin grow by 0.1 ln(stretch) + 1 (the YaRN
    paper's formulas, Peng et al. 2023)."""
    if rot < 0 or rot % 2:
        raise ValueError("rot must be even")
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    factor = 1.0
    if by_parts:
        factor = 0.1 * math.log(stretch) + 1.0 if stretch > 1.0 else 1.0
        keep = [min(1.0, max(0.0, (length * x / (2 * math.pi) - slow) / (fast - slow))) for x in f]
        f = [x / stretch * (1 - k) + x * k for x, k in zip(f, keep)]
    else:
        f = [x / stretch for x in f]
    device = device or torch.cuda.current_device()
    return torch.tensor(f, dtype=torch.float64, device=device), factor


def rope_append(qkv: torch.Tensor, cache: KVCache | KVCache8, position: torch.Tensor, slot: torch.Tensor,
                freq: torch.Tensor, heads: int, interleaved: bool = False, factor: float = 1.0,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rotate the queries and keys of ``qkv`` [T][(heads + 2 * cache.heads) *
    head_dim] and append keys and values to the cache (q4_rope_append).
    2 * len(freq) elements of each head turn.  Returns the queries
    [T][heads][head_dim] (``out`` may be the query part of qkv itself).  Into a
    KVCache8 keys and values go quantised (q4_rope_append8)."""
    dev = _current_device()
    if cache._on != dev:
        _elsewhere("cache", cache._on, dev)
    qp, T, n, stride = _rows(qkv, "qkv", cache.dtype, dev)
    if n != (heads + 2 * cache.heads) * cache.head_dim:
        raise ValueError(f"qkv rows have {n} elements, not (heads + 2 * cache heads) * head_dim")
    if out is None:
        out = _empty((T, heads, cache.head_dim), cache.dtype, qkv.device, stream)
        op, ostride = out.data_ptr(), heads * cache.head_dim
    else:
        op, To, no, ostride = _rows(out, "out", cache.dtype, dev)
        if To != T or no != heads * cache.head_dim:
            raise ValueError("out must be T rows of heads * head_dim")
    _ok(cache._append(qp, stride, T, heads, 2 * freq.numel(), ROPE_INTERLEAVED if interleaved else ROPE_HALF,
                      _array(freq, "freq", torch.float64, dev), factor, _array(position, "position", torch.int32, dev, T),
                      _array(slot, "slot", torch.int64, dev, T), op, ostride, cache._ref,
                      _raw_stream(stream, dev)), cache._append_name)
    return out


def cache_read(cache: KVCache8, table: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor, T: int,
               out: tuple[torch.Tensor, torch.Tensor] | None = None, out_dtype=None, stream=None):
    """Reads tokens back from an 8-bit cache (q4_cache_read8): (k, v), T rows
    [heads][head_dim] each, of the cache's dtype or float32.  Rows q_start[b] ..
    q_start[b + 1] are request b's last tokens of the kv_len[b] it holds, in
    order: all of them where q_start is the running sum of kv_len."""
    if type(cache) is not KVCache8:
        raise TypeError("cache must be a KVCache8: a 16-bit cache holds its values as they are")
    dev = _current_device()
    if cache._on != dev:
        _elsewhere("cache", cache._on, dev)
    B = kv_len.numel()
    tp, ts, width = _table(table, B, dev)
    row = cache.heads * cache.head_dim
    if out is None:
        shape, dtype = (T, cache.heads, cache.head_dim), out_dtype or cache.dtype
        out = _empty(shape, dtype, table.device, stream), _empty(shape, dtype, table.device, stream)
        kp, vp, ks, vs = out[0].data_ptr(), out[1].data_ptr(), row, row
    else:
        kp, Tk, nk, ks = _rows(out[0], "out", out[0].dtype, dev)
        vp, Tv, nv, vs = _rows(out[1], "out", out[0].dtype, dev)
        if Tk != T or Tv != T or nk != row or nv != row:
            raise ValueError("out must be two tensors of T rows of heads * head_dim")
    _ok(_lib.q4_cache_read8(cache._ref, tp, ts, width, _array(q_start, "q_start", torch.int32, dev, B + 1),
                            _array(kv_len, "kv_len", torch.int32, dev, B), B, T, kp, ks, vp, vs,
                            _DTYPE.get(out[0].dtype, -1), _raw_stream(stream, dev)), "q4_cache_read8")
    return out


def attention_workspace_bytes(max_fresh: int, heads: int, kv_heads: int, head_dim: int, eight_bit: bool = False) -> int:
    fn = _lib.q4_attention8_workspace_bytes if eight_bit else _lib.q4_attention_workspace_bytes
    return int(fn(max_fresh, heads, kv_heads, head_dim))


def attention_workspace(max_fresh: int, heads: int, kv_heads: int, head_dim: int,
                        device=None, eight_bit: bool = False) -> torch.Tensor | None:
    """A zero-filled workspace for attention (not shared with the products'),
    ``eight_bit``: over a KVCache8."""
    return _zeros(attention_workspace_bytes(max_fresh, heads, kv_heads, head_dim, eight_bit), device)


def attention(q: torch.Tensor, cache: KVCache | KVCache8, table: torch.Tensor, q_start: torch.Tensor,
              kv_len: torch.Tensor, max_fresh: int, scale: float | None = None, window: int = 0,
              out: torch.Tensor | None = None, out_dtype=None, return_lse: bool = False,
              lse: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None, _call=None):
    """Attention of each request's new tokens over its cache (q4_attention;
    q4_attention8 over a KVCache8).

    q [T][heads][head_dim]; request b's rows are q_start[b]..q_start[b + 1],
    its keys the kv_len[b] first tokens of table row b, its own new ones last.
    ``window`` > 0: each token sees that many keys, itself included.  Returns
    o [T][heads][head_dim] (q's type, or float32), with ``return_lse`` also the
    f32 log-sum-exp [T][heads].  Keep one ``ws`` (attention_workspace) per
    stream: without it each call allocates and zero-fills tens of megabytes."""
    dev = _current_device()
    if cache._on != dev:
        _elsewhere("cache", cache._on, dev)
    qp, T, n, stride = _rows(q, "q", cache.dtype, dev)
    D = cache.head_dim
    if q.dim() != 3 or q.shape[2] != D:
        raise ValueError(f"q must be [T][heads][{D}]")
    heads = q.shape[1]
    B = kv_len.numel()
    tp, ts, width = _table(table, B, dev)
    if out is None:
        out = _empty((T, heads, D), out_dtype or cache.dtype, q.device, stream)
        op, ostride = out.data_ptr(), n
    else:
        op, To, no, ostride = _rows(out, "out", out.dtype, dev)
        if To != T or no != n:
            raise ValueError("out must be T rows of heads * head_dim")
    if return_lse and lse is None:
        lse = _empty((T, heads), torch.float32, q.device, stream)
    if ws is None:
        with _on(stream if stream is not None else torch.cuda.current_stream()):
            ws = attention_workspace(max_fresh, heads, cache.heads, D, q.device, cache._eight_bit)
    _ok((_call or cache._attend)(qp, stride, T, heads, cache._ref, tp, ts, width, _array(q_start, "q_start", torch.int32, dev, B + 1),
              _array(kv_len, "kv_len", torch.int32, dev, B), B, max_fresh, D ** -0.5 if scale is None else scale, window,
              op, _DTYPE.get(out.dtype, -1), ostride,
              0 if lse is None else _array(lse, "lse", torch.float32, dev, T * heads),
              *_ws(ws), _raw_stream(stream, dev)), cache._attend_name)
    return (out, lse) if lse is not None else out


def attention_timeout_selftest(q: torch.Tensor, cache: KVCache | KVCache8, table: torch.Tensor, q_start: torch.Tensor,
                               kv_len: torch.Tensor, max_fresh: int, out: torch.Tensor, ws: torch.Tensor,
                               stream=None) -> None:
    attention(q, cache, table, q_start, kv_len, max_fresh, out=out, ws=ws, stream=stream,
              _call=cache._attend_selftest)


def check(stream=None) -> int:
    """Synchronise and return the library status (raises nothing)."""
    return int(_lib.q4_check(_stream(stream)))
