"""Refusals of the 8-bit cache's entry points: every bad argument is answered on
the host, before any CUDA call (CPU only; the pointers are never dereferenced)."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "weight_only_int4_group_gb300", "libq4.so")
P = 4096
BAD, UNSUP, MISALIGNED = 1, 2, 3
F32, BF16, F16 = 0, 1, 2


class Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_exp", "v_exp")] + [
        ("code", ctypes.c_int), ("type", ctypes.c_int)] + [
        (n, ctypes.c_int64) for n in ("blocks", "heads", "block_size", "head_dim", "block_stride",
                                      "head_stride", "token_stride")]


CACHE = dict(k=P, v=2 * P, k_exp=P, v_exp=2 * P, code=0, type=BF16, blocks=10, heads=2, block_size=16, head_dim=64,
             block_stride=2048, head_stride=1024, token_stride=64)
BAD_CACHES = [
    *((({n: None}, BAD)) for n in ("k", "v", "k_exp", "v_exp")), (dict(blocks=0), BAD), (dict(heads=0), BAD),
    (dict(block_size=0), BAD), (dict(head_dim=0), BAD), (dict(type=F32), UNSUP), (dict(type=7), UNSUP),
    (dict(code=2), UNSUP), (dict(code=-1), UNSUP),
    (dict(blocks=2 ** 31), UNSUP), (dict(block_size=24), UNSUP), (dict(block_size=8), UNSUP),
    (dict(head_dim=144, token_stride=144), UNSUP), (dict(head_dim=56), UNSUP), (dict(head_dim=72, token_stride=80), UNSUP),
    (dict(k=P + 8), MISALIGNED), (dict(v=2 * P + 2), MISALIGNED),
    (dict(token_stride=72, head_stride=1152, block_stride=2304), MISALIGNED),
    (dict(token_stride=48), BAD),      # shorter than a token
    (dict(head_stride=512), BAD),      # heads overlap
    (dict(block_stride=1024), BAD),    # blocks overlap
    (dict(block_stride=-2048), BAD), (dict(block_stride=2 ** 60), BAD),
    (dict(v=P), BAD), (dict(v_exp=P), BAD), (dict(v_exp=P + 19), BAD), (dict(k_exp=2 * P + 19), BAD),
]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        import __graft_entry__
        __graft_entry__.build()
    x = ctypes.CDLL(LIB)
    V, I, Z, S, F, C = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int, ctypes.c_float,
                        ctypes.POINTER(Cache))
    x.q4_rope_append8.argtypes = [V, I, I, I, I, S, V, F, V, V, V, I, C, V]
    x.q4_cache_read8.argtypes = [C, V, I, I, V, V, I, I, V, I, V, I, S, V]
    x.q4_attention8.argtypes = [V, I, I, I, C, V, I, I, V, V, I, I, F, I, V, S, I, V, V, Z, V]
    x.q4_attention8_workspace_bytes.argtypes = [I, I, I, I]
    x.q4_attention8_workspace_bytes.restype = Z
    return x


def call(fn, good, **kw):
    a = dict(good, **kw)
    return fn(*(ctypes.byref(Cache(**v)) if n == "cache" and v is not None else v for n, v in a.items()))


APPEND = dict(qkv=P, stride=512, T=3, Hq=4, rot=64, style=0, freq=P, factor=1.0, position=P, slot=P, out=P,
              q_stride=256, cache=CACHE, stream=None)


@pytest.mark.parametrize("change,status", [
    *(({n: None}, BAD) for n in ("qkv", "freq", "position", "slot", "out", "cache")),
    *(({n: v}, BAD) for n in ("T", "Hq") for v in (0, -1)),
    (dict(rot=63), BAD), (dict(rot=66), BAD), (dict(rot=-2), BAD), (dict(style=2), BAD),
    (dict(T=2 ** 31 - 1), UNSUP), (dict(T=2 ** 31), UNSUP), (dict(Hq=65537), UNSUP),
    (dict(stride=504), BAD), (dict(q_stride=248), BAD), (dict(stride=2 ** 31), UNSUP), (dict(q_stride=2 ** 31), UNSUP),
    (dict(stride=516), MISALIGNED), (dict(q_stride=260), MISALIGNED), (dict(qkv=P + 2), MISALIGNED), (dict(out=P + 8), MISALIGNED),
    *((dict(cache=dict(CACHE, **c)), s) for c, s in BAD_CACHES),
], ids=str)
def test_append_refusals(lib, change, status):
    assert call(lib.q4_rope_append8, APPEND, **change) == status


READ = dict(cache=CACHE, table=P, table_stride=8, width=8, q_start=P, kv_len=P, B=4, T=9, k_out=P, k_stride=128, v_out=P,
            v_stride=128, ot=BF16, stream=None)


@pytest.mark.parametrize("change,status", [
    *(({n: None}, BAD) for n in ("cache", "table", "q_start", "kv_len", "k_out", "v_out")),
    *(({n: v}, BAD) for n in ("T", "B", "width") for v in (0, -1)),
    (dict(table_stride=7), BAD), (dict(ot=F16), UNSUP), (dict(ot=5), UNSUP),
    (dict(T=2 ** 31 - 1), UNSUP), (dict(B=2 ** 31), UNSUP), (dict(table_stride=2 ** 50), UNSUP),
    (dict(width=2 ** 28, table_stride=2 ** 28), UNSUP),
    (dict(k_stride=120), BAD), (dict(v_stride=0), BAD), (dict(v_stride=2 ** 31), UNSUP),
    (dict(k_stride=132), MISALIGNED), (dict(k_out=P + 8), MISALIGNED), (dict(v_out=P + 2), MISALIGNED),
    *((dict(cache=dict(CACHE, **c)), s) for c, s in BAD_CACHES),
], ids=str)
def test_read_refusals(lib, change, status):
    assert call(lib.q4_cache_read8, READ, **change) == status


ATTN = dict(q=P, q_stride=256, T=5, Hq=4, cache=CACHE, table=P, table_stride=8, width=8, q_start=P, kv_len=P, B=4,
            max_fresh=2, scale=0.1, window=0, o=P, ot=BF16, o_stride=256, lse=None, ws=P, wsb=1 << 40, stream=None)


@pytest.mark.parametrize("change,status", [
    *(({n: None}, BAD) for n in ("q", "cache", "table", "q_start", "kv_len", "o")),
    *(({n: v}, BAD) for n in ("T", "B", "Hq", "max_fresh", "width") for v in (0, -1)),
    (dict(Hq=3), BAD), (dict(table_stride=7), BAD), (dict(window=-1), BAD), (dict(scale=float("nan")), BAD),
    (dict(scale=float("inf")), BAD), (dict(q_stride=248), BAD), (dict(o_stride=0), BAD),
    (dict(ot=F16), UNSUP), (dict(T=2 ** 30), UNSUP), (dict(B=2 ** 31), UNSUP), (dict(max_fresh=2 ** 31), UNSUP),
    (dict(width=2 ** 27, table_stride=2 ** 27), UNSUP), (dict(q_stride=2 ** 31), UNSUP),
    (dict(q=P + 8), MISALIGNED), (dict(o=P + 2), MISALIGNED), (dict(ws=P + 4), MISALIGNED), (dict(q_stride=260), MISALIGNED),
    (dict(lse=P + 2), MISALIGNED),
    *((dict(cache=dict(CACHE, **c)), s) for c, s in BAD_CACHES),
], ids=str)
def test_attention_refusals(lib, change, status):
    assert call(lib.q4_attention8, ATTN, **change) == status


@pytest.mark.parametrize("sizes", [(0, 4, 2, 64), (1, 3, 2, 64), (1, 4, 0, 64), (1, 4, 2, 72), (1, 4, 2, 144), (1, 1 << 17, 1, 64)])
def test_workspace_of_bad_sizes(lib, sizes):
    assert lib.q4_attention8_workspace_bytes(*sizes) == 0
