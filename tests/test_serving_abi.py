"""Refusals of the serving operators: every bad argument is answered on the
host, before any CUDA call (CPU only; the pointers are never dereferenced)."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "weight_only_int4_group_gb300", "libq4.so")
P = 4096
BAD, UNSUP, MISALIGNED = 1, 2, 3
F32, BF16, F16 = 0, 1, 2


class Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("type", ctypes.c_int)] + [
        (n, ctypes.c_int64) for n in ("blocks", "heads", "block_size", "head_dim", "block_stride",
                                      "head_stride", "token_stride")]


CACHE = dict(k=P, v=P, type=BF16, blocks=10, heads=2, block_size=16, head_dim=64,
             block_stride=2048, head_stride=1024, token_stride=64)
BAD_CACHES = [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(blocks=0), BAD), (dict(heads=0), BAD),
    (dict(block_size=0), BAD), (dict(head_dim=0), BAD), (dict(type=F32), UNSUP), (dict(type=7), UNSUP),
    (dict(blocks=2 ** 31), UNSUP), (dict(block_size=24), UNSUP), (dict(block_size=8), UNSUP),
    (dict(head_dim=136, token_stride=136), UNSUP), (dict(head_dim=60), UNSUP), (dict(k=P + 8), MISALIGNED),
    (dict(v=P + 2), MISALIGNED), (dict(token_stride=68, head_stride=1088, block_stride=2176), MISALIGNED),
    (dict(token_stride=56), BAD),      # shorter than a token
    (dict(head_stride=512), BAD),      # heads overlap
    (dict(block_stride=1024), BAD),    # blocks overlap
    (dict(block_stride=-2048), BAD), (dict(block_stride=2 ** 60), BAD),
]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        import __graft_entry__
        __graft_entry__.build()
    x = ctypes.CDLL(LIB)
    V, I, Z, S, F, C = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int, ctypes.c_float,
                        ctypes.POINTER(Cache))
    x.q4_cache_plan.argtypes = [V, V, I, I, V, I, I, V, V, I, I, V, V, V, V, V, V]
    x.q4_rope_append.argtypes = [V, I, I, I, I, S, V, F, V, V, V, I, C, V]
    x.q4_attention.argtypes = [V, I, I, I, C, V, I, I, V, V, I, I, F, I, V, S, I, V, V, Z, V]
    x.q4_attention_workspace_bytes.argtypes = [I, I, I, I]
    x.q4_attention_workspace_bytes.restype = Z
    return x


def call(fn, good, order, **kw):
    a = dict(good, **kw)
    args = [ctypes.byref(Cache(**a[n])) if n == "cache" and a[n] is not None else a[n] for n in order]
    return fn(*args)


PLAN = dict(cached=P, fresh=P, B=4, S=16, table=P, stride=8, width=8, free=P, count=P, cap=9, T=5,
            q_start=P, kv_len=P, position=P, slot=P, counts=P, stream=None)


@pytest.mark.parametrize("change,status", [
    *(({n: None}, BAD) for n in ("cached", "fresh", "table", "free", "count", "q_start", "kv_len", "position",
                                 "slot", "counts")),
    *(({n: v}, BAD) for n in ("B", "S", "width", "cap", "T") for v in (0, -1)),
    (dict(stride=7), BAD), (dict(B=16385), UNSUP), (dict(T=2 ** 31), UNSUP), (dict(cap=2 ** 31), UNSUP),
    (dict(width=2 ** 28, stride=2 ** 28), UNSUP), (dict(stride=2 ** 50), UNSUP),
], ids=str)
def test_plan_refusals(lib, change, status):
    assert call(lib.q4_cache_plan, PLAN, list(PLAN), **change) == status


ROPE = dict(qkv=P, stride=512, T=3, Hq=4, rot=64, style=0, freq=P, factor=1.0, position=P, slot=P, out=P,
            q_stride=256, cache=CACHE, stream=None)


@pytest.mark.parametrize("change,status", [
    *(({n: None}, BAD) for n in ("qkv", "freq", "position", "slot", "out", "cache")),
    (dict(T=0), BAD), (dict(Hq=0), BAD), (dict(rot=-2), BAD), (dict(rot=63), BAD), (dict(rot=66), BAD),
    (dict(style=2), BAD), (dict(stride=504), BAD), (dict(q_stride=248), BAD), (dict(T=2 ** 31), UNSUP),
    (dict(qkv=P + 8), MISALIGNED), (dict(out=P + 4), MISALIGNED), (dict(stride=516), MISALIGNED),
    (dict(q_stride=260), MISALIGNED), (dict(stride=2 ** 40), UNSUP), (dict(Hq=10 ** 6), UNSUP),
    *((dict(cache=dict(CACHE, **c)), s) for c, s in BAD_CACHES),
], ids=str)
def test_rope_refusals(lib, change, status):
    assert call(lib.q4_rope_append, ROPE, list(ROPE), **change) == status


ATTN = dict(q=P, q_stride=256, T=3, Hq=4, cache=CACHE, table=P, stride=8, width=8, q_start=P, kv_len=P, B=2,
            max_fresh=1, scale=0.125, window=0, o=P, ot=BF16, o_stride=256, lse=None, ws=P, wsb=1 << 30, stream=None)


@pytest.mark.parametrize("change,status", [
    *(({n: None}, BAD) for n in ("q", "cache", "table", "q_start", "kv_len", "o")),
    *(({n: 0}, BAD) for n in ("T", "B", "Hq", "width", "max_fresh")),
    (dict(Hq=3), BAD), (dict(stride=7), BAD), (dict(window=-1), BAD), (dict(scale=float("nan")), BAD),
    (dict(scale=float("inf")), BAD), (dict(q_stride=248), BAD), (dict(o_stride=248), BAD),
    (dict(ot=F16), UNSUP), (dict(ot=9), UNSUP), (dict(T=2 ** 30), UNSUP), (dict(B=2 ** 31), UNSUP),
    (dict(width=2 ** 28, stride=2 ** 28), UNSUP), (dict(q=P + 8), MISALIGNED), (dict(o=P + 8), MISALIGNED),
    (dict(ws=P + 8), MISALIGNED), (dict(q_stride=260), MISALIGNED), (dict(o_stride=260), MISALIGNED),
    (dict(lse=P + 2), MISALIGNED),
    *((dict(cache=dict(CACHE, **c)), s) for c, s in BAD_CACHES),
], ids=str)
def test_attention_refusals(lib, change, status):
    assert call(lib.q4_attention, ATTN, list(ATTN), **change) == status


def test_workspace_bytes_of_invalid_sizes(lib):
    for sizes in ((0, 8, 1, 64), (1, 0, 1, 64), (1, 8, 3, 64), (1, 8, 0, 64), (1, 8, 1, 136), (1, 8, 1, 12)):
        assert lib.q4_attention_workspace_bytes(*sizes) == 0


@pytest.mark.gpu
def test_short_workspace_and_wrong_tensors_are_refused():
    import torch
    import weight_only_int4_group_gb300 as q4
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = q4.KVCache.empty(4, 2, 16, 64)
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    table, start, kv = torch.zeros((1, 2), **i32), torch.tensor([0, 1], **i32), torch.zeros(1, **i32)
    ws = q4.attention_workspace(1, 4, 2, 64)
    with pytest.raises(q4.Q4Error):
        q4.attention(q, cache, table, start, kv, 1, ws=ws[:-16])
    for bad in (dict(q=q.float()), dict(q=q[:, :, :32]), dict(table=table.long()), dict(q_start=start[:1]),
                dict(q=q.half()), dict(kv_len=kv.cpu())):
        a = dict(dict(q=q, cache=cache, table=table, q_start=start, kv_len=kv, max_fresh=1, ws=ws), **bad)
        with pytest.raises((ValueError, q4.Q4Error)):
            q4.attention(**a)
    with pytest.raises(ValueError):
        q4.KVCache(cache.k, cache.v.half())
    with pytest.raises(ValueError):
        q4.KVCache(cache.k, cache.v.transpose(0, 1))
    qkv = torch.zeros((1, 8 * 64), dtype=torch.bfloat16, device="cuda")
    pos, slot = torch.zeros(1, **i32), torch.zeros(1, dtype=torch.int64, device="cuda")
    freq, _ = q4.rope_frequencies(64)
    for bad in (dict(heads=3), dict(freq=freq.float()), dict(slot=pos), dict(position=slot), dict(qkv=qkv[:, :256])):
        a = dict(dict(qkv=qkv, cache=cache, position=pos, slot=slot, freq=freq, heads=4), **bad)
        with pytest.raises((ValueError, q4.Q4Error)):
            q4.rope_append(**a)
    with pytest.raises((ValueError, q4.Q4Error)):
        q4.cache_plan(kv, kv, table, start, start, 16, 0)
    with pytest.raises(ValueError):
        q4.cache_plan(kv, start, table, start, start, 16, 1)
    assert q4.check() == q4.OK


def test_debug_library_exports_the_same(lib):
    """Both builds carry the operators (loaded in a child: one process, one build)."""
    other = os.path.join(os.path.dirname(LIB), "libq4_debug.so")
    if not os.path.exists(other):
        pytest.skip("the bounds-checked build is not there")
    code = f"import ctypes; l = ctypes.CDLL({other!r}); l.q4_cache_plan; l.q4_rope_append; l.q4_attention"
    subprocess.run([sys.executable, "-c", code], check=True)


@pytest.mark.parametrize("source", ["serve.cuh", "attention.cuh", "attention.cu", "attention_tc.cu", "cache.cu", "gemv.cu"])
def test_kernels_that_start_early_load_coherently(source):
    """They are resident while the kernel that writes their inputs may still
    run: no load of the non-coherent path, which asks for data that nothing
    writes as long as the kernel lives."""
    text = open(os.path.join(ROOT, "weight_only_int4_group_gb300", "csrc", source)).read()
    code = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    assert not re.search(r"__ldg\b|ld\.global\.nc|__restrict__", code)


@pytest.mark.parametrize("Hq,heads", [(1, 1), (4, 2), (64, 1), (1000, 2)])
def test_attention_refuses_rows_whose_tiles_pass_32_bits(lib, Hq, heads):
    """Row indices run on to the end of a tile of 256 rows."""
    good = dict(ATTN, Hq=Hq, q_stride=Hq * 64, o_stride=Hq * 64, cache=dict(CACHE, heads=heads))
    for rows in (2 ** 31 - 1, 2 ** 31 - 256, 2 ** 31 - 513):
        assert call(lib.q4_attention, good, list(ATTN), T=rows // Hq if Hq < 1000 else 2147483) == UNSUP


PLAN_APART = dict(PLAN, **{n: P * i for i, n in enumerate(("cached", "fresh", "table", "free", "count", "q_start", "kv_len",
                                                           "position", "slot", "counts"), 1)})


@pytest.mark.parametrize("out", ["table", "q_start", "kv_len", "position", "slot", "counts"])
@pytest.mark.parametrize("other", ["cached", "fresh", "table", "free", "count", "q_start", "kv_len", "position", "slot", "counts"])
def test_plan_refuses_outputs_over_other_arrays(lib, out, other):
    """kv_len over cached would be the tempting one: CTAs read the lengths
    again after some of them have been written."""
    if out == other:
        return
    size = dict(table=(3 * 8 + 8) * 4, q_start=20, kv_len=16, position=20, slot=40, counts=16)[out]
    for at in (PLAN_APART[out], PLAN_APART[out] + size - 4):
        assert call(lib.q4_cache_plan, PLAN_APART, list(PLAN), **{other: at}) == BAD


def test_plan_checks_every_row_of_a_wide_table(lib):
    """Rows of a table whose stride is far above its width."""
    wide = dict(PLAN_APART, table=P * 100, stride=P // 4)
    for at, name in ((P * 101 + 28, "cached"), (P * 101 - 4, "kv_len"), (P * 103 + 31 - 3, "fresh")):
        assert call(lib.q4_cache_plan, wide, list(PLAN), **{name: at}) == BAD
