"""The 8-bit cache's kernels write nothing outside their buffers: guard bytes
around every output, and the suites once more against the bounds-checked
library in a child process."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

from cache8_ref import CODES, Requests8, raw
from test_gpu_canaries import DEBUG_LIB, UNDER_DEBUG, Guarded

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def q4():
    import weight_only_int4_group_gb300 as m
    return m


def guarded(shape, dtype, fill=None):
    size = torch.Size(shape).numel() * torch.empty((), dtype=dtype).element_size()
    g = Guarded(size)
    t = g.view(dtype, shape)
    if fill is not None:
        t.view(torch.uint8).copy_(fill.contiguous().view(torch.uint8))
    return g, t


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_guard_bytes(dtype, code):
    """Ragged sizes: cache, exponents, queries, rows read back, outputs and workspace."""
    m = q4()
    for lengths, D, S, heads, kv in (([(7, 25), (0, 1), (16, 3), (100, 33)], 80, 16, 6, 2), ([(63, 1), (5, 1)], 64, 32, 5, 5),
                                     ([(200, 70)], 128, 48, 8, 1)):
        r = Requests8(lengths, heads, kv, D, S, dtype, code, seed=3)
        parts = [guarded(x.shape, x.dtype, x) for x in (r.k, r.v, r.k_exp, r.v_exp)]
        cache = m.KVCache8(*(t for _, t in parts), dtype)
        T = r.T
        slot = torch.tensor([int(r.table[b, p // S]) * S + p % S for b, (c, n) in enumerate(lengths) for p in range(c, c + n)],
                            device="cuda")
        pos = torch.tensor([p for c, n in lengths for p in range(c, c + n)], dtype=torch.int32, device="cuda")
        qkv = torch.randn(T, (heads + 2 * kv) * D, device="cuda").to(dtype)
        freq, _ = m.rope_frequencies(D)
        gq, q = guarded((T, heads, D), dtype)
        m.rope_append(qkv, cache, pos, slot, freq, heads, out=q)
        outs = [guarded((T, kv, D), t) for t in (dtype, dtype)]
        m.cache_read(cache, r.table, r.q_start, r.kv_len, T, out=tuple(t for _, t in outs))
        go, o = guarded((T, heads, D), dtype)
        gl, lse = guarded((T, heads), torch.float32)
        nb = m.attention_workspace_bytes(r.max_fresh, heads, kv, D, eight_bit=True)
        gw, ws = guarded((nb,), torch.uint8, torch.zeros(nb, dtype=torch.uint8, device="cuda"))
        m.attention(q, cache, r.table, r.q_start, r.kv_len, r.max_fresh, out=o, lse=lse, return_lse=True, ws=ws)
        assert m.check() == m.OK
        for i, g in enumerate([gq, go, gl, gw, *(g for g, _ in parts), *(g for g, _ in outs)]):
            g.assert_guards(f"{lengths}, buffer {i}")
        # the last tokens read back are the appended ones' values, and finite
        assert torch.isfinite(outs[1][1]).all() and raw(cache.k).numel()


@pytest.mark.skipif(UNDER_DEBUG, reason="already running against the debug library")
def test_suites_under_debug_build():
    assert os.path.exists(DEBUG_LIB), "libq4_debug.so is missing: run __graft_entry__.build()"
    env = dict(os.environ, Q4_LIBRARY=DEBUG_LIB)
    names = ["test_gpu_cache8.py", "test_gpu_attention8.py", "test_gpu_cache8_guard.py"]
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider",
                        *(os.path.join(ROOT, "tests", n) for n in names)], cwd=ROOT, env=env, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
