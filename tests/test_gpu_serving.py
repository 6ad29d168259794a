"""The serving operators together, as examples/attention_block.py runs them:
a mixed batch against 64 bits, and decoding token by token against the whole
prompt at once.  And none of them writes outside its buffers: guard bytes
around every output, and the suites once more against the bounds-checked
library in a child process."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

from serving_ref import Requests, assert_attention, attention_reference, rope_reference
from test_gpu_canaries import DEBUG_LIB, UNDER_DEBUG, Guarded

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def q4():
    import weight_only_int4_group_gb300 as m
    return m


def dense(w):
    """The weight matrix a QWeight stands for, in 64 bits."""
    packed, scale, zero = q4().unpack(w.data, w.N, w.K)
    codes = torch.stack([packed & 15, packed >> 4], -1).view(w.N, w.K).double()
    rep = lambda t: t.double().repeat_interleave(128, 1)  # noqa: E731
    return (codes - rep(zero)) * rep(scale)


def test_attention_block_against_64_bits():
    from attention_block import AttentionBlock, Server
    heads, kv, D, hidden = 4, 2, 64, 256
    server = Server(3, 60, 16, 12)
    block = AttentionBlock(hidden, heads, kv, D, 40, 60, dtype=torch.float16)
    block.cache.k.fill_(float("nan"))
    block.cache.v.fill_(float("nan"))
    wq, wo = dense(block.qkv), dense(block.o)
    past = [torch.zeros(0, hidden, device="cuda", dtype=torch.float64) for _ in range(3)]
    for fresh in ([30, 1, 7], [1, 1, 1], [1, 40, 1], [3, 0, 1]):
        x = torch.randn(sum(fresh), hidden, device="cuda").half()
        y = block(x, server, server.plan(torch.tensor(fresh, dtype=torch.int32, device="cuda"), len(x)))
        assert q4().check() == q4().OK
        for b, part in enumerate(x.split(fresh)):
            past[b] = torch.cat([past[b], part.double()])
        for b, part in enumerate(y.split(fresh)):
            if not fresh[b]:
                continue
            L = len(past[b])
            z = (past[b] @ wq.T).view(L, heads + 2 * kv, D)
            z[:, :heads + kv] = rope_reference(z[:, :heads + kv], torch.arange(L, device="cuda"), block.freq, D,
                                               False, 1.0)
            k, v = (t.permute(1, 0, 2)[None] for t in (z[:, heads:heads + kv], z[:, heads + kv:]))
            # as one block of L tokens per request
            q = z[L - fresh[b]:, :heads].float()
            o, *_ = attention_reference(q, k, v, torch.zeros(1, 1, device="cuda"), [0, fresh[b]], [L], D ** -0.5, 0)
            ref = o.reshape(fresh[b], -1) @ wo.T
            # five roundings to f16 in a row (2^-11 each), scores of order 1
            err = (part.double() - ref).norm() / ref.norm()
            assert err < 16 * 2.0 ** -11, float(err)


def test_decoding_equals_the_whole_prompt():
    from attention_block import AttentionBlock, Server
    heads, kv, D, hidden, L = 8, 1, 128, 512, 150
    x = torch.randn(L, hidden, device="cuda").half()
    ys = []
    for chunks in ([L], [1] * 20 + [100] + [1] * 30, [64, 64, 22]):
        server = Server(1, 12, 16, 12)
        block = AttentionBlock(hidden, heads, kv, D, max(chunks), 12, dtype=torch.float16)
        ys.append(torch.cat([block(p, server, server.plan(torch.tensor([len(p)], dtype=torch.int32, device="cuda"),
                                                          len(p))) for p in x.split(chunks)]))
        assert server.length.item() == L and server.free_count.item() == 12 - 10
    assert q4().check() == q4().OK
    for y in ys[1:]:
        assert (y.double() - ys[0].double()).norm() / ys[0].double().norm() < 16 * 2.0 ** -11


def test_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "attention_block.py"), "--steps", "3"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "lengths [703, 36, 4, 259]" in r.stdout


@pytest.mark.parametrize("many", [False, True])
def test_attention_right_behind_its_plan(many):
    """Nothing between the plan and the attention that reads its lengths and
    table; the lengths change from step to step, in a graph."""
    m = q4()
    B, heads, kv, D, S, W = 40, 8, 2, 64, 16, 8
    n = 9 if many else 2
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(31)
    k, v = (torch.randn((B * W, kv, S, D), generator=g, device="cuda").half() for _ in range(2))
    cache, ws = m.KVCache(k, v), m.attention_workspace(n, heads, kv, D)
    cached, fresh = torch.zeros(B, **i32), torch.zeros(B, **i32)
    table, count = torch.full((B, W), -1, **i32), torch.full((1,), B * W, **i32)
    free = torch.randperm(B * W, generator=g, device="cuda").int()
    T = B * n
    q = torch.randn((T, heads, D), generator=g, device="cuda").half()
    plan, o = m.CachePlan.empty(B, T), torch.empty_like(q)

    def step():
        m.cache_plan(cached, fresh, table, free, count, S, T, out=plan)
        m.attention(q, cache, table, plan.q_start, plan.kv_len, n, out=o, ws=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(12):
        cached.copy_(torch.randint(0, W * S - n, (B,), generator=g, device="cuda"))
        fresh.copy_(torch.randint(0, n + 1, (B,), generator=g, device="cuda"))
        # the blocks that the requests hold, and the pool of the others
        held = ((cached + S - 1) // S).tolist()
        pool, at = torch.randperm(B * W, generator=g, device="cuda").int(), 0
        table.fill_(-1)
        for b, h in enumerate(held):
            table[b, :h] = pool[at:at + h]
            at += h
        free[:B * W - at] = pool[at:]
        count.fill_(B * W - at)
        torch.cuda.synchronize()
        graph.replay()
        assert m.check() == m.OK
        start, total = plan.q_start.tolist(), plan.kv_len.tolist()
        assert total == (cached + fresh).tolist()
        ref = attention_reference(q, k, v, table, start, total, D ** -0.5, 0)
        used = start[-1]
        assert_attention(o[:used], None, [t[:used] for t in ref], f"step {i}")


def test_a_refused_request_keeps_its_history():
    """Two blocks for two requests: the step in which the first needs another
    one refuses it, and when a block comes back it goes on from its length."""
    from attention_block import AttentionBlock, Server
    heads, kv, D, hidden = 4, 2, 64, 256
    i32 = dict(dtype=torch.int32, device="cuda")

    def fresh(*n):
        return torch.tensor(n, **i32)

    x = torch.randn(64, hidden, device="cuda").half()
    ys = {}
    for short in (False, True):
        server = Server(2, 2 if short else 4, 16, 4)
        block = AttentionBlock(hidden, heads, kv, D, 16, 4, dtype=torch.float16)
        block(x[:26], server, server.plan(fresh(16, 10), 26))
        assert server.length.tolist() == [16, 10] and server.refused.item() == 0
        y1 = block(x[26:28], server, server.plan(fresh(1, 1), 2))
        if short:
            assert server.length.tolist() == [16, 11] and server.refused.item() == 1
            assert (y1[0] == 0).all()
            server.free_blocks[0], server.free_count[0] = 3, 1  # a block comes back
            y1[:1] = block(x[26:27], server, server.plan(fresh(1, 0), 1))
        assert server.length.tolist() == [17, 11]
        y2 = block(x[28:30], server, server.plan(fresh(1, 1), 2))
        assert server.length.tolist() == [18, 12] and server.refused.item() == 0
        assert q4().check() == q4().OK
        ys[short] = torch.cat([y1, y2])
    # one row at a time or two: the products may round differently, twice, to f16
    assert (ys[True].double() - ys[False].double()).norm() <= 4 * 2.0 ** -11 * ys[False].double().norm()


# ------------------------------------------------------------------ guards
@pytest.mark.parametrize("lengths", [[(700, 1), (40, 1), (0, 1)], [(700, 60), (40, 133), (0, 1)]], ids=["few", "many"])
@pytest.mark.parametrize("D", [64, 80, 128])
def test_attention_stays_inside(lengths, D):
    m = q4()
    r = Requests(lengths, 6, 2, D, 16, torch.bfloat16, seed=D)
    cache = m.KVCache(r.k, r.v)
    ins = [t.clone() for t in (r.q, r.table, r.q_start, r.kv_len)]
    nws = m.attention_workspace_bytes(r.max_fresh, 6, 2, D)
    ws = Guarded(nws, fill=0)
    for dt in (torch.bfloat16, torch.float32):
        o, lse = Guarded(r.q.numel() * dt.itemsize), Guarded(r.T * 6 * 4)
        m.attention(r.q, cache, r.table, r.q_start, r.kv_len, r.max_fresh, out=o.view(dt, r.q.shape),
                    lse=lse.view(torch.float32, (r.T, 6)), ws=ws.view())
        assert m.check() == m.OK
        for g, n in ((o, "o"), (lse, "lse"), (ws, "workspace")):
            g.assert_guards(n)
        assert torch.isfinite(o.view(dt).float()).all()
    for a, b in zip(ins, (r.q, r.table, r.q_start, r.kv_len)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 37, 900])
def test_rope_stays_inside(T):
    m = q4()
    H, KV, D, S = 3, 2, 80, 16
    blocks = -(-T // S)
    nb = blocks * KV * S * D * 2
    k, v, q = Guarded(nb), Guarded(nb), Guarded(T * H * D * 2)
    shape = (blocks, KV, S, D)
    cache = m.KVCache(k.view(torch.float16, shape), v.view(torch.float16, shape))
    qkv = torch.randn(T, (H + 2 * KV) * D, device="cuda").half()
    freq, _ = m.rope_frequencies(D)
    slot = torch.arange(blocks * S - 1, blocks * S - 1 - T, -1, device="cuda")
    for inter in (False, True):
        m.rope_append(qkv, cache, torch.arange(T, dtype=torch.int32, device="cuda"), slot, freq, H,
                      interleaved=inter, out=q.view(torch.float16, (T, H, D)))
        assert m.check() == m.OK
        for g, n in ((k, "k"), (v, "v"), (q, "q")):
            g.assert_guards(n)


@pytest.mark.parametrize("B", [1, 50, 1000])
def test_plan_stays_inside(B):
    m = q4()
    i32 = dict(dtype=torch.int32, device="cuda")
    W, S = 5, 16
    cached = (torch.arange(B, **i32) * 7) % 60
    fresh = (torch.arange(B, **i32) * 5) % 40
    T = max(1, int(fresh.sum()) - 3)
    table = Guarded(B * W * 4)
    out = [Guarded(n) for n in (4 * (B + 1), 4 * B, 4 * T, 8 * T, 16)]
    p = m.CachePlan(*(g.view(d) for g, d in zip(out, (torch.int32, torch.int32, torch.int32, torch.int64, torch.int32))))
    free = torch.arange(B * 3, **i32)
    m.cache_plan(cached, fresh, table.view(torch.int32, (B, W)), free, torch.full((1,), B * 2, **i32), S, T, out=p)
    assert m.check() == m.OK
    for i, g in enumerate([table, *out]):
        g.assert_guards(str(i))


@pytest.mark.skipif(UNDER_DEBUG, reason="this is the outer run")
def test_suites_with_the_bounds_checked_library():
    env = dict(os.environ, Q4_LIBRARY=DEBUG_LIB)
    files = [os.path.join("tests", f) for f in ("test_gpu_serving.py", "test_gpu_cache.py", "test_gpu_attention.py")]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", *files],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-1000:]


@pytest.mark.parametrize("pad", [0, 8, 72])
@pytest.mark.parametrize("heads,kv", [(3, 3), (8, 2), (16, 2), (32, 1), (40, 1)])
@pytest.mark.parametrize("D", [64, 80, 128])
def test_attention_stores_end_at_the_rows(heads, kv, D, pad):
    """Groups of 1, 4, 8, 32 and 40 query heads, requests of rows on both sides
    of multiples of 32 and 128, outputs inside wider rows: whole rows of the
    first four leave by tensor copies of 32.  Padding between the rows, rows of
    no request and the bytes around the buffer stay as they were."""
    m = q4()
    g = heads // kv
    news = [max(1, x // g) for x in (31, 32, 33, 64, 127, 128, 129, 256, 257)] + [1, 2, 40]
    r = Requests([(i * 29 % 90, n) for i, n in enumerate(news)], heads, kv, D, 16, torch.float16, seed=D + heads)
    T, row, tail = r.T, heads * D, 5
    q = torch.cat([r.q, torch.randn_like(r.q[:1]).expand(tail, -1, -1)])
    o = Guarded((T + tail) * (row + pad) * 2)
    wide = o.view(torch.float16, (T + tail, row + pad))
    before = wide.view(torch.int16).clone()
    lse = Guarded((T + tail) * heads * 4)
    m.attention(q, m.KVCache(r.k, r.v), r.table, r.q_start, r.kv_len, r.max_fresh,
                out=wide[:, :row].unflatten(1, (heads, D)), lse=lse.view(torch.float32, (T + tail, heads)))
    assert m.check() == m.OK
    o.assert_guards("o")
    lse.assert_guards("lse")
    after = wide.view(torch.int16)
    assert torch.equal(after[:, row:], before[:, row:]) and torch.equal(after[T:], before[T:])
    assert_attention(wide[:T, :row].unflatten(1, (heads, D)), None, r.reference(), f"{heads}/{kv} {D}")


@pytest.mark.parametrize("lengths", [[(20000, 1)], [(20000, 2)], [(12000, 7)], [(9000, 13), (9000, 40)]], ids=str)
def test_the_workspace_counters_return_to_zero(lengths):
    """All of them: those of every level of the streaming kernel's tree too."""
    m = q4()
    for kv in (1, 2):
        r = Requests(lengths, 8, kv, 64, 32, torch.bfloat16, seed=25)
        ws = m.attention_workspace(r.max_fresh, 8, kv, 64)
        for _ in range(2):
            m.attention(r.q, m.KVCache(r.k, r.v), r.table, r.q_start, r.kv_len, r.max_fresh, ws=ws)
            assert m.check() == m.OK
            assert not ws[:131072].any()
        assert ws[131072:].any()  # the items were split
