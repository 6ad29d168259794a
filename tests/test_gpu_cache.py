"""q4_cache_plan against a plan in Python integers, and q4_rope_append against
the rotation in 64 bits (one rounding of the output type, plus the f32 sine,
cosine and products: 2^-20 of the pair's magnitude)."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from serving_ref import U, plan_reference, rope_reference

pytestmark = pytest.mark.gpu


def q4():
    import weight_only_int4_group_gb300 as m
    return m


# ------------------------------------------------------------------- plan
def plan_case(cached, fresh, S, W, free, spare=4, T=None, seed=0, holes=False):
    rng = np.random.default_rng(seed)
    B = len(cached)
    T = T or max(1, sum(max(0, f) for f in fresh))
    table = np.full((B, W), -9)
    nxt = 1000
    for b in range(B):
        for j in range(min(W, -(-max(0, cached[b]) // S))):
            table[b, j] = -1 if holes and rng.random() < 0.3 else nxt
            nxt += 1
    stack = rng.permutation(500000)[:max(1, free + spare)] + 10
    return dict(cached=cached, fresh=fresh, table=table, free_blocks=stack, free_count=free, S=S, T=T)


def check_plan(c):
    m = q4()
    ref = plan_reference(**c)

    def dev(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")

    table, free = dev(c["table"]), dev(c["free_blocks"])
    cached, fresh, count = dev(c["cached"]), dev(c["fresh"]), dev([c["free_count"]])
    for _ in range(2):  # a repeated call gives the same
        p = m.cache_plan(cached, fresh, table, free, count, c["S"], c["T"])
        assert m.check() == m.OK
        assert table.tolist() == ref["table"].tolist()
        for k in ("q_start", "kv_len", "counts", "position", "slot"):
            assert getattr(p, k).tolist() == list(ref[k]), k
    assert count.item() == c["free_count"] and free.tolist() == c["free_blocks"].tolist()


@pytest.mark.parametrize("S", [1, 16, 48, 64])
@pytest.mark.parametrize("B", [1, 2, 33, 600, 1500])
def test_plan(B, S):
    rng = np.random.default_rng(B * 100 + S)
    cached = rng.integers(0, 5 * S + 40, B).tolist()
    fresh = rng.integers(0, 2 * S + 3, B).tolist()
    W = (7 * S + 43) // S + 2
    need = sum(-(-(c + f) // S) - -(-c // S) for c, f in zip(cached, fresh))
    for free in (need, need + 5, need // 2, 0):
        for extra in (0, 1, 700):
            check_plan(plan_case(cached, fresh, S, W, free, T=max(1, sum(fresh)) + extra, seed=B, holes=free == need + 5))


@pytest.mark.parametrize("cached,fresh", [
    ([0], [1]), ([0], [0]), ([16], [0]), ([15], [1]), ([16], [1]), ([17], [500]),
    ([-1, 5], [3, 2]), ([5, 5], [-4, 2]), ([3, 100000, 4], [1, 1, 1]),
    ([2 ** 31 - 1, 0], [2 ** 31 - 1, 1]), ([0, 0, 0], [0, 0, 7]),
])
def test_plan_edges(cached, fresh):
    for T in (1, 5, 600):
        for free in (0, 1, 40):
            check_plan(plan_case([min(c, 2 ** 31 - 1) for c in cached], fresh, 16, 40, free, T=T))


def test_plan_keeps_serving_requests_that_need_no_block():
    check_plan(plan_case([5, 16, 3, 32, 4], [1, 20, 2, 1, 1], 16, 8, 1))


def test_plan_free_count_is_cut_to_the_stack():
    c = plan_case([0, 0], [40, 40], 16, 8, 3, spare=0)
    c["free_count"] = 1000
    check_plan(c)
    c["free_count"] = -3
    check_plan(c)


def test_plan_of_the_most_requests():
    B = 16384
    check_plan(plan_case([i % 50 for i in range(B)], [1] * B, 16, 4, B, seed=1))


def test_plan_in_a_graph_follows_its_inputs():
    m = q4()
    table = torch.full((3, 6), -1, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    cached, fresh = torch.zeros(3, **i32), torch.ones(3, **i32)
    free, count = torch.arange(20, **i32), torch.full((1,), 20, **i32)
    out = m.CachePlan.empty(3, 8)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.cache_plan(cached, fresh, table, free, count, 16, 8, out=out)
    ref_table = np.full((3, 6), -1)
    c, n = np.zeros(3, int), 20
    for step in range(20):
        f = np.array([1, step % 3, 2])
        fresh.copy_(torch.tensor(f))
        g.replay()
        ref = plan_reference(c, f, ref_table, np.arange(20), n, 16, 8)
        assert out.slot.tolist() == list(ref["slot"]) and table.tolist() == ref["table"].tolist()
        assert out.counts.tolist() == ref["counts"]
        ref_table, n, c = ref["table"], ref["counts"][2], c + f
        cached.copy_(out.kv_len)
        count.copy_(out.counts[2:3])


def test_plan_arrays_between_the_tables_rows():
    """The room between a wide table's rows is nobody's: arrays may lie there."""
    m = q4()
    c = plan_case([5, 16, 30], [20, 1, 9], 16, 4, 8)
    ref = plan_reference(**c)
    i32 = dict(dtype=torch.int32, device="cuda")
    buf = torch.full((3, 64), -3, **i32)
    table = buf[:, :4]
    table.copy_(torch.tensor(c["table"]))
    out = m.CachePlan.empty(3, c["T"])
    out.kv_len, cached = buf[0, 4:7], buf[1, 61:64]
    cached.copy_(torch.tensor(c["cached"]))
    m.cache_plan(cached, torch.tensor(c["fresh"], **i32), table, torch.tensor(c["free_blocks"], **i32),
                 torch.tensor([c["free_count"]], **i32), 16, c["T"], out=out)
    assert m.check() == m.OK
    assert table.tolist() == ref["table"].tolist() and out.slot.tolist() == list(ref["slot"])
    assert out.kv_len.tolist() == ref["kv_len"] and cached.tolist() == c["cached"]
    with pytest.raises(m.Q4Error):
        out.kv_len = buf[1, 3:6]
        m.cache_plan(cached, torch.tensor(c["fresh"], **i32), table, torch.tensor(c["free_blocks"], **i32),
                     torch.tensor([c["free_count"]], **i32), 16, c["T"], out=out)


# ------------------------------------------------------------------- rope
def rope_case(T, heads, kv, D, rot, S, dtype, inter, seed=0, reach=5000, token_major=False, in_place=False,
              skip=False, factor=1.0, freq=None):
    m = q4()
    g = torch.Generator().manual_seed(seed)
    W = (heads + 2 * kv) * D
    pad = 16
    wide = torch.randn(T, W + pad, generator=g).to(dtype).cuda()
    qkv = wide[:, :W]
    before = qkv.clone()
    blocks = -(-T // S) + 2
    shape = (blocks, S, kv, D) if token_major else (blocks, kv, S, D)
    mk = [torch.randn(shape, generator=g).to(dtype).cuda() for _ in range(2)]
    k, v = (t.transpose(1, 2) if token_major else t for t in mk)
    k0, v0 = k.clone(), v.clone()
    pos = torch.randint(0, reach, (T,), generator=g, dtype=torch.int32)
    slot = torch.randperm(blocks * S, generator=g)[:T]
    if skip:
        slot[::3] = torch.tensor([-1, blocks * S, -2 ** 62, 2 ** 62])[torch.arange(len(slot[::3])) % 4]
    if freq is None:
        freq, _ = m.rope_frequencies(rot)
    pos, slot = pos.cuda(), slot.cuda()
    out = qkv[:, :heads * D].unflatten(1, (heads, D)) if in_place else None
    q = m.rope_append(qkv, m.KVCache(k, v), pos, slot, freq, heads, interleaved=inter, factor=factor, out=out)
    assert m.check() == m.OK
    x = before.reshape(T, heads + 2 * kv, D)
    ref = rope_reference(x[:, :heads + kv], pos, freq, rot, inter, factor)
    size = torch.zeros_like(ref)
    if rot:
        a = x[:, :heads + kv, :rot].double()
        pairs = (a[..., 0::2], a[..., 1::2]) if inter else a.split(rot // 2, -1)
        mag = torch.hypot(*pairs) * abs(factor)
        size[..., :rot] = mag.repeat_interleave(2, -1) if inter else torch.cat([mag, mag], -1)
    allow = U[dtype] * ref.abs() + 2.0 ** -19 * size + (2.0 ** -24) * (size > 0)
    err = (q.double() - ref[:, :heads]).abs()
    assert (err <= allow[:, :heads]).all(), float((err - allow[:, :heads]).max())
    assert torch.equal(q[..., rot:], x[:, :heads, rot:])
    # the cache: appended rows, everything else untouched
    for t in range(T):
        s = int(slot[t])
        if 0 <= s < blocks * S:
            b, o = s // S, s % S
            e = (k[b, :, o].double() - ref[t, heads:]).abs()
            assert (e <= allow[t, heads:]).all(), t
            assert torch.equal(k[b, :, o, rot:], x[t, heads:heads + kv, rot:])
            assert torch.equal(v[b, :, o], x[t, heads + kv:])
            k0[b, :, o], v0[b, :, o] = k[b, :, o], v[b, :, o]
    assert torch.equal(k, k0) and torch.equal(v, v0)
    if not in_place:
        assert torch.equal(qkv, before)
    else:
        assert torch.equal(qkv[:, heads * D:], before[:, heads * D:])


DT = [torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (128, 2), (128, 0), (64, 64), (80, 80), (80, 40), (96, 48),
                                   (96, 36), (8, 8), (16, 6), (120, 30), (72, 72)])
def test_rope(D, rot, inter, dtype):
    rope_case(9, 6, 2, D, rot, 16, dtype, inter, seed=D + rot)


@pytest.mark.parametrize("T", [1, 2, 3, 5, 31, 130, 700, 1300])
def test_rope_token_counts(T):
    rope_case(T, 4, 1, 64, 64, 16, torch.float16, False, seed=T)
    rope_case(T, 1, 1, 128, 64, 48, torch.bfloat16, True, seed=T, token_major=True)


@pytest.mark.parametrize("heads,kv", [(64, 8), (32, 32), (1, 1), (200, 1), (7, 7)])
def test_rope_heads(heads, kv):
    rope_case(6, heads, kv, 128, 128, 32, torch.bfloat16, False, seed=heads)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_in_place_and_skipped_slots(inter):
    rope_case(40, 4, 2, 64, 32, 16, torch.bfloat16, inter, in_place=True)
    rope_case(40, 4, 2, 64, 64, 16, torch.float16, inter, skip=True)


def test_rope_scaled_and_far_positions():
    m = q4()
    for stretch, parts in ((8.0, False), (32.0, True)):
        f, factor = m.rope_frequencies(128, stretch=stretch, by_parts=parts)
        rope_case(20, 4, 1, 128, 128, 16, torch.float16, False, freq=f, factor=factor, reach=131072)
    rope_case(20, 4, 1, 128, 128, 16, torch.float16, False, reach=2 ** 31 - 1)


def test_rope_frequencies():
    m = q4()
    f, factor = m.rope_frequencies(64)
    assert factor == 1.0 and f.shape == (32,) and f.dtype == torch.float64
    assert np.allclose(f.cpu().numpy(), 10000.0 ** (-np.arange(32) / 32), rtol=1e-14)
    g, factor = m.rope_frequencies(64, stretch=16.0, by_parts=True)
    ratio = (g / f).cpu().numpy()
    assert ratio[0] == 1.0 and abs(ratio[-1] - 1 / 16) < 1e-12 and (np.diff(ratio) <= 1e-12).all()
    assert abs(factor - (0.1 * math.log(16) + 1)) < 1e-12
    g, factor = m.rope_frequencies(64, stretch=4.0)
    assert factor == 1.0 and np.allclose((g / f).cpu().numpy(), 0.25)


@pytest.mark.parametrize("T", [2999, 3000, 3001, 3003])
@pytest.mark.parametrize("inter", [False, True])
def test_rope_of_many_tokens(T, inter):
    """Several tokens per CTA, with a last CTA of fewer; in place too."""
    rope_case(T, 3, 2, 64, 32, 16, torch.bfloat16, inter, seed=T)
    rope_case(T, 4, 1, 80, 80, 48, torch.float16, inter, seed=T, in_place=True, token_major=True)


@pytest.mark.parametrize("T", [2999, 3001, 3003])
def test_rope_of_many_tokens_stays_inside(T):
    from test_gpu_canaries import Guarded
    m = q4()
    H, KV, D, S = 3, 2, 80, 16
    blocks = -(-T // S)
    nb = blocks * KV * S * D * 2
    k, v, q = Guarded(nb), Guarded(nb), Guarded(T * H * D * 2)
    cache = m.KVCache(*(t.view(torch.float16, (blocks, KV, S, D)) for t in (k, v)))
    qkv = torch.randn(T, (H + 2 * KV) * D, device="cuda").half()
    freq, _ = m.rope_frequencies(D)
    slot = torch.arange(blocks * S - 1, blocks * S - 1 - T, -1, device="cuda")
    slot[5::7] = blocks * S  # one past the cache
    for inter in (False, True):
        m.rope_append(qkv, cache, torch.arange(T, dtype=torch.int32, device="cuda"), slot, freq, H,
                      interleaved=inter, out=q.view(torch.float16, (T, H, D)))
        assert m.check() == m.OK
        for g, n in ((k, "k"), (v, "v"), (q, "q")):
            g.assert_guards(n)
