"""q4_rope_append8 and q4_cache_read8 against the definition in 64 bits: types,
layouts, head sizes, runs from one token to several blocks, blocks begun and
continued, scales that grow, values of no finite magnitude, skipped slots,
strides, streams and graphs.  Tolerances: cache8_ref.py."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from cache8_ref import CODES, MOST, RANGE, Requests8, check_append, exponents, numbers, random_cache, raw, rope_reference, runs, values

pytestmark = pytest.mark.gpu
DT = [torch.bfloat16, torch.float16]
REL = 2.0 ** -19


def q4():
    import weight_only_int4_group_gb300 as m
    return m


def slots_of(lengths, S, blocks, seed=0):
    """Slots and positions of requests' new tokens over shuffled blocks."""
    pool = np.random.default_rng(seed).permutation(blocks).tolist()
    slot, pos = [], []
    for c, n in lengths:
        first = c // S
        ids = [pool.pop() for _ in range(-(-(c + n) // S) - first)]
        slot += [ids[p // S - first] * S + p % S for p in range(c, c + n)]
        pos += range(c, c + n)
    return torch.tensor(slot, dtype=torch.int64, device="cuda"), torch.tensor(pos, dtype=torch.int32, device="cuda")


def clones(cache):
    return [(cache.k.clone(), cache.k_exp.clone()), (cache.v.clone(), cache.v_exp.clone())]


def append(lengths, heads, kv, D, S, dtype, code, rot=None, inter=False, factor=1.0, seed=0, token_major=False,
           edit=None, scale=1.0, exps=(-7, -3)):
    m = q4()
    g = torch.Generator().manual_seed(seed)
    rot = D if rot is None else rot
    blocks = sum(-(-(c + n) // S) - c // S for c, n in lengths) + 2
    slot, pos = slots_of(lengths, S, blocks, seed)
    cache = m.KVCache8(*random_cache(blocks, kv, S, D, code, g, token_major=token_major, exps=exps), dtype)
    T = len(slot)
    qkv = (torch.randn(T, (heads + 2 * kv) * D, generator=g) * scale).to(dtype).cuda()
    if edit:
        edit(qkv.view(T, heads + 2 * kv, D), slot)
    freq = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).cuda()
    before = clones(cache)
    q = m.rope_append(qkv, cache, pos, slot, freq, heads, interleaved=inter, factor=factor)
    assert m.check() == m.OK
    after = clones(cache)
    x = rope_reference(qkv.view(T, heads + 2 * kv, D)[:, :heads + kv], pos, freq, rot, inter, factor)
    u = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[dtype]
    want = x[:, :heads]
    if torch.isfinite(want).all():
        # r bounds the rotation's error, 2^-20 (|x| + |p|) factor with both at most the
        # head's largest; then one rounding of what is computed, by u of it or, in
        # binary16's subnormals, 2^-25
        r = abs(factor) * 2.0 ** -19 * qkv.view(T, -1, D)[:, :heads].double().abs().amax(-1, keepdim=True)
        assert ((q.double() - want).abs() <= r + u * (want.abs() + r) + 2.0 ** -24).all(), "queries"
    check_append(before[0], after[0], x[:, heads:], slot, dtype, REL if rot else 0)
    check_append(before[1], after[1], qkv.view(T, -1, D)[:, heads + kv:].double(), slot, dtype, 0)
    return cache, slot, before, after


LENGTHS = [
    [(0, 1)], [(15, 1)], [(16, 1)], [(0, 16)], [(0, 17)], [(5, 40)],
    [(3, 2), (100, 1), (0, 1), (31, 3)],
    [(i * 37 % 500, 1) for i in range(70)],
    [(0, 130), (50, 1), (63, 66), (64, 65), (1, 200)],
]


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda x: str(x)[:24])
def test_append(lengths, dtype, code):
    append(lengths, 8, 2, 128, 16, dtype, code, seed=len(lengths))


@pytest.mark.parametrize("S", [16, 32, 48, 64, 80, 128, 256, 400])
@pytest.mark.parametrize("token_major", [False, True])
def test_block_sizes_and_layouts(S, token_major):
    for code in CODES:
        append([(S - 1, 2), (0, 2 * S + 5), (S, 1), (7, S)], 4, 2, 64, S, torch.float16, code, seed=S, token_major=token_major)


@pytest.mark.parametrize("D,rot", [(16, 16), (32, 8), (48, 20), (64, 64), (80, 40), (96, 2), (112, 112), (128, 0), (128, 64)])
@pytest.mark.parametrize("inter", [False, True])
def test_heads_and_rotations(D, rot, inter):
    for heads, kv, code in ((3, 3, CODES[0]), (40, 20, CODES[1]), (7, 1, CODES[0])):
        append([(10, 30), (100000, 1), (2 ** 30, 3)], heads, kv, D, 16, torch.bfloat16, code, rot=rot, inter=inter,
               factor=1.3, seed=D + rot)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", DT)
def test_token_by_token_growth(dtype, code):
    """A block filled one token at a time with growing magnitudes: each append
    is checked against the state before it."""
    m = q4()
    g = torch.Generator().manual_seed(1)
    S, D = 32, 64
    cache = m.KVCache8(*random_cache(2, 1, S, D, code, g), dtype)
    freq, _ = m.rope_frequencies(D)
    exact = torch.zeros(S, D, dtype=torch.float64, device="cuda")
    for o in range(S):
        x = (torch.randn(1, 3 * D, generator=g) * 1.3 ** o * 1e-2).to(dtype).cuda()
        slot, pos = torch.tensor([S + o], device="cuda"), torch.tensor([o], dtype=torch.int32, device="cuda")
        before = clones(cache)
        m.rope_append(x, cache, pos, slot, freq, 1)
        after = clones(cache)
        check_append(before[1], after[1], x.view(1, 3, D)[:, 2:].double(), slot, dtype, 0)
        check_append(before[0], after[0], rope_reference(x.view(1, 3, D)[:, 1:2], pos, freq, D, False, 1.0), slot, dtype, REL)
        exact[o] = x.view(3, D)[2].double()
    # all roundings of a value together: under one step of the last scale (int8)
    if code == torch.int8:
        err = (values(cache.v, cache.v_exp, dtype)[1, 0] - exact).abs()
        assert float(err.max()) <= 2.0 ** (int(cache.v_exp[1, 0]) - 127)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", DT)
def test_border_and_special_values(dtype, code):
    """Peaks on the codes' end and one step beside it, zeros, values too small
    and too large for the range, infinities and NaN."""
    top = MOST[code]
    lo, hi = RANGE[code, dtype]
    info = torch.finfo(dtype)

    def edit(x, slot):
        v = x[:, -1]  # the one value head
        v.clamp_(-1, 1)
        v[0, 3] = top / 64
        v[1, 3] = top / 64 * (1 + info.eps)
        v[2, 3] = -top / 64 * (1 - info.eps)
        v[3] = 0
        v[4] = info.tiny
        v[5, 7], v[5, 8] = info.max, -info.max
        v[6, 5], v[6, 6], v[6, 7] = math.inf, -math.inf, math.nan
        v[7] = math.nan
        v[8] = -math.inf
        v[9] = torch.arange(x.shape[2], device="cuda") + 0.5  # ties
        v[9, 0] = top

    cache, slot, _, after = append([(0, 1)] * 12, 1, 1, 64, 16, dtype, code, edit=edit)
    e = exponents(cache.v_exp[slot // 16, 0], code, dtype).tolist()
    assert e[0] == -6 and e[1] == -5 and e[2] == -6 and e[3] == lo and e[7] == lo and e[8] == lo
    codes = numbers(cache.v)[slot // 16, 0, 0]
    assert codes[6, 5] == top and codes[6, 6] == -top and codes[6, 7] == 0 and (codes[7] == 0).all() and (codes[8] == -top).all()
    got = values(cache.v, cache.v_exp, dtype)
    fin = got[slot // 16, 0, 0]
    assert torch.equal(fin.to(dtype).double(), fin), "values are numbers of the 16-bit type"


@pytest.mark.parametrize("code", CODES)
def test_skipped_slots_and_padding(code):
    """Rows without a slot, alone and between others, leave the cache alone; their
    queries are rotated all the same."""
    m = q4()
    g = torch.Generator().manual_seed(3)
    S, D, blocks = 16, 64, 6
    cache = m.KVCache8(*random_cache(blocks, 2, S, D, code, g), torch.float16)
    slot = torch.tensor([-1, 0, 1, -1, 35, -7, blocks * S, blocks * S + 1, 2 ** 40, 48, 49, 50, -1, -1], device="cuda")
    T = len(slot)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    qkv = torch.randn(T, (4 + 4) * D, generator=g).half().cuda()
    freq, _ = m.rope_frequencies(D)
    before = clones(cache)
    q = m.rope_append(qkv, cache, pos, slot, freq, 4)
    after = clones(cache)
    x = rope_reference(qkv.view(T, 8, D)[:, :6], pos, freq, D, False, 1.0)
    assert float((q.double() - x[:, :4]).abs().max()) < 1e-2
    check_append(before[0], after[0], x[:, 4:], slot, torch.float16, REL)
    check_append(before[1], after[1], qkv.view(T, 8, D)[:, 6:].double(), slot, torch.float16, 0)
    assert runs(slot, S, blocks * S) == [(1, 2), (4, 1), (9, 3)]


@pytest.mark.parametrize("inter", [False, True])
def test_in_place_queries(inter):
    """q_out may be qkv itself."""
    m = q4()
    g = torch.Generator().manual_seed(4)
    for D, T, heads in ((128, 300, 64), (64, 5, 3), (80, 33, 9)):
        slot, pos = slots_of([(0, T)], 32, -(-T // 32))
        freq, _ = m.rope_frequencies(D)
        qkv = torch.randn(T, (heads + 2) * D, generator=g).bfloat16().cuda()
        caches = [m.KVCache8(*(t.clone() for t in random_cache(-(-T // 32), 1, 32, D, torch.int8, torch.Generator().manual_seed(5))))
                  for _ in range(2)]
        want = m.rope_append(qkv, caches[0], pos, slot, freq, heads, interleaved=inter)
        rows = qkv[:, :heads * D]
        m.rope_append(qkv, caches[1], pos, slot, freq, heads, interleaved=inter, out=rows)
        assert torch.equal(rows.reshape(T, heads, D), want)
        assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)


@pytest.mark.parametrize("D,rot", [(80, 40), (96, 2), (128, 120), (64, 0)])
def test_in_place_queries_whose_pairs_lie_apart(D, rot):
    """The same where a pair's elements belong to different threads' pieces."""
    m = q4()
    g = torch.Generator().manual_seed(8)
    T, heads = 70, 20
    slot, pos = slots_of([(0, T)], 16, -(-T // 16))
    freq = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).cuda()
    qkv = torch.randn(T, (heads + 2) * D, generator=g).half().cuda()
    caches = [m.KVCache8.empty(-(-T // 16), 1, 16, D, dtype=torch.float16) for _ in range(2)]
    want = m.rope_append(qkv, caches[0], pos, slot, freq, heads)
    rows = qkv[:, :heads * D]
    m.rope_append(qkv, caches[1], pos, slot, freq, heads, out=rows)
    assert torch.equal(rows.reshape(T, heads, D), want)
    for n in ("k_exp", "v_exp"):
        assert torch.equal(getattr(caches[0], n), getattr(caches[1], n))
    live = slot.cpu()
    for x, y in ((caches[0].k, caches[1].k), (caches[0].v, caches[1].v)):
        assert torch.equal(x.transpose(1, 2).reshape(-1, D).cpu()[live], y.transpose(1, 2).reshape(-1, D).cpu()[live])


def test_many_heads():
    """More heads than one CTA's share of each kind, several times over."""
    append([(5, 2)], 20000, 600, 16, 16, torch.bfloat16, torch.int8, seed=9)
    append([(0, 1), (17, 1)], 3, 300, 128, 16, torch.float16, torch.float8_e4m3fn, seed=10)


def test_queries_agree_with_the_16_bit_append():
    m = q4()
    g = torch.Generator().manual_seed(6)
    T, D, S = 100, 128, 16
    slot, _ = slots_of([(0, T)], S, 7)
    pos = torch.randint(0, 2 ** 31 - 1, (T,), generator=g, dtype=torch.int32).cuda()
    qkv = torch.randn(T, 10 * D, generator=g).half().cuda()
    freq, factor = m.rope_frequencies(D, stretch=8.0, by_parts=True)
    a = m.rope_append(qkv, m.KVCache.empty(7, 1, S, D, torch.float16), pos, slot, freq, 8, factor=factor)
    b = m.rope_append(qkv, m.KVCache8.empty(7, 1, S, D, dtype=torch.float16), pos, slot, freq, 8, factor=factor)
    # each within 2^-20 of the pair's size and its own rounding
    assert float((a.double() - b.double()).abs().max()) <= 2 ** -10 * float(qkv.abs().max())
    assert float((a != b).float().mean()) < 0.01


def test_empty_append():
    m = q4()
    cache = m.KVCache8.empty(2, 1, 16, 64)
    freq, _ = m.rope_frequencies(64)
    with pytest.raises(ValueError):
        m.rope_append(torch.empty(0, 3 * 64, dtype=torch.bfloat16, device="cuda"), cache,
                      torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), freq, 1)


# ------------------------------------------------------------------ reading back
def check_read(r, back, dtype, out_dtype=None, **kw):
    """back: rows per request (its last tokens)."""
    m = q4()
    start = np.concatenate([[0], np.cumsum(back)])
    qs = torch.tensor(start, dtype=torch.int32, device="cuda")
    got = m.cache_read(r.cache(), r.table, qs, r.kv_len, int(start[-1]), out_dtype=out_dtype, **kw)
    assert m.check() == m.OK
    S = r.k.shape[2]
    for g, full in zip(got, r.values()):
        assert g.dtype == (out_dtype or dtype)
        for b, n in enumerate(back):
            rows = g[start[b]:start[b + 1]].double()
            for i, p in enumerate(range(r.total[b] - n, r.total[b])):
                want = full[int(r.table[b, p // S]), :, p % S] if p >= 0 else torch.zeros_like(rows[i])
                assert torch.equal(rows[i], want), (b, p)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", DT)
def test_read(dtype, code):
    for S, D, kv, major in ((16, 128, 2, False), (48, 80, 3, True), (32, 16, 1, False), (64, 64, 4, True)):
        r = Requests8([(0, 1), (37, 0), (0, 0), (15, 2), (64, 60), (1, 0)], kv, kv, D, S, dtype, code, seed=S, token_major=major,
                      exps=RANGE[code, dtype])
        check_read(r, r.total, dtype)
        check_read(r, [0, 1, 0, 2, 100, 1], dtype)
        check_read(r, [0, 0, 0, 0, 1, 0], dtype, torch.float32)
        check_read(r, [4, 0, 3, 17, 0, 2], dtype)  # rows before the first token


def test_read_many_requests():
    """More requests than a look, empty ones among them."""
    r = Requests8([(i * 7 % 40, 0) for i in range(200)], 1, 1, 64, 16, torch.float16, torch.int8, seed=9)
    check_read(r, r.total, torch.float16)
    r = Requests8([(1 if i % 50 == 49 else 0, 0) for i in range(3000)], 1, 1, 16, 16, torch.float16, torch.int8, seed=9)
    check_read(r, r.total, torch.float16)


def test_read_leaves_other_rows():
    """Rows before the first request's and behind the last's; strided outputs."""
    m = q4()
    r = Requests8([(20, 0), (5, 0)], 2, 2, 64, 16, torch.float16, torch.int8)
    qs = torch.tensor([3, 23, 28], dtype=torch.int32, device="cuda")
    big = [torch.full((40, 200), 7.0, dtype=torch.float16, device="cuda") for _ in "kv"]
    out = tuple(b[:, 8:136] for b in big)
    m.cache_read(r.cache(), r.table, qs, r.kv_len, 40, out=out)
    want = m.cache_read(r.cache(), r.table, qs - 3, r.kv_len, 25)
    for b, o, w in zip(big, out, want):
        assert torch.equal(o[3:28], w.flatten(1))
        keep = torch.ones_like(b, dtype=torch.bool)
        keep[3:28, 8:136] = False
        assert (b[keep] == 7).all()


def test_read_bad_tables_and_lengths():
    """Blocks outside the cache give zeros; lengths are cut to the table and rows
    to T, whatever the device arrays hold."""
    m = q4()
    r = Requests8([(40, 0), (40, 0)], 1, 1, 64, 16, torch.float16, torch.int8, width_extra=0)
    full = r.values()[0]
    r.table[0, 1] = -1
    r.table[1, 2] = 10 ** 9
    qs = torch.tensor([0, 40, 80], dtype=torch.int32, device="cuda")
    k, _ = m.cache_read(r.cache(), r.table, qs, r.kv_len, 80)
    assert (k[16:32] == 0).all() and (k[72:80] == 0).all() and torch.equal(k[:16].double(), full[int(r.table[0, 0])].transpose(0, 1))
    for lens, starts in (([10 ** 9, -5], [0, 40, 80]), ([2 ** 31 - 1] * 2, [0, 10 ** 9, 2 ** 31 - 1]),
                         ([40, 40], [-9, 90, 5]), ([40, 40], [80, 40, 0]), ([0, 0], [0, 40, 80])):
        out = tuple(torch.full((80, 64), 3.0, dtype=torch.float16, device="cuda") for _ in "kv")
        m.cache_read(r.cache(), r.table, torch.tensor(starts, dtype=torch.int32, device="cuda"),
                     torch.tensor(lens, dtype=torch.int32, device="cuda"), 80, out=out)
        assert m.check() == m.OK
        if lens == [0, 0]:
            assert (out[0] == 0).all() and (out[1] == 0).all()


@pytest.mark.parametrize("code", CODES)
def test_streams_and_graphs(code):
    """Append and read-back on a side stream and replayed from a graph give the
    eager bits; the second replay finds the scales of the first."""
    m = q4()
    D, S, T = 128, 16, 45
    slot, pos = slots_of([(3, T)], S, 4)
    freq, _ = m.rope_frequencies(D)
    qkv = torch.randn(T, 6 * D, generator=torch.Generator().manual_seed(0)).half().cuda()
    table = torch.tensor([[int(slot[0]) // S, *(int(s) // S for s in slot[13::16])]], dtype=torch.int32, device="cuda")
    qs = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    n = torch.tensor([T + 3], dtype=torch.int32, device="cuda")

    def fresh():
        return m.KVCache8(*random_cache(4, 2, S, D, code, torch.Generator().manual_seed(1)), torch.float16)

    def step(cache, **kw):
        q = m.rope_append(qkv, cache, pos, slot, freq, 2, **kw)
        return (q, *m.cache_read(cache, table, qs, n, T, **kw))

    eager = fresh()
    want = step(eager)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    c2 = fresh()
    torch.cuda.synchronize()
    got = step(c2, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    c3 = fresh()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(c3)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert torch.equal(raw(c3.k), raw(eager.k)) and torch.equal(c3.v_exp, eager.v_exp)


def test_repeated_append_is_the_same():
    """The same tokens again change nothing more."""
    cache, *_ = append([(5, 20)], 2, 1, 64, 16, torch.float16, torch.int8, seed=8)
    m = q4()
    one = clones(cache)
    g = torch.Generator().manual_seed(8)
    slot, pos = slots_of([(5, 20)], 16, 4, 8)
    random_cache(4, 1, 16, 64, torch.int8, g)
    qkv = torch.randn(20, 4 * 64, generator=g).half().cuda()
    freq = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).cuda()
    m.rope_append(qkv, cache, pos, slot, freq, 2)
    two = clones(cache)
    for (a, b), (c, d) in zip(one, two):
        assert torch.equal(raw(a), raw(c)) and torch.equal(b, d)


@pytest.mark.parametrize("far", ["blocks", "heads", "tokens"])
def test_offsets_past_32_bits(far):
    """A cache whose codes lie more than 2^32 apart gives what a dense one gives:
    append, reading back, attention with few and with many rows."""
    m = q4()
    blocks, heads, S, D = 6, 2, 16, 64
    shape = (blocks, heads, S, D)
    dense = [1024 * heads, 1024, D]
    stride = list(dense)
    i = ("blocks", "heads", "tokens").index(far)
    n = shape[i]
    stride[i] = -(-(2 ** 32 + 2 ** 20) // (n - 1) // 16) * 16
    if far == "heads":
        stride[0] = 1024
    if far == "tokens":
        stride[0], stride[1] = heads * D, D
    size = sum((a - 1) * b for a, b in zip(shape, stride)) + D
    assert size > 2 ** 32
    big = []
    for _ in "kv":
        big.append(torch.zeros(size, dtype=torch.int8, device="cuda").as_strided(shape, stride + [1]))
    exps = [torch.zeros(blocks, heads, dtype=torch.uint8, device="cuda") for _ in range(4)]
    wide = m.KVCache8(*big, *exps[:2])
    near = m.KVCache8(*(torch.zeros(shape, dtype=torch.int8, device="cuda") for _ in "kv"), *exps[2:])
    g = torch.Generator().manual_seed(12)
    T = blocks * S - 3
    table = torch.tensor([[4, 1, 5, 0, 3, 2]], dtype=torch.int32, device="cuda")
    place = torch.arange(T, device="cuda")
    slot = table[0].long()[place // S] * S + place % S
    freq, _ = m.rope_frequencies(D)
    qkv = torch.randn(T, (6 + 2 * heads) * D, generator=g).bfloat16().cuda()
    q = [m.rope_append(qkv, c, place.int(), slot, freq, 6) for c in (wide, near)]
    assert torch.equal(*q)
    assert torch.equal(wide.k, near.k) and torch.equal(wide.v, near.v)
    assert torch.equal(exps[0], exps[2]) and torch.equal(exps[1], exps[3])
    kv = torch.tensor([T], dtype=torch.int32, device="cuda")
    for rows in (1, 4, T):
        start = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        a, b = (m.cache_read(c, table, start, kv, rows) for c in (wide, near))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        a, b = (m.attention(q[0][T - rows:], c, table, start, kv, rows) for c in (wide, near))
        assert torch.equal(a, b) and a.isfinite().all()
    assert m.check() == m.OK
