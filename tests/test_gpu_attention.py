"""q4_attention against the definition in 64 bits: types, head layouts,
lengths from one token up, odd sizes, both cache layouts, windows, rows that
see nothing, stale NaN in the cache, strides, splits over CTAs, streams,
graphs and a shared workspace.  Tolerances: serving_ref.py."""
from __future__ import annotations

import math

import pytest
import torch

from serving_ref import Requests, assert_attention

pytestmark = pytest.mark.gpu


def q4():
    import weight_only_int4_group_gb300 as m
    return m


def run(r, window=0, scale=None, out_dtype=None, ws=None, max_fresh=None, **kw):
    m = q4()
    cache = m.KVCache(r.k, r.v)
    o, lse = m.attention(r.q, cache, r.table, r.q_start, r.kv_len, max_fresh or r.max_fresh, scale=scale,
                         window=window, out_dtype=out_dtype, return_lse=True, ws=ws, **kw)
    assert m.check() == m.OK
    return o, lse


def check(r, window=0, scale=None, **kw):
    o, lse = run(r, window, scale, **kw)
    assert_attention(o, lse, r.reference(scale, window), f"{r.lengths} window {window}")
    return o, lse


DT = [torch.bfloat16, torch.float16]
# (cached, fresh) of each request
FEW = [
    [(0, 1)],
    [(15, 1)], [(16, 1)], [(17, 1)],
    [(127, 1)], [(128, 1)], [(129, 1)],
    [(776, 1)],
    [(5000, 1)],
    [(3, 2), (100, 1), (0, 1), (31, 3)],
    [(0, 0), (64, 1), (0, 0), (7, 1), (300, 0)],
    [(i * 37 % 500, 1) for i in range(70)],
]
MANY = [
    [(0, 17)], [(0, 128)], [(0, 129)], [(5, 64)],
    [(0, 300)], [(777, 100)], [(1000, 257)],
    [(0, 130), (50, 1), (0, 0), (400, 65), (3, 33)],
    [(127, 1), (128, 128), (129, 2)],
]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("lengths", FEW, ids=lambda x: str(x)[:24])
@pytest.mark.parametrize("heads,kv", [(8, 1), (4, 4), (14, 2)])
def test_few_rows(lengths, heads, kv, dtype):
    check(Requests(lengths, heads, kv, 128, 16, dtype, seed=len(lengths)))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("lengths", MANY, ids=lambda x: str(x)[:24])
@pytest.mark.parametrize("heads,kv", [(8, 1), (2, 2), (14, 2)])
def test_many_rows(lengths, heads, kv, dtype):
    check(Requests(lengths, heads, kv, 128, 16, dtype, seed=len(lengths)))


@pytest.mark.parametrize("D", [8, 16, 40, 64, 72, 80, 96, 112, 120, 128])
@pytest.mark.parametrize("lengths", [[(200, 1), (33, 1)], [(200, 40), (0, 150)]], ids=["few", "many"])
def test_head_dims(D, lengths):
    for dtype in DT:
        check(Requests(lengths, 6, 2, D, 32, dtype, seed=D))


@pytest.mark.parametrize("S", [16, 32, 48, 64, 80, 128, 256, 400])
@pytest.mark.parametrize("token_major", [False, True])
def test_block_sizes_and_layouts(S, token_major):
    for lengths in ([(S, 1), (2 * S + 1, 1), (S - 2, 1)], [(S - 1, 70), (3 * S, 20), (0, 5)]):
        check(Requests(lengths, 8, 2, 64, S, torch.float16, seed=S, token_major=token_major))


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 128, 129, 1000, 2 ** 31 - 1, 2 ** 40])
@pytest.mark.parametrize("lengths", [[(500, 1), (20, 1), (0, 1)], [(500, 140), (0, 260), (90, 1)]],
                         ids=["few", "many"])
def test_windows(window, lengths):
    check(Requests(lengths, 8, 2, 128, 16, torch.bfloat16, seed=3), window)


@pytest.mark.parametrize("heads", [1, 3, 16, 17, 64, 100, 128, 200])
def test_one_kv_head_for_all(heads):
    for lengths in ([(90, 1), (300, 1)], [(90, 5), (0, 9)]):
        check(Requests(lengths, heads, 1, 64, 16, torch.bfloat16, seed=heads))


@pytest.mark.parametrize("lengths", [[(40, 1), (0, 2)], [(40, 30), (0, 200)]], ids=["few", "many"])
@pytest.mark.parametrize("dtype", DT)
def test_f32_output_and_scales(lengths, dtype):
    r = Requests(lengths, 4, 2, 128, 16, dtype, seed=5)
    for scale in (0.0, 0.3, -0.2, 1e-6):
        o, lse = run(r, scale=scale, out_dtype=torch.float32)
        assert o.dtype == torch.float32
        assert_attention(o, lse, r.reference(scale), f"scale {scale}")


@pytest.mark.parametrize("lengths", [[(400, 1), (70, 1)], [(400, 200), (70, 33)]], ids=["few", "many"])
def test_peaked_and_growing_scores(lengths):
    """Scores of hundreds whose maximum keeps rising along the keys, so that
    earlier sums have to be scaled down again and again."""
    r = Requests(lengths, 4, 1, 64, 16, torch.float16, seed=6, q_scale=8.0)
    check(r)
    r.q.fill_(1.0)
    S = r.k.shape[2]
    for b, L in enumerate(r.total):
        for j in range(L):
            r.k[r.table[b, j // S].item(), :, j % S] = j / 16
    check(r)
    check(r, scale=-0.125)


@pytest.mark.parametrize("many", [False, True])
def test_rows_that_see_nothing(many):
    """More new tokens than the length says: the first rows stand before the
    first key.  A length of 0 (a request that was not served) leaves all."""
    m = q4()
    n = 150 if many else 4
    r = Requests([(0, n), (60, n), (0, n)], 4, 2, 64, 16, torch.bfloat16, seed=7)
    short = [n - 3, 60 + n, 0]
    r.kv_len.copy_(torch.tensor(short, dtype=torch.int32))
    o, lse = run(r)
    assert (o[:3] == 0).all() and torch.isinf(lse[:3]).all()
    assert (o[2 * n:] == 0).all() and torch.isinf(lse[2 * n:]).all()
    r.total = short
    ref = r.reference()
    assert_attention(o, lse, ref, "short")
    assert m.check() == m.OK


@pytest.mark.parametrize("many", [False, True])
def test_blocks_outside_the_cache_read_as_zeros(many):
    n = 40 if many else 1
    r = Requests([(100, n)], 8, 1, 64, 16, torch.float16, seed=8)
    bad = [0, 3]
    for i, x in zip(bad, (-5, r.k.shape[0])):
        blk = r.table[0, i].item()
        r.k[blk] = 0
        r.v[blk] = 0
    ref = r.reference()
    r.table[0, 0], r.table[0, 3] = -5, r.k.shape[0]
    assert_attention(*run(r), ref, "bad blocks")


@pytest.mark.parametrize("many", [False, True])
def test_bad_lengths_stay_inside(many):
    """Lengths past the table and row ranges past T are cut; rows of no
    request keep what they held."""
    m = q4()
    n = 50 if many else 1
    r = Requests([(30, n), (30, n)], 4, 1, 64, 16, torch.float16, seed=9, width_extra=0)
    r.k.nan_to_num_(0.0)
    r.v.nan_to_num_(0.0)
    r.kv_len[1] = 2 ** 31 - 1
    r.q_start[2] = 2 ** 31 - 1
    o, _ = run(r)
    assert torch.isfinite(o.float()).all()
    r.q_start[:] = -7
    out = torch.full_like(r.q, 3.0)
    run(r, out=out)
    assert (out == 3.0).all()
    assert m.check() == m.OK


@pytest.mark.parametrize("lengths", [[(300, 1), (50, 1)], [(300, 40), (50, 130)]], ids=["few", "many"])
def test_strided_rows_and_padding(lengths):
    """Queries inside wider rows (a qkv product's output), outputs inside
    wider rows, and token rows behind the last request left alone."""
    m = q4()
    r = Requests(lengths, 8, 2, 64, 16, torch.bfloat16, seed=10)
    T, pad = r.T, 3
    wide = torch.full((T + pad, 8 * 64 + 256), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:T, :8 * 64] = r.q.view(T, -1)
    q = wide[:, :8 * 64].unflatten(1, (8, 64))
    ow = torch.full((T + pad, 8 * 64 + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out = ow[:, :8 * 64].unflatten(1, (8, 64))
    m.attention(q, m.KVCache(r.k, r.v), r.table, r.q_start, r.kv_len, r.max_fresh, out=out)
    assert m.check() == m.OK
    assert_attention(out[:T], None, r.reference(), "strided")
    assert (ow[T:] == 7.0).all() and (ow[:, 8 * 64:] == 7.0).all()


@pytest.mark.parametrize("lengths", [[(9000, 1)], [(6000, 1), (10, 1), (3001, 1)], [(4000, 70)], [(3000, 300), (5, 1)]],
                         ids=str)
def test_split_items_are_deterministic(lengths):
    r = Requests(lengths, 8, 1, 128, 16, torch.bfloat16, seed=11)
    m = q4()
    ws = m.attention_workspace(r.max_fresh, 8, 1, 128)
    o, lse = check(r, ws=ws)
    for _ in range(5):
        o2, lse2 = run(r, ws=ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert not ws[:16384].any()


def test_the_hint_only_picks_the_kernel():
    for lengths in (FEW[9], MANY[7]):
        r = Requests(lengths, 8, 2, 128, 16, torch.float16, seed=12)
        for hint in (1, 2, 3, 40, 100000):
            check(r, max_fresh=hint)


def test_one_workspace_for_any_sequence_of_calls():
    m = q4()
    ws = m.attention_workspace(1000, 16, 2, 128)
    for i, lengths in enumerate((MANY[7], FEW[11], MANY[5], FEW[8], MANY[7])):
        r = Requests(lengths, 16, 2, (128, 64, 80)[i % 3], 16, DT[i % 2], seed=i)
        check(r, ws=ws)


def test_on_another_stream_and_in_a_graph():
    m = q4()
    for lengths in ([(700, 1), (40, 1)], [(700, 60), (40, 130)]):
        r = Requests(lengths, 8, 2, 128, 16, torch.bfloat16, seed=13)
        cache = m.KVCache(r.k, r.v)
        ref = r.reference()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        o = m.attention(r.q, cache, r.table, r.q_start, r.kv_len, r.max_fresh, stream=s)
        assert m.check(s) == m.OK
        assert_attention(o, None, ref, "stream")
        ws = m.attention_workspace(r.max_fresh, 8, 2, 128)
        out = torch.empty_like(r.q)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.attention(r.q, cache, r.table, r.q_start, r.kv_len, r.max_fresh, out=out, ws=ws)
        for _ in range(2):
            out.fill_(math.nan)
            g.replay()
            assert m.check() == m.OK
            assert_attention(out, None, ref, "graph")


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes and 2^31 elements: its first and last blocks."""
    m = q4()
    H, S, D = 8, 64, 128
    blocks = (1 << 31) // (H * S * D) + 3
    k = torch.zeros((blocks, H, S, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    for lengths in ([(90, 1)], [(90, 30)]):
        r = Requests(lengths, H, H, D, S, torch.bfloat16, seed=14)
        ids = r.table[0, :2].long() if lengths[0][1] == 1 else r.table[0, :2].long()
        far = torch.tensor([blocks - 1, 0], device="cuda")
        k[far], v[far] = r.k[ids], r.v[ids]
        ref = r.reference()
        r.k, r.v = k, v
        r.table[0, :2] = far.int()
        assert_attention(*run(r), ref, "far")


def test_bounded_waits_report_a_timeout():
    """With its copies switched off the tensor-core kernel stops after its
    wait limit, writes nothing, and the same SMs' tensor memory works again."""
    m = q4()
    r = Requests([(300, 60), (0, 200)], 8, 2, 128, 16, torch.bfloat16, seed=15)
    ws = m.attention_workspace(r.max_fresh, 8, 2, 128)
    out = torch.full_like(r.q, 5.0)
    m.attention_timeout_selftest(r.q, m.KVCache(r.k, r.v), r.table, r.q_start, r.kv_len, r.max_fresh, out, ws)
    assert m.check() == m.ERR_TIMEOUT
    assert (out == 5.0).all()
    ws.zero_()
    check(r, ws=ws)
    one = Requests([(30, 1)], 8, 2, 128, 16, torch.bfloat16, seed=15)
    with pytest.raises(m.Q4Error):
        m.attention_timeout_selftest(one.q, m.KVCache(one.k, one.v), one.table, one.q_start, one.kv_len, 1,
                                        torch.empty_like(one.q), ws)


@pytest.mark.parametrize("lengths", [[(20000, 1)], [(20000, 2)], [(20000, 3)], [(12000, 7)], [(9000, 13), (9000, 40)]],
                         ids=str)
@pytest.mark.parametrize("D", [64, 128])
def test_long_chains_of_parts(lengths, D):
    """One KV head, so that many workers share an item: the tree of the
    streaming kernel (three levels) and the joins of the tensor-core kernel
    with at most 32, 64 and 128 rows."""
    m = q4()
    r = Requests(lengths, 8, 1, D, 32, torch.bfloat16, seed=16)
    ws = m.attention_workspace(r.max_fresh, 8, 1, D)
    o, lse = check(r, ws=ws)
    for _ in range(3):
        o2, lse2 = run(r, ws=ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("many", [False, True])
def test_hundreds_of_requests(many):
    """More than 32 requests take the other way of finding a worker's share."""
    lengths = [(i * 53 % 400, (1 + i * 7 % 30 if many else 1) if i % 5 else 0) for i in range(333)]
    check(Requests(lengths, 4, 2, 64, 16, torch.float16, seed=17))


def test_an_empty_batch_writes_nothing():
    m = q4()
    for hint in (1, 100):
        r = Requests([(5, 1), (7, 1)], 8, 2, 64, 16, torch.bfloat16, seed=18)
        r.q_start.zero_()
        out = torch.full_like(r.q, 9.0)
        run(r, out=out, max_fresh=hint)
        assert (out == 9.0).all()
        assert m.check() == m.OK


@pytest.mark.parametrize("step", [0.5, 1.0, 3.0, 7.9, 8.1, 30.0])
@pytest.mark.parametrize("dtype", DT)
def test_scores_that_rise_by_tiles(step, dtype):
    """Every tile of 128 keys scores `step` (in powers of two) above the one
    before: weights under a stale reference grow to the limits of the type."""
    r = Requests([(1500, 200), (0, 700)], 4, 2, 64, 16, dtype, seed=19)
    r.q.fill_(1.0)
    S = r.k.shape[2]
    for b, L in enumerate(r.total):
        for j in range(L):
            r.k[r.table[b, j // S].item(), :, j % S] = 0.0
            r.k[r.table[b, j // S].item(), :, j % S, 0] = round(step * (j // 128) * 8) / 8 * 0.6875
    check(r, scale=1.0)
    check(r, scale=1.0, window=300)


@pytest.mark.parametrize("lengths", [[(3000, 1)], [(12000, 2)], [(700, 1), (5000, 1), (90, 2)]], ids=str)
def test_joins_add_this_calls_parts(lengths):
    """Call after call through one workspace, each with other queries: a join
    that took a part of the call before, or one not yet there, would show."""
    m = q4()
    r = Requests(lengths, 8, 1, 64, 16, torch.bfloat16, seed=21)
    cache, ws = m.KVCache(r.k, r.v), m.attention_workspace(r.max_fresh, 8, 1, 64)
    g = torch.Generator(device="cuda").manual_seed(22)
    qs = [torch.randn(r.q.shape, generator=g, device="cuda").bfloat16() for _ in range(40)]
    outs = [m.attention(q, cache, r.table, r.q_start, r.kv_len, r.max_fresh, ws=ws) for q in qs]
    assert m.check() == m.OK
    for i in (0, 1, 20, 39):
        r.q = qs[i]
        assert_attention(outs[i], None, r.reference(), f"call {i}")
    for q, o in zip(qs, outs):
        alone = m.attention(q, cache, r.table, r.q_start, r.kv_len, r.max_fresh, ws=ws)
        assert m.check() == m.OK and torch.equal(alone, o)


@pytest.mark.parametrize("recycled", [False, True])
@pytest.mark.parametrize("window", [1, 5, 16, 33, 100, 128, 200, 1000])
@pytest.mark.parametrize("lengths", [[(500, 1), (20, 3), (1300, 1)], [(500, 140), (90, 33), (0, 400)], [(3000, 20)]],
                         ids=["few", "many", "split"])
def test_nothing_before_a_window_reaches_the_output(lengths, window, recycled):
    """Keys and values that have left every row's window are NaN; ``recycled``:
    the blocks that hold nothing else are other requests' or gone."""
    for dtype, hint in ((torch.bfloat16, None), (torch.float16, 1), (torch.float16, 1000)):
        r = Requests(lengths, 8, 2, 64 if hint else 128, 16, dtype, seed=20)
        ref = r.reference(window=window)
        S = r.k.shape[2]
        for b, (cached, _) in enumerate(lengths):
            out = max(0, cached - window + 1)  # keys that no row sees any more
            for j in range(-(-out // S)):
                blk, m = r.table[b, j].item(), min(S, out - j * S)
                r.k[blk, :, :m] = math.nan
                r.v[blk, :, :m] = math.nan
                if recycled and m == S:
                    r.table[b, j] = (-1, 2 ** 31 - 1, r.table[b, 0].item())[j % 3]
        o, lse = run(r, window, max_fresh=hint)
        assert_attention(o, lse, ref, f"{lengths} window {window}")


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dtype", DT)
def test_many_small_weights_beside_a_large_one(dtype, many):
    """65536 keys of weight e^-17.5 (2^-25.2) and value 1 beside one of weight 1
    and value 0: the output is the small ones' share, 0.0016, and nothing if
    their weights round to nothing.  Allowed: each weight off by u of itself,
    or in binary16 by half its smallest number, 2^-25, under a reference of
    2^7 at least; f32 sums of 4096 steps, each off by 2^-24 of the row's sum
    (near 1 throughout) and 2^-23 of the output's, 2^-10 in all."""
    m = q4()
    S, L, D = 64, 65537, 64
    B, heads, n = (160, 8, 32) if many else (1300, 1, 1)
    blocks = -(-L // S)
    k = torch.zeros((blocks, 1, S, D), dtype=dtype, device="cuda")
    v = torch.ones_like(k)
    k[0, 0, 0, 0], v[0, 0, 0] = 17.5, 0.0
    q = torch.zeros((B * n, heads, D), dtype=dtype, device="cuda")
    q[..., 0] = 1.0
    i32 = dict(dtype=torch.int32, device="cuda")
    # every request reads the same blocks
    table = torch.arange(blocks, **i32).expand(B, blocks).contiguous()
    start, kv = torch.arange(B + 1, **i32) * n, torch.full((B,), L, **i32)
    o, lse = m.attention(q, m.KVCache(k, v), table, start, kv, n, scale=1.0, out_dtype=torch.float32, return_lse=True)
    assert m.check() == m.OK
    seen = (L - n + torch.arange(n, device="cuda", dtype=torch.float64)).view(1, n, 1)
    small = seen * math.exp(-17.5)
    exact = (small / (1 + small))[..., None]
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    allow = (u + 2.0 ** -10) * exact + (L * 2.0 ** -32 if dtype == torch.float16 else 0.0)
    err = (o.view(B, n, heads, D).double() - exact).abs()
    assert (err <= allow).all(), float((err / exact).max())
    err = (lse.view(B, n, heads).double() - 17.5 - torch.log1p(small)).abs()
    assert (err <= 2.0 ** -12 + 36 * 2.0 ** -18).all(), float(err.max())


@pytest.mark.parametrize("top", [2.0 ** 12, 2.0 ** 20, 2.0 ** 24, 2.0 ** 28, 2.0 ** 32])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dtype", DT)
def test_large_scores_pick_their_key(dtype, many, top):
    """Scores up to `top`, each a power of two away from the next: the largest
    one a row sees takes all, its value comes out (one weight, rounded once)."""
    n = 200 if many else 2
    r = Requests([(300, n), (0, n)], 4, 2, 64, 16, dtype, seed=23)
    g = torch.Generator().manual_seed(24)
    S = r.k.shape[2]
    r.q.zero_()
    r.q[..., 0] = 2.0 ** 15
    for sign in (1.0, -1.0):
        for b, L in enumerate(r.total):
            # 2^15 * key: top * (1 - i / 64), in any order; every 64th key is as large as another
            level = torch.arange(L)[torch.randperm(L, generator=g)] % 64
            for j in range(L):
                row = r.k[r.table[b, j // S].item(), :, j % S]
                row.zero_()
                row[:, 0] = sign * (1.0 - level[j].item() / 64) * 2.0
        scale = top / 2.0 ** 16
        o, lse = run(r, scale=scale, out_dtype=torch.float32)
        for b, L in enumerate(r.total):
            t0, t1 = r.start[b], r.start[b + 1]
            ids = r.table[b, :-(-L // S)].long()
            for c in range(2):
                k = r.k[ids, c].reshape(-1, 64)[:L, 0].double()
                v = r.v[ids, c].reshape(-1, 64)[:L].double()
                s = (2.0 ** 15 * scale) * k.expand(t1 - t0, L)
                place = torch.arange(L - (t1 - t0), L, device="cuda")[:, None]
                s = torch.where(torch.arange(L, device="cuda") <= place, s, -math.inf)
                best = (s == s.amax(1, keepdim=True)).double()  # the next one is e^-64 away at least
                want = best @ v / best.sum(1, keepdim=True)
                size = best @ v.abs() / best.sum(1, keepdim=True)
                u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
                for h in (2 * c, 2 * c + 1):
                    err = (o[t0:t1, h].double() - want).abs()
                    assert (err <= (u + 2.0 ** -16) * size).all(), (sign, b, float(err.max()))
                    exact = s.amax(1) + torch.log(best.sum(1))
                    assert ((lse[t0:t1, h].double() - exact).abs() <= 2.0 ** -22 * (1 + exact.abs())).all()
