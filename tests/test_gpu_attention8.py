"""q4_attention8 against the definition in 64 bits over the values that the
codes stand for: codes, types, head layouts, lengths from one token up, odd
sizes, both cache layouts, windows, rows that see nothing, garbage in unused
codes, scales far apart, splits over CTAs, streams, graphs, shared workspaces.
Tolerances: serving_ref.py (weights are rounded to 16 bits there too)."""
from __future__ import annotations

import pytest
import torch

from cache8_ref import CODES, Requests8, raw
from serving_ref import assert_attention

pytestmark = pytest.mark.gpu
DT = [torch.bfloat16, torch.float16]


def q4():
    import weight_only_int4_group_gb300 as m
    return m


def run(r, window=0, scale=None, out_dtype=None, ws=None, max_fresh=None, **kw):
    m = q4()
    o, lse = m.attention(r.q, r.cache(), r.table, r.q_start, r.kv_len, max_fresh or r.max_fresh, scale=scale,
                         window=window, out_dtype=out_dtype, return_lse=True, ws=ws, **kw)
    assert m.check() == m.OK
    return o, lse


def check(r, window=0, scale=None, **kw):
    o, lse = run(r, window, scale, **kw)
    assert_attention(o, lse, r.reference(scale, window), f"{r.lengths} window {window}")
    return o, lse


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


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("lengths", FEW, ids=lambda x: str(x)[:24])
@pytest.mark.parametrize("heads,kv", [(8, 1), (4, 4), (14, 2), (16, 1)])
def test_few_rows(lengths, heads, kv, dtype, code):
    check(Requests8(lengths, heads, kv, 128, 16, dtype, code, seed=len(lengths)))


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("lengths", MANY, ids=lambda x: str(x)[:24])
@pytest.mark.parametrize("heads,kv", [(8, 1), (2, 2), (14, 2)])
def test_many_rows(lengths, heads, kv, dtype, code):
    check(Requests8(lengths, heads, kv, 128, 16, dtype, code, seed=len(lengths)))


@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("lengths", [[(200, 1), (33, 1)], [(200, 40), (0, 150)]], ids=["few", "many"])
def test_head_dims(D, lengths):
    for dtype in DT:
        for code in CODES:
            check(Requests8(lengths, 6, 2, D, 32, dtype, code, seed=D))


@pytest.mark.parametrize("S", [16, 32, 48, 64, 80, 128, 256, 400])
@pytest.mark.parametrize("token_major", [False, True])
def test_block_sizes_and_layouts(S, token_major):
    for code in CODES:
        for lengths in ([(S, 1), (2 * S + 1, 1), (S - 2, 1)], [(S - 1, 70), (3 * S, 20), (0, 5)]):
            check(Requests8(lengths, 8, 2, 64, S, torch.float16, code, seed=S, token_major=token_major))


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 128, 129, 1000, 2 ** 31 - 1, 2 ** 40])
@pytest.mark.parametrize("lengths", [[(500, 1), (20, 1), (0, 1)], [(500, 140), (0, 260), (90, 1)]],
                         ids=["few", "many"])
def test_windows(window, lengths):
    check(Requests8(lengths, 8, 2, 128, 16, torch.bfloat16, torch.int8, seed=3), window)
    check(Requests8(lengths, 4, 4, 64, 32, torch.float16, torch.float8_e4m3fn, seed=4), window)


@pytest.mark.parametrize("heads", [1, 3, 9, 16, 17, 33, 64, 100, 128, 200])
def test_one_kv_head_for_all(heads):
    for code in CODES:
        for lengths in ([(90, 1), (300, 1)], [(90, 5), (0, 9)]):
            check(Requests8(lengths, heads, 1, 64, 16, torch.bfloat16, code, seed=heads))


@pytest.mark.parametrize("lengths", [[(40, 1), (0, 2)], [(40, 30), (0, 200)]], ids=["few", "many"])
@pytest.mark.parametrize("dtype", DT)
def test_f32_output_and_scales(lengths, dtype):
    r = Requests8(lengths, 4, 2, 128, 16, dtype, torch.int8, seed=5)
    for scale in (0.0, 0.3, -0.2, 1e-6):
        o, lse = run(r, scale=scale, out_dtype=torch.float32)
        assert o.dtype == torch.float32
        assert_attention(o, lse, r.reference(scale), f"scale {scale}")


@pytest.mark.parametrize("lengths", [[(400, 1), (70, 1)], [(400, 200), (70, 33)]], ids=["few", "many"])
@pytest.mark.parametrize("code", CODES)
def test_peaked_and_growing_scores(lengths, code):
    """Scores of hundreds whose maximum keeps rising along the keys."""
    r = Requests8(lengths, 4, 1, 64, 16, torch.float16, code, seed=6, q_scale=8.0)
    check(r)
    r.q.fill_(1.0)
    for b, L in enumerate(r.total):
        for j in range(L):
            blk = r.table[b, j // 16].item()
            e = max(0, (j // 16).bit_length() - 3)
            r.k_exp[blk] = 127 + e
            value = torch.tensor(j / 16 / 2 ** e, device="cuda")
            raw(r.k)[blk, :, j % 16] = raw(value.round().to(torch.int8) if code == torch.int8 else value.to(code)).item()
    check(r)
    check(r, scale=-0.125)


@pytest.mark.parametrize("lengths", [[(700, 1), (70, 2)], [(700, 100), (70, 33)]], ids=["few", "many"])
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", DT)
def test_scales_far_apart(lengths, dtype, code):
    """Blocks whose values differ by many powers of two, and keys likewise: a
    large scale with a negligible weight may not cost the others' precision."""
    span = (-12, 6) if dtype == torch.float16 else (-30, 20)
    r = Requests8(lengths, 4, 2, 128, 16, dtype, code, seed=11, exps=span)
    r.k_exp.copy_(torch.randint(127 - 10, 127 - 3, r.k_exp.shape, device="cuda"))
    check(r)
    # the largest values only where the weights are smallest
    r.q.fill_(1.0)
    raw(r.k).fill_(raw(torch.ones((), device="cuda").to(code)).item())
    r.k_exp.fill_(127)
    r.v_exp.fill_(127 + span[0])
    for b, L in enumerate(r.total):
        blk = r.table[b, 1].item()
        r.v_exp[blk] = 127 + span[1]
        raw(r.k)[blk] = raw(torch.full((), -1.0, device="cuda").to(code)).item()
    check(r)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("code", CODES)
def test_rows_that_see_nothing(many, code):
    n = 150 if many else 4
    r = Requests8([(0, n), (60, n), (0, n)], 4, 2, 64, 16, torch.bfloat16, code, seed=7)
    short = [n - 3, 60 + n, 0]
    r.kv_len.copy_(torch.tensor(short, dtype=torch.int32))
    o, lse = run(r)
    assert (o[:3] == 0).all() and torch.isinf(lse[:3]).all()
    assert (o[2 * n:] == 0).all() and torch.isinf(lse[2 * n:]).all()
    r.total = short
    assert_attention(o, lse, r.reference(), "short")


@pytest.mark.parametrize("many", [False, True])
def test_hint_does_not_change_what_is_computed(many):
    """Any number of new tokens is right with either kernel."""
    r = Requests8([(300, 40), (20, 1), (0, 9)], 8, 2, 128, 16, torch.bfloat16, torch.int8, seed=8)
    ws = q4().attention_workspace(1 if not many else 64, 8, 2, 128, eight_bit=True)
    check(r, max_fresh=1 if not many else 64, ws=ws)


def test_equals_the_16_bit_attention_within_rounding():
    """The same values in a 16-bit cache."""
    m = q4()
    for lengths in ([(900, 1), (33, 2)], [(900, 200), (0, 70)]):
        for code in CODES:
            r = Requests8(lengths, 8, 2, 128, 16, torch.bfloat16, code, seed=2)
            k, v = (x.to(torch.bfloat16) for x in r.values())
            o8, l8 = run(r, out_dtype=torch.float32)
            o, l = m.attention(r.q, m.KVCache(k, v), r.table, r.q_start, r.kv_len, r.max_fresh, return_lse=True,
                               out_dtype=torch.float32)
            # 2 * 2^-8 on the weights
            assert ((o8 - o).abs() <= 2 ** -7 * v.double().abs().nan_to_num().max()).all()
            assert ((l8 - l).abs() <= 1e-4).all()


def test_rows_of_no_request_and_strides():
    m = q4()
    for lengths, pad in (([(50, 1), (9, 1)], 3), ([(50, 60), (9, 30)], 5)):
        r = Requests8(lengths, 4, 2, 64, 16, torch.float16, torch.float8_e4m3fn, seed=1)
        T = r.T + pad
        qbig = torch.zeros(T, 4 * 64 + 8, dtype=torch.float16, device="cuda")
        qbig[:r.T, :256] = r.q.flatten(1)
        obig = torch.full((T, 4 * 64 + 16), 5.0, dtype=torch.float16, device="cuda")
        m.attention(qbig[:, :256].unflatten(1, (4, 64)), r.cache(), r.table, r.q_start, r.kv_len, r.max_fresh,
                    out=obig[:, :256].unflatten(1, (4, 64)))
        want, _ = run(r)
        assert torch.equal(obig[:r.T, :256].unflatten(1, (4, 64)), want)
        assert (obig[r.T:] == 5).all() and (obig[:, 256:] == 5).all()


def test_bad_device_data():
    """Table entries outside the cache are keys of score 0 and value 0; lengths and
    row starts of any kind stay within the buffers."""
    m = q4()
    for lengths in ([(60, 1), (40, 2)], [(60, 50), (40, 70)]):
        r = Requests8(lengths, 4, 2, 64, 16, torch.bfloat16, torch.int8, seed=4)
        r.table[0, 1] = -3
        r.table[1, 0] = 2 ** 31 - 1
        good = r.table.clone()
        # the reference: a spare block of zeros in their place
        spare = next(i for i in range(r.k.shape[0]) if i not in set(good[good >= 0].tolist()))
        raw(r.k)[spare] = 0
        raw(r.v)[spare] = 0
        o, lse = run(r)
        r.table[0, 1] = r.table[1, 0] = spare
        assert_attention(o, lse, r.reference(), "outside")
        for lens, starts in (([10 ** 9, -5], r.start), ([2 ** 31 - 1] * 2, [0, 10 ** 9, 2 ** 31 - 1]),
                             (r.total, [-9, 90, 5]), (r.total, [r.T, 1, 0])):
            m.attention(r.q, r.cache(), good, torch.tensor(starts, dtype=torch.int32, device="cuda"),
                        torch.tensor(lens, dtype=torch.int32, device="cuda"), r.max_fresh)
            assert m.check() == m.OK


def test_long_context_split_over_all_workers():
    for heads, kv in ((1, 1), (8, 1), (16, 1)):
        check(Requests8([(70000, 1)], heads, kv, 128, 64, torch.bfloat16, torch.int8, seed=heads))
    check(Requests8([(30000, 3), (5, 1)], 8, 1, 64, 16, torch.float16, torch.float8_e4m3fn, seed=5))
    check(Requests8([(9000, 300)], 4, 1, 128, 16, torch.bfloat16, torch.float8_e4m3fn, seed=5))


def test_one_workspace_for_calls_of_both_kinds_and_repeats():
    m = q4()
    sizes = [(1, [(5000, 1)]), (150, [(700, 150), (3, 20)]), (1, [(i * 13, 1) for i in range(40)]), (40, [(2000, 40)])]
    ws = max((m.attention_workspace(n, 8, 2, 128, eight_bit=e) for n, _ in sizes for e in (False, True)),
             key=lambda t: t.numel())
    outs = {}
    for turn in range(2):
        for i, (n, lengths) in enumerate(sizes):
            r = Requests8(lengths, 8, 2, 128, 16, torch.bfloat16, CODES[i % 2], seed=i)
            o, lse = check(r, ws=ws)
            k, v = (x.to(torch.bfloat16) for x in r.values())
            m.attention(r.q, m.KVCache(k, v), r.table, r.q_start, r.kv_len, r.max_fresh, ws=ws)
            if turn:
                assert torch.equal(outs[i][0], o) and torch.equal(outs[i][1], lse)
            outs[i] = (o, lse)
    torch.cuda.synchronize()
    assert int(ws[:131072].count_nonzero()) == 0


def test_streams_and_graphs():
    m = q4()
    for lengths in ([(3000, 1), (100, 1)], [(3000, 90), (100, 33)]):
        r = Requests8(lengths, 8, 2, 128, 16, torch.bfloat16, torch.int8, seed=9)
        want, wl = run(r)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        o, l = m.attention(r.q, r.cache(), r.table, r.q_start, r.kv_len, r.max_fresh, return_lse=True, stream=side)
        side.synchronize()
        assert torch.equal(o, want) and torch.equal(l, wl)
        ws = m.attention_workspace(r.max_fresh, 8, 2, 128, eight_bit=True)
        cache = r.cache()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o, l = m.attention(r.q, cache, r.table, r.q_start, r.kv_len, r.max_fresh, return_lse=True, ws=ws)
        for _ in range(3):
            o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want) and torch.equal(l, wl)
        # other lengths in the same graph
        r.kv_len.copy_(torch.tensor([2000 + lengths[0][1], lengths[1][1]], dtype=torch.int32))
        r.total = r.kv_len.tolist()
        graph.replay()
        torch.cuda.synchronize()
        assert_attention(o, l, r.reference(), "replayed")
    assert m.check() == m.OK


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", DT)
def test_bounded_waits_report_a_timeout(dtype, code):
    """A copy that never comes ends the kernel's waits, all roles leave, nothing is
    written, and the context goes on."""
    m = q4()
    r = Requests8([(300, 150), (7, 20)], 8, 2, 128, 16, dtype, code, seed=14)
    ws = m.attention_workspace(r.max_fresh, 8, 2, 128, eight_bit=True)
    out = torch.full_like(r.q, 5.0)
    m.attention_timeout_selftest(r.q, r.cache(), r.table, r.q_start, r.kv_len, r.max_fresh, out, ws)
    assert m.check() == m.ERR_TIMEOUT
    assert (out == 5.0).all()
    ws.zero_()
    check(r, ws=ws)
    one = Requests8([(30, 1)], 8, 2, 128, 16, dtype, code, seed=15)
    with pytest.raises(m.Q4Error):
        m.attention_timeout_selftest(one.q, one.cache(), one.table, one.q_start, one.kv_len, 1, torch.empty_like(one.q), ws)


MIDDLE = [  # heads, KV heads, dims, lengths: 17 to 32 rows per KV head
    (16, 2, 128, [(i * 37 % 500, 1 + i % 4) for i in range(40)]),
    (16, 2, 128, [(i * 53 % 90, 3 + i % 2) for i in range(31)]),
    (20, 1, 64, [(i * 61 % 700, 1) for i in range(70)]),
    (32, 1, 128, [(i * 61 % 700, i % 2) for i in range(70)]),
    (4, 4, 96, [(i * 29 % 300, 1 + i * 7 % 32) for i in range(20)]),
    (64, 8, 128, [(5000 + 3 * i, 4) for i in range(8)]),
    (24, 8, 48, [(40000, 9)] + [(0, 0)] * 6 + [(3, 9)]),
]


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("case", MIDDLE, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{len(c[3])}")
def test_up_to_32_rows(case, dtype, code):
    """Both kernels' side of the requests times heads that choose between them, with
    one workspace, and with windows."""
    heads, kv, D, lengths = case
    ws = q4().attention_workspace(max(n for _, n in lengths), heads, kv, D, eight_bit=True)
    for part in (lengths, lengths[:3]):
        r = Requests8(part, heads, kv, D, 32, dtype, code, seed=len(part))
        for window in (0, 19):
            check(r, window, ws=ws, max_fresh=max(n for _, n in lengths))


def test_a_workspace_serves_smaller_steps():
    m = q4()
    for D in (16, 64, 80, 128):
        for GQ in (1, 2, 3, 5, 8, 11, 16, 17, 31, 32, 33, 64):
            size = [m.attention_workspace_bytes(n, 2 * GQ, 2, D, eight_bit=True) for n in (*range(1, 40), 64, 1000, 10 ** 6)]
            assert size[0] > 0 and size == sorted(size), (D, GQ)
    ws = m.attention_workspace(512, 64, 8, 128, eight_bit=True)
    for n in (1, 2, 4, 40, 4):
        check(Requests8([(500, n)] * 8, 64, 8, 128, 16, torch.bfloat16, torch.int8, seed=n), ws=ws)


@pytest.mark.parametrize("code", CODES)
def test_up_to_32_rows_repeat_and_use_every_scale(code):
    """The same bits at each call, splits over many warps; keys and values of all
    the scales of bf16; queries past 2^80 against zero codes."""
    r = Requests8([(3000, 4)] * 8, 64, 8, 128, 16, torch.bfloat16, code, seed=5)
    ws = q4().attention_workspace(4, 64, 8, 128, eight_bit=True)
    a, la = run(r, ws=ws)
    for _ in range(5):
        b, lb = run(r, ws=ws)
        assert torch.equal(a, b) and torch.equal(la, lb)
    r = Requests8([(200, 4)] * 64, 8, 1, 128, 16, torch.bfloat16, code, seed=6, exps=(-30, 20))
    r.k_exp.copy_(torch.randint(127 - 10, 127 - 3, r.k_exp.shape, device="cuda"))
    check(r)
    raw(r.k).zero_()
    r.k_exp.fill_(127 + 48)
    r.q.fill_(2.0 ** 127)
    check(r)


@pytest.mark.parametrize("n", [1, 2, 40])
@pytest.mark.parametrize("code", CODES)
def test_large_queries_against_empty_codes(n, code):
    """Queries of 2^127 and keys that are all 0 under the largest scale: all
    scores are 0 and each visible key has the same weight.  (n rows: all kernels.)"""
    from cache8_ref import RANGE
    for scale in (None, -0.125):
        r = Requests8([(100, n)], 8, 1, 128, 16, torch.bfloat16, code, seed=4)
        raw(r.k).zero_()
        r.k_exp.fill_(127 + RANGE[code, torch.bfloat16][1])
        r.q.fill_(2.0 ** 127)
        o, lse = check(r, scale=scale)
        # the sum of up to 140 equal weights, f32
        want = torch.log(torch.arange(101, 101 + n, device="cuda", dtype=torch.float64))
        assert ((lse.double() - want[:, None]).abs() <= 2.0 ** -18).all()


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", DT)
def test_every_code_and_exponent(dtype, code):
    """All 254 or 255 codes, subnormal e4m3 among them, under every exponent of
    the range, come to the output exactly: one visible key per request."""
    from cache8_ref import RANGE
    lo, hi = RANGE[code, dtype]
    for D, n in ((64, 1), (128, 40)):
        es = list(range(lo, hi + 1))
        r = Requests8([(0, n)] * len(es), 8, 1, D, 16, dtype, code, seed=3)
        codes = torch.arange(256, device="cuda").to(torch.uint8)
        if code == torch.int8:
            codes = codes[codes != 0x80]
        else:
            codes = codes[(codes & 0x7F) != 0x7F]
        raw(r.k).zero_()
        for b, e in enumerate(es):
            # every token of the request holds the same value row
            for j in range(-(-n // 16)):
                blk = r.table[b, j].item()
                r.v_exp[blk] = 127 + e
                raw(r.v)[blk, 0] = codes[(torch.arange(D, device="cuda") + b * D) % len(codes)]
        o, _ = run(r, out_dtype=torch.float32)
        vals = r.values()[1]
        for b in range(len(es)):
            want = vals[r.table[b, 0].item(), 0, 0]
            got = o[r.start[b]:r.start[b + 1]].double()
            # equal weights sum to 1 within 2^-22 (a sum of at most 40 of them in f32)
            assert ((got - want).abs() <= want.abs() * 2.0 ** -20).all(), (es[b], n)


def test_two_streams_at_once():
    """Calls on two streams, each with its workspace, and an append beside them."""
    m = q4()
    rs = [Requests8(ls, 8, 2, 128, 16, torch.bfloat16, c, seed=i) for i, (ls, c) in
          enumerate([([(9000, 1), (40, 1)], CODES[0]), ([(3000, 120)], CODES[1])])]
    want = [run(r)[0] for r in rs]
    streams = [torch.cuda.Stream() for _ in rs]
    spaces = [m.attention_workspace(r.max_fresh, 8, 2, 128, eight_bit=True) for r in rs]
    caches = [r.cache() for r in rs]
    torch.cuda.synchronize()
    for _ in range(20):
        outs = [m.attention(r.q, c, r.table, r.q_start, r.kv_len, r.max_fresh, ws=w, stream=s)
                for r, c, w, s in zip(rs, caches, spaces, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want)) and m.check() == m.OK


@pytest.mark.parametrize("code", CODES)
def test_attention_block_example(code):
    """The example's block with an 8-bit cache: decoding token by token is near the
    same block over 16 bits (its codes are within 2^-4 of each value, or a step)."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    from attention_block import AttentionBlock, Server
    outs = []
    for c in (None, code):
        server = Server(2, 20, 16, 8)
        block = AttentionBlock(256, 4, 2, 64, 40, 20, dtype=torch.float16, code=c)
        g = torch.Generator(device="cuda").manual_seed(1)
        for fresh in ([30, 5], [1, 1], [1, 0], [3, 1]):
            x = torch.randn(sum(fresh), 256, generator=g, device="cuda").half()
            y = block(x, server, server.plan(torch.tensor(fresh, dtype=torch.int32, device="cuda"), len(x)))
        outs.append(y.float())
    assert q4().check() == q4().OK and torch.isfinite(outs[1]).all()
    # values are off by 2^-4 of themselves at most (e4m3; int8 in blocks of normal
    # numbers less), weights by factors of as little on scores near 1
    rel = float((outs[0] - outs[1]).norm() / outs[0].norm())
    assert rel < 2.0 ** -3, rel


@pytest.mark.parametrize("code", CODES)
def test_a_layer_in_8_bits(code):
    """Plan, quantising append, attention and read-back together, as a server
    runs them: a prompt step, then decode steps in a graph."""
    m = q4()
    heads, kv, D, S, B = 8, 2, 128, 16, 3
    prompts = [70, 5, 33]
    i32 = dict(dtype=torch.int32, device="cuda")
    length, table = torch.zeros(B, **i32), torch.full((B, 12), -1, **i32)
    free, count = torch.arange(36, **i32), torch.full((1,), 36, **i32)
    cache = m.KVCache8.empty(36, kv, S, D, code)
    freq, factor = m.rope_frequencies(D)
    ws = m.attention_workspace(max(prompts), heads, kv, D, eight_bit=True)
    g = torch.Generator(device="cuda").manual_seed(0)

    def step(x, fresh, T, most, plan=None):
        p = m.cache_plan(length, fresh, table, free, count, S, T, out=plan)
        length.copy_(p.kv_len)
        count.copy_(p.counts[2:3])
        q = m.rope_append(x, cache, p.position, p.slot, freq, heads, factor=factor)
        return q, m.attention(q, cache, table, p.q_start, p.kv_len, most, ws=ws), p

    def reference(q, p):
        from serving_ref import attention_reference
        start = torch.cumsum(torch.cat([torch.zeros(1, **i32), p.kv_len]), 0).int()
        k, v = m.cache_read(cache, table, start, p.kv_len, int(start[-1]))
        # the values read back as requests' own blocks of a 64-bit cache
        L = p.kv_len.tolist()
        W = max(L)
        kk, vv = (torch.zeros(B, kv, W, D, dtype=torch.float64, device="cuda") for _ in "kv")
        for b in range(B):
            kk[b, :, :L[b]] = k[start[b]:start[b + 1]].double().transpose(0, 1)
            vv[b, :, :L[b]] = v[start[b]:start[b + 1]].double().transpose(0, 1)
        return attention_reference(q, kk, vv, torch.arange(B, device="cuda")[:, None], p.q_start.tolist(), L, D ** -0.5, 0)

    x = torch.randn(sum(prompts), (heads + 2 * kv) * D, generator=g, device="cuda").bfloat16()
    q, o, p = step(x, torch.tensor(prompts, **i32), len(x), max(prompts))
    assert_attention(o, None, reference(q, p), "prompt")
    x, one = x[:B].clone(), torch.ones(B, **i32)
    plan = m.CachePlan.empty(B, B)
    step(x, one, B, 1, plan)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, o, p = step(x, one, B, 1, plan)
    for _ in range(20):
        x.normal_(generator=g)
        graph.replay()
        assert_attention(o, None, reference(q, p), "decode")
    assert length.tolist() == [n + 21 for n in prompts] and m.check() == m.OK


def within(r, o, few, window=0):
    """o (f32) against the definition, where weights carry 11 bits with few rows
    whatever the type, and the type's with many: off by (u + e) sum p |v| / sum p
    (serving_ref.py), with nothing added that small values could hide behind."""
    from serving_ref import U, attention_reference
    args = (*r.values(), r.table, r.start, r.total, r.q.shape[2] ** -0.5, window)
    want, _, typed, _ = attention_reference(r.q, *args)
    free = attention_reference(r.q.float(), *args)[2]  # e sum p |v| / sum p: no weight is rounded
    limit = free + (typed - free) * (2.0 ** -11 / U[r.dtype] if few else 1.0)
    err = (o.double() - want).abs()
    assert not torch.isnan(err).any() and (err <= limit).all(), float((err / limit.clamp(min=1e-300)).max())


@pytest.mark.parametrize("n", [4, 8, 16, 40])
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", DT)
def test_blocks_outside_the_cache_beside_the_smallest_scales(dtype, code, n):
    """Their values are 0, whatever the scales of the blocks beside them."""
    from cache8_ref import RANGE
    lo = RANGE[code, dtype][0]
    r = Requests8([(150, n)] * 8, 16, 8, 64, 16, dtype, code, seed=n, exps=(lo, lo + 2), q_scale=0.25)
    r.k_exp.copy_(torch.randint(127 - 7, 127 - 3, r.k_exp.shape, device="cuda"))
    used = set(r.table[r.table < r.k.shape[0]].tolist())
    spare = next(i for i in range(r.k.shape[0]) if i not in used)
    raw(r.k)[spare] = 0
    raw(r.v)[spare] = 0
    r.table[:4, 0] = -1
    r.table[4:, 5] = 2 ** 31 - 1
    o, _ = run(r, out_dtype=torch.float32)
    r.table[:4, 0] = spare
    r.table[4:, 5] = spare
    within(r, o, n <= 16)


@pytest.mark.parametrize("n", [4, 8, 16, 40])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", DT)
def test_a_large_scale_whose_codes_are_zero(dtype, code, D, n):
    """One block's value scale lies 8 to 96 powers of two above the others', and all
    its codes but dim 0's are 0: the other dims hold the small values, wherever the
    block stands and however the keys are split, with equal scores and others."""
    from cache8_ref import RANGE
    lo, hi = RANGE[code, dtype]
    for q_scale, at in ((0.0, 4), (0.25, 0), (0.25, 9)):  # at: the block, of 10
        r = Requests8([(159 - n + b % 2, n) for b in range(8)], 16, 8, D, 16, dtype, code, seed=n, q_scale=q_scale)
        r.k_exp.copy_(torch.randint(127 - 7, 127 - 3, r.k_exp.shape, device="cuda"))
        r.v_exp.fill_(127 + lo)
        for b in range(8):
            blk = r.table[b, at].item()
            r.v_exp[blk] = 127 + min(hi, lo + 8 + b * (hi - lo - 8) // 7 + b % 2)
            raw(r.v)[blk, :, :, 1:] = 0
        o, _ = run(r, out_dtype=torch.float32)
        within(r, o, n <= 16)
    # seven scales in turn, two requests
    r = Requests8([(2000, n), (700, n)], 2, 1, D, 32, dtype, code, seed=5, q_scale=0.25)
    r.k_exp.copy_(torch.randint(127 - 7, 127 - 3, r.k_exp.shape, device="cuda"))
    r.v_exp.copy_(127 + lo + (torch.arange(len(r.v_exp), device="cuda") % 7 * (hi - lo) // 6)[:, None])
    raw(r.v)[torch.arange(len(r.v), device="cuda") % 7 > 0, :, :, 8:] = 0
    o, _ = run(r, out_dtype=torch.float32)
    within(r, o, n <= 8)


@pytest.mark.parametrize("n", [4, 8, 16, 40])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("code", CODES)
def test_small_query_elements_beside_large_ones(code, D, n):
    """Query elements 2^28 to 2^120 times as large as the others meet zero codes:
    the scores come from the small ones."""
    r = Requests8([(100 + b, n) for b in range(8)], 16, 8, D, 16, torch.bfloat16, code, seed=n)
    raw(r.k)[:, :, :, :2] = 0
    for b, e in enumerate((28, 31, 32, 33, 36, 40, 60, 120)):
        rows = r.q[r.start[b]:r.start[b + 1]]
        rows[..., 0] = 1.5 * 2.0 ** e
        rows[:, ::3, 1] = -2.0 ** (e - 5)
        rows[:, 1::4, :2] = 0.25  # and heads without one
    o, lse = run(r, out_dtype=torch.float32)
    ref = r.reference()
    assert_attention(o, lse, ref, f"{n}")
    within(r, o, n <= 16)
    # elements as small as 2^-100, that large codes bring back
    r.q *= 2.0 ** -100
    r.q[r.start[7]:] *= 2.0 ** -20
    r.k_exp.fill_(127 + 48)
    check(r, scale=2.0 ** 45 * D ** -0.5)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("heads,kv,D", [(8, 1, 128), (14, 2, 64), (4, 4, 80)])
def test_few_rows_keep_11_bits_of_the_weights(heads, kv, D, dtype, code):
    """Of bf16 caches too, and whether items are split or not."""
    for lengths in ([(776, 1)], [(5000, 1), (3, 2)], [(i * 37 % 500, 1) for i in range(33)], [(90, 2), (0, 1), (17, 2)]):
        r = Requests8(lengths, heads, kv, D, 16, dtype, code, seed=len(lengths), q_scale=0.5)
        within(r, run(r, out_dtype=torch.float32)[0], True)
        within(r, run(r, window=33, out_dtype=torch.float32)[0], True, 33)
