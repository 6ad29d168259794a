"""Serving with the KV cache in 8 bits: the rotary append that quantises keys and
values as it writes them, reading tokens back, and attention over such a cache.

The cache holds int8 codes (to +-127) or e4m3 numbers (to +-448) and one
power-of-two scale 2^e for each (block of tokens, head), keys and values apart,
stored as the byte e + 127.  A token appended to a block that holds others
already can only raise its scale; the codes held are then rounded again.

Each case is run through the library's calls (``own``) or through plain torch
operations in 32 bits.  Shapes are those of the two layers this repository
benchmarks (64 query heads on 8 KV heads of 128; 32 heads of 128) and small
generic ones.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
GQA = {"heads": 64, "kv_heads": 8, "dim": 128}  # the 70B-shaped layer
MHA = {"heads": 32, "kv_heads": 32, "dim": 128}  # the 7B-shaped layer
MOST = {"int8": 127.0, "e4m3": 448.0}  # the largest code
# the exponents that keep every value a number of the 16-bit type
RANGE = {("int8", "f16"): (-24, 9), ("e4m3", "f16"): (-15, 7),
         ("int8", "bf16"): (-48, 48), ("e4m3", "bf16"): (-48, 48)}


# ------------------------------------------------------------------ cases
def _append(name, requests, cached, fresh, model, rot, interleaved, block, dtype, code):
    return {"name": name, "op": "append", "requests": requests, "cached_lo": cached[0], "cached_hi": cached[1],
            "fresh_lo": fresh[0], "fresh_hi": fresh[1], **model, "rot": rot, "interleaved": interleaved,
            "block": block, "dtype": dtype, "code": code}


def _read(name, requests, cached, model, block, dtype, code):
    return {"name": name, "op": "read", "requests": requests, "cached_lo": cached[0], "cached_hi": cached[1],
            "fresh_lo": 0, "fresh_hi": 0, **model, "block": block, "dtype": dtype, "code": code}


def _attention(name, requests, cached, fresh, model, block, dtype, code, window=0, lse=False):
    return {"name": name, "op": "attention", "requests": requests, "cached_lo": cached[0],
            "cached_hi": cached[1], "fresh_lo": fresh[0], "fresh_hi": fresh[1], **model,
            "block": block, "dtype": dtype, "code": code, "window": window, "lse": lse}


def listed():
    return [
        # the smallest decode step: one new token for each of four users, half of each head rotated in pairs
        _append("append 4 decoding", 4, (100, 4000), (1, 1), MHA, 64, True, 16, "f16", "int8"),
        # a prompt chunk of odd length that begins inside a block
        _append("append 1001 in 3 chunks", 3, (5, 8000), (300, 367), MHA, 128, False, 32, "bf16", "e4m3"),
        # a large prefill step, far into long contexts
        _append("append 8192 in 4 chunks", 4, (0, 100000), (2048, 2048), GQA, 128, False, 64, "bf16", "int8"),
        # one request's tokens for a layer that works on 16 bits
        _read("read 777", 1, (777, 777), MHA, 16, "f16", "int8"),
        # requests that leave the card for a while
        _read("read 24 requests", 24, (900, 8100), GQA, 64, "bf16", "e4m3"),
        # one user decoding: latency
        _attention("attention 1 decoding", 1, (776, 776), (1, 1), MHA, 16, "f16", "int8"),
        # an ordinary decode batch of ragged lengths
        _attention("attention 32 decoding", 32, (100, 8191), (1, 1), GQA, 16, "bf16", "e4m3"),
        # a long-context decode batch: the cache is gigabytes
        _attention("attention 48 decoding long", 48, (1000, 24575), (1, 1), GQA, 64, "bf16", "int8"),
        # a few drafted tokens per request, a small model with a sliding window
        _attention("attention 16 drafted window", 16, (10, 6000), (4, 4),
                   {"heads": 16, "kv_heads": 4, "dim": 64}, 32, "f16", "e4m3", window=1024, lse=True),
        # one chunk of a long prompt
        _attention("attention chunk 512 after 16384", 1, (16384, 16384), (512, 512), GQA, 16, "bf16", "int8"),
        # a whole prompt at once
        _attention("attention prompt 4096", 1, (0, 0), (4096, 4096), MHA, 16, "f16", "e4m3"),
        # continuous batching: prompt chunks and decodes in one step
        _attention("attention mixed", 12, (50, 4000), (1, 160), GQA, 16, "bf16", "e4m3"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "attention", "attention", "attention", "attention"])
    block = rng.choice([16, 32, 48, 64])
    dtype, code = rng.choice(["bf16", "f16"]), rng.choice(["int8", "e4m3"])
    kv = rng.choice([1, 2, 4, 8])
    model = {"heads": kv * rng.choice([1, 2, 4, 7, 8]), "kv_heads": kv,
             "dim": rng.choice([64, 80, 96, 128, 128])}
    lo = _log_int(rng, 1, 2000)
    if op == "append":
        requests = _log_int(rng, 1, 64)
        cached = (lo, lo + _log_int(rng, 1, 100000))
        n = 1 if rng.random() < 0.4 else _log_int(rng, 1, 8192 // requests)
        rot = rng.choice([model["dim"], model["dim"] // 2])
        return _unnamed(_append("", requests, cached, (min(n, rng.randint(1, 3)), n), model, rot, rng.random() < 0.5,
                                block, dtype, code))
    if op == "read":
        return _unnamed(_read("", _log_int(rng, 1, 24), (lo, lo + _log_int(rng, 1, 6000)), model, block, dtype, code))
    window = rng.choice([0, 0, 0, _log_int(rng, 1, 4096)])
    kind = rng.choice(["decode", "decode", "draft", "chunk", "prompt"])
    if kind == "decode":
        sizes = (_log_int(rng, 1, 48), (lo, lo + _log_int(rng, 1, 20000)), (1, 1))
    elif kind == "draft":
        sizes = (_log_int(rng, 1, 32), (lo, lo + _log_int(rng, 1, 6000)), (1, rng.randint(2, 8)))
    elif kind == "chunk":
        sizes = (rng.randint(1, 12), (lo, lo + _log_int(rng, 1, 4000)), (1, _log_int(rng, 16, 160)))
    else:
        n = _log_int(rng, 100, 2048)
        sizes = (1, (0, 0) if rng.random() < 0.5 else (777, 777), (n, n))
    return _unnamed(_attention("", *sizes, model, block, dtype, code, window, rng.random() < 0.25))


def _unnamed(case):
    del case["name"]
    return case


def _lengths(case):
    """The (cached, new) token counts of the case's requests; prepare() shuffles them."""
    n = case["requests"]
    d = max(1, n - 1)
    cached = [case["cached_lo"] + (case["cached_hi"] - case["cached_lo"]) * i // d for i in range(n)]
    fresh = [case["fresh_lo"] + (case["fresh_hi"] - case["fresh_lo"]) * (i * 7 % n) // d
             for i in range(n)]
    if n == 1:
        fresh = [case["fresh_hi"]]
    return cached, fresh


def _blocks(n, block):
    return -(-n // block)


# ------------------------------------------------------------------ inputs
def _codes(case, shape, gen):
    """Codes as blocks of normal keys or values hold them."""
    if case["code"] == "int8":
        x = torch.empty(shape, dtype=torch.float16, device="cuda").normal_(0.0, 36.0, generator=gen)
        return x.round_().clamp_(-127, 127).to(torch.int8)
    x = torch.empty(shape, dtype=torch.float16, device="cuda").normal_(0.0, 120.0, generator=gen)
    return x.clamp_(-448, 448).to(torch.float8_e4m3fn)


def _exponents(case, shape, gen):
    """e + 127 for entries near 1: 2^-5 for int8 codes, 2^-7 for e4m3, one more or less here and there."""
    e = 127 - (5 if case["code"] == "int8" else 7)
    return torch.randint(e - 1, e + 2, shape, generator=gen, device="cuda", dtype=torch.uint8)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)

    def ints(a, dtype=torch.int32):
        return torch.from_numpy(np.asarray(a)).to(device=dev, dtype=dtype)

    def normal(*shape):
        return torch.empty(shape, dtype=DTYPES[case["dtype"]], device=dev).normal_(generator=gen)

    block, kv, dim = case["block"], case["kv_heads"], case["dim"]
    cached, fresh = (np.asarray(a) for a in _lengths(case))
    order = rng.permutation(len(cached))
    cached, fresh = cached[order], fresh[order]
    last = cached + fresh
    width = int(_blocks(int(last.max()), block))
    # the blocks that the case touches: an append's from the first new token's on
    first = cached // block if case["op"] == "append" else np.zeros_like(cached)
    held = -(-last // block)
    total = int((held - first).sum()) + 3
    pool = rng.permutation(total)
    table = np.full((len(cached), width), -1)
    at = 0
    for i in range(len(cached)):
        n = int(held[i] - first[i])
        table[i, first[i]:held[i]] = pool[at:at + n]
        at += n
    start = np.concatenate([[0], np.cumsum(fresh)])
    s = {"case": case, "table": ints(table), "kv_len": ints(last), "q_start": ints(start), "T": int(start[-1]),
         "k": _codes(case, (total, kv, block, dim), gen), "v": _codes(case, (total, kv, block, dim), gen),
         "k_exp": _exponents(case, (total, kv), gen), "v_exp": _exponents(case, (total, kv), gen)}
    if case["op"] == "append":
        req = np.repeat(np.arange(len(cached)), fresh)
        position = np.arange(s["T"]) - start[req] + cached[req]
        slot = table[req, position // block].astype(np.int64) * block + position % block
        f = 10000.0 ** (-np.arange(0, case["rot"], 2, dtype=np.float64) / case["rot"])
        # read back: all tokens of the blocks that were written
        back = np.concatenate([[0], np.cumsum(last - first * block)])
        s.update(qkv=normal(s["T"], (case["heads"] + 2 * kv) * dim), position=ints(position),
                 slot=ints(slot, torch.int64), freq=torch.from_numpy(f).to(dev), back=ints(back), rows=int(back[-1]))
    elif case["op"] == "read":
        back = np.concatenate([[0], np.cumsum(last)])
        s.update(back=ints(back), rows=int(back[-1]))
    else:
        s.update(q=normal(s["T"], case["heads"], dim), longest=int(last.max()), max_fresh=int(fresh.max()))
    if own:
        import weight_only_int4_group_gb300 as q4
        s["cache"] = q4.KVCache8(s["k"], s["v"], s["k_exp"], s["v_exp"], DTYPES[case["dtype"]])
        if case["op"] == "attention":
            s["ws"] = q4.attention_workspace(s["max_fresh"], case["heads"], kv, dim, eight_bit=True)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if own:
        return {"append": _append_own, "read": _read_own, "attention": _attention_own}[case["op"]](state, case)
    return {"append": _append_plain, "read": _read_plain, "attention": _attention_plain}[case["op"]](state, case)


def _append_own(s, case):
    import weight_only_int4_group_gb300 as q4
    q = q4.rope_append(s["qkv"], s["cache"], s["position"], s["slot"], s["freq"], heads=case["heads"],
                       interleaved=case["interleaved"])
    return [q, *q4.cache_read(s["cache"], s["table"], s["back"], s["kv_len"], s["rows"])]


def _read_own(s, case):
    import weight_only_int4_group_gb300 as q4
    return list(q4.cache_read(s["cache"], s["table"], s["back"], s["kv_len"], s["rows"]))


def _attention_own(s, case):
    import weight_only_int4_group_gb300 as q4
    return q4.attention(s["q"], s["cache"], s["table"], s["q_start"], s["kv_len"], s["max_fresh"],
                        window=case["window"], return_lse=case["lse"], ws=s["ws"])


def _bytes(codes):
    """The codes as a type that can be indexed."""
    return codes.view(torch.uint8)


def _numbers(raw, case):
    return raw.view(torch.int8 if case["code"] == "int8" else torch.float8_e4m3fn).float()


def _rounded(x, case):
    """Codes of x, which is in codes' units."""
    if case["code"] == "int8":
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _scale(e):
    return torch.ldexp(torch.ones((), device=e.device), e)


def _append_plain(s, case):
    h, kv, dim, rot, block = (case[k] for k in ("heads", "kv_heads", "dim", "rot", "block"))
    T = s["T"]
    x = s["qkv"].view(T, h + 2 * kv, dim)
    # whole turns leave in 64 bits: 32 lose the angles of far positions
    turns = s["position"].double()[:, None] * (s["freq"] / (2 * math.pi))
    angle = ((turns - turns.round()) * (2 * math.pi)).float()
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    qk = x[:, :h + kv, :rot].float()
    a, b = (qk[..., 0::2], qk[..., 1::2]) if case["interleaved"] else qk.split(rot // 2, dim=-1)
    a, b = a * cos - b * sin, a * sin + b * cos
    qk = torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1)
    qk = torch.cat([qk, x[:, :h + kv, rot:].float()], -1)
    blk, off = s["slot"] // block, s["slot"] % block
    _store_plain(s["k"], s["k_exp"], qk[:, h:], blk, off, case)
    _store_plain(s["v"], s["v_exp"], x[:, h + kv:].float(), blk, off, case)
    return [qk[:, :h].to(x.dtype), *_read_plain(s, case)]


def _store_plain(codes, exps, new, blk, off, case):
    """Quantise the rows ``new`` [T][kv][dim] into their blocks."""
    n, kv, block, _ = codes.shape
    lo, hi = RANGE[case["code"], case["dtype"]]
    peak = torch.zeros(n, kv, device=new.device).scatter_reduce_(0, blk[:, None].expand(-1, kv), new.abs().amax(-1), "amax")
    begin = torch.full((n,), block, device=new.device).scatter_reduce_(0, blk, off, "amin")
    m, e = torch.frexp(peak)  # peak = m 2^e, m in [1/2, 1)
    m0, e0 = math.frexp(MOST[case["code"]])
    need = torch.where(peak > 0, e - e0 + (m > m0), lo).clamp(lo, hi)
    old = exps.int() - 127
    e = torch.where((begin == 0)[:, None], need, torch.maximum(need, old))
    e = torch.where((begin == block)[:, None], old, e)  # blocks without a new token
    kept = _rounded(codes.float() * _scale(old - e)[:, :, None, None], case)
    codes.copy_(kept)
    exps.copy_((e + 127).to(torch.uint8))
    _bytes(codes)[blk, :, off] = _bytes(_rounded(new * _scale(-e[blk])[:, :, None], case))


def _read_plain(s, case):
    block, dtype = case["block"], DTYPES[case["dtype"]]
    back, kv_len = s["back"].long(), s["kv_len"].long()
    t = torch.arange(s["rows"], device=back.device)
    req = torch.searchsorted(back[1:], t, right=True)
    place = kv_len[req] - (back[req + 1] - t)
    blk, off = s["table"].long()[req, place // block], place % block
    return [(_numbers(_bytes(s[n])[blk, :, off], case) * _scale(s[n + "_exp"][blk].int() - 127)[:, :, None]).to(dtype)
            for n in ("k", "v")]


def _attention_plain(s, case):
    h, kv, dim, block = (case[k] for k in ("heads", "kv_heads", "dim", "block"))
    B, T, n, L, g = case["requests"], s["T"], s["max_fresh"], s["longest"], h // kv
    dev = s["q"].device
    start, kv_len = s["q_start"].long(), s["kv_len"].long()
    fresh = start[1:] - start[:-1]
    # the requests side by side, padded to the longest
    j, i = torch.arange(L, device=dev), torch.arange(n, device=dev)
    at = s["table"].long()[:, j // block].clamp(min=0)
    k, v = (_numbers(_bytes(s[x])[at, :, j % block], case).mul_(_scale(s[x + "_exp"][at].int() - 127)[..., None])
            for x in ("k", "v"))  # [B][L][kv][dim]
    q = s["q"][(start[:-1, None] + i).clamp(max=T - 1)].float()  # [B][n][h][dim]
    q = q.view(B, n, kv, g, dim).permute(0, 2, 3, 1, 4).reshape(B, kv, g * n, dim)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(dim ** -0.5).view(B, kv, g, n, L)
    pos = (kv_len - fresh)[:, None] + i  # a new token's place in its request
    hidden = (j > pos[..., None]) | (j >= kv_len[:, None, None])
    if case["window"]:
        hidden |= j <= pos[..., None] - case["window"]
    score.masked_fill_(hidden[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score.view(B, kv, g * n, L), v.transpose(1, 2)).view(B, kv, g, n, dim)
    o = torch.where(total > 0, o / total, 0.0)
    lse = torch.log(total) + top
    t = torch.arange(T, device=dev)
    req = torch.searchsorted(start[1:], t, right=True)
    row = t - start[req]
    o = o[req, :, :, row].reshape(T, h, dim).to(s["q"].dtype)
    return (o, lse[req, :, :, row].reshape(T, h)) if case["lse"] else o


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _append_exact, "read": _read_exact, "attention": _attention_exact}[case["op"]](s, case)


def _values(codes, exps):
    """All numbers that a cache stands for."""
    return codes.double() * torch.exp2(exps.double() - 127)[:, :, None, None]


def _nearest(x, case):
    """x in 64 bits to the nearest code, ties to the even one."""
    if case["code"] == "int8":
        return x.round().clamp(-127, 127)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return ((x / step).round() * step).clamp(-448, 448)


def _append_exact(s, case):
    """Each pair as a complex number times e^(i position frequency), and block by block the scale's rule."""
    h, kv, dim, rot, block = (case[k] for k in ("heads", "kv_heads", "dim", "rot", "block"))
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["position"].double()[:, None] * s["freq"])
    x = s["qkv"].double().view(s["T"], h + 2 * kv, dim)
    for head in range(h + kv):
        y = x[:, head, :rot]
        first = y[:, 0::2] if case["interleaved"] else y[:, :rot // 2]
        second = y[:, 1::2] if case["interleaved"] else y[:, rot // 2:]
        z = torch.complex(first.contiguous(), second.contiguous()) * turn
        if case["interleaved"]:
            y[:, 0::2], y[:, 1::2] = z.real, z.imag
        else:
            y[:, :rot // 2], y[:, rot // 2:] = z.real, z.imag
    lo, hi = RANGE[case["code"], case["dtype"]]
    held, slots = [], s["slot"].tolist()
    t0 = 0
    full = {n: _values(s[n], s[n + "_exp"]) for n in ("k", "v")}
    while t0 < len(slots):
        b, o = divmod(slots[t0], block)
        t1 = t0 + 1
        while t1 < len(slots) and slots[t1] == slots[t0] + t1 - t0 and o + t1 - t0 < block:
            t1 += 1
        held.append((b, o, t0, t1))
        t0 = t1
    for n, at in (("k", h), ("v", h + kv)):
        for b, o, t0, t1 in held:
            new = x[t0:t1, at:at + kv].transpose(0, 1)  # [kv][tokens][dim]
            peak = new.abs().amax((1, 2))
            e = torch.where(peak > 0, torch.ceil(torch.log2(peak / MOST[case["code"]])), lo).clamp(lo, hi)
            if o:
                e = torch.maximum(e, s[n + "_exp"][b].double() - 127)
            unit = torch.exp2(e)[:, None, None]
            full[n][b, :, :o] = _nearest(full[n][b, :, :o] / unit, case) * unit
            full[n][b, :, o:o + t1 - t0] = _nearest(new / unit, case) * unit
    return [x[:, :h].contiguous(), *_gathered(s, case, full)]


def _gathered(s, case, full):
    """The rows to be read, request by request."""
    block, back, out = case["block"], s["back"].tolist(), {"k": [], "v": []}
    for b, last in enumerate(s["kv_len"].tolist()):
        place = torch.arange(last - (back[b + 1] - back[b]), last, device="cuda")
        ids = s["table"][b].long()[place // block]
        for n in out:
            out[n].append(full[n][ids, :, place % block])
    return [torch.cat(out["k"]), torch.cat(out["v"])]


def _read_exact(s, case):
    return _gathered(s, case, {n: _values(s[n], s[n + "_exp"]) for n in ("k", "v")})


def _attention_exact(s, case):
    """Request by request and KV head by KV head, the definition."""
    h, kv, dim, block = (case[k] for k in ("heads", "kv_heads", "dim", "block"))
    g = h // kv
    start, kv_len = s["q_start"].tolist(), s["kv_len"].tolist()
    o = torch.zeros(s["T"], h, dim, dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], h), -math.inf, dtype=torch.float64, device="cuda")
    raw = {n: s[n].view(torch.uint8) for n in ("k", "v")}
    for b in range(case["requests"]):
        t0, t1, L = start[b], start[b + 1], kv_len[b]
        ids = s["table"][b, :_blocks(L, block)].long()
        key = torch.arange(L, device="cuda")
        place = torch.arange(L - (t1 - t0), L, device="cuda")[:, None]
        seen = key <= place
        if case["window"]:
            seen &= key > place - case["window"]
        for c in range(kv):
            k, v = (_values(raw[n][ids, c:c + 1].view(s[n].dtype), s[n + "_exp"][ids, c:c + 1]).reshape(-1, dim)[:L]
                    for n in ("k", "v"))
            for head in range(c * g, c * g + g):
                a = (s["q"][t0:t1, head].double() @ k.T) / math.sqrt(dim)
                a = torch.where(seen, a, -math.inf)
                lse[t0:t1, head] = torch.logsumexp(a, 1)
                o[t0:t1, head] = torch.softmax(a, 1) @ v
    return (o, lse) if case["lse"] else o


# ------------------------------------------------------------------ the floor
def work(case):
    """Bytes of each input read once and each output written once, and the
    products' operations; no path can do with less."""
    cached, fresh = _lengths(case)
    B, T, block = case["requests"], sum(fresh), case["block"]
    kv, dim, heads = case["kv_heads"], case["dim"], case["heads"]
    token = 2 * kv * dim  # codes of a token's keys and values, in bytes
    if case["op"] == "read":
        rows = sum(cached)
        blocks = sum(_blocks(c, block) for c in cached)
        return {"bytes": rows * 3 * token + blocks * (4 + 2 * kv) + 4 * (2 * B + 1), "flops": rows * token}
    if case["op"] == "append":
        old = sum(c % block for c in cached)  # held in the blocks that the new tokens enter
        blocks = sum(_blocks(c + n, block) - c // block for c, n in zip(cached, fresh))
        row = (heads + 2 * kv) * dim * 2
        # qkv in, q and codes out; then the written blocks' codes in, their values out
        return {"bytes": T * (row + 2 * heads * dim + token + 12) + 8 * (case["rot"] // 2) + 2 * blocks * kv
                + (T + old) * 3 * token + blocks * (4 + 2 * kv) + 4 * (2 * B + 1),
                "flops": T * (heads + kv) * case["rot"] * 3 + (2 * T + old) * token}
    pairs, keys = 0, 0
    for c, n in zip(cached, fresh):
        first = max(0, c + 1 - case["window"]) if case["window"] else 0
        keys += c + n - first
        if case["window"]:
            pairs += sum(min(c + i + 1, case["window"]) for i in range(n))
        else:
            pairs += n * c + n * (n + 1) // 2
    row = heads * dim
    blocks = sum(_blocks(c + n, block) for c, n in zip(cached, fresh))
    return {"bytes": 4 * T * row + keys * token + blocks * (4 + 2 * kv) + 4 * (2 * B + 1)
            + (4 * T * heads if case["lse"] else 0),
            "flops": 4 * pairs * row}
