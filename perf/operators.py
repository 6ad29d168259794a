"""The serving operators around the W4A16 products, as a decoder's attention
block runs them: a step's plan over a blocked KV cache, the rotary positions
with the cache append, and the attention of each request's new tokens over
everything it has in the cache.

Each case is run through the library's calls (``own``) or through plain torch
operations in 32 bits.  Shapes are those of the two layers this repository
benchmarks (64 query heads on 8 KV heads of 128: qkv 10240x8192; 32 heads of
128: qkv 12288x4096) and small generic ones.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
GQA = {"heads": 64, "kv_heads": 8, "dim": 128}  # the 70B-shaped layer
MHA = {"heads": 32, "kv_heads": 32, "dim": 128}  # the 7B-shaped layer


# ------------------------------------------------------------------ cases
def _plan(name, requests, cached, fresh, block):
    return {"name": name, "op": "plan", "requests": requests, "cached_lo": cached[0],
            "cached_hi": cached[1], "fresh_lo": fresh[0], "fresh_hi": fresh[1], "block": block}


def _rope(name, tokens, model, rot, interleaved, scaled, reach, block, dtype):
    return {"name": name, "op": "rope", "tokens": tokens, **model, "rot": rot,
            "interleaved": interleaved, "scaled": scaled, "reach": reach, "block": block,
            "dtype": dtype}


def _attention(name, requests, cached, fresh, model, block, dtype, window=0, lse=False):
    return {"name": name, "op": "attention", "requests": requests, "cached_lo": cached[0],
            "cached_hi": cached[1], "fresh_lo": fresh[0], "fresh_hi": fresh[1], **model,
            "block": block, "dtype": dtype, "window": window, "lse": lse}


def listed():
    return [
        # a few users decoding: one new token each, once per step
        _plan("plan 8 decoding", 8, (3, 2000), (1, 1), 16),
        # a full server: a thousand requests, prompt chunks among the decodes
        _plan("plan 1024 ragged", 1024, (0, 8000), (1, 31), 16),
        # the smallest decode step, half of each head rotated in pairs
        _rope("rope 4 tokens", 4, MHA, 64, True, False, 4096, 16, "f16"),
        # a prompt chunk of odd length
        _rope("rope 1001 tokens", 1001, MHA, 128, False, False, 8192, 16, "f16"),
        # a large prefill step with positions scaled for a long context
        _rope("rope 8192 tokens scaled", 8192, GQA, 128, False, True, 131072, 64, "bf16"),
        # one user decoding: latency
        _attention("attention 1 decoding", 1, (776, 776), (1, 1), MHA, 16, "f16"),
        # an ordinary decode batch of ragged lengths
        _attention("attention 32 decoding", 32, (100, 8191), (1, 1), GQA, 16, "bf16"),
        # a long-context decode batch: the cache is gigabytes
        _attention("attention 48 decoding long", 48, (1000, 24575), (1, 1), GQA, 64, "bf16"),
        # a few drafted tokens per request, a small model with a sliding window
        _attention("attention 16 drafted window", 16, (10, 6000), (4, 4),
                   {"heads": 16, "kv_heads": 4, "dim": 64}, 32, "f16", window=1024, lse=True),
        # one chunk of a long prompt
        _attention("attention chunk 512 after 16384", 1, (16384, 16384), (512, 512), GQA, 16, "bf16"),
        # a whole prompt at once
        _attention("attention prompt 4096", 1, (0, 0), (4096, 4096), MHA, 16, "f16"),
        # continuous batching: prompt chunks and decodes in one step
        _attention("attention mixed", 12, (50, 4000), (1, 160), GQA, 16, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "rope", "attention", "attention", "attention", "attention"])
    block = rng.choice([16, 32, 64])
    dtype = rng.choice(["bf16", "f16"])
    if op == "plan":
        lo = rng.randint(0, 200)
        return _unnamed(_plan("", _log_int(rng, 1, 1024), (lo, lo + _log_int(rng, 1, 7800)),
                              (1, _log_int(rng, 1, 31)), block))
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 128])
        kv = rng.choice([1, 4, 8])
        model = {"heads": kv * rng.choice([1, 4, 7, 8]), "kv_heads": kv, "dim": dim}
        return _unnamed(_rope("", _log_int(rng, 1, 8192), model, rng.choice([dim, dim // 2]),
                              rng.random() < 0.5, rng.random() < 0.5,
                              rng.choice([2048, 8192, 131072]), block, dtype))
    kv = rng.choice([1, 2, 4, 8])
    model = {"heads": kv * rng.choice([1, 2, 4, 7, 8]), "kv_heads": kv,
             "dim": rng.choice([64, 80, 96, 128, 128])}
    window = rng.choice([0, 0, 0, _log_int(rng, 1, 4096)])
    kind = rng.choice(["decode", "decode", "draft", "chunk", "prompt"])
    if kind == "decode":
        lo = _log_int(rng, 1, 2000)
        sizes = (_log_int(rng, 1, 48), (lo, lo + _log_int(rng, 1, 20000)), (1, 1))
    elif kind == "draft":
        lo = _log_int(rng, 1, 2000)
        sizes = (_log_int(rng, 1, 32), (lo, lo + _log_int(rng, 1, 6000)), (1, rng.randint(2, 8)))
    elif kind == "chunk":
        lo = rng.randint(0, 500)
        sizes = (rng.randint(1, 12), (lo, lo + _log_int(rng, 1, 4000)), (1, _log_int(rng, 16, 160)))
    else:
        n = _log_int(rng, 100, 2048)
        sizes = (1, (0, 0) if rng.random() < 0.5 else (777, 777), (n, n))
    return _unnamed(_attention("", *sizes, model, block, dtype, window, rng.random() < 0.25))


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
def _frequencies(rot, scaled):
    """Radians per position of each rotated pair (64 bits) and the factor on
    cos and sin; ``scaled`` stretches a 4096-token model by 32 by parts: pairs
    that turn less than once over its length are slowed by 32, those that turn
    over 32 times kept, a ramp between."""
    base, stretch, length = 10000.0, 32.0, 4096.0
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if not scaled:
        return f, 1.0
    turns = length * f / (2 * math.pi)
    keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
    return f / stretch * (1 - keep) + f * keep, 0.1 * math.log(stretch) + 1.0


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)

    def ints(a, dtype=torch.int32):
        return torch.from_numpy(np.asarray(a)).to(device=dev, dtype=dtype)

    def normal(*shape):
        return torch.empty(shape, dtype=DTYPES[case["dtype"]], device=dev).normal_(generator=gen)

    block = case["block"]
    if case["op"] == "rope":
        T, kv, dim = case["tokens"], case["kv_heads"], case["dim"]
        nb = _blocks(T, block) + 2
        freq, factor = _frequencies(case["rot"], case["scaled"])
        s = {"qkv": normal(T, (case["heads"] + 2 * kv) * dim),
             "k": normal(nb, kv, block, dim), "v": normal(nb, kv, block, dim),
             "position": ints(rng.integers(0, case["reach"], T)),
             "slot": ints(rng.permutation(nb * block)[:T], torch.int64),
             "freq": torch.from_numpy(freq).to(dev), "factor": factor}
    else:
        cached, fresh = (np.asarray(a) for a in _lengths(case))
        order = rng.permutation(len(cached))
        cached, fresh = cached[order], fresh[order]
        last = cached + fresh
        width = int(_blocks(int(last.max()), block))
        start = np.concatenate([[0], np.cumsum(fresh)])
        s = {"T": int(start[-1])}
        held = -(-(cached if case["op"] == "plan" else last) // block)
        total = int((-(-last // block)).sum()) + 100
        pool = rng.permutation(total)
        table = np.full((len(cached), width), -1)
        at = 0
        for i, n in enumerate(held):
            table[i, :n] = pool[at:at + n]
            at += n
        s["table"] = ints(table)
        if case["op"] == "plan":
            s.update(cached=ints(cached), fresh=ints(fresh), free=ints(pool[at:]),
                     free_count=ints([total - at]))
        else:
            kv, dim = case["kv_heads"], case["dim"]
            s.update(q=normal(s["T"], case["heads"], dim), k=normal(total, kv, block, dim),
                     v=normal(total, kv, block, dim), q_start=ints(start), kv_len=ints(last),
                     longest=int(last.max()), max_fresh=int(fresh.max()))
    if own and case["op"] != "plan":
        import weight_only_int4_group_gb300 as q4
        s["cache"] = q4.KVCache(s["k"], s["v"])
        if case["op"] == "attention":
            s["ws"] = q4.attention_workspace(s["max_fresh"], case["heads"], case["kv_heads"], case["dim"])
    s["case"] = case
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if own:
        return {"plan": _plan_own, "rope": _rope_own, "attention": _attention_own}[case["op"]](state, case)
    return {"plan": _plan_plain, "rope": _rope_plain, "attention": _attention_plain}[case["op"]](state, case)


def _plan_own(s, case):
    import weight_only_int4_group_gb300 as q4
    p = q4.cache_plan(s["cached"], s["fresh"], s["table"], s["free"], s["free_count"], case["block"], s["T"])
    return [s["table"], p.q_start, p.kv_len, p.position, p.slot, p.counts]


def _plan_plain(s, case):
    block, T = case["block"], s["T"]
    cached, fresh, table, free = (s[k].long() for k in ("cached", "fresh", "table", "free"))
    last = cached + fresh
    have, need = (cached + block - 1) // block, (last + block - 1) // block
    taken = torch.cumsum(need - have, 0)
    served = ((need == have) | (taken <= s["free_count"])) & (need <= table.shape[1])
    first = taken - (need - have)
    q_start = torch.nn.functional.pad(torch.cumsum(fresh, 0), (1, 0))
    j = torch.arange(table.shape[1], device=table.device)
    new = (j >= have[:, None]) & (j < need[:, None]) & served[:, None]
    at = s["free_count"] - 1 - (first[:, None] + j - have[:, None])
    table = torch.where(new, free[at.clamp(0, free.numel() - 1)], table)
    t = torch.arange(T, device=table.device)
    req = torch.searchsorted(q_start[1:], t, right=True)
    pos = cached[req] + t - q_start[req]
    slot = torch.where(served[req], table[req, pos // block] * block + pos % block, -1)
    kv_len = torch.where(served, last, 0)
    used = torch.where(served, need - have, 0).sum()
    counts = torch.stack([q_start[-1], torch.where(served, fresh, 0).sum(), s["free_count"][0] - used,
                          (~served).sum()])
    return [table.int(), q_start.int(), kv_len.int(), pos.int(), slot, counts.int()]


def _rope_own(s, case):
    import weight_only_int4_group_gb300 as q4
    q = q4.rope_append(s["qkv"], s["cache"], s["position"], s["slot"], s["freq"], heads=case["heads"],
                       interleaved=case["interleaved"], factor=s["factor"])
    return [q, s["k"], s["v"]]


def _rope_plain(s, case):
    h, kv, dim, rot, block = (case[k] for k in ("heads", "kv_heads", "dim", "rot", "block"))
    T = case["tokens"]
    x = s["qkv"].view(T, h + 2 * kv, dim)
    angle = s["position"].float()[:, None] * s["freq"].float()
    cos = (torch.cos(angle) * s["factor"])[:, None]
    sin = (torch.sin(angle) * s["factor"])[:, None]
    qk = x[:, :h + kv, :rot].float()
    a, b = (qk[..., 0::2], qk[..., 1::2]) if case["interleaved"] else qk.split(rot // 2, dim=-1)
    a, b = a * cos - b * sin, a * sin + b * cos
    qk = torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1)
    qk = torch.cat([qk.to(x.dtype), x[:, :h + kv, rot:]], -1)
    at, off = s["slot"] // block, s["slot"] % block
    s["k"][at, :, off] = qk[:, h:]
    s["v"][at, :, off] = x[:, h + kv:]
    return [qk[:, :h].contiguous(), s["k"], s["v"]]


def _attention_own(s, case):
    import weight_only_int4_group_gb300 as q4
    return q4.attention(s["q"], s["cache"], s["table"], s["q_start"], s["kv_len"], s["max_fresh"],
                        window=case["window"], return_lse=case["lse"], ws=s["ws"])


def _attention_plain(s, case):
    h, kv, dim, block = (case[k] for k in ("heads", "kv_heads", "dim", "block"))
    B, T, n, L, g = case["requests"], s["T"], s["max_fresh"], s["longest"], h // kv
    dev = s["q"].device
    start, kv_len = s["q_start"].long(), s["kv_len"].long()
    fresh = start[1:] - start[:-1]
    # the requests side by side, padded to the longest
    j, i = torch.arange(L, device=dev), torch.arange(n, device=dev)
    at = s["table"].long()[:, j // block].clamp(min=0)
    k = s["k"][at, :, j % block].float()  # [B][L][kv][dim]
    v = s["v"][at, :, j % block].float()
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
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    return _rope_exact(s, case) if case["op"] == "rope" else _attention_exact(s, case)


def _rope_exact(s, case):
    """Each pair as a complex number times factor * e^(i position frequency)."""
    h, kv, dim, rot, block = (case[k] for k in ("heads", "kv_heads", "dim", "rot", "block"))
    turn = torch.polar(torch.full((), s["factor"], dtype=torch.float64, device="cuda"),
                       s["position"].double()[:, None] * s["freq"])
    x = s["qkv"].double().view(case["tokens"], h + 2 * kv, dim)
    for head in range(h + kv):
        y = x[:, head, :rot]
        first = y[:, 0::2] if case["interleaved"] else y[:, :rot // 2]
        second = y[:, 1::2] if case["interleaved"] else y[:, rot // 2:]
        z = torch.complex(first.contiguous(), second.contiguous()) * turn
        if case["interleaved"]:
            y[:, 0::2], y[:, 1::2] = z.real, z.imag
        else:
            y[:, :rot // 2], y[:, rot // 2:] = z.real, z.imag
    k, v = s["k"].double(), s["v"].double()
    for head in range(kv):
        k[s["slot"] // block, head, s["slot"] % block] = x[:, h + head]
        v[s["slot"] // block, head, s["slot"] % block] = x[:, h + kv + head]
    return [x[:, :h].contiguous(), k, v]


def _attention_exact(s, case):
    """Request by request and KV head by KV head, the definition."""
    h, kv, dim, block = (case[k] for k in ("heads", "kv_heads", "dim", "block"))
    g = h // kv
    start, kv_len = s["q_start"].tolist(), s["kv_len"].tolist()
    o = torch.zeros(s["T"], h, dim, dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], h), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(case["requests"]):
        t0, t1, L = start[b], start[b + 1], kv_len[b]
        ids = s["table"][b, :_blocks(L, block)].long()
        key = torch.arange(L, device="cuda")
        place = torch.arange(L - (t1 - t0), L, device="cuda")[:, None]
        seen = key <= place
        if case["window"]:
            seen &= key > place - case["window"]
        for c in range(kv):
            k = s["k"][ids, c].reshape(-1, dim)[:L].double()
            v = s["v"][ids, c].reshape(-1, dim)[:L].double()
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
    if case["op"] == "rope":
        row = (case["heads"] + 2 * case["kv_heads"]) * case["dim"] * 2
        turned = (case["heads"] + case["kv_heads"]) * case["rot"]
        return {"bytes": case["tokens"] * (2 * row + 12) + 8 * (case["rot"] // 2),
                "flops": case["tokens"] * turned * 3}
    cached, fresh = _lengths(case)
    B, T, block = case["requests"], sum(fresh), case["block"]
    if case["op"] == "plan":
        new = sum(_blocks(c + n, block) - _blocks(c, block) for c, n in zip(cached, fresh))
        old = sum(1 for c in cached if c % block)
        return {"bytes": 8 * B + 4 * old + 8 * new + 4 * (2 * B + 1) + 12 * T + 20, "flops": 0}
    pairs, keys = 0, 0
    for c, n in zip(cached, fresh):
        first = max(0, c + 1 - case["window"]) if case["window"] else 0
        keys += c + n - first
        if case["window"]:
            pairs += sum(min(c + i + 1, case["window"]) for i in range(n))
        else:
            pairs += n * c + n * (n + 1) // 2
    row = case["heads"] * case["dim"]
    return {"bytes": 2 * (2 * T * row + 2 * keys * case["kv_heads"] * case["dim"])
            + 4 * sum(_blocks(c + n, block) for c, n in zip(cached, fresh)) + 4 * (2 * B + 1)
            + (4 * T * case["heads"] if case["lse"] else 0),
            "flops": 4 * pairs * row}
