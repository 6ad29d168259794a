"""Plain 64-bit references of the serving operators and their inputs (CPU or
GPU tensors; loops over requests and heads, nothing shared with the library).

Tolerance of an attention output, derived from what the kernels round: the
weights p = exp(s - max) are rounded once to the cache's type (relative error
u: 2^-8 bf16, 2^-11 f16), everything else is f32.  With A = sum p |v| / sum p,
    |o - o_ref| <= (u + e) A + u |o_ref|,   e = 2 (exp(2 d) - 1) + 2^-16
where d bounds the error of a score: head_dim f32 additions of products whose
magnitudes sum to at most S = max_j sum_d |q_d k_jd| * scale, each off by at
most 2^-22 of that; the last term is the output's own rounding (none for f32
outputs), and 2^-16 covers the exponentials (2^-21) and the f32 sums.  The
log-sum-exp is within d + 2^-18 (1 + |lse| + |max s|)."""
from __future__ import annotations

import math

import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 0.0}


def plan_reference(cached, fresh, table, free_blocks, free_count, S, T):
    """The plan in Python integers: dict of arrays."""
    B, W = table.shape
    table = table.copy()
    avail = max(0, min(int(free_count), len(free_blocks)))
    q_start, kv_len, served_tokens, unserved, taken, used, run = [], [], 0, 0, 0, 0, 0
    position, slot = np.zeros(T, np.int64), np.full(T, -1, np.int64)
    for b in range(B):
        c, f = int(cached[b]), int(fresh[b])
        bad = c < 0 or f < 0
        n = 0 if bad else f
        fits = not bad and c + f <= W * S
        have, need = -(-max(c, 0) // S), -(-max(c + f, 0) // S)
        nb = need - have if fits else 0
        served = fits and run + n <= T and (nb == 0 or taken + nb <= avail)
        q_start.append(min(run, T))
        kv_len.append(c + f if served else 0)
        if served:
            for j in range(have, need):
                table[b, j] = free_blocks[avail - 1 - (taken + j - have)]
            used += nb
            served_tokens += n
        else:
            unserved += 1
        for i in range(n):
            if run + i >= T:
                break
            p = c + i
            if served:
                position[run + i] = p
            if served and table[b, p // S] >= 0:
                slot[run + i] = int(table[b, p // S]) * S + p % S
        run += n
        taken += nb
    q_start.append(min(run, T))
    return {"table": table, "q_start": q_start, "kv_len": kv_len, "position": position, "slot": slot,
            "counts": [q_start[-1], served_tokens, avail - used, unserved]}


def rope_reference(x, position, freq, rot, interleaved, factor):
    """x [T][heads][D] (any float type) rotated, in 64 bits."""
    y = x.double().clone()
    angle = position.double()[:, None, None] * freq.double()
    cos, sin = torch.cos(angle) * factor, torch.sin(angle) * factor
    if interleaved:
        a, b = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        h = rot // 2
        a, b = y[..., :h].clone(), y[..., h:rot].clone()
        y[..., :h], y[..., h:rot] = a * cos - b * sin, a * sin + b * cos
    return y


def attention_reference(q, k, v, table, q_start, kv_len, scale, window):
    """(o, lse, tolerance of o before output rounding, tolerance of lse), all
    64 bits.  k, v: [blocks][heads][S][D]."""
    T, H, D = q.shape
    Hkv, S = k.shape[1], k.shape[2]
    G = H // Hkv
    u = U[q.dtype]
    o = torch.zeros(T, H, D, dtype=torch.float64, device=q.device)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=q.device)
    tol, ltol = torch.zeros_like(o), torch.zeros_like(lse)
    for b, L in enumerate(kv_len):
        t0, t1 = q_start[b], q_start[b + 1]
        n = t1 - t0
        if n == 0 or L == 0:
            continue
        ids = table[b, :-(-L // S)].long()
        j = torch.arange(L, device=q.device)
        place = torch.arange(L - n, L, device=q.device)[:, None]
        seen = j <= place
        if window:
            seen &= j > place - window
        some = seen.any(1)
        for c in range(Hkv):
            kk = k[ids, c].reshape(-1, D)[:L].double()
            vv = v[ids, c].reshape(-1, D)[:L].double()
            for h in range(c * G, (c + 1) * G):
                qq = q[t0:t1, h].double()
                s = torch.where(seen, qq @ kk.T * scale, -math.inf)
                mag = torch.where(seen, qq.abs() @ kk.abs().T * abs(scale), 0.0).amax(1)
                top = torch.where(some, s.amax(1), 0.0)
                p = torch.exp(s - top[:, None])
                z = p.sum(1)
                z1 = torch.where(some, z, 1.0)[:, None]
                o[t0:t1, h] = p @ vv / z1
                lse[t0:t1, h] = torch.where(some, torch.log(z) + top, -math.inf)
                d = D * 2.0 ** -22 * mag
                e = 2 * torch.expm1(2 * d) + 2.0 ** -16
                tol[t0:t1, h] = (u + e)[:, None] * (p @ vv.abs()) / z1
                ltol[t0:t1, h] = d + 2.0 ** -18 * (1 + torch.where(some, lse[t0:t1, h], 0.0).abs() + top.abs())
    return o, lse, tol, ltol


def assert_attention(got, lse, ref, where=""):
    o, l, tol, ltol = ref
    allow = tol + U[got.dtype] * o.abs() + 2.0 ** -24  # the smallest f16 step rounds by 2^-25
    err = (got.double() - o).abs()
    assert not torch.isnan(err).any(), f"{where}: NaN"
    worst = float((err / allow).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"{where}: error {worst:.3g} of the tolerance"
    if lse is not None:
        assert torch.equal(torch.isinf(lse), torch.isinf(l)), f"{where}: empty rows"
        fin = ~torch.isinf(l)
        lw = ((lse.double() - l)[fin].abs() / ltol[fin])
        assert lw.numel() == 0 or float(lw.max()) <= 1.0, f"{where}: lse {float(lw.max()):.3g}"


class Requests:
    """Requests of given (cached, fresh) lengths over a shuffled cache.  Cache
    entries that belong to no request, and those behind a request's end, are
    NaN; table entries past the last block are out of range."""

    def __init__(self, lengths, heads, kv_heads, D, S, dtype, seed=0, spare=3, token_major=False,
                 width_extra=2, q_scale=1.0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.lengths = lengths
        total = [c + n for c, n in lengths]
        nb = [-(-L // S) for L in total]
        blocks = sum(nb) + spare
        pool = rng.permutation(blocks)
        W = max(nb) + width_extra
        table = np.full((len(lengths), max(W, 1)), 2 ** 31 - 1)
        k = torch.full((blocks, kv_heads, S, D), math.nan)
        v = torch.full((blocks, kv_heads, S, D), math.nan)
        at = 0
        for b, L in enumerate(total):
            ids = pool[at:at + nb[b]]
            table[b, :nb[b]] = ids
            at += nb[b]
            for j, i in enumerate(ids):
                m = min(S, L - j * S)
                k[i, :, :m] = torch.randn(kv_heads, m, D, generator=g)
                v[i, :, :m] = torch.randn(kv_heads, m, D, generator=g)
        k, v = k.to(dtype), v.to(dtype)
        if token_major:
            k = k.transpose(1, 2).contiguous().to(device).transpose(1, 2)
            v = v.transpose(1, 2).contiguous().to(device).transpose(1, 2)
        self.k, self.v = k.to(device), v.to(device)
        start = np.concatenate([[0], np.cumsum([n for _, n in lengths])])
        self.T = int(start[-1])
        self.q = (torch.randn(max(self.T, 1), heads, D, generator=g) * q_scale).to(dtype).to(device)
        self.start, self.total = start.tolist(), total
        self.table = torch.from_numpy(table.astype(np.int32)).to(device)
        self.q_start = torch.from_numpy(start.astype(np.int32)).to(device)
        self.kv_len = torch.tensor(total, dtype=torch.int32, device=device)
        self.max_fresh = max(1, max(n for _, n in lengths))

    def reference(self, scale=None, window=0):
        scale = self.q.shape[2] ** -0.5 if scale is None else scale
        return attention_reference(self.q, self.k, self.v, self.table, self.start, self.total, scale, window)
