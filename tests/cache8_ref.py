"""Plain 64-bit references of the 8-bit cache's operators and their inputs.

Tolerance of a quantised key: the rotation is f32, y = x cos + p sin of the pair
(x, p).  The angle is off by 2^-24 of a turn (2^-21.3 rad) at any position, sine
and cosine by 2^-22 of 1, their product with the factor and the two products and
the sum by 2^-24 each: together under 2^-20 (|x| + |p|) factor, and that is at
most 2^-19 of the largest magnitude of the run (a pair keeps its length, so
|x| + |p| <= 2 max |y|, but for the factor, which scales all).  Quantising adds
half a step."""
from __future__ import annotations

import math

import numpy as np
import torch

from serving_ref import attention_reference, rope_reference  # noqa: F401

MOST = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
RANGE = {(torch.int8, torch.float16): (-24, 9), (torch.float8_e4m3fn, torch.float16): (-15, 7),
         (torch.int8, torch.bfloat16): (-48, 48), (torch.float8_e4m3fn, torch.bfloat16): (-48, 48)}
CODES = [torch.int8, torch.float8_e4m3fn]


def exponents(exp, code, dtype):
    """The exponents that the bytes stand for."""
    lo, hi = RANGE[code, dtype]
    return (exp.long() - 127).clamp(lo, hi)


def numbers(codes):
    return codes.float().double()


def values(codes, exp, dtype):
    """[blocks][heads][S][D] in 64 bits."""
    e = exponents(exp, codes.dtype, dtype).double()
    return numbers(codes) * torch.exp2(e)[:, :, None, None]


def half_step(y, code):
    """Half the distance of the codes around y (|y| within the codes)."""
    if code == torch.int8:
        return torch.full_like(y, 0.5)
    return torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 4)


def nearest(y, code):
    """y in the scale's units to the nearest code, ties to even (64 bits)."""
    step = 2 * half_step(y.clamp(-MOST[code], MOST[code]), code)
    return (torch.round(y / step) * step).clamp(-MOST[code], MOST[code])


def needed(peak, code, dtype):
    lo, hi = RANGE[code, dtype]
    if not peak > 0:
        return lo
    e = math.ceil(math.log2(peak / MOST[code]))
    while peak <= MOST[code] * 2.0 ** (e - 1):
        e -= 1
    while peak > MOST[code] * 2.0 ** e:
        e += 1
    return min(max(e, lo), hi)


def runs(slot, S, slots):
    """(first row, rows) of the runs, and of single rows without a slot none."""
    out, t = [], 0
    slot = slot.tolist()
    while t < len(slot):
        n = 1
        if 0 <= slot[t] < slots:
            while t + n < len(slot) and slot[t + n] == slot[t] + n and (slot[t] + n) % S:
                n += 1
            out.append((t, n))
        t += n
    return out


def check_append(before, after, x, slot, dtype, rel):
    """One kind (keys or values).  before, after: (codes, exps) clones; x [T][heads][D]
    in 64 bits, known to rel of its run's largest magnitude.  Everything outside the
    runs stays; scales follow the rule; codes held are rounded again exactly; the
    new ones are nearest."""
    (c0, e0), (c1, e1) = before, after
    code, S = c0.dtype, c0.shape[2]
    lo, hi = RANGE[code, dtype]
    want_c, want_e = numbers(c0), e0.clone()
    known = torch.ones(c0.shape[:3], dtype=torch.bool, device=c0.device)
    got = numbers(c1)
    for t, n in runs(slot, S, c0.shape[0] * S):
        b, o = divmod(int(slot[t]), S)
        for h in range(c0.shape[1]):
            y = x[t:t + n, h]
            fin = torch.where(torch.isfinite(y), y.abs(), 0.0)
            peak = float(fin.max())
            old = int(exponents(e0[b, h], code, dtype)) if o else lo
            e = int(e1[b, h]) - 127
            assert max(old, needed(peak * (1 - rel), code, dtype)) <= e <= max(old, needed(peak * (1 + rel), code, dtype)), \
                f"run at row {t}, head {h}: exponent {e}, peak {peak}, before {old}"
            want_e[b, h] = e + 127
            if o:
                want_c[b, h, :o] = nearest(want_c[b, h, :o] * 2.0 ** (old - e), code)
            known[b, h, o:o + n] = False
            z = torch.nan_to_num(y * 2.0 ** -e, nan=0.0)
            clamped = z.clamp(-MOST[code], MOST[code])
            new = got[b, h, o:o + n]
            if rel == 0:
                assert torch.equal(new, nearest(z, code)), f"run at row {t}, head {h}"
            else:
                off = peak * 2.0 ** -e * rel
                assert ((new - clamped).abs() <= half_step(clamped.abs() + off, code) + off).all(), f"run at row {t}, head {h}"
    assert torch.equal(want_e, e1), "exponents outside the runs"
    # bits of what was not written: NaN codes among it stay as they are
    same = (got == want_c) | (torch.isnan(got) & torch.isnan(want_c))
    assert same[known].all(), "codes outside the runs, or codes held"


def random_cache(blocks, heads, S, D, code, gen, spread=36.0, exps=(-7, -3), token_major=False, device="cuda"):
    """(k, v, k_exp, v_exp) of normal codes."""
    def codes():
        x = torch.randn(blocks, S, heads, D, generator=gen) if token_major else torch.randn(blocks, heads, S, D, generator=gen)
        x = (x * spread).clamp(-127, 127)
        x = (x.round().to(torch.int8) if code == torch.int8 else x.to(code)).to(device)
        return x.transpose(1, 2) if token_major else x

    def e():
        return torch.randint(exps[0] + 127, exps[1] + 128, (blocks, heads), generator=gen, dtype=torch.uint8).to(device)
    return codes(), codes(), e(), e()


def raw(codes):
    """Bytes of codes, in place (float8 tensors cannot be indexed)."""
    return codes.view(torch.uint8)


class Requests8:
    """Requests of given (cached, fresh) lengths over a shuffled 8-bit cache.
    Codes of no request and behind a request's end are garbage (-128, or e4m3's
    NaN), their exponents' bytes 255; table entries past the last block are out of
    range."""

    def __init__(self, lengths, heads, kv_heads, D, S, dtype, code, seed=0, spare=3, token_major=False,
                 width_extra=2, q_scale=1.0, exps=(-7, -3), device="cuda"):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.lengths, self.dtype = lengths, dtype
        total = [c + n for c, n in lengths]
        nb = [-(-L // S) for L in total]
        blocks = sum(nb) + spare
        pool = rng.permutation(blocks)
        table = np.full((len(lengths), max(max(nb) + width_extra, 1)), 2 ** 31 - 1)
        self.k, self.v, self.k_exp, self.v_exp = random_cache(blocks, kv_heads, S, D, code, g, exps=exps,
                                                              token_major=token_major, device=device)
        junk = 0x80 if code == torch.int8 else 0x7F
        at = 0
        for b, L in enumerate(total):
            ids = pool[at:at + nb[b]]
            table[b, :nb[b]] = ids
            at += nb[b]
            if L % S:
                for x in (self.k, self.v):
                    raw(x)[int(ids[-1]), :, L % S:] = junk
        rest = torch.from_numpy(pool[at:].copy()).to(device)
        for x in (self.k, self.v):
            raw(x)[rest] = junk
        for x in (self.k_exp, self.v_exp):
            x[rest] = 255
        start = np.concatenate([[0], np.cumsum([n for _, n in lengths])])
        self.T = int(start[-1])
        self.q = (torch.randn(max(self.T, 1), heads, D, generator=g) * q_scale).to(dtype).to(device)
        self.start, self.total = start.tolist(), total
        self.table = torch.from_numpy(table.astype(np.int32)).to(device)
        self.q_start = torch.from_numpy(start.astype(np.int32)).to(device)
        self.kv_len = torch.tensor(total, dtype=torch.int32, device=device)
        self.max_fresh = max(1, max(n for _, n in lengths))

    def cache(self):
        import weight_only_int4_group_gb300 as q4
        return q4.KVCache8(self.k, self.v, self.k_exp, self.v_exp, self.dtype)

    def values(self):
        return values(self.k, self.k_exp, self.dtype), values(self.v, self.v_exp, self.dtype)

    def reference(self, scale=None, window=0):
        scale = self.q.shape[2] ** -0.5 if scale is None else scale
        return attention_reference(self.q, *self.values(), self.table, self.start, self.total, scale, window)

