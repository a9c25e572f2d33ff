"""Plain references of the attention-side operators, in Python and 64-bit torch
on the CPU, written from their definitions.

Tolerances count roundings. With u = 2^-23 for a rounding or a truncation of a
32-bit value to 24 bits, a score of D products summed in T terms is off by at
most (T D + 4) u times the sum S of its products' magnitudes, so a probability's
relative error is below 2 (T D + 4) u S (numerator and denominator); the sum over
n keys and its joins add (n + 64) u, the two-term probabilities of bf16 calls
2^-15 (where one bf16 term is used, with a sum of the same rounded terms: 2^-8 in
each of the two, 2^-7), all of them relative to A = sum p |v|. The output's own rounding adds
eps / 2 of its type relative to the value.

These are relative errors, and 32-bit numbers end at 2^-126: a probability below
it, a term of one, or a product p v, counts as zero in exp2 and in the matrix
instructions. Of a key's p (at most 1, the largest p being 1 and the sum of all at
least 1) at most 2^-126 is lost whole or 2 * 2^-126 in its lower terms, that is
3 * 2^-126 |v|, and of its up to three products at most 2^-126 each; n keys thus lose
below n 2^-124 (max |v| + 1), which is added as an absolute term.
"""
import math

import torch

U = 2.0 ** -23
LIMIT = 448.0
LOW_EXP = -100


def map_blocks(lens, starts, free, table, block, max_tokens):
    """(table, slots, cu, used) as Python lists."""
    table = [list(r) for r in table]
    mb = len(table[0])
    cu, slots, used = [0], [-1] * max_tokens, 0
    at = 0
    for b, ln in enumerate(lens):
        ln, st = max(ln, 0), max(starts[b], 0) if starts else 0
        have = min(-(-st // block), mb)
        want = max(min(-(-(st + ln) // block), mb), have)
        if free is not None:
            for k in range(have, mb):
                table[b][k] = free[at + k - have] if k < want and at + k - have < len(free) else -1
            at += want - have
            used += want - have
        for i in range(ln):
            p = st + i
            ident = table[b][p // block] if p // block < mb else -1
            if cu[-1] + i < max_tokens and ident >= 0 and ident * block + p % block < 2 ** 31:
                slots[cu[-1] + i] = ident * block + p % block
        cu.append(cu[-1] + ln)
    return table, slots, cu, used


def e4m3(y):
    """float64 values rounded to e4m3, ties to even; the values, not bits."""
    size = y.abs()
    step = torch.exp2(torch.floor(torch.log2(torch.where(size > 0, size, 1.0))).clamp_min(-6) - 3)
    return torch.round(y / step) * step


def decode(bits):
    b = bits.to(torch.int64)
    e, f = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e > 0, (1 + f / 8) * torch.exp2((e - 7).double()), f / 8 * 2.0 ** -6)
    v = torch.where((b & 127) == 127, torch.nan, v)
    return torch.where(b >= 128, -v, v)


def write(values, scale, x, slots):
    """Writes rows x [T, H, D] (float64) into the cache ``values`` [N, bs, H, D] with
    ``scale`` [N, H], both float64, in place: run by run, from the definition."""
    n, bs, h, _ = values.shape
    i = 0
    while i < len(slots):
        s = int(slots[i])
        if not 0 <= s < n * bs:
            i += 1
            continue
        blk, off = divmod(s, bs)
        run = 1
        while i + run < len(slots) and off + run < bs and int(slots[i + run]) == s + run:
            run += 1
        rows = x[i:i + run]
        ok = torch.isfinite(rows)
        amax = torch.where(ok, rows.abs(), 0.0).amax(-1).amax(0)
        for k in range(h):
            a = float(amax[k])
            e = LOW_EXP if a == 0 else max(LOW_EXP, math.ceil(math.log2(a / LIMIT)))
            while a > LIMIT * 2.0 ** e:
                e += 1
            while e > LOW_EXP and a <= LIMIT * 2.0 ** (e - 1):
                e -= 1
            sc = 2.0 ** e
            if off and float(scale[blk, k]) >= sc:
                sc = float(scale[blk, k])
            elif off:
                values[blk, :off, k] = e4m3(values[blk, :off, k] / sc) * sc
            # behind the new tokens the bytes stay, so their values follow the scale
            values[blk, off + run:, k] *= sc / float(scale[blk, k])
            scale[blk, k] = sc
            values[blk, off:off + run, k] = torch.where(ok[:, k], e4m3(torch.where(ok[:, k], rows[:, k], 0.0) / sc) * sc, torch.nan)
        i += run


def attend(q, k, v, seen, scale, dtype, terms, one_term=False):
    """(values, tolerance) of queries q [m, D] over keys k, v [n, D] with seen [m, n]
    (bool), all float64."""
    m, d = q.shape
    if not k.shape[0] or not bool(seen.any()):
        return torch.zeros(m, d, dtype=torch.float64), torch.zeros(m, d, dtype=torch.float64)
    any_key = seen.any(0)
    k = torch.where(any_key[:, None], k, 0.0)
    s = scale * (q @ k.T)
    mag = torch.where(seen, scale * (q.abs() @ k.abs().T), 0.0).amax(-1, keepdim=True)
    s = torch.where(seen, s, -torch.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top > -torch.inf, top, 0.0))
    tot = p.sum(-1, keepdim=True)
    p = p / torch.where(tot > 0, tot, 1.0)
    o = torch.stack([torch.where(seen[i][:, None], v, 0.0).mul(p[i][:, None]).sum(0) for i in range(m)]) \
        if bool(torch.isnan(v).any()) else p @ v
    a = p @ torch.nan_to_num(v).abs()
    half, extra = (2.0 ** -8, 2.0 ** -15) if dtype == "bf16" else (2.0 ** -24, 2.0 ** -23)
    extra = 2.0 ** -7 if one_term else extra
    rel = 2 * (terms * d + 4) * U * mag + (k.shape[0] + 64) * U + extra
    low = k.shape[0] * 2.0 ** -124 * (float(torch.nan_to_num(v, posinf=0, neginf=0).abs().max()) + 1)
    return o, half * o.abs() + rel * a * (1 + half) + low


def cache_attention(q, kv, vv, table, lens, ptable, plens, q_len, rows, scale, dtype):
    """(values, tolerance) [B*rows*q_len, Hq, D]; kv and vv the cache's values [N, bs,
    Hkv, D] in float64, the tables and lengths lists."""
    n, bs, hk, d = kv.shape
    hq = q.shape[1]
    grp = hq // hk
    o, tol = torch.zeros_like(q), torch.zeros_like(q)

    def gather(row, length):
        length = min(max(length, 0), len(row) * bs)
        at = [(row[p // bs], p % bs) for p in range(length)]
        ok = torch.tensor([0 <= b < n for b, _ in at], dtype=torch.bool)
        b = torch.tensor([b if 0 <= b < n else 0 for b, _ in at], dtype=torch.int64)
        p = torch.tensor([p for _, p in at], dtype=torch.int64)
        return kv[b, p], vv[b, p], ok

    for r in range(len(lens)):
        k, v, ok = gather(table[r], lens[r])
        own = k.shape[0]
        if ptable is not None:
            pk, pv, pok = gather(ptable[r // rows], plens[r // rows])
            k, v, ok = torch.cat([pk, k]), torch.cat([pv, v]), torch.cat([pok, ok])
        extra = k.shape[0] - own
        for i in range(q_len):
            seen = ok & (torch.arange(k.shape[0]) < extra + own - (q_len - 1) + i)
            seen = seen | (ok & (torch.arange(k.shape[0]) < extra))
            for h in range(hk):
                at = r * q_len + i, slice(h * grp, (h + 1) * grp)
                vals = torch.where(seen[:, None], v[:, h], 0.0)
                keys = torch.where(seen[:, None], k[:, h], 0.0)
                o[at], tol[at] = attend(q[at], keys, vals, seen.expand(grp, -1), scale, dtype,
                                        3 if dtype == "f32" else 1)
    return o, tol


def cross_attention(q, k, v, lens, mask, scale, dtype):
    # bf16 calls of more than 32 columns (rows * grouped heads; 16 for head sizes from 80
    # to 128) round probabilities to bf16
    """(values, tolerance) for q [B, R, Hq, D], k, v [B, S, Hkv, D] in float64."""
    b, rows, hq, d = q.shape
    hk = k.shape[2]
    grp = hq // hk
    o, tol = torch.zeros_like(q), torch.zeros_like(q)
    for i in range(b):
        at = torch.arange(k.shape[1])
        if lens is not None:
            at = at[: max(0, min(int(lens[i]), k.shape[1]))]
        if mask is not None:
            at = at[mask[i, at] != 0]
        for h in range(hk):
            sl = slice(h * grp, (h + 1) * grp)
            x = q[i, :, sl].reshape(-1, d)
            seen = torch.ones(x.shape[0], at.numel(), dtype=torch.bool)
            y, t = attend(x, k[i, at, h], v[i, at, h], seen, scale, dtype, 1,
                          dtype == "bf16" and rows * grp > (16 if 64 < d <= 128 else 32))
            o[i, :, sl], tol[i, :, sl] = y.view(rows, grp, d), t.view(rows, grp, d)
    return o, tol


def check(got, want, tol, what):
    got = got.detach().double().cpu()
    bad = torch.isnan(got) != torch.isnan(want)
    assert not bool(bad.any()), f"{what}: NaN in other places: {torch.nonzero(bad)[:4].tolist()}"
    off = (got - want).abs()
    inf = torch.isinf(want)
    off = torch.where(torch.isnan(want) | (inf & (got == want)), 0.0, off)
    over = off > tol
    worst = float((off / tol.clamp_min(1e-300))[~torch.isnan(off)].max()) if off.numel() else 0.0
    assert not bool(over.any()), (f"{what}: {int(over.sum())} of {off.numel()} outside, worst {worst:.3g} "
                                  f"tolerances, first at {torch.nonzero(over)[0].tolist()}: "
                                  f"{got[over][:3].tolist()}, not {want[over][:3].tolist()}")
