"""The attention-side operators around the beam step, as measured cases.

A decoder that searches with this library runs, besides the search itself and
the cache's reorder, four operators per step or prompt:

  map    block tables and slot maps from request lengths
  write  K and V of new tokens into the 8-bit paged cache (e4m3 values, one
         power-of-two scale for each block of tokens and head)
  cache  attention of an item's beams over that cache: the prompt that the
         beams share, then each beam's own generated positions
  cross  attention of an item's rows to its encoder's states

``run`` computes them in plain torch, or, where ``own`` is true, through the
library. Sizes are the benchmark's (Transformer-base, Llama-3-8B-shaped, wide,
verify) or generic.
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
LIMIT = 448.0       # the largest e4m3 value
LOW_EXP = -100      # the smallest scale exponent

# handles by their configuration: a program makes them once, for any inputs
_handles = {}


def listed():
    return [
        # the slots of one more token for each of the 32 beams of the Llama-shaped search
        dict(name="map_step", op="map", n=32, mean=1, start=1100, block=16, empty=False),
        # block tables and slots of a large ragged batch of prompts that arrive at once
        dict(name="map_prompts", op="map", n=4096, mean=1000, start=0, block=16, empty=True),
        # a Llama-shaped decode step writes its 32 beams' new position, inside partly filled blocks
        dict(name="write_step", op="write", n=32, mean=1, start=100, block=16, heads=8, dim=128,
             dtype="bf16", empty=False),
        # eight ragged prompts around 1000 tokens enter the cache
        dict(name="write_prompts", op="write", n=8, mean=1000, start=0, block=16, heads=8, dim=128,
             dtype="bf16", empty=False),
        # one Llama-shaped decode step in the middle of the 200-step search, prompts around 1000
        dict(name="cache_llama", op="cache", batch=8, rows=4, q_len=1, heads=32, kv_heads=8, dim=128,
             block=16, prompt=1000, gen=100, dtype="bf16", empty=False),
        # the same search over long ragged documents
        dict(name="cache_long", op="cache", batch=8, rows=4, q_len=1, heads=32, kv_heads=8, dim=128,
             block=16, prompt=32000, gen=200, dtype="bf16", empty=False),
        # blockwise verify: 8 proposed positions of 64 ragged sequences, causal, no shared prompt
        dict(name="cache_verify", op="cache", batch=64, rows=1, q_len=8, heads=8, kv_heads=8, dim=64,
             block=16, prompt=0, gen=500, dtype="bf16", empty=False),
        # the wide search's step in fp32: 16 beams, 16 heads of 64, a short source as the prompt
        dict(name="cache_wide", op="cache", batch=16, rows=16, q_len=1, heads=16, kv_heads=16, dim=64,
             block=16, prompt=60, gen=128, dtype="f32", empty=False),
        # Transformer-base decode step in fp32: 4 beams look at a sentence of about 30 tokens
        dict(name="cross_tbase", op="cross", batch=32, rows=4, heads=8, kv_heads=8, dim=64, length=30,
             dtype="f32", mask=False, empty=False),
        # a decode step over long encoder states (audio frames) with padding given as a mask
        dict(name="cross_long", op="cross", batch=16, rows=4, heads=16, kv_heads=16, dim=64,
             length=1500, dtype="bf16", mask=True, empty=False),
        # the wide search's beams over a long fp32 source, one item with no source at all
        dict(name="cross_wide", op="cross", batch=16, rows=16, heads=16, kv_heads=16, dim=64,
             length=1000, dtype="f32", mask=False, empty=True),
        # scoring whole given targets: every target position at once, grouped heads
        dict(name="cross_score", op="cross", batch=8, rows=1024, heads=32, kv_heads=8, dim=128,
             length=2048, dtype="bf16", mask=False, empty=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["map", "write", "cache", "cross"])
    empty = rng.random() < 0.3
    if op == "map":
        n = _log(rng, 1, 4096)
        start = rng.choice([0, _log(rng, 1, 4000)])
        return dict(op=op, n=n, mean=_log(rng, 1, max(2, min(8000, 4000000 // n))), start=start,
                    block=rng.choice([8, 16, 24, 32, 64, 128]), empty=empty)
    heads, dim, dtype = rng.choice([1, 2, 3, 8, 16]), rng.choice([32, 64, 80, 96, 128, 256]), rng.choice(["f32", "bf16"])
    block = rng.choice([8, 16, 24, 32, 64])
    if op == "write":
        n, start = _log(rng, 1, 256), rng.choice([0, _log(rng, 1, 1000)])
        mean = 1 if rng.random() < 0.5 else _log(rng, 2, max(3, min(4000, 30000000 // (n * heads * dim))))
        return dict(op=op, n=n, mean=mean, start=start, block=block, heads=heads, dim=dim, dtype=dtype, empty=empty)
    group = rng.choice([1, 2, 4, 7])
    if op == "cache":
        batch, rows, q_len = _log(rng, 1, 64), rng.choice([1, 2, 4, 5, 16]), rng.choice([1, 1, 1, 3, 8])
        gen = _log(rng, 8, 1000 if rows * batch * heads * dim < 400000 else 100)
        prompt = rng.choice([0, _log(rng, 1, max(2, min(32000, 200000000 // (batch * heads * dim))))])
        return dict(op=op, batch=batch, rows=rows, q_len=q_len, heads=heads * group, kv_heads=heads, dim=dim,
                    block=block, prompt=prompt, gen=gen, dtype=dtype, empty=empty)
    batch = _log(rng, 1, 64)
    length = _log(rng, 1, max(2, min(16000, 100000000 // (batch * heads * dim))))
    rows = rng.choice([1, 4, 8, 16, _log(rng, 17, max(18, min(2048, 30000000000 // (batch * heads * group * dim * length))))])
    return dict(op=op, batch=batch, rows=rows, heads=heads * group, kv_heads=heads, dim=dim, length=length,
                dtype=dtype, mask=rng.random() < 0.4, empty=empty)


def _spread(n, mean, empty):
    """n ragged lengths around a mean, whose sum depends on nothing else; with ``empty`` they begin at 0."""
    if n == 1 or mean == 0 or (mean == 1 and not empty):
        return [mean] * n
    lo = 0 if empty else (mean + 1) // 2
    return [lo + round(2 * (mean - lo) * i / (n - 1)) for i in range(n)]


def _up(a, b):
    return -(-a // b)


def _blocks(case):
    """The lengths of a case and the block counts that follow from them, as the host knows them."""
    if case["op"] == "cache":
        prompt = _spread(case["batch"], case["prompt"], case["empty"])
        gen = _spread(case["batch"] * case["rows"], case["gen"], False)
        return prompt, [max(g, case["q_len"]) for g in gen]
    return _spread(case["n"], case["mean"], case["empty"]), _spread(case["n"], case["start"], case["empty"])


def work(case):
    op = case["op"]
    if op == "map":
        lens, starts = _blocks(case)
        mb = _up(max(lens) + max(starts), case["block"])
        new = sum(_up(a, case["block"]) for a in lens)
        return {"bytes": 4 * (2 * case["n"] * (2 if case["start"] else 1) + new + case["n"] * mb + sum(lens)),
                "flops": 2 * sum(lens)}
    e = 4 if case["dtype"] == "f32" else 2
    if op == "write":
        lens, _ = _blocks(case)
        row = case["heads"] * case["dim"] * 2
        return {"bytes": sum(lens) * (row * (e + 1) + 4) + sum(lens) * row * (e + 1), "flops": 6 * sum(lens) * row}
    if op == "cache":
        prompt, gen = _blocks(case)
        q = case["batch"] * case["rows"] * case["q_len"] * case["heads"] * case["dim"]
        seen = case["rows"] * sum(prompt) + sum(gen)
        return {"bytes": (sum(prompt) + sum(gen)) * case["kv_heads"] * case["dim"] * 2 + 2 * q * e,
                "flops": 4 * seen * case["q_len"] * case["heads"] * case["dim"]}
    lens = _spread(case["batch"], case["length"], case["empty"])
    q = case["batch"] * case["rows"] * case["heads"] * case["dim"]
    return {"bytes": sum(lens) * case["kv_heads"] * case["dim"] * 2 * e + 2 * q * e,
            "flops": 4 * case["rows"] * sum(lens) * case["heads"] * case["dim"]}


def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _shuffled(values, g):
    t = torch.tensor(values, dtype=torch.int32, device=DEVICE)
    return t[torch.randperm(len(values), generator=g, device=DEVICE)]


def _pool(n, block, heads, dim, g):
    """A filled 8-bit pool [n, block, heads, dim] (e4m3 bits) and its scales [n, heads]."""
    bits = torch.empty((n, block, heads, dim), dtype=torch.uint8, device=DEVICE)
    step = max(1, (1 << 26) // (block * heads * dim))
    for a in range(0, n, step):
        x = torch.randn((min(n, a + step) - a, block, heads, dim), generator=g, device=DEVICE) * 100
        bits[a:a + step] = x.clamp_(-LIMIT, LIMIT).to(torch.float8_e4m3fn).view(torch.uint8)
    e = torch.randint(-8, -5, (n, heads), generator=g, device=DEVICE, dtype=torch.int32)
    return bits, _two(e)


def _two(e):
    """2**e as float32, exactly, for whole e in -126..127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _table(counts, width, ids):
    """Rows of block ids: row r takes the next counts[r] of ``ids``, -1 behind them."""
    k = torch.arange(width, device=DEVICE)[None]
    base = (torch.cumsum(counts, 0) - counts)[:, None]
    return torch.where(k < counts[:, None], ids[(base + k).clamp_max(max(0, ids.numel() - 1))] if ids.numel() else -1, -1).to(torch.int32)


def _positions(first, count):
    """The rows and positions of ragged runs: run r covers first[r] .. first[r] + count[r] - 1."""
    row = torch.repeat_interleave(torch.arange(count.numel(), device=DEVICE), count)
    base = torch.cumsum(count, 0) - count
    return row, first[row] + torch.arange(row.numel(), device=DEVICE) - base[row]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "map":
        lens, starts = _blocks(case)
        mb = max(1, _up(max(lens) + max(starts), case["block"]))
        s["lens"] = _shuffled(lens, g)
        s["free"] = torch.randperm(max(1, sum(_up(a, case["block"]) for a in lens) + case["n"]), generator=g,
                                   device=DEVICE).to(torch.int32)
        s["starts"] = _shuffled(starts, g) if case["start"] else None
        s["table"] = torch.full((case["n"], mb), -1, dtype=torch.int32, device=DEVICE)
        if case["start"]:
            have = (s["starts"].long() + case["block"] - 1) // case["block"]
            total = sum(_up(a, case["block"]) for a in starts)
            s["table"] = _table(have, mb, torch.randperm(total, generator=g, device=DEVICE) + s["free"].numel())
        s["tokens"] = sum(lens) + 64    # the slot map's capacity; its end is padding
        if own:
            s["handle"] = _handle("map", case["n"], case["block"], mb, s["tokens"])
        return s
    dt = DTYPES[case["dtype"]]
    if op == "write":
        lens, starts = _blocks(case)
        bs, h, d = case["block"], case["heads"], case["dim"]
        ln, st = _shuffled(lens, g).long(), _shuffled(starts, g).long()
        first = st // bs                    # the first block that a row writes into
        count = torch.where(ln > 0, (st + ln + bs - 1) // bs - first, 0)
        n = sum(_up(a, bs) + 1 for a in lens)
        width = max(_up(a, bs) + 1 for a in lens)
        table = _table(count, width, torch.randperm(n, generator=g, device=DEVICE))
        row, pos = _positions(st, ln)
        s["slots"] = (table[row, pos // bs - first[row]].long() * bs + pos % bs).to(torch.int32)
        if case["n"] > 8 and case["mean"] == 1:
            s["slots"][3::8] = -1           # beams that have ended write nothing
        row, pos = _positions(first * bs, torch.where(ln > 0, st + ln - first * bs, 0))
        s["reads"] = (table[row, pos // bs - first[row]].long() * bs + pos % bs).to(torch.int32)
        for name in ("k", "v"):
            s[name + "_pool"], s[name + "_scale"] = _pool(n, bs, h, d, g)
            x = torch.randn((sum(lens), h, d), generator=g, device=DEVICE)
            x *= torch.exp(0.7 * torch.randn((sum(lens), h, 1), generator=g, device=DEVICE))
            s[name] = x.to(dt)
        if own:
            s["handle"] = _cache(s)
        return s
    d, hk, hq = case["dim"], case["kv_heads"], case["heads"]
    if op == "cache":
        bs, b, w = case["block"], case["batch"], case["rows"]
        prompt, gen = _blocks(case)
        s["prompt_lens"], s["lens"] = _shuffled(prompt, g), _shuffled(gen, g)
        pn, gn = [(t.long() + bs - 1) // bs for t in (s["prompt_lens"], s["lens"])]
        np_, ng = sum(_up(a, bs) for a in prompt), sum(_up(a, bs) for a in gen)
        ids = torch.randperm(np_ + ng, generator=g, device=DEVICE)
        s["prompt_table"] = _table(pn, max(1, _up(max(prompt), bs)), ids[:np_])
        s["table"] = _table(gn, _up(max(gen), bs), ids[np_:])
        for name in ("k", "v"):
            s[name + "_pool"], s[name + "_scale"] = _pool(np_ + ng, bs, hk, d, g)
        s["q"] = (1.5 * torch.randn((b * w * case["q_len"], hq, d), generator=g, device=DEVICE)).to(dt)
        if own:
            s["pool"] = _cache(s)
            s["handle"] = _handle("cache", b, w, case["q_len"], hq, hk, d, bs, s["table"].shape[1],
                                  s["prompt_table"].shape[1] if case["prompt"] else 0, case["dtype"])
        return s
    b, lens = case["batch"], _spread(case["batch"], case["length"], case["empty"])
    n = max(1, max(lens))
    s["lens"] = _shuffled(lens, g)
    s["k"] = torch.randn((b, n, hk, d), generator=g, device=DEVICE).to(dt)
    s["v"] = torch.randn((b, n, hk, d), generator=g, device=DEVICE).to(dt)
    s["q"] = (1.5 * torch.randn((b, case["rows"], hq, d), generator=g, device=DEVICE)).to(dt)
    s["mask"] = None
    if case["mask"]:
        s["mask"] = (torch.rand((b, n), generator=g, device=DEVICE) < 0.9).to(torch.uint8)
    if own:
        s["handle"] = _handle("cross", b, case["rows"], hq, hk, d, n, case["dtype"])
    return s


def _handle(op, *key):
    if (op, key) not in _handles:
        import beam_search_step_amd as bs
        if op == "map":
            n, block, mb, tokens = key
            h = bs.BlockMap(n, block, mb, tokens)
        elif op == "cache":
            b, w, q_len, hq, hk, d, block, mb, pmb, dtype = key
            h = bs.CacheAttention(b, w, hq, hk, d, block, mb, max_prompt_blocks=pmb, q_len=q_len, dtype=dtype)
        else:
            b, rows, hq, hk, d, n, dtype = key
            h = bs.CrossAttention(b, rows, hq, hk, d, n, dtype=dtype)
        _handles[op, key] = h
    return _handles[op, key]


def _cache(s):
    import beam_search_step_amd as bs
    return bs.QuantCache(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])


def run(s):
    op = s["case"]["op"]
    if own:
        if op == "map":
            table, slots, cu, used = s["handle"](s["lens"], s["free"], starts=s["starts"], table=s["table"])
            return {"table": table, "slots": slots, "cu": cu, "used": used}
        if op == "write":
            s["handle"].write(s["k"], s["v"], s["slots"])
            k, v = s["handle"].read(s["reads"], s["case"]["dtype"])
            return {"k": k, "v": v}
        if op == "cache":
            return s["handle"](s["q"], s["pool"], s["table"], s["lens"],
                               **(dict(prompt_table=s["prompt_table"], prompt_lens=s["prompt_lens"]) if s["case"]["prompt"] else {}))
        return s["handle"](s["q"], s["k"], s["v"], lens=s["lens"], mask=s["mask"])
    return {"map": _plain_map, "write": _plain_write, "cache": _plain_cache, "cross": _plain_cross}[op](s)


def _plain_map(s):
    bs, table, free = s["case"]["block"], s["table"], s["free"]
    n, mb = table.shape
    ln = s["lens"].long()
    st = s["starts"].long() if s["starts"] is not None else torch.zeros_like(ln)
    cu = torch.zeros(n + 1, dtype=torch.int64, device=ln.device)
    cu[1:] = torch.cumsum(ln, 0)
    have = (st + bs - 1) // bs
    want = ((st + ln + bs - 1) // bs).clamp_max(mb)
    new = (want - have).clamp_min(0)
    k = torch.arange(mb, device=ln.device)[None]
    at = (torch.cumsum(new, 0) - new - have)[:, None] + k
    fresh = torch.where((k < want[:, None]) & (at < free.numel()), free[at.clamp(0, free.numel() - 1)], -1)
    table = torch.where(k < have[:, None], table, fresh)
    i = torch.arange(s["tokens"], device=ln.device)
    r = torch.searchsorted(cu[1:], i, right=True).clamp_max(n - 1)
    p = st[r] + i - cu[r]
    b = table[r, (p // bs).clamp(0, mb - 1)].long()
    slots = torch.where((i < cu[-1]) & (p // bs < mb) & (b >= 0), b * bs + p % bs, -1)
    return {"table": table.to(torch.int32), "slots": slots.to(torch.int32), "cu": cu.to(torch.int32), "used": new.sum()[None].to(torch.int32)}


def _plain_store(pool, scale, x, slots):
    n, bs, h, d = pool.shape
    x, at = x.float()[slots >= 0], slots[slots >= 0].long()
    block, off = at // bs, at % bs
    amax = torch.zeros((n, h), device=x.device)
    amax.scatter_reduce_(0, block[:, None].expand(-1, h), x.abs().amax(-1), "amax")
    first = torch.full((n,), bs, device=x.device)
    first.scatter_reduce_(0, block, off, "amin")
    m, e = torch.frexp(amax / 512)          # amax = m * 2**(e + 9), m in [0.5, 1), and 448 = 0.875 * 2**9
    need = _two(torch.where(amax > 0, (e + (m > 0.875)).clamp_min(LOW_EXP), LOW_EXP))
    grown = torch.where((first == 0)[:, None], need, torch.maximum(scale, need))
    t = torch.nonzero(first < bs).squeeze(1)
    old = pool[t].view(torch.float8_e4m3fn).float() * (scale[t] / grown[t])[:, None, :, None]
    old = old.to(torch.float8_e4m3fn).view(torch.uint8)
    earlier = torch.arange(bs, device=x.device)[None] < first[t][:, None]
    pool[t] = torch.where(earlier[:, :, None, None], old, pool[t])
    scale[t] = grown[t]
    pool.view(n * bs, h, d)[at] = (x / scale[block][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(pool, scale, blocks):
    """The values that the blocks of a pool stand for, in 32 bits."""
    return pool[blocks].view(torch.float8_e4m3fn).float() * scale[blocks][..., None, :, None]


def _plain_write(s):
    out = {}
    at = s["reads"].long()
    for name in ("k", "v"):
        pool, scale = s[name + "_pool"], s[name + "_scale"]
        _plain_store(pool, scale, s[name], s["slots"])
        n, bs, h, d = pool.shape
        x = pool.view(n * bs, h, d)[at].view(torch.float8_e4m3fn).float() * scale[at // bs][:, :, None]
        out[name] = x.to(s[name].dtype)
    return out


def _softmax_values(score, seen, v):
    """softmax over the seen keys, times their values; zeros where nothing is seen."""
    score = torch.where(seen, score, -torch.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > -torch.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total > 0, total, 1.0)


def _plain_cache(s):
    c = s["case"]
    b, w, n, hk, d, bs = c["batch"], c["rows"], c["q_len"], c["kv_heads"], c["dim"], c["block"]
    grp = c["heads"] // hk
    dev = s["q"].device
    # queries of a row: [b, w, hk, n * grp, d]
    q = s["q"].float().view(b, w, n, hk, grp, d).permute(0, 1, 3, 2, 4, 5).reshape(b, w, hk, n * grp, d)
    keys = []
    for table, lens, per in ((s["prompt_table"], s["prompt_lens"], 1), (s["table"], s["lens"], w)):
        at = table.long().clamp_min(0)
        length = at.shape[1] * bs
        k, v = (_values(s[x + "_pool"], s[x + "_scale"], at).view(b, per, length, hk, d).transpose(2, 3).contiguous() for x in ("k", "v"))
        keys.append((k, v, lens.long().view(b, per, 1, 1, 1), torch.arange(length, device=dev)))
    (pk, pv, plen, pi), (k, v, ln, i) = keys
    # the prompt's keys are the same for all rows of an item
    flat = q.transpose(1, 2).reshape(b, hk, w * n * grp, d)
    ps = torch.matmul(flat, pk[:, 0].transpose(-1, -2)).view(b, hk, w, n * grp, -1).transpose(1, 2)
    score = torch.cat([ps, torch.matmul(q, k.transpose(-1, -2))], -1) / math.sqrt(d)
    back = (n - 1 - torch.arange(n, device=dev)).repeat_interleave(grp)[:, None]     # positions that a query may not see yet
    seen = torch.cat([(pi < plen).expand(b, w, hk, n * grp, -1), (i < ln - back).expand(b, w, hk, n * grp, -1)], -1)
    score = torch.where(seen, score, -torch.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > -torch.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p[..., pi.numel():], v)
    pp = p[..., : pi.numel()].transpose(1, 2).reshape(b, hk, w * n * grp, -1)
    o += torch.matmul(pp, pv[:, 0]).view(b, hk, w, n * grp, d).transpose(1, 2)
    o /= torch.where(total > 0, total, 1.0)
    return o.view(b, w, hk, n, grp, d).permute(0, 1, 3, 2, 4, 5).reshape(b * w * n, hk * grp, d).to(s["q"].dtype)


def _plain_cross(s):
    b, rows, hq, d = s["q"].shape
    n, hk = s["k"].shape[1:3]
    grp = hq // hk
    q = s["q"].float().view(b, rows, hk, grp, d).permute(0, 2, 1, 3, 4).reshape(b, hk, rows * grp, d)
    k, v = (s[x].float().transpose(1, 2).contiguous() for x in ("k", "v"))
    seen = torch.arange(n, device=q.device)[None] < s["lens"].long()[:, None]
    if s["mask"] is not None:
        seen = seen & (s["mask"] != 0)
    o = _softmax_values(torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d), seen[:, None, None], v)
    return o.view(b, hk, rows, grp, d).permute(0, 2, 1, 3, 4).reshape(b, rows, hq, d).to(s["q"].dtype)


# the same from the definitions, in 64 bits

def _e4m3(y):
    """The nearest value with 3 fraction bits and exponents from -6 on, ties to even."""
    size = y.abs()
    step = torch.exp2(torch.floor(torch.log2(torch.where(size > 0, size, 1.0))).clamp_min(-6) - 3)
    return torch.round(y / step) * step


def _decode(bits):
    """e4m3 bits as 64-bit values: sign, 4 exponent bits of bias 7, 3 fraction bits."""
    b = bits.to(torch.int64)
    e, f = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e > 0, (1 + f / 8) * torch.exp2((e - 7).double()), f / 8 * 2.0 ** -6)
    return torch.where(b >= 128, -v, v)


def _attend(q, k, v):
    """Attention of q [m, d] to k, v [n, d] in 64 bits."""
    if not k.shape[0]:
        return torch.zeros_like(q)
    p = torch.softmax(q @ k.T / q.shape[1] ** 0.5, -1)
    return p @ v


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "map":
        return None
    if op == "write":
        bs = case["block"]
        out = {}
        for name in ("k", "v"):
            x, old = s[name].double(), _decode(s[name + "_pool"]) * s[name + "_scale"].double()[:, None, :, None]
            n = old.shape[0]
            fresh = torch.full((n * bs,), -1, dtype=torch.int64, device=DEVICE)
            kept = s["slots"].long() >= 0
            fresh[s["slots"].long()[kept]] = torch.arange(x.shape[0], device=DEVICE)[kept]
            new = (fresh >= 0).view(n, bs)
            val = torch.where(new[:, :, None, None], x[fresh.clamp_min(0)].view(old.shape), old)
            amax = torch.where(new[:, :, None], val.abs().amax(-1), 0.0).amax(1)
            e = torch.where(amax > 0, torch.ceil(torch.log2(amax / LIMIT)), -torch.inf).clamp_min(LOW_EXP)
            scale = torch.exp2(e)
            from_start = new[:, 0]
            scale = torch.where(from_start[:, None], scale, torch.maximum(scale, s[name + "_scale"].double()))
            scale = torch.where(new.any(1)[:, None], scale, s[name + "_scale"].double())
            val = _e4m3(val / scale[:, None, :, None]) * scale[:, None, :, None]
            out[name] = val.view(n * bs, *val.shape[2:])[s["reads"].long()]
        return out
    grp, hk, q = case["heads"] // case["kv_heads"], case["kv_heads"], s["q"].double()
    out = torch.zeros_like(q)
    if op == "cross":
        if case["batch"] * hk > 600 and case["rows"] * case["length"] > 1 << 20:
            return None
        for b in range(case["batch"]):
            at = torch.arange(int(s["lens"][b]), device=DEVICE)
            if s["mask"] is not None:
                at = at[s["mask"][b, : at.numel()] != 0]
            k, v = s["k"][b, at].double(), s["v"][b, at].double()
            for h in range(hk):
                x = q[b, :, h * grp:(h + 1) * grp]
                out[b, :, h * grp:(h + 1) * grp] = _attend(x.reshape(-1, x.shape[-1]), k[:, h], v[:, h]).view(x.shape)
        return out
    bs, w, n = case["block"], case["rows"], case["q_len"]
    if case["batch"] * w * n * hk > 20000:
        return None

    def rows_of(table, length):
        t = table[: _up(length, bs)].long()
        return [(_decode(s[x + "_pool"][t]) * s[x + "_scale"][t].double()[:, None, :, None]).reshape(-1, hk, q.shape[-1])[:length] for x in ("k", "v")]

    for b in range(case["batch"]):
        pk, pv = rows_of(s["prompt_table"][b], int(s["prompt_lens"][b]))
        for r in range(b * w, (b + 1) * w):
            length = int(s["lens"][r])
            k, v = rows_of(s["table"][r], length)
            k, v = torch.cat([pk, k]), torch.cat([pv, v])
            for i in range(n):
                to = k.shape[0] - (n - 1 - i)
                x = q[r * n + i].view(hk, grp, -1)
                score = torch.matmul(x, k[:to].permute(1, 2, 0)) / x.shape[-1] ** 0.5
                out[r * n + i] = torch.matmul(torch.softmax(score, -1), v[:to].transpose(0, 1)).view(hk * grp, -1)
    return out
