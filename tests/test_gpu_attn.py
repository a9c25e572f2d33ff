"""The attention-side operators on an MI355X against plain 64-bit references
(tests/attn_ref.py, where the tolerances are derived)."""
import math
import os
import random

import pytest

import attn_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dev():
    import beam_search_step_amd as bs
    bs.attn_library()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    torch.cuda.set_device(0)
    # an earlier test's CPU timing leaves the process on one core, where a pool of
    # threads for the references would only wait for itself
    threads = torch.get_num_threads()
    torch.set_num_threads(min(threads, len(os.sched_getaffinity(0))))
    yield torch.device("cuda", 0)
    torch.set_num_threads(threads)


DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def say(*a):
    print(*a, flush=True)


# --- block tables and slot maps ---------------------------------------------

@pytest.mark.parametrize("n,block,mean,start,short,seed", [
    (1, 16, 1, 0, 0, 0), (1, 1, 5, 0, 0, 1), (3, 16, 40, 0, 0, 2), (7, 24, 100, 50, 0, 3),
    (32, 16, 1, 130, 0, 4), (513, 8, 30, 0, 0, 5), (1025, 16, 3, 70, 0, 6), (5, 128, 3000, 0, 0, 7),
    (40, 16, 60, 20, 25, 8), (9, 3, 17, 5, 0, 9),
])
def test_map_blocks(dev, n, block, mean, start, short, seed):
    import beam_search_step_amd as bs
    rng = random.Random(seed)
    lens = [rng.choice([0, rng.randint(0, 2 * mean), mean, -3]) for _ in range(n)]
    starts = [rng.choice([0, rng.randint(0, 2 * start), -1]) for _ in range(n)] if start else None
    mb = max(1, -(-(2 * mean + 2 * start) // block) - (1 if n > 20 else 0))  # some rows do not fit
    free = rng.sample(range(10 * n * mb), n * mb)
    if short:
        free = free[:short]                                # the list runs out
    table = [[rng.randint(-1, 5) for _ in range(mb)] for _ in range(n)]
    total = sum(max(0, x) for x in lens)
    for cap in (total + 37, max(0, total - 3)):
        say("map", n, block, mean, start, cap)
        m = bs.BlockMap(n, block, mb, cap)
        t = i32(table, dev)
        got = m(i32(lens, dev), i32(free, dev), starts=None if starts is None else i32(starts, dev),
                table=t)
        want = ref.map_blocks(lens, starts, free, table, block, cap)
        for g, w, what in zip(got, want, ("table", "slots", "cu")):
            assert g.tolist() == w, what
        assert got[3].tolist() == [want[3]]
        # without a free list the table is read only
        t = i32(table, dev)
        got = m(i32(lens, dev), starts=None if starts is None else i32(starts, dev), table=t)
        want = ref.map_blocks(lens, starts, None, table, block, cap)
        assert t.tolist() == table and got[1].tolist() == want[1] and got[2].tolist() == want[2]
        assert got[3].tolist() == [0]


def test_map_blocks_with_an_empty_free_list(dev):
    import beam_search_step_amd as bs
    m = bs.BlockMap(3, 4, 2, 8)
    table, slots, cu, used = m(i32([2, 0, 5], dev), torch.empty(0, dtype=torch.int32, device=dev))
    assert table.tolist() == [[-1, -1]] * 3 and slots.tolist() == [-1] * 8
    assert cu.tolist() == [0, 2, 2, 7] and used.tolist() == [3]


# --- the 8-bit cache ----------------------------------------------------------

def make_cache(dev, n, block, heads, dim, seed, pad=0):
    """A QuantCache of random content and the same as float64 values and scales."""
    import beam_search_step_amd as bs
    g = torch.Generator().manual_seed(seed)
    parts, vals, scales = [], [], []
    for _ in range(2):
        bits = torch.randint(0, 256, (n, block, heads, dim), generator=g, dtype=torch.uint8)
        bits[(bits & 127) == 127] = 0x35
        sc = torch.exp2(torch.randint(-9, 0, (n, heads), generator=g).float())
        full = torch.zeros((n, block + pad, heads, dim + 0), dtype=torch.uint8, device=dev)
        pool = full[:, :block]
        pool.copy_(bits)
        parts.append((pool, sc.to(dev)))
        vals.append(ref.decode(bits) * sc.double()[:, None, :, None])
        scales.append(sc.double())
    (k, ks), (v, vs) = parts
    return bs.QuantCache(k, v, ks, vs), vals, scales


def assert_cache(cache, vals, scales, what):
    for pool, sc, v, s in ((cache.k, cache.k_scale, vals[0], scales[0]),
                           (cache.v, cache.v_scale, vals[1], scales[1])):
        assert torch.equal(sc.double().cpu(), s), f"{what}: scales"
        got = ref.decode(pool.cpu().view(torch.uint8)) * s[:, None, :, None]
        off = torch.nonzero(~((got == v) | (torch.isnan(got) & torch.isnan(v))))
        first = [(i, float(got[tuple(i)]), float(v[tuple(i)]), float(s[i[0], i[2]])) for i in off[:4].tolist()]
        assert not len(off), f"{what}: {len(off)} values differ: {first}"


def rows_of(n, heads, dim, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, heads, dim), generator=g)
    x = x * torch.exp(2 * torch.randn((n, heads, 1), generator=g))
    return x.to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block,heads,dim,pad", [
    (16, 2, 128, 0), (16, 3, 64, 2), (1, 2, 32, 0), (24, 1, 80, 0), (128, 2, 16, 1), (8, 5, 256, 0),
    (70, 1, 48, 0),
])
def test_write(dev, dtype, block, heads, dim, pad):
    n = 12
    say("write", dtype, block, heads, dim)
    cache, vals, scales = make_cache(dev, n, block, heads, dim, 3, pad)
    rng = random.Random(block * dim)
    ids = rng.sample(range(n), n)
    # a run over several blocks, a run inside a block, single tokens, skips
    slots = [ids[0] * block + p for p in range(block)] + [ids[1] * block + p for p in range(max(1, block // 2))]
    slots += [-1, n * block, n * block + 5]
    if block > 2:
        slots += [ids[2] * block + p for p in range(block // 3, block - 1)]
        slots += [ids[3] * block + block - 1, ids[4] * block, ids[5] * block + 1]
    slots += [-7]
    x = [rows_of(len(slots), heads, dim, dtype, 5 + i) for i in range(2)]
    for step in range(2):
        if step and block > 2:  # later positions of some blocks, small and large
            slots = [ids[5] * block + 2, ids[1] * block + block // 2]
            x = [rows_of(2, heads, dim, dtype, 9 + i) * (64.0 if step else 1) for i in range(2)]
        cache.write(x[0].to(dev), x[1].to(dev), i32(slots, dev))
        for i in range(2):
            ref.write(vals[i], scales[i], x[i].double(), slots)
        torch.cuda.synchronize()
        assert_cache(cache, vals, scales, f"step {step}")
    if pad:  # what lies between the blocks is left alone
        full = torch.as_strided(cache.k, (n, block + pad, heads, dim),
                                (cache.k.stride(0), cache.k.stride(1), dim, 1))
        assert int(full[:, block:].sum()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_write_long_lists_and_strided_rows(dev, dtype):
    """Chunks of 64 tokens: runs that cross them, blocks of 100 and of 16 positions."""
    import beam_search_step_amd as bs
    for block, tokens in ((16, 3001), (100, 2050)):
        heads, dim, n = 4, 64, tokens // block + 2
        cache, vals, scales = make_cache(dev, n, block, heads, dim, 4)
        perm = random.Random(7).sample(range(n), n)
        slots = [perm[i // block] * block + i % block for i in range(tokens)]
        slots[500] = slots[1100] = -1
        qkv = rows_of(tokens, 3 * heads, dim, dtype, 11).to(dev)
        say("write", dtype, block, tokens)
        cache.write(qkv[:, heads:2 * heads], qkv[:, 2 * heads:], i32(slots, dev))
        ref.write(vals[0], scales[0], qkv[:, heads:2 * heads].double().cpu(), slots)
        ref.write(vals[1], scales[1], qkv[:, 2 * heads:].double().cpu(), slots)
        assert_cache(cache, vals, scales, f"block {block}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_write_edges(dev, dtype):
    """Zeros, amax at and just above 448 * 2^e, infinities and NaN, tiny and huge values,
    growth that rounds earlier subnormals."""
    block, heads, dim = 8, 1, 16
    cache, vals, scales = make_cache(dev, 10, block, heads, dim, 8)
    up = float(torch.nextafter(torch.tensor(448.0), torch.tensor(1e9))) if dtype == "f32" else 450.0
    rows = [[0.0] * 16, [448.0] + [1.0] * 15, [up] + [1.0] * 15, [math.inf, -math.inf, math.nan, 3.0] + [0.01] * 12,
            [1e-36] * 16, [3e38, -1e30] + [0.0] * 14, [math.nan] * 16, [-0.0, 2.0 ** -9 * 1.5] + [0.4375] * 14]
    x = torch.tensor(rows).view(8, 1, 16).to(DT[dtype])
    slots = [i * block for i in range(8)]
    for step in range(2):
        say("edges", dtype, step)
        cache.write(x.to(dev), x.flip(0).contiguous().to(dev), i32(slots, dev))
        ref.write(vals[0], scales[0], x.double(), slots)
        ref.write(vals[1], scales[1], x.flip(0).double(), slots)
        assert_cache(cache, vals, scales, f"step {step}")
        slots = [i * block + 1 for i in range(8)]
        x = x.roll(3, 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_read(dev, dtype):
    cache, vals, _ = make_cache(dev, 9, 12, 3, 48, 2)
    slots = [0, 107, 108, -1, 5, 5, 60, 2 ** 31 - 1, -2 ** 31]
    k, v = cache.read(i32(slots, dev), dtype)
    for got, val in ((k, vals[0]), (v, vals[1])):
        flat = val.view(9 * 12, 3, 48)
        want = torch.stack([flat[s] if 0 <= s < 108 else torch.zeros(3, 48, dtype=torch.float64) for s in slots])
        assert torch.equal(got.double().cpu(), want)
    k, v = cache.read(i32([], dev), dtype)
    assert k.shape == (0, 3, 48)


# --- attention over the 8-bit cache -----------------------------------------

def cache_case(dev, batch, rows, q_len, heads, kv_heads, dim, block, prompt, gen, dtype, seed,
               holes=False, scale=None, nan_behind=False):
    import beam_search_step_amd as bs
    rng = random.Random(seed)
    plens = [rng.choice([prompt, rng.randint(0, prompt), 0]) for _ in range(batch)] if prompt else None
    lens = [rng.choice([gen, rng.randint(0, gen), max(0, gen - 1)]) for _ in range(batch * rows)]
    lens[0] = gen
    if batch * rows > 2:
        lens[2] = 0
    mb, pmb = -(-gen // block) + 1, (-(-prompt // block) if prompt else 0)
    n = batch * rows * mb + batch * pmb
    cache, vals, _ = make_cache(dev, n, block, kv_heads, dim, seed)
    ids = rng.sample(range(n), n)
    table = [[ids.pop() for _ in range(mb)] for _ in range(batch * rows)]
    ptable = [[ids.pop() for _ in range(pmb)] for _ in range(batch)] if prompt else None
    if holes:  # entries that are no blocks
        table[0][0] = -1
        table[-1][-1] = n + 3
        if ptable:
            ptable[0][pmb // 2] = -5
    if nan_behind:  # positions past the lengths hold NaN
        for t, ls in ((table, lens), (ptable or [], plens or [])):
            for row, ln in zip(t, ls):
                for p in range(ln, len(row) * block):
                    if 0 <= row[p // block] < n:
                        for pool in (cache.k, cache.v):
                            pool[row[p // block], p % block] = 0x7f
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn((batch * rows * q_len, heads, dim), generator=g) * 0.3).to(DT[dtype])
    scale = dim ** -0.5 if scale is None else scale
    say("cache", batch, rows, q_len, heads, kv_heads, dim, block, prompt, gen, dtype)
    att = bs.CacheAttention(batch, rows, heads, kv_heads, dim, block, mb, pmb, q_len, dtype, scale)
    kw = dict(prompt_table=i32(ptable, dev), prompt_lens=i32(plens, dev)) if prompt else {}
    out = att(q.to(dev), cache, i32(table, dev), i32(lens, dev), **kw)
    want, tol = ref.cache_attention(q.double(), *vals, table, lens, ptable, plens, q_len, rows, scale, dtype)
    ref.check(out, want, tol, "cache attention")
    if batch * rows > 2 and not prompt:
        assert not out[2 * q_len:3 * q_len].any()     # nothing seen: zeros
    return att


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", [
    (2, 4, 1, 8, 2, 128, 16, 100, 20), (3, 2, 1, 4, 4, 64, 16, 0, 70), (1, 1, 1, 1, 1, 16, 16, 0, 1),
    (2, 3, 1, 6, 2, 80, 24, 50, 33), (2, 2, 1, 2, 1, 256, 8, 40, 17), (1, 16, 1, 2, 2, 64, 32, 300, 40),
    (2, 5, 1, 14, 2, 96, 1, 37, 9), (4, 1, 8, 2, 2, 64, 16, 0, 130), (2, 3, 5, 4, 1, 32, 16, 20, 31),
    (1, 2, 64, 2, 1, 64, 7, 9, 100), (1, 1, 1, 16, 1, 48, 100, 0, 1500), (2, 1, 3, 7, 1, 112, 16, 700, 5),
    (1, 16, 1, 8, 2, 128, 16, 520, 30), (1, 8, 8, 4, 4, 128, 16, 130, 40),
])
def test_cache_attention(dev, case, dtype):
    cache_case(dev, *case, dtype, seed=sum(case))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", [
    (2, 3, 1, 2, 2, 128, 16, 90, 200), (1, 1, 1, 1, 1, 96, 32, 0, 1300), (2, 1, 1, 3, 3, 48, 16, 30, 65),
    (1, 1, 1, 2, 2, 128, 16, 33, 600), (4, 64, 1, 8, 8, 64, 16, 40, 20), (4, 64, 1, 16, 8, 64, 16, 17, 70),
    (2, 128, 2, 8, 8, 128, 16, 0, 35), (2, 128, 1, 8, 8, 112, 16, 33, 40), (32, 1, 1, 8, 8, 64, 16, 0, 300),
    (32, 1, 1, 16, 8, 128, 16, 0, 270), (32, 1, 1, 8, 8, 128, 32, 0, 333), (32, 1, 3, 8, 8, 80, 16, 0, 290),
])
def test_cache_attention_of_one_column_and_of_many_units(dev, case, dtype):
    cache_case(dev, *case, dtype, seed=sum(case))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [16, 5])
def test_cache_attention_skips_bad_entries_and_what_lies_behind(dev, dtype, block):
    cache_case(dev, 2, 2, 1, 4, 2, 64, block, 90, 50, dtype, 77, holes=True, nan_behind=True)
    cache_case(dev, 2, 1, 4, 4, 2, 64, block, 0, 50, dtype, 78, holes=True, nan_behind=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cache_attention_nan_under_a_causal_mask(dev, dtype):
    """A NaN value at a verified position reaches the queries that see it, and no others."""
    import beam_search_step_amd as bs
    q_len, block, dim, gen = 6, 16, 64, 45
    cache, vals, _ = make_cache(dev, 3, block, 1, dim, 5)
    pos = gen - 3                                   # seen by the last three queries
    cache.v[pos // block, pos % block, 0, 7] = 0x7f
    vals[1][pos // block, pos % block, 0, 7] = math.nan
    cache.k[(gen - 1) // block, (gen - 1) % block, 0, 3] = 0x7f   # its score: the last query's alone
    vals[0][(gen - 1) // block, (gen - 1) % block, 0, 3] = math.nan
    q = torch.randn((q_len, 2, dim), generator=torch.Generator().manual_seed(3)).to(DT[dtype])
    att = bs.CacheAttention(1, 1, 2, 1, dim, block, 3, q_len=q_len, dtype=dtype)
    out = att(q.to(dev), cache, i32([[0, 1, 2]], dev), i32([gen], dev))
    want, tol = ref.cache_attention(q.double(), *vals, [[0, 1, 2]], [gen], None, None, q_len, 1,
                                    dim ** -0.5, dtype)
    assert torch.isnan(want[5]).all() and not torch.isnan(want[:3]).any()
    assert torch.isnan(want[3, 0]).sum() == 1
    ref.check(out, want, tol, "causal NaN")


@pytest.mark.parametrize("scale", [1e-3, 3.0])
def test_cache_attention_scale(dev, scale):
    cache_case(dev, 2, 2, 1, 4, 2, 64, 16, 60, 40, "f32", 5, scale=scale)


# --- cross attention -----------------------------------------------------------

def cross_case(dev, batch, rows, heads, kv_heads, dim, keys, dtype, seed, lens="ragged", mask=False,
               layout="bshd", max_rows=None, max_keys=None):
    import beam_search_step_amd as bs
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((batch, rows, heads, dim), generator=g)).to(DT[dtype])
    k, v = [torch.randn((batch, keys, kv_heads, dim), generator=g).to(DT[dtype]) for _ in range(2)]
    ln = None
    if lens == "ragged":
        ln = [rng.choice([keys, rng.randint(0, keys)]) for _ in range(batch)]
        ln[0] = keys
        if batch > 1:
            ln[1] = 0
    mk = (torch.rand((batch, keys), generator=g) < 0.6).to(torch.uint8) if mask else None
    if mask and batch > 2:
        mk[2] = 0                                 # a mask that leaves nothing
    kd, vd = k.clone(), v.clone()                 # what is not seen holds NaN and infinities
    for b in range(batch):
        bad = torch.zeros(keys, dtype=torch.bool)
        if ln is not None:
            bad[ln[b]:] = True
        if mk is not None:
            bad |= mk[b] == 0
        kd[b, bad] = math.nan
        vd[b, bad] = math.inf
    if layout == "bhsd":
        kd, vd = [x.transpose(1, 2).contiguous().to(dev).transpose(1, 2) for x in (kd, vd)]
    else:
        kd, vd = kd.to(dev), vd.to(dev)
    say("cross", batch, rows, heads, kv_heads, dim, keys, dtype, lens, mask, layout)
    att = bs.CrossAttention(batch, max_rows or rows, heads, kv_heads, dim, max_keys or max(keys, 1), dtype)
    out = att(q.to(dev), kd, vd, lens=None if ln is None else i32(ln, dev),
              mask=None if mk is None else mk.to(dev))
    want, tol = ref.cross_attention(q.double(), k.double(), v.double(), ln, mk, dim ** -0.5, dtype)
    ref.check(out, want, tol, "cross attention")
    return att, out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", [
    (2, 4, 8, 8, 64, 30), (1, 1, 1, 1, 16, 1), (3, 16, 4, 4, 64, 129), (2, 5, 6, 2, 80, 77),
    (2, 1, 4, 1, 256, 300), (1, 40, 2, 2, 128, 260), (2, 33, 14, 2, 96, 50), (1, 200, 2, 1, 64, 513),
    (1, 3, 2, 2, 128, 3001), (2, 130, 4, 2, 128, 333), (1, 70, 3, 3, 32, 64), (1, 257, 1, 1, 112, 96),
])
def test_cross_attention(dev, case, dtype):
    cross_case(dev, *case, dtype, seed=sum(case))


@pytest.mark.parametrize("case", [(32, 130, 8, 8, 64, 270), (16, 300, 8, 8, 128, 131), (32, 70, 16, 8, 80, 33)])
@pytest.mark.parametrize("mask", [False, True])
def test_cross_attention_of_many_rows_and_items(dev, case, mask):
    cross_case(dev, *case, "bf16", seed=sum(case), mask=mask)


@pytest.mark.parametrize("rows", [70, 600])
def test_cross_attention_rising_scores(dev, rows):
    """Scores that rise and fall by hundreds along the keys: the point that they are
    taken from has to follow."""
    import beam_search_step_amd as bs
    g = torch.Generator().manual_seed(rows)
    q, k, v = [torch.randn(s, generator=g) for s in ((1, rows, 2, 64), (1, 700, 2, 64), (1, 700, 2, 64))]
    k[0, :, :, 0] = torch.linspace(-40, 40, 700)[:, None] * torch.tensor([1.0, -1.0])
    k[0, 300:340, :, 0] = 60.0
    q[..., 0] = 40.0
    q[:, ::3, :, 0] = 0.0
    q, k, v = [x.to(torch.bfloat16) for x in (q, k, v)]
    say("rising", rows)
    out = bs.CrossAttention(1, rows, 2, 2, 64, 700, "bf16")(q.to(dev), k.to(dev), v.to(dev))
    want, tol = ref.cross_attention(q.double(), k.double(), v.double(), None, None, 0.125, "bf16")
    ref.check(out, want, tol, "rising scores")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [4, 150])
def test_cross_attention_masks_and_layouts(dev, dtype, rows):
    cross_case(dev, 4, rows, 4, 2, 64, 100, dtype, 5, mask=True)
    cross_case(dev, 4, rows, 4, 2, 128, 70, dtype, 6, mask=True, lens=None, layout="bhsd")
    cross_case(dev, 3, rows, 4, 2, 64, 65, dtype, 7, lens=None, max_rows=rows + 9, max_keys=500)
    cross_case(dev, 2, rows, 2, 2, 48, 0, dtype, 8, lens=None)


def test_cross_attention_infinite_scores(dev):
    """-inf in a seen key: the score is -inf or NaN as its products say."""
    import beam_search_step_amd as bs
    k = torch.zeros(1, 40, 1, 64)
    k[0, 3, 0, 5] = -math.inf
    q = torch.zeros(1, 1, 1, 64)
    q[0, 0, 0] = 1.0
    v = torch.randn(1, 40, 1, 64, generator=torch.Generator().manual_seed(1))
    for dtype in ("bf16", "f32"):
        a, b, c = [x.to(DT[dtype]) for x in (q, k, v)]
        att = bs.CrossAttention(1, 1, 1, 1, 64, 40, dtype)
        out = att(a.to(dev), b.to(dev), c.to(dev))
        want, tol = ref.cross_attention(a.double(), b.double(), c.double(), None, None, 0.125, dtype)
        ref.check(out, want, tol, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows, keys", [(1, 1), (3, 40), (3, 3000), (150, 70)])
def test_cross_attention_nan_is_not_lost(dev, dtype, rows, keys):
    """A NaN query makes its own row NaN, and a seen NaN key its item's rows, also where
    every score of a row is NaN."""
    import beam_search_step_amd as bs
    g = torch.Generator().manual_seed(rows + keys)
    q, k, v = [torch.randn(s, generator=g).to(DT[dtype]) for s in ((3, rows, 2, 64), (3, keys, 2, 64), (3, keys, 2, 64))]
    q[0, rows // 2, 1, 5] = math.nan
    k[2, keys - 1, 0, 9] = math.nan
    say("nan", dtype, rows, keys)
    out = bs.CrossAttention(3, rows, 2, 2, 64, keys, dtype)(q.to(dev), k.to(dev), v.to(dev))
    want, tol = ref.cross_attention(q.double(), k.double(), v.double(), None, None, 0.125, dtype)
    assert torch.isnan(want).sum() == 64 * (1 + rows)
    ref.check(out, want, tol, "NaN")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [16, 5])
@pytest.mark.parametrize("heads, q_len, prompt, gen", [(2, 1, 0, 1), (4, 1, 30, 9), (2, 1, 40, 700), (2, 3, 0, 20)])
def test_cache_attention_nan_is_not_lost(dev, dtype, block, heads, q_len, prompt, gen):
    import beam_search_step_amd as bs
    mb, pmb = -(-gen // block), -(-prompt // block)
    cache, vals, _ = make_cache(dev, 2 * mb + pmb, block, 2, 64, 3)
    table = [list(range(mb)), list(range(mb, 2 * mb))]
    ptable = [list(range(2 * mb, 2 * mb + pmb))] if prompt else None
    q = torch.randn((2 * q_len, heads, 64), generator=torch.Generator().manual_seed(4)).to(DT[dtype])
    q[0, 1, 5] = math.nan
    at = table[1][0], 0, 1, 9                     # seen by every query of the second row
    cache.k[at] = 0x7f
    vals[0][at] = math.nan
    say("nan", dtype, block, heads, q_len, prompt, gen)
    att = bs.CacheAttention(1, 2, heads, 2, 64, block, mb, pmb, q_len, dtype)
    kw = dict(prompt_table=i32(ptable, dev), prompt_lens=i32([prompt], dev)) if prompt else {}
    out = att(q.to(dev), cache, i32(table, dev), i32([gen, gen], dev), **kw)
    want, tol = ref.cache_attention(q.double(), *vals, table, [gen, gen], ptable, [prompt] if prompt else None,
                                    q_len, 2, 0.125, dtype)
    assert torch.isnan(want).sum() == 64 * (1 + q_len * heads // 2)
    ref.check(out, want, tol, "NaN")


# --- the operators together ---------------------------------------------------

def test_search_with_a_quantised_paged_cache(dev):
    """A whole small search: prompts mapped and written, then per step map, write,
    attend over prompt and own positions, attend to the encoder, bs_step, and the
    reorder with copy on write. Every row's cached values stand for its own
    lineage's rows, and both attentions match their references on those values.

    A value is rounded once at its block's scale s and, where a later token grew
    the scale, once more at each larger one. Rounding to a larger power of two only
    moves subnormals, by at most 2^-10 of that scale, and the scales double at
    least, so a value is off by at most 2^-4 |x| + 2^-9 s."""
    import beam_search_step_amd as bs
    for dtype, block, seed in (("bf16", 4, 1), ("f32", 16, 2)):
        B, W, V, T, layers, hq, hk, d = 2, 3, 23, 13, 2, 4, 2, 32
        R, dt = B * W, DT[dtype]
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        plens, slens = [9, 6], [5, 11]
        search = bs.BeamSearch(B, W, V, T, eos_id=3, dtype="f32", stop="never")
        paged = bs.PagedKV(search, block)
        own = B * paged.blocks_per_item                       # the prompt's blocks lie behind
        pmb = -(-max(plens) // block)
        caches = [bs.QuantCache.empty(own + B * pmb, block, hk, d) for _ in range(layers)]
        pmap = bs.BlockMap(B, block, pmb, sum(plens) + 5)
        ptable, pslots, _, used = pmap(i32(plens, dev), i32(list(range(own, own + B * pmb)), dev))
        assert int(used) == sum(-(-p // block) for p in plens)
        praw = [[rnd(sum(plens), hk, d).to(dt) for _ in range(2)] for _ in range(layers)]
        for c, (k, v) in zip(caches, praw):
            c.write(k.to(dev), v.to(dev), pslots)
        enc = [[rnd(B, max(slens), hk, d).to(dt) for _ in range(2)] for _ in range(layers)]
        att = bs.CacheAttention(B, W, hq, hk, d, block, paged.max_blocks, pmb, dtype=dtype)
        cross = bs.CrossAttention(B, W, hq, hk, d, max(slens), dtype=dtype)
        smap = bs.BlockMap(R, block, paged.max_blocks, R)
        head = rnd(hq * d, V) * 2
        raw = [[[torch.zeros(0, hk, d) for _ in range(2)] for _ in range(R)] for _ in range(layers)]
        live = [w == 0 for _ in range(B) for w in range(W)]
        copies = 0
        for t in range(1, T + 1):
            say("search", dtype, "step", t)
            lens = [int(x) for x in live]
            _, slots, _, _ = smap(i32(lens, dev), starts=i32([t - 1] * R, dev), table=paged)
            rows = [r for r in range(R) if live[r]]
            # the map packs the live rows; so do their keys and values
            logits = torch.zeros(R, V)
            for layer in range(layers):
                k, v = [(rnd(R, hk, d) * math.exp(float(rnd(1)))).to(dt) for _ in range(2)]
                q = rnd(R, hq, d).to(dt)
                caches[layer].write(k[rows].to(dev), v[rows].to(dev), slots)
                for r in rows:
                    raw[layer][r] = [torch.cat([a, b[r:r + 1].float()]) for a, b in zip(raw[layer][r], (k, v))]
                seen = i32([t * x for x in lens], dev)
                o = att(q.to(dev), caches[layer], paged, seen, prompt_table=ptable, prompt_lens=i32(plens, dev))
                c = caches[layer]
                vals = [ref.decode(p.cpu()) * s.double().cpu()[:, None, :, None]
                        for p, s in ((c.k, c.k_scale), (c.v, c.v_scale))]
                table = paged.table().tolist()
                want, tol = ref.cache_attention(q.double(), *vals, table, [t * x for x in lens],
                                                ptable.tolist(), plens, 1, W, d ** -0.5, dtype)
                ref.check(o, want, tol, f"step {t} layer {layer} cache attention")
                x = cross(q.view(B, W, hq, d).to(dev), *[e.to(dev) for e in enc[layer]], lens=i32(slens, dev))
                want, tol = ref.cross_attention(q.view(B, W, hq, d).double(), *[e.double() for e in enc[layer]],
                                                slens, None, d ** -0.5, dtype)
                ref.check(x, want, tol, f"step {t} layer {layer} cross attention")
                for which, (pool, s) in enumerate(zip(vals, (c.k_scale.double().cpu(), c.v_scale.double().cpu()))):
                    for r in rows:
                        at = [(table[r][p // block], p % block) for p in range(t)]
                        got = torch.stack([pool[a] for a in at])
                        sc = torch.stack([s[a[0]] for a in at])[..., None]
                        x0 = raw[layer][r][which].double()
                        assert bool(((got - x0).abs() <= 2.0 ** -4 * x0.abs() + 2.0 ** -9 * sc).all()), \
                            f"step {t} layer {layer} row {r}"
                logits += (o.float().cpu().view(R, -1) + x.float().cpu().view(R, -1)) @ head
            bi, _, sc, dn = search.step(logits.to(dev))
            bi, sc, dn = bi.cpu().view(-1), sc.cpu().view(-1), dn.cpu()
            paged.reorder_quant(caches, t)
            parent = [r // W * W + int(bi[r]) for r in range(R)]
            raw = [[raw[layer][parent[r]] for r in range(R)] for layer in range(layers)]
            live = [float(sc[r]) > -math.inf and not dn[r // W] for r in range(R)]
            if t % block:
                for b in range(B):
                    ps = [parent[r] for r in range(b * W, b * W + W) if live[r]]
                    copies += len(ps) - len(set(ps))
            if not any(live):
                break
        assert copies > 0, "the search made no copies on write"
        assert paged.status()[0] == 0


def test_reorder_refuses_other_caches(dev):
    import beam_search_step_amd as bs
    search = bs.BeamSearch(2, 2, 10, 8, dtype="f32")
    paged = bs.PagedKV(search, 4)
    n = 2 * paged.blocks_per_item
    good = bs.QuantCache.empty(n, 4, 2, 16)
    search.step(torch.randn(4, 10, device=dev))
    before = paged.table().tolist()
    for bad in ([bs.QuantCache.empty(n, 8, 2, 16)], [bs.QuantCache.empty(n - 1, 4, 2, 16)],
                [good, bs.QuantCache.empty(n, 4, 1, 16)], [good, bs.QuantCache.empty(n + 1, 4, 2, 16)]):
        with pytest.raises(bs.BeamStepError) as e:
            paged.reorder_quant(bad, 1)
        assert e.value.status == bs.BS_EINVAL
    with pytest.raises(bs.BeamStepError) as e:
        paged.reorder_quant([good], 2)
    assert e.value.status == bs.BS_ESTATE
    assert paged.table().tolist() == before
    paged.reorder_quant([good], 1)
    with pytest.raises(bs.BeamStepError):     # the step is reordered already
        paged.reorder_quant([good], 1)


def test_wrappers_refuse(dev):
    import beam_search_step_amd as bs
    m = bs.BlockMap(3, 4, 2, 8)
    ok, free = i32([1, 2, 3], dev), i32([0, 1, 2, 3], dev)
    for args, kw in (((ok.cpu(), free), {}), ((ok.long(), free), {}), ((ok[:2], free), {}),
                     ((ok, free.cpu()), {}), ((ok,), {}), ((ok, free), dict(starts=ok)),
                     ((ok, free), dict(starts=ok, table=torch.zeros(3, 3, dtype=torch.int32, device=dev))),
                     ((ok, free), dict(table=torch.zeros(2, 2, dtype=torch.int32, device=dev)))):
        with pytest.raises(ValueError):
            m(*args, **kw)
    c = bs.QuantCache.empty(4, 8, 2, 32)
    x = torch.zeros(5, 2, 32, device=dev)
    sl = i32([0, 1, 2, 3, 4], dev)
    for a in ((x, x[:4], sl), (x.half(), x.half(), sl), (x, x.bfloat16(), sl), (x.cpu(), x.cpu(), sl),
              (x, x, sl[:4]), (x, x, sl.long()), (x[:, :, :16], x[:, :, :16], sl)):
        with pytest.raises(ValueError):
            c.write(*a)
    with pytest.raises(ValueError):
        bs.QuantCache(c.k, c.v[:3], c.k_scale, c.v_scale)
    with pytest.raises(ValueError):
        bs.QuantCache(c.k, c.v, c.k_scale[:, :1], c.v_scale)
    with pytest.raises(bs.BeamStepError):     # head_dim 24 is no multiple of 16
        d = bs.QuantCache.empty(4, 8, 2, 24)
        d.write(torch.zeros(5, 2, 24, device=dev), torch.zeros(5, 2, 24, device=dev), sl)
    att = bs.CacheAttention(2, 1, 4, 2, 32, 8, 3, dtype="f32")
    q, table, lens = torch.zeros(2, 4, 32, device=dev), torch.zeros(2, 3, dtype=torch.int32, device=dev), i32([1, 1], dev)
    for a, kw in (((q[:1], c, table, lens), {}), ((q.bfloat16(), c, table, lens), {}),
                  ((q, c, table[:, :2], lens), {}), ((q, c, table[:1], lens), {}), ((q, c, table, lens[:1]), {}),
                  ((q, c, table, lens), dict(prompt_lens=lens)),
                  ((q, c, table, lens), dict(out=torch.zeros(2, 4, 32)))):
        with pytest.raises(ValueError):
            att(*a, **kw)
    with pytest.raises(bs.BeamStepError):     # a cache of another block size
        att(q, bs.QuantCache.empty(4, 16, 2, 32), table, lens)
    with pytest.raises(bs.BeamStepError):     # a prompt, though none was configured
        att(q, c, table, lens, prompt_table=torch.zeros(2, 0, dtype=torch.int32, device=dev), prompt_lens=lens)
    cr = bs.CrossAttention(2, 3, 4, 2, 32, 10, dtype="f32")
    q, k = torch.zeros(2, 3, 4, 32, device=dev), torch.zeros(2, 9, 2, 32, device=dev)
    for a, kw in (((torch.zeros(2, 4, 4, 32, device=dev), k, k), {}), ((q, torch.zeros(2, 11, 2, 32, device=dev), k), {}),
                  ((q, k, k[:, :8]), {}), ((q, k, torch.zeros(2, 2, 9, 32, device=dev).transpose(1, 2)), {}),
                  ((q, k, k), dict(mask=torch.zeros(2, 8, dtype=torch.uint8, device=dev))),
                  ((q, k, k), dict(mask=torch.zeros(2, 9, dtype=torch.int32, device=dev))),
                  ((q, k, k), dict(lens=i32([1], dev)))):
        with pytest.raises(ValueError):
            cr(*a, **kw)
    for bad in (torch.zeros(2, 9, 2, 33, device=dev)[..., :32], torch.zeros(2, 9, 2, 36, device=dev)[..., 1:33]):
        with pytest.raises(bs.BeamStepError):  # rows that are not 16-byte aligned
            cr(q, bad, bad)


def test_a_captured_step_replays(dev):
    """Map, write and both attentions captured once; every replay, with new inputs in the
    captured tensors and eager work in between, gives the eager result's bits."""
    import beam_search_step_amd as bs
    B, W, hq, hk, d, block, mb, S = 2, 3, 8, 2, 64, 16, 4, 300
    R = B * W
    stream = torch.cuda.Stream()
    g = torch.Generator(device=dev).manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g, device=dev).bfloat16()  # noqa: E731
    table = i32([[r * mb + k for k in range(mb)] for r in range(R)], dev)
    ptable = i32([[R * mb + b * 40 + k for k in range(40)] for b in range(B)], dev)
    n = R * mb + B * 40
    base = [torch.randint(0, 120, (n, block, hk, d), generator=g, device=dev, dtype=torch.uint8) for _ in range(2)]
    st = dict(starts=i32([0] * R, dev), lens=i32([1] * R, dev), seen=i32([1] * R, dev), plens=i32([640, 333], dev),
              q=rnd(R, hq, d), k=rnd(R, hk, d), v=rnd(R, hk, d), ek=rnd(B, S, hk, d), ev=rnd(B, S, hk, d),
              elens=i32([300, 170], dev))

    def make(stream):
        cache = bs.QuantCache(*[b.clone() for b in base], *[torch.ones(n, hk, device=dev) for _ in range(2)],
                              stream=stream)
        return (bs.BlockMap(R, block, mb, R + 2, stream=stream), cache,
                bs.CacheAttention(B, W, hq, hk, d, block, mb, 40, stream=stream),
                bs.CrossAttention(B, W, hq, hk, d, S, stream=stream))

    def step(objs):
        m, cache, att, cross = objs
        slots = m(st["lens"], starts=st["starts"], table=table)[1]
        cache.write(st["k"], st["v"], slots)
        a = att(st["q"], cache, table, st["seen"], prompt_table=ptable, prompt_lens=st["plens"])
        c = cross(st["q"].view(B, W, hq, d), st["ek"], st["ev"], lens=st["elens"])
        return a, c

    eager, captured = make(None), make(stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = step(captured)
    for t in range(20, 26):
        st["starts"].fill_(t)
        st["seen"].fill_(t + 1)
        for name in ("q", "k", "v", "ek"):
            st[name].copy_(rnd(*st[name].shape))
        torch.cuda.synchronize()
        say("replay", t)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        want = step(eager)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y), f"replay at {t}"
        assert torch.equal(eager[1].k, captured[1].k) and torch.equal(eager[1].v_scale, captured[1].v_scale)


def test_two_handles_on_two_streams(dev):
    """Calls issued in turn on two streams give the bits that each gives alone."""
    import beam_search_step_amd as bs
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    g = torch.Generator(device=dev).manual_seed(9)
    data, alone, handles = [], [], []
    for s in streams:
        q = torch.randn(4, 5, 8, 128, generator=g, device=dev).bfloat16()
        k, v = [torch.randn(4, 900, 8, 128, generator=g, device=dev).bfloat16() for _ in range(2)]
        data.append((q, k, v))
        handles.append(bs.CrossAttention(4, 5, 8, 8, 128, 900, stream=s))
    torch.cuda.synchronize()
    for h, x in zip(handles, data):
        alone.append(h(*x))
    torch.cuda.synchronize()
    alone = [a.clone() for a in alone]
    outs = [[torch.empty_like(a) for _ in range(12)] for a in alone]
    torch.cuda.synchronize()
    for i in range(12):
        for j in range(2):
            handles[j](*data[j], out=outs[j][i])
    torch.cuda.synchronize()
    for j in range(2):
        for o in outs[j]:
            assert torch.equal(o, alone[j])


def test_offsets_beyond_32_bits(dev):
    """Blocks whose byte offsets pass 2^31 and 2^32."""
    import beam_search_step_amd as bs
    block, hk, d = 64, 8, 128
    n = (1 << 32) // (block * hk * d) + 40
    cache = bs.QuantCache.empty(n, block, hk, d)
    ids = [n - 1, n // 2 + 3, 0, n - 7]
    slots = [b * block + p for b in ids for p in range(block)]
    x = [rows_of(len(slots), hk, d, "bf16", i) for i in range(2)]
    cache.write(x[0].to(dev), x[1].to(dev), i32(slots, dev))
    k, v = cache.read(i32(slots, dev))
    vals = []
    for raw, got in ((x[0], k), (x[1], v)):
        small = torch.zeros(4, block, hk, d, dtype=torch.float64)
        ref.write(small, torch.ones(4, hk, dtype=torch.float64), raw.double(), list(range(4 * block)))
        assert torch.equal(got.double().cpu().view(small.shape), small)
        vals.append(small)
    q = torch.randn(1, 8, d, generator=torch.Generator().manual_seed(4)).bfloat16()
    att = bs.CacheAttention(1, 1, 8, hk, d, block, 4)
    out = att(q.to(dev), cache, i32([ids], dev), i32([250], dev))
    want, tol = ref.cache_attention(q.double(), *vals, [[0, 1, 2, 3]], [250], None, None, 1, 1, d ** -0.5, "bf16")
    ref.check(out, want, tol, "far blocks")


@pytest.mark.parametrize("rows", [3, 70])
@pytest.mark.parametrize("shift", [22, 24])
def test_cross_attention_of_keys_far_apart(dev, rows, shift):
    """Keys 2^shift elements apart (a batch-inner cache of many items): a key's offset
    passes 2^31 bytes."""
    import beam_search_step_amd as bs
    keys, d = 129, 64
    g = torch.Generator().manual_seed(shift + rows)
    q, k, v = [torch.randn(s, generator=g).bfloat16() for s in ((1, rows, 1, d), (1, keys, 1, d), (1, keys, 1, d))]
    step = 1 << shift
    pool = torch.empty((keys - 1) * step + 2 * d, dtype=torch.bfloat16, device=dev)
    kd, vd = [pool[o:].as_strided((1, keys, 1, d), (step, step, d, 1)) for o in (0, d)]
    kd.copy_(k.to(dev))
    vd.copy_(v.to(dev))
    say("far keys", rows, shift)
    out = bs.CrossAttention(1, rows, 1, 1, d, keys)(q.to(dev), kd, vd)
    want, tol = ref.cross_attention(q.double(), k.double(), v.double(), None, None, 0.125, "bf16")
    ref.check(out, want, tol, "far keys")
