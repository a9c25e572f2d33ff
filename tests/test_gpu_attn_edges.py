"""Edges of the attention-side operators on an MI355X: infinite scores and values,
head sizes above 128, scales of blocks that nobody reads, and calls across streams.
References and tolerances are those of tests/attn_ref.py; cross attention is held to
the bound of two-term probabilities at every number of columns."""
import math
import os
import random

import pytest

import attn_ref as ref
from test_gpu_attn import cache_case, i32, make_cache, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def dev():
    import beam_search_step_amd as bs
    bs.attn_library()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    torch.cuda.set_device(0)
    threads = torch.get_num_threads()
    torch.set_num_threads(min(threads, len(os.sched_getaffinity(0))))
    yield torch.device("cuda", 0)
    torch.set_num_threads(threads)


def cross_want(q, k, v, lens, mask, scale, dtype):
    """ref.cross_attention with the two-term bound, whatever the number of columns."""
    b, rows, hq, d = q.shape
    hk = k.shape[2]
    grp = hq // hk
    o, tol = torch.zeros_like(q), torch.zeros_like(q)
    for i in range(b):
        at = torch.arange(k.shape[1] if lens is None else max(0, min(int(lens[i]), k.shape[1])))
        if mask is not None:
            at = at[mask[i, at] != 0]
        for h in range(hk):
            sl = slice(h * grp, (h + 1) * grp)
            x = q[i, :, sl].reshape(-1, d)
            y, t = ref.attend(x, k[i, at, h], v[i, at, h], torch.ones(x.shape[0], at.numel(), dtype=torch.bool),
                              scale, dtype, 1)
            o[i, :, sl], tol[i, :, sl] = y.view(rows, grp, d), t.view(rows, grp, d)
    return o, tol


def cross_case(dev, batch, rows, heads, kv_heads, dim, keys, dtype, seed, mask=False):
    import beam_search_step_amd as bs
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((batch, rows, heads, dim), generator=g).to(DT[dtype])
    k, v = [torch.randn((batch, keys, kv_heads, dim), generator=g).to(DT[dtype]) for _ in range(2)]
    ln = [keys] + [rng.randint(0, keys) for _ in range(batch - 1)]
    mk = (torch.rand((batch, keys), generator=g) < 0.6).to(torch.uint8) if mask else None
    kd, vd = k.clone(), v.clone()                 # what is not seen holds NaN and infinities
    for b in range(batch):
        kd[b, ln[b]:], vd[b, ln[b]:] = math.nan, math.inf
        if mask:
            kd[b, mk[b] == 0], vd[b, mk[b] == 0] = math.inf, math.nan
    say("cross", batch, rows, heads, kv_heads, dim, keys, dtype, mask)
    out = bs.CrossAttention(batch, rows, heads, kv_heads, dim, keys, dtype)(
        q.to(dev), kd.to(dev), vd.to(dev), lens=i32(ln, dev), mask=None if mk is None else mk.to(dev))
    want, tol = cross_want(q.double(), k.double(), v.double(), ln, mk, dim ** -0.5, dtype)
    ref.check(out, want, tol, "cross attention")


# --- one bound at every number of columns ----------------------------------------

@pytest.mark.parametrize("case", [
    (2, 20, 2, 2, 128, 300), (1, 64, 1, 1, 128, 1403), (3, 9, 8, 2, 64, 200), (1, 150, 4, 2, 64, 700),
    (2, 300, 2, 1, 128, 513), (1, 5, 7, 1, 96, 77), (32, 260, 8, 8, 64, 130), (1, 40, 1, 1, 256, 900),
])
def test_probabilities_keep_their_bits_at_every_number_of_columns(dev, case):
    """The same bound for 5 and for hundreds of columns: fp32 arithmetic, rounded once."""
    cross_case(dev, *case, "bf16", seed=sum(case), mask=case[1] % 2 == 0)


# --- infinite scores and values -----------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows, keys", [(1, 40), (1, 3000), (70, 40), (70, 3000), (300, 700)])
@pytest.mark.parametrize("dim", [64, 256])
def test_one_key_of_a_score_of_minus_infinity(dev, dtype, rows, keys, dim):
    """It has no weight: the mean of the others. Scores of the others are 0, so
    probabilities are exactly equal; n terms in two parts, their sum and the output."""
    import beam_search_step_amd as bs
    k = torch.zeros(1, keys, 1, dim)
    k[0, keys // 2, 0, 5] = -math.inf
    v = torch.randn(1, keys, 1, dim, generator=torch.Generator().manual_seed(1)).to(DT[dtype])
    q = torch.ones(1, rows, 1, dim, dtype=DT[dtype], device=dev)
    say("-inf key", dtype, rows, keys, dim)
    out = bs.CrossAttention(1, rows, 1, 1, dim, keys, dtype)(q, k.to(DT[dtype]).to(dev), v.to(dev))
    others = torch.cat([v[0, :keys // 2, 0], v[0, keys // 2 + 1:, 0]]).double()
    want = others.mean(0)
    half, extra = (2.0 ** -8, 2.0 ** -15) if dtype == "bf16" else (2.0 ** -24, 2.0 ** -23)
    tol = half * want.abs() + (extra + (keys + 64) * ref.U) * others.abs().mean(0) * (1 + half)
    ref.check(out[0, :, 0], want.expand(rows, -1), tol.expand(rows, -1), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows, keys", [(1, 1), (1, 40), (1, 3000), (70, 40), (70, 3000)])
def test_every_score_minus_infinity_gives_zeros(dev, dtype, rows, keys):
    """Whatever the values hold."""
    import beam_search_step_amd as bs
    k = torch.zeros(1, keys, 1, 64)
    k[..., 5] = -math.inf
    v = torch.ones(1, keys, 1, 64)
    v[0, :, 0, 7], v[0, keys // 2, 0, 8], v[0, 0, 0, 9] = math.nan, math.inf, -math.inf
    q = torch.ones(1, rows, 1, 64)
    say("all -inf", dtype, rows, keys)
    out = bs.CrossAttention(1, rows, 1, 1, 64, keys, dtype)(*[x.to(DT[dtype]).to(dev) for x in (q, k, v)])
    assert torch.equal(out, torch.zeros_like(out))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block, prompt, gen", [(16, 0, 5), (16, 40, 9), (5, 30, 700), (16, 0, 1500)])
def test_every_score_minus_infinity_over_the_cache_gives_zeros(dev, dtype, block, prompt, gen):
    """Finite queries and keys whose products pass the range of fp32."""
    import beam_search_step_amd as bs
    mb, pmb = -(-gen // block), -(-prompt // block)
    cache, _, _ = make_cache(dev, mb + pmb, block, 1, 64, 2)
    cache.k.zero_()
    cache.k[..., 3] = 0x7e                          # 448
    cache.k_scale.fill_(2.0 ** 20)
    cache.v[..., 7] = 0x7f                          # NaN
    q = torch.zeros(1, 2, 64, dtype=DT[dtype], device=dev)
    q[..., 3] = -3e38
    att = bs.CacheAttention(1, 1, 2, 1, 64, block, mb, pmb, dtype=dtype)
    kw = dict(prompt_table=i32([list(range(mb, mb + pmb))], dev), prompt_lens=i32([prompt], dev)) if prompt else {}
    say("all -inf", dtype, block, prompt, gen)
    out = att(q, cache, i32([list(range(mb))], dev), i32([gen], dev), **kw)
    assert torch.equal(out, torch.zeros_like(out))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 70])
@pytest.mark.parametrize("keys, dead", [(40, 20), (3000, 1536), (3000, 2900)])
def test_a_nan_value_of_no_weight_is_nan_however_keys_are_split(dev, dtype, rows, keys, dead):
    """0 * NaN: the first `dead` keys have a score of -inf and a NaN value."""
    import beam_search_step_amd as bs
    k = torch.zeros(1, keys, 1, 64)
    k[0, :dead, 0, 5] = -math.inf
    v = torch.ones(1, keys, 1, 64)
    v[0, :dead, 0, 7] = math.nan
    q = torch.ones(1, rows, 1, 64)
    say("NaN of no weight", dtype, rows, keys, dead)
    out = bs.CrossAttention(1, rows, 1, 1, 64, keys, dtype)(*[x.to(DT[dtype]).to(dev) for x in (q, k, v)]).cpu()
    assert bool(torch.isnan(out[..., 7]).all())
    rest = torch.cat([out[..., :7], out[..., 8:]], -1).double()
    assert bool(((rest - 1).abs() <= 2.0 ** -8 + 2.0 ** -15).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 20, 70])
@pytest.mark.parametrize("keys", [1, 4, 7, 3000])
def test_infinite_values(dev, dtype, rows, keys):
    """A seen value of +-inf with some weight is the output, and NaN where both meet."""
    import beam_search_step_amd as bs
    v = torch.ones(1, keys, 1, 64)
    v[0, keys // 2, 0, 7], v[0, 0, 0, 9] = math.inf, -math.inf
    v[0, 0, 0, 11], v[0, keys - 1, 0, 11] = math.inf, -math.inf
    q, k = torch.ones(1, rows, 1, 64), torch.zeros(1, keys, 1, 64)
    say("inf values", dtype, rows, keys)
    out = bs.CrossAttention(1, rows, 1, 1, 64, keys, dtype)(*[x.to(DT[dtype]).to(dev) for x in (q, k, v)]).cpu()[0, :, 0]
    assert bool((out[:, 7] == math.inf).all()) and bool((out[:, 9] == -math.inf).all())
    assert bool((out[:, 11] == -math.inf).all() if keys == 1 else torch.isnan(out[:, 11]).all())
    rest = torch.cat([out[:, :7], out[:, 12:]], -1).double()
    assert bool(((rest - 1).abs() <= 2.0 ** -8 + 2.0 ** -15).all())


@pytest.mark.parametrize("bits", [0x7f800001, 0x7f80ffff, 0xff800001, 0x7fc00000])
def test_every_nan_of_an_fp32_query_is_nan(dev, bits):
    """Also one whose payload lies in the low half, over keys that all have one sign."""
    import beam_search_step_amd as bs
    for sign in (0, 0x80):
        cache, _, _ = make_cache(dev, 2, 16, 1, 64, 3)
        cache.k.fill_(0x38 | sign)                  # +-1
        q = torch.ones(1, 1, 64)
        q.view(torch.int32)[0, 0, 5] = bits - (1 << 32) if bits >> 31 else bits
        assert bool(torch.isnan(q[0, 0, 5]))
        out = bs.CacheAttention(1, 1, 1, 1, 64, 16, 2, dtype="f32")(q.to(dev), cache, i32([[0, 1]], dev), i32([20], dev))
        assert bool(torch.isnan(out).all()), (hex(bits), sign)


# --- scales of blocks that are not read -----------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [16, 5])
@pytest.mark.parametrize("scale", [math.nan, math.inf, 2.0 ** 127])
def test_scales_of_blocks_that_no_table_names(dev, dtype, block, scale):
    """Block 0 was never written; tables have holes and lengths end inside a tile."""
    import beam_search_step_amd as bs
    gen, dim, n = 40, 64, 12
    cache, vals, _ = make_cache(dev, n, block, 2, dim, 6)
    cache.k_scale[0], cache.v_scale[0] = scale, scale
    mb = -(-gen // block)
    table = [list(range(1, 1 + mb)), [-1] + list(range(2, 1 + mb)), list(range(1, mb)) + [n + 7]]
    lens = [gen, gen, 1]
    q = torch.randn(3, 4, dim, generator=torch.Generator().manual_seed(8)).to(DT[dtype])
    say("scales", dtype, block, scale)
    out = bs.CacheAttention(3, 1, 4, 2, dim, block, mb, dtype=dtype)(q.to(dev), cache, i32(table, dev), i32(lens, dev))
    want, tol = ref.cache_attention(q.double(), *vals, table, lens, None, None, 1, 1, dim ** -0.5, dtype)
    ref.check(out, want, tol, "scales")


# --- head sizes above 128 ---------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mask", [False, True])
@pytest.mark.parametrize("case", [
    (2, 40, 1, 1, 256, 129), (2, 200, 2, 2, 256, 77), (1, 60, 3, 1, 144, 333), (2, 70, 2, 1, 208, 100),
    (1, 130, 1, 1, 240, 1000), (1, 36, 2, 2, 256, 3001), (3, 5, 8, 2, 144, 50), (2, 1, 16, 1, 208, 700),
])
def test_cross_attention_of_heads_above_128(dev, case, mask, dtype):
    cross_case(dev, *case, dtype, seed=sum(case), mask=mask)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", [
    (2, 3, 1, 4, 2, 256, 16, 90, 40), (1, 2, 5, 4, 1, 208, 32, 70, 33), (2, 1, 8, 2, 2, 256, 16, 0, 300),
    (1, 16, 1, 4, 2, 144, 16, 520, 30), (1, 1, 1, 1, 1, 240, 48, 0, 1300), (1, 8, 3, 6, 2, 256, 32, 200, 50),
])
def test_cache_attention_of_heads_above_128(dev, case, dtype):
    cache_case(dev, *case, dtype, seed=sum(case))


# --- streams ----------------------------------------------------------------------------

def stream_of(t):
    """The raw stream whose pool a tensor's memory belongs to."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no segment")


def test_what_an_object_allocates_belongs_to_its_stream(dev):
    """Otherwise the allocator may hand over memory that the current stream still uses,
    and fills on the current stream may come after the first write."""
    import beam_search_step_amd as bs
    s = torch.cuda.Stream()
    m = bs.BlockMap(2, 4, 3, 8, stream=s)
    m(i32([3, 5], dev), i32([0, 1, 2, 3], dev))
    c = bs.QuantCache.empty(6, 4, 2, 64, stream=s)
    own = [m.cu, m.slots, m.used, m._table, c.k, c.v, c.k_scale, c.v_scale,
           bs.CacheAttention(2, 1, 4, 2, 64, 4, 3, stream=s).out,
           bs.CrossAttention(2, 3, 4, 2, 64, 9, stream=s)._buf]
    torch.cuda.synchronize()
    assert [stream_of(t) for t in own] == [s.cuda_stream] * len(own)


def busy(n=40):
    """Some tens of milliseconds of work on the current stream."""
    x = torch.full((4096, 4096), 2.0 ** -12, device="cuda")
    for _ in range(n):
        x = x @ x
    return x


def test_a_cache_made_for_a_stream_while_the_current_one_is_busy(dev):
    import beam_search_step_amd as bs
    s = torch.cuda.Stream()
    x = [torch.randn(8, 2, 64, generator=torch.Generator().manual_seed(i)).to(dev) for i in range(2)]
    slots = i32(list(range(8)), dev)
    torch.cuda.synchronize()
    keep = busy()
    c = bs.QuantCache.empty(3, 4, 2, 64, stream=s)
    c.write(*x, slots)
    first = c.read(slots)
    s.synchronize()
    first = [t.cpu() for t in first]
    torch.cuda.synchronize()
    again = [t.cpu() for t in c.read(slots)]
    del keep
    for t, a, b in zip(x, first, again):
        assert torch.equal(a, b)
        assert bool(((a - t.cpu()).abs() <= 2.0 ** -4 * t.cpu().abs() + 2.0 ** -9).all())


def attentions(dev):
    """Two handles and a call of both on given inputs."""
    import beam_search_step_amd as bs
    cache, _, _ = make_cache(dev, 4, 16, 2, 64, 7)
    att, cross = bs.CacheAttention(2, 1, 4, 2, 64, 16, 2), bs.CrossAttention(2, 1, 4, 2, 64, 50)
    table, lens = i32([[0, 1], [2, 3]], dev), i32([20, 32], dev)
    torch.cuda.synchronize()
    return lambda q, k, v: (att(q, cache, table, lens), cross(q.view(2, 1, 4, 64), k, v))


def attention_inputs(dev, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    return [torch.randn(s, generator=g, device=dev).bfloat16() for s in ((2, 4, 64), (2, 50, 2, 64), (2, 50, 2, 64))]


def test_handles_made_under_another_stream_keep_in_order_with_the_current_one(dev):
    """Without a stream of their own they wait for what the current stream made, and it
    waits for them."""
    call = attentions(dev)
    s = torch.cuda.Stream()
    data = [attention_inputs(dev, i) for i in range(4)]
    want = []
    for d in data:
        want.append([o.clone() for o in call(*d)])
    ins = [torch.zeros_like(x) for x in data[0]]
    torch.cuda.synchronize()
    got = []
    with torch.cuda.stream(s):
        keep = busy()
        for d in data:
            for x, y in zip(ins, d):
                x.copy_(y)
            got.append([o.clone() for o in call(*ins)])
    torch.cuda.synchronize()
    del keep
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_handles_made_under_another_stream_and_captured(dev):
    """Their stream joins the capture; the null stream cannot, and is refused."""
    default, a, b = attentions(dev), torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(a):
        call = attentions(dev)
    ins = attention_inputs(dev, 0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=b):
        with pytest.raises(ValueError, match="capture"):
            default(*ins)
        outs = call(*ins)
    for i in range(1, 5):
        for x, y in zip(ins, attention_inputs(dev, i)):
            x.copy_(y)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        want = default(*ins)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), f"replay {i}"



def test_maps_and_caches_without_a_stream_follow_the_current_one(dev):
    """Their memory may be freed while another stream still uses it: that stream is
    recorded."""
    import beam_search_step_amd as bs
    s = torch.cuda.Stream()
    for _ in range(3):
        m, c = bs.BlockMap(2, 4, 3, 8), bs.QuantCache.empty(6, 4, 2, 64)
        x = torch.randn(8, 2, 64, device=dev)
        lens, free = i32([3, 5], dev), i32([4, 1, 2, 3], dev)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            keep = busy()
            table, slots, cu, used = [t.clone() for t in m(lens, free)]
            c.write(x, x, m.slots)
            k, v = c.read(slots)
        at = [m._table.data_ptr(), c.k.data_ptr()]
        del m, c
        other = [torch.full((2, 3), 9, dtype=torch.int32, device=dev), torch.full((6, 4, 2, 64), 77, dtype=torch.uint8, device=dev)]
        pending = not s.query()
        say("still busy:", pending)
        torch.cuda.synchronize()
        assert not pending or at[0] != other[0].data_ptr() and at[1] != other[1].data_ptr(), "memory in use was handed over"
        assert table.tolist() == [[4, -1, -1], [1, 2, -1]] and cu.tolist() == [0, 3, 8]
        assert bool(((k - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -9).all()) and torch.equal(k, v)
        del keep


# --- handles wider than their calls ---------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch, rows, q_len, heads, kv_heads, dim, block, prompt", [
    (2, 3, 1, 4, 2, 64, 16, 40), (1, 2, 4, 8, 2, 128, 24, 100), (3, 1, 1, 2, 2, 256, 32, 33), (16, 16, 1, 8, 8, 64, 16, 20),
])
def test_cache_attention_of_a_handle_much_wider_than_its_lengths(dev, dtype, batch, rows, q_len, heads, kv_heads, dim,
                                                                 block, prompt):
    """Tables of thousands of entries (wider than the handle asks for) of which few are
    used, queries inside wider rows, then the same handle without a prompt and with
    nothing at all."""
    import beam_search_step_amd as bs
    rng = random.Random(batch * dim)
    R, mb, pmb = batch * rows, 700, 900
    used, pused = -(-30 // block), -(-prompt // block)
    n = R * used + batch * pused
    cache, vals, _ = make_cache(dev, n, block, kv_heads, dim, 4)
    ids = rng.sample(range(n), n)
    table = [[ids.pop() for _ in range(used)] + [-1] * (mb + 5 - used) for _ in range(R)]
    ptable = [[ids.pop() for _ in range(pused)] + [-1] * (pmb - pused) for _ in range(batch)]
    lens, plens = [rng.randint(0, 30) for _ in range(R)], [rng.randint(0, prompt) for _ in range(batch)]
    wide = torch.randn((R * q_len, 3 * heads, dim), generator=torch.Generator().manual_seed(6)).to(DT[dtype])
    q = wide[:, heads:2 * heads]
    say("wide handle", batch, rows, q_len, heads, dim, block, dtype)
    att = bs.CacheAttention(batch, rows, heads, kv_heads, dim, block, mb, pmb, q_len, dtype)
    td, pd, qd = i32(table, dev), i32(ptable, dev), wide.to(dev)[:, heads:2 * heads]
    for p in (True, False):
        kw = dict(prompt_table=pd, prompt_lens=i32(plens, dev)) if p else {}
        out = att(qd, cache, td, i32(lens, dev), **kw)
        want, tol = ref.cache_attention(q.double(), *vals, table, lens, ptable if p else None, plens if p else None,
                                        q_len, rows, dim ** -0.5, dtype)
        ref.check(out, want, tol, f"prompt {p}")
    out = att(qd, cache, td, i32([0] * R, dev), prompt_table=pd, prompt_lens=i32([-4] * batch, dev))
    assert torch.equal(out, torch.zeros_like(out))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cross_attention_of_a_handle_much_wider_than_its_calls(dev, dtype):
    """One handle, from one row and key to its limits, strided queries, in any order."""
    import beam_search_step_amd as bs
    B, hq, hk, d = 2, 4, 2, 64
    att = bs.CrossAttention(B, 300, hq, hk, d, 3000, dtype)
    for rows, keys in ((300, 3000), (1, 1), (7, 0), (0, 5), (9, 3000), (300, 3), (1, 3000)):
        g = torch.Generator().manual_seed(rows + keys)
        wide = torch.randn((B, rows, 3 * hq, d), generator=g).to(DT[dtype])
        k, v = [torch.randn((B, keys, hk, d), generator=g).to(DT[dtype]) for _ in range(2)]
        say("wide handle", rows, keys, dtype)
        out = att(wide.to(dev)[:, :, hq:2 * hq], k.to(dev), v.to(dev))
        assert out.shape == (B, rows, hq, d)
        want, tol = cross_want(wide[:, :, hq:2 * hq].double(), k.double(), v.double(), None, None, d ** -0.5, dtype)
        if rows:
            ref.check(out, want, tol, f"{rows} rows, {keys} keys")
