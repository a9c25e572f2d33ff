"""Edges of libbeamattn.so and its binding that need no GPU: every call below is
refused on the host."""
import ctypes

import pytest

import beam_search_step_amd as bs
from beam_search_step_amd import attn


@pytest.mark.parametrize("scale", [1e-50, 1e-38, 1e30])
def test_scales_that_fp32_does_not_hold_are_refused(scale):
    """Below 1e-37 scale * log2(e) loses bits or is zero, and zero times the -inf of a
    key that is not seen is NaN."""
    h = ctypes.c_void_p(123)
    L = bs.attn_library()
    for create, cfg in ((L.bs_cache_attn_create, attn.bs_cache_attn_config(1, 1, 1, 1, 1, 64, 16, 1, 0, 1, scale)),
                        (L.bs_cross_attn_create, attn.bs_cross_attn_config(1, 1, 1, 1, 64, 8, 1, scale))):
        assert create(ctypes.addressof(cfg), None, ctypes.addressof(h)) == bs.BS_EINVAL
        assert h.value is None


def paged_kv(device, rows=4, block=16, entries=3, h=None):
    """A PagedKV as the binding sees it, without a device behind it."""
    from types import SimpleNamespace
    p = bs.PagedKV.__new__(bs.PagedKV)
    p.search = SimpleNamespace(B=rows // 2, W=2, device=device)
    p.block_size, p.max_blocks, p._addr, p.h = block, entries, 1 << 20, h
    return p


def test_the_table_of_a_closed_paged_cache_is_refused():
    """Its memory is freed."""
    torch = pytest.importorskip("torch")
    dev = torch.device("meta")
    p = paged_kv(dev)
    with pytest.raises(ValueError, match="closed"):
        attn._table_arg(p, 4, dev, 16)
    p.h = 1
    try:
        assert attn._table_arg(p, 4, dev, 16) == (1 << 20, 3)
    finally:
        p.h = None


def test_the_table_of_a_paged_cache_of_another_block_size_is_refused():
    torch = pytest.importorskip("torch")
    dev = torch.device("meta")
    p = paged_kv(dev, h=1)
    try:
        with pytest.raises(ValueError, match="blocks of 16"):
            attn._table_arg(p, 4, dev, 8)
    finally:
        p.h = None


def test_caches_and_streams_of_another_device_are_refused():
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace
    p = paged_kv(torch.device("cuda", 0))
    with pytest.raises(ValueError, match="cuda:1"):
        p.reorder_quant([SimpleNamespace(device=torch.device("cuda", d)) for d in (0, 1)], 1)
    attn._check_stream(None, torch.device("cuda", 0))
    attn._check_stream(SimpleNamespace(device=torch.device("cuda", 0)), torch.device("cuda", 0))
    with pytest.raises(ValueError, match="cuda:1"):
        attn._check_stream(SimpleNamespace(device=torch.device("cuda", 1)), torch.device("cuda", 0))


def test_counts_that_an_int32_does_not_hold_are_refused():
    """They would reach the library cut to 32 bits."""
    torch = pytest.importorskip("torch")
    dev = torch.device("meta")
    big = (1 << 32) + 8
    m = bs.BlockMap.__new__(bs.BlockMap)
    m.n, m.block_size, m.max_blocks, m.device, m._table = 4, 16, 8, dev, None
    lens = torch.zeros(4, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError, match="free_blocks"):
        m(lens, torch.empty(big, dtype=torch.int32, device=dev))
    with pytest.raises(ValueError, match="table"):
        attn._table_arg(torch.empty((1, big), dtype=torch.int32, device=dev), 1, dev, 16)
    c = bs.QuantCache.__new__(bs.QuantCache)
    c.device, c.heads, c.head_dim, c.stream = dev, 1, 16, None
    x, slots = torch.empty((big, 1, 16), dtype=torch.bfloat16, device=dev), torch.empty(big, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError, match="slots"):
        c.write(x, x, slots)
    with pytest.raises(ValueError, match="slots"):
        c.read(slots)
    for kw in (dict(batch=big), dict(rows=big), dict(heads=big), dict(max_blocks=big), dict(block_size=-big)):
        a = dict(batch=1, rows=1, heads=1, kv_heads=1, head_dim=64, block_size=16, max_blocks=4)
        a.update(kw)
        with pytest.raises(ValueError, match="int32"):
            bs.CacheAttention(**a)
    with pytest.raises(ValueError, match="int32"):
        bs.CrossAttention(1, 1, 1, 1, 64, big)
    with pytest.raises(ValueError, match="int32"):
        attn._int32(n_blocks=4, block_size=big)
