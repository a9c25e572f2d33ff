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
