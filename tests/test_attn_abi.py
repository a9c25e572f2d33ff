"""libbeamattn.so without a GPU: its exports, struct layouts and the arguments
it refuses before it touches a device."""
import ctypes
import subprocess

import pytest

import beam_search_step_amd as bs
from beam_search_step_amd import attn


def test_exports_match_the_header():
    out = subprocess.run(["nm", "-D", "--defined-only", attn.ATTN_LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    names = [(ln.split()[-2], ln.split()[-1]) for ln in out.splitlines()]
    assert sorted(n for t, n in names if t == "T") == bs.attn_functions()
    assert not [n for t, n in names if t == "W" and not n.startswith("_")]
    with open(attn.ATTN_LIB_PATH, "rb") as f:
        assert b"amdgcn-amd-amdhsa--gfx950" in f.read()


def test_struct_layouts():
    assert ctypes.sizeof(attn.bs_kvq_desc) == 64
    assert attn.bs_kvq_desc.n_blocks.offset == 32 and attn.bs_kvq_desc.block_stride.offset == 48
    assert ctypes.sizeof(attn.bs_cache_attn_config) == 48
    assert attn.bs_cache_attn_config.scale.offset == 40
    assert ctypes.sizeof(attn.bs_cross_attn_config) == 40
    assert attn.bs_cross_attn_config.scale.offset == 32
    assert ctypes.sizeof(attn.bs_cross_kv) == 40


# device addresses that are never read: every call below is refused on the host
P = 1 << 20


def _map(**kw):
    a = dict(stream=None, n=4, block_size=16, max_blocks=8, starts=None, lens=P, free=P, n_free=4,
             table=P, cu=P, slots=P, max_tokens=10, used=P)
    a.update(kw)
    return bs.attn_library().bs_map_blocks(*a.values())


@pytest.mark.parametrize("kw", [
    dict(n=0), dict(n=65536), dict(block_size=0), dict(max_blocks=0), dict(n_free=-1),
    dict(max_tokens=-1), dict(block_size=1 << 16, max_blocks=1 << 15), dict(lens=None),
    dict(table=None), dict(cu=None), dict(used=None), dict(slots=None), dict(free=None),
])
def test_map_blocks_refuses(kw):
    assert _map(**kw) == bs.BS_EINVAL


def _desc(**kw):
    a = dict(k=P, v=P, k_scale=P, v_scale=P, n_blocks=10, block_size=16, kv_heads=2, head_dim=64,
             block_stride=16 * 128, pos_stride=128)
    a.update(kw)
    return attn.bs_kvq_desc(*a.values())


BAD_DESC = [
    dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(n_blocks=0),
    dict(block_size=0), dict(kv_heads=0), dict(head_dim=0), dict(head_dim=8), dict(head_dim=72),
    dict(head_dim=272, pos_stride=1024, block_stride=16384), dict(n_blocks=1 << 27, block_size=16),
    dict(pos_stride=112), dict(pos_stride=136), dict(block_stride=15 * 128 + 112),
    dict(block_stride=16 * 128 + 8), dict(k=P + 8), dict(v=P + 1), dict(k_scale=P + 2),
    dict(pos_stride=1 << 26, block_stride=1 << 31),
]


@pytest.mark.parametrize("kw", BAD_DESC)
def test_every_call_refuses_a_bad_cache(kw):
    L, d = bs.attn_library(), _desc(**kw)
    r = ctypes.addressof(d)
    assert L.bs_kvq_write(None, r, 0, P, P, 128, P, 4) == bs.BS_EINVAL
    assert L.bs_kvq_read(None, r, 0, P, 4, P, P) == bs.BS_EINVAL


@pytest.mark.parametrize("args", [
    (2, P, P, 128, P, 4), (-1, P, P, 128, P, 4), (0, None, P, 128, P, 4), (0, P, None, 128, P, 4),
    (0, P, P, 127, P, 4), (0, P, P, 130, P, 4), (1, P, P, 132, P, 4), (0, P, P, 128, None, 4),
    (0, P, P, 128, P, -1), (0, P + 8, P, 128, P, 4), (0, P, P + 4, 128, P, 4),
])
def test_write_refuses(args):
    d = _desc()
    assert bs.attn_library().bs_kvq_write(None, ctypes.addressof(d), *args) == bs.BS_EINVAL


@pytest.mark.parametrize("args", [
    (2, P, 4, P, P), (0, None, 4, P, P), (0, P, -1, P, P), (0, P, 4, None, P), (0, P, 4, P, None),
    (0, P, 4, P + 8, P), (0, P, 4, P, P + 4),
])
def test_read_refuses(args):
    d = _desc()
    assert bs.attn_library().bs_kvq_read(None, ctypes.addressof(d), *args) == bs.BS_EINVAL


def test_empty_lists_are_nothing_to_do():
    L, d = bs.attn_library(), _desc()
    assert L.bs_kvq_write(None, ctypes.addressof(d), 0, None, None, 128, None, 0) == bs.BS_OK
    assert L.bs_kvq_read(None, ctypes.addressof(d), 0, None, 0, None, None) == bs.BS_OK


def _cache_cfg(**kw):
    a = dict(batch=2, rows=4, q_len=1, heads=8, kv_heads=2, head_dim=64, block_size=16,
             max_blocks=4, max_prompt_blocks=3, dtype=1, scale=0.125)
    a.update(kw)
    return attn.bs_cache_attn_config(*a.values())


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(rows=0), dict(q_len=0), dict(q_len=65), dict(batch=1024, rows=64),
    dict(heads=0), dict(heads=7), dict(kv_heads=0), dict(kv_heads=-2), dict(head_dim=24),
    dict(head_dim=512), dict(block_size=0), dict(max_blocks=0), dict(max_prompt_blocks=-1),
    dict(block_size=1 << 20, max_blocks=1 << 11), dict(block_size=1 << 20, max_prompt_blocks=1 << 11),
    dict(dtype=2), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")),
])
def test_cache_attn_create_refuses(kw):
    h = ctypes.c_void_p(123)
    cfg = _cache_cfg(**kw)
    assert bs.attn_library().bs_cache_attn_create(ctypes.addressof(cfg), None,
                                                  ctypes.addressof(h)) == bs.BS_EINVAL
    assert h.value is None


def _cross_cfg(**kw):
    a = dict(batch=2, max_rows=4, heads=8, kv_heads=2, head_dim=64, max_keys=100, dtype=1,
             scale=0.125)
    a.update(kw)
    return attn.bs_cross_attn_config(*a.values())


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(max_rows=0), dict(heads=0), dict(heads=9), dict(kv_heads=0),
    dict(batch=65536, kv_heads=1), dict(head_dim=24), dict(head_dim=272), dict(max_keys=0),
    dict(max_keys=1 << 30), dict(max_rows=1 << 25), dict(dtype=3), dict(scale=0.0),
    dict(scale=float("nan")),
])
def test_cross_attn_create_refuses(kw):
    h = ctypes.c_void_p(123)
    cfg = _cross_cfg(**kw)
    assert bs.attn_library().bs_cross_attn_create(ctypes.addressof(cfg), None,
                                                  ctypes.addressof(h)) == bs.BS_EINVAL
    assert h.value is None


def test_null_handles_are_refused():
    L = bs.attn_library()
    d = _desc()
    kv = attn.bs_cross_kv(P, P, 64, 64, 64)
    assert L.bs_cache_attn_create(None, None, None) == bs.BS_EINVAL
    assert L.bs_cross_attn_create(None, None, None) == bs.BS_EINVAL
    assert L.bs_cache_attn(None, ctypes.addressof(d), P, 512, P, 4, P, None, None, P) == bs.BS_EINVAL
    assert L.bs_cross_attn(None, P, 512, 1, ctypes.addressof(kv), 1, None, None, 0, P) == bs.BS_EINVAL
    assert L.bs_kvq_reorder(None, ctypes.addressof(d), 1, 1) == bs.BS_EINVAL
    L.bs_cache_attn_destroy(None)
    L.bs_cross_attn_destroy(None)


def test_row_layouts_are_checked():
    import torch
    rows = attn._head_rows
    t = torch.zeros(6, 2, 64)
    assert rows(t, "x", (6,), 2, 64) == 128
    assert rows(torch.zeros(6, 3, 64)[:, :2], "x", (6,), 2, 64) == 192
    assert rows(torch.zeros(3, 2, 2, 64), "x", (3, 2), 2, 64) == 128
    assert rows(torch.zeros(1, 2, 64), "x", (1,), 2, 64) == 128
    bad = [torch.zeros(5, 2, 64), torch.zeros(6, 2, 65)[:, :, :64], torch.zeros(6, 64, 2).transpose(1, 2),
           torch.zeros(6, 2, 128)[:, :, ::2], torch.zeros(6, 128)]
    for x in bad:
        with pytest.raises(ValueError):
            rows(x, "x", (6,), 2, 64)
    with pytest.raises(ValueError):  # the rows of two items unevenly spaced
        rows(torch.zeros(3, 3, 2, 64)[:, :2], "x", (3, 2), 2, 64)


def test_sizes_whose_counters_would_pass_31_bits_are_refused():
    L, h, d = bs.attn_library(), ctypes.c_void_p(1), _desc()
    most = (1 << 31) - (1 << 21)
    assert _map(block_size=1, max_blocks=most + 1) == bs.BS_EINVAL
    assert _map(max_tokens=most + 1) == bs.BS_EINVAL
    assert L.bs_kvq_write(None, ctypes.addressof(d), 0, P, P, 128, P, most + 1) == bs.BS_EINVAL
    for kw in (dict(block_size=1 << 20, max_blocks=1 << 10), dict(block_size=1 << 20, max_prompt_blocks=1 << 10),
               dict(batch=1, rows=65535, heads=65535, kv_heads=1), dict(batch=1, rows=1025, heads=65532, kv_heads=2)):
        cfg = _cache_cfg(**kw)
        assert L.bs_cache_attn_create(ctypes.addressof(cfg), None, ctypes.addressof(h)) == bs.BS_EINVAL, kw
        assert h.value is None
