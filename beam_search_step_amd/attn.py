"""Python binding of libbeamattn.so (the C ABI in include/beamattn.h): block and
slot maps, the 8-bit paged cache, attention over it, and cross attention.

As in the package's main module, this marshals arguments only; every operator
runs in the library's HIP kernels, and the checks here keep a kernel within the
caller's tensors, whose sizes the library cannot see.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re
from typing import Optional, Sequence

import beam_search_step_amd as _bs

ATTN_LIB_PATH = os.path.join(_bs.HERE, "libbeamattn.so")
ATTN_HEADER = os.path.join(os.path.dirname(_bs.HERE), "include", "beamattn.h")


class bs_kvq_desc(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("n_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("block_stride", ctypes.c_int64), ("pos_stride", ctypes.c_int64),
    ]


class bs_cache_attn_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "rows", "q_len", "heads", "kv_heads", "head_dim", "block_size", "max_blocks",
        "max_prompt_blocks", "dtype")] + [("scale", ctypes.c_double)]


class bs_cross_attn_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "max_rows", "heads", "kv_heads", "head_dim", "max_keys", "dtype")] + [
            ("scale", ctypes.c_double)]


class bs_cross_kv(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + [
        (n, ctypes.c_int64) for n in ("batch_stride", "pos_stride", "head_stride")]


_lib = None


def attn_library() -> ctypes.CDLL:
    """The loaded libbeamattn.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        _bs.library()
        if not os.path.exists(ATTN_LIB_PATH):
            raise ImportError(f"{ATTN_LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(ATTN_LIB_PATH)
        P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        L.bs_map_blocks.argtypes = [P, i32, i32, i32, P, P, P, i32, P, P, P, i32, P]
        L.bs_kvq_write.argtypes = [P, P, i32, P, P, i64, P, i32]
        L.bs_kvq_read.argtypes = [P, P, i32, P, i32, P, P]
        L.bs_kvq_reorder.argtypes = [P, P, i32, i32]
        L.bs_cache_attn_create.argtypes = [P, P, P]
        L.bs_cache_attn.argtypes = [P, P, P, i64, P, i32, P, P, P, P]
        L.bs_cross_attn_create.argtypes = [P, P, P]
        L.bs_cross_attn.argtypes = [P, P, i64, i32, P, i32, P, P, i64, P]
        for name in ("bs_map_blocks", "bs_kvq_write", "bs_kvq_read", "bs_kvq_reorder",
                     "bs_cache_attn_create", "bs_cache_attn", "bs_cross_attn_create",
                     "bs_cross_attn"):
            getattr(L, name).restype = ctypes.c_int
        for name in ("bs_cache_attn_destroy", "bs_cross_attn_destroy"):
            getattr(L, name).argtypes = [P]
            getattr(L, name).restype = None
        _lib = L
    return _lib


def attn_functions() -> list:
    """Names of the functions include/beamattn.h declares."""
    with open(ATTN_HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(bs_[a-z_]+)\s*\(", text)))


_torch = None


def _t():
    """torch, imported at the first use."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _torch_dtypes():
    torch = _t()
    return {"f32": torch.float32, "bf16": torch.bfloat16}


_MOST = 2 ** 31 - 1  # the largest count that the library takes


def _int32(**values) -> None:
    """Refuses values that ctypes would cut to 32 bits."""
    for name, v in values.items():
        if not -_MOST <= v <= _MOST:
            raise ValueError(f"{name}: {v} is no int32")


def _need(t, what: str, device, dtype, shape=None):
    """A tensor on the device, of the type and, when a shape is given, contiguous and of it."""
    if t.device == device and t.dtype is dtype and (
            shape is None or (t.shape == shape and t.is_contiguous())):
        return
    if t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{what}: dtype {t.dtype}, expected {dtype}")
    raise ValueError(f"{what}: a contiguous tensor of shape {list(shape)} is needed, not "
                     f"{list(t.shape)}")


def _head_rows(t, what: str, lead: tuple, heads: int, dim: int) -> int:
    """Elements between the rows of a tensor [*lead, heads, dim] whose rows are
    contiguous and evenly spaced."""
    if t.shape != (*lead, heads, dim):
        raise ValueError(f"{what}: shape {list(t.shape)}, expected {[*lead, heads, dim]}")
    if t.is_contiguous():
        return heads * dim
    st = t.stride()
    if (dim > 1 and st[-1] != 1) or (heads > 1 and st[-2] != dim):
        raise ValueError(f"{what}: the heads of a row must be contiguous")
    n = [(s, k) for s, k in zip(lead, st) if s > 1]
    for (_, a), (s, b) in zip(n, n[1:]):
        if a != s * b:
            raise ValueError(f"{what}: rows must be evenly spaced")
    return n[-1][1] if n else heads * dim


def _on_device(device, stream, fn, *args):
    """fn(raw stream, *args) with the device as the current one, on the given stream
    or the device's current stream."""
    torch = _t()
    if stream is not None:
        raw = stream.cuda_stream
    else:
        raw = torch._C._cuda_getCurrentRawStream(device.index)
    if torch.cuda.current_device() == device.index:
        return fn(raw, *args)
    with torch.cuda.device(device):
        return fn(raw, *args)


def _gpu_device(stream):
    torch = _t()
    return stream.device if stream is not None else torch.device("cuda", torch.cuda.current_device())


def _check_stream(stream, device) -> None:
    if stream is not None and stream.device != device:
        raise ValueError(f"stream: on {stream.device}, expected {device}")


def _record_use(device, *tensors) -> None:
    """Tells the allocator that an object's memory is used on the current stream too, where
    that is another than the one it was made under."""
    torch = _t()
    if not torch.cuda.is_current_stream_capturing():
        now = torch.cuda.current_stream(device)
        for t in tensors:
            t.record_stream(now)


def _memory_of(stream):
    """Allocations (and fills) inside belong to the stream that was given to an object: its
    kernels run there, and the allocator orders reuse by stream."""
    return contextlib.nullcontext() if stream is None else _t().cuda.stream(stream)


class _Handle:
    """A handle of the library, whose calls are all on one stream: the one given, or the
    current one of the time when it was made. In the second case a call under another
    stream is kept in order with that: a caller who names no stream expects the current one's
    order."""

    h = None

    def _create(self, fn, cfg, stream):
        torch = _t()
        self.device = _gpu_device(stream)
        self._made_on = None if stream is not None else torch.cuda.current_stream(self.device)
        self._raw = (self._made_on if stream is None else stream).cuda_stream
        self._current = torch._C._cuda_getCurrentRawStream
        h = ctypes.c_void_p()
        _bs._check(_on_device(self.device, stream, lambda raw: fn(
            ctypes.addressof(cfg), raw, ctypes.addressof(h))), fn.__name__)
        self.h = h.value

    def _call(self, fn, *args) -> int:
        made = self._made_on
        if made is None or self._current(self.device.index) == self._raw:
            return fn(self.h, *args)
        torch = _t()
        now = torch.cuda.current_stream(self.device)
        if self._raw == 0 and torch.cuda.is_current_stream_capturing():
            raise ValueError("made under the null stream, which no capture can hold: make it "
                             "under another stream, or give it one")
        made.wait_stream(now)
        status = fn(self.h, *args)
        now.wait_stream(made)
        return status


def _table_arg(table, rows: int, device, block_size: int):
    """(address, entries per row) of a block table: a tensor, or a PagedKV's own."""
    if isinstance(table, _bs.PagedKV):
        if not table.h:  # its device memory is freed
            raise ValueError("table: the PagedKV is closed")
        if table.block_size != block_size:
            raise ValueError(f"table: blocks of {table.block_size} positions, {block_size} needed")
        if table.search.B * table.search.W != rows:
            raise ValueError(f"table: {table.search.B * table.search.W} rows, {rows} needed")
        if table.search.device != device:
            raise ValueError(f"table: on {table.search.device}, expected {device}")
        return table._addr, table.max_blocks
    _need(table, "table", device, _t().int32)
    shape = table.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] > _MOST or not table.is_contiguous():
        raise ValueError(f"table: a contiguous tensor [{rows}, entries] is needed, not "
                         f"{list(shape)}")
    return table.data_ptr(), shape[1]


class BlockMap:
    """Block tables and slot maps for n requests (bs_map_blocks).

    ``map(lens, free_blocks, starts=None, table=None)`` returns (table, slots,
    cu, used): int32 tensors [n, max_blocks], [max_tokens], [n + 1] and [1].
    The table is the one given (updated in place), or the map's own when the
    requests are new; without ``free_blocks`` it is only read and may be a
    PagedKV. The other three are the map's own, written again by every call.
    """

    def __init__(self, n, block_size, max_blocks, max_tokens, stream=None):
        torch = _t()
        self.n, self.block_size, self.max_blocks, self.max_tokens = n, block_size, max_blocks, max_tokens
        if not (1 <= n <= 65535 and block_size >= 1 and max_blocks >= 1 and max_tokens >= 0
                and block_size * max_blocks <= 2 ** 31 - 2 ** 21
                and max_tokens <= 2 ** 31 - 2 ** 21):
            raise ValueError(f"BlockMap({n}, {block_size}, {max_blocks}, {max_tokens})")
        self._fn = attn_library().bs_map_blocks
        self.device = _gpu_device(stream)
        self.stream = stream
        kw = dict(dtype=torch.int32, device=self.device)
        with _memory_of(stream):
            self.cu = torch.empty(n + 1, **kw)
            self.slots = torch.empty(max_tokens, **kw)
            self.used = torch.empty(1, **kw)
        self._cu, self._used = self.cu.data_ptr(), self.used.data_ptr()
        self._slots = self.slots.data_ptr() or None
        self._table = None
        self._current = torch._C._cuda_getCurrentRawStream
        self._raw = self._current(self.device.index)

    def __call__(self, lens, free_blocks=None, starts=None, table=None):
        torch = _t()
        i32, dev = torch.int32, self.device
        _need(lens, "lens", dev, i32, (self.n,))
        if starts is not None:
            _need(starts, "starts", dev, i32, (self.n,))
        n_free = 0
        if free_blocks is not None:
            _need(free_blocks, "free_blocks", dev, i32)
            if free_blocks.dim() != 1 or not free_blocks.is_contiguous():
                raise ValueError("free_blocks: a contiguous list is needed")
            if isinstance(table, _bs.PagedKV):
                raise ValueError("a PagedKV's table is only read: no free_blocks")
            n_free = free_blocks.numel()
            if n_free > _MOST:
                raise ValueError(f"free_blocks: {n_free} entries, at most {_MOST}")
        if table is None:
            if starts is not None or free_blocks is None:
                raise ValueError("table: needed with starts, and without free_blocks")
            if self._table is None:
                with _memory_of(self.stream):
                    self._table = torch.empty((self.n, self.max_blocks), dtype=i32, device=dev)
            table = self._table
        at, width = _table_arg(table, self.n, dev, self.block_size)
        if width != self.max_blocks:
            raise ValueError(f"table: {width} entries per row, expected {self.max_blocks}")
        if self.stream is None and self._current(dev.index) != self._raw:
            _record_use(dev, self.cu, self.slots, self.used,
                        *(() if self._table is None else (self._table,)))
        # an empty list is a list still: any address will do
        free = None if free_blocks is None else free_blocks.data_ptr() or self._used
        _bs._check(_on_device(dev, self.stream, self._fn, self.n, self.block_size,
                              self.max_blocks, _bs._ptr(starts), lens.data_ptr(), free, n_free,
                              at, self._cu, self._slots, self.max_tokens, self._used),
                   "bs_map_blocks")
        return table, self.slots, self.cu, self.used


class QuantCache:
    """One layer's 8-bit paged cache over the caller's tensors.

    k, v: uint8 or float8_e4m3fn [n_blocks, block_size, kv_heads, head_dim]
    (e4m3 bytes; blocks and positions may be strided); k_scale, v_scale: float32
    [n_blocks, kv_heads]. ``QuantCache.empty(...)`` allocates and fills them, on the
    stream that it is given.
    ``write(k, v, slots)`` rounds new tokens into their slots, ``read(slots,
    dtype)`` returns what slots hold; both run on the given or current stream.
    """

    def __init__(self, k, v, k_scale, v_scale, stream=None):
        torch = _t()
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k, v: two pools [n_blocks, block_size, kv_heads, head_dim] of one "
                             "shape, type and strides are needed")
        n, bs, h, d = k.shape
        _int32(n_blocks=n, block_size=bs, kv_heads=h, head_dim=d)
        if not k.is_cuda:
            raise ValueError("k: a GPU tensor is needed")
        if k.dtype not in (torch.uint8, torch.float8_e4m3fn):
            raise ValueError(f"k: dtype {k.dtype}, expected uint8 or float8_e4m3fn")
        if k.stride(3) != 1 or (h > 1 and k.stride(2) != d):
            raise ValueError("k, v: the heads of a position must be contiguous")
        self.device = k.device
        _check_stream(stream, self.device)
        _need(v, "v", self.device, k.dtype)
        _need(k_scale, "k_scale", self.device, torch.float32, (n, h))
        _need(v_scale, "v_scale", self.device, torch.float32, (n, h))
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.heads, self.head_dim, self.block_size, self.n_blocks = h, d, bs, n
        self.stream = stream
        pos = k.stride(1) if bs > 1 else h * d
        block = k.stride(0) if n > 1 else max((bs - 1) * pos + h * d, bs * pos)
        self.desc = bs_kvq_desc(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(),
                                v_scale.data_ptr(), n, bs, h, d, block, pos)
        self._ref = ctypes.addressof(self.desc)
        self._dtypes = _torch_dtypes()
        self._current = torch._C._cuda_getCurrentRawStream
        self._raw = self._current(self.device.index)
        self._write, self._read = attn_library().bs_kvq_write, attn_library().bs_kvq_read

    @classmethod
    def empty(cls, n_blocks, block_size, kv_heads, head_dim, device=None, stream=None):
        torch = _t()
        kw = dict(device=device if device is not None else _gpu_device(stream))
        with _memory_of(stream):
            pools = [torch.zeros((n_blocks, block_size, kv_heads, head_dim), dtype=torch.uint8,
                                 **kw) for _ in range(2)]
            scales = [torch.ones((n_blocks, kv_heads), dtype=torch.float32, **kw)
                      for _ in range(2)]
        return cls(*pools, *scales, stream=stream)

    def write(self, k, v, slots) -> None:
        torch = _t()
        n = k.shape[0]
        f32 = k.dtype is torch.float32
        dt = torch.float32 if f32 else torch.bfloat16
        _need(k, "k", self.device, dt)
        _need(v, "v", self.device, dt)
        stride = _head_rows(k, "k", (n,), self.heads, self.head_dim)
        if _head_rows(v, "v", (n,), self.heads, self.head_dim) != stride:
            raise ValueError("k, v: rows must be equally spaced")
        _need(slots, "slots", self.device, torch.int32)
        if slots.dim() != 1 or slots.shape[0] < n or n > _MOST or not slots.is_contiguous():
            raise ValueError(f"slots: a contiguous list of at least {n} (and {n} at most {_MOST}) "
                             "is needed")
        if self.stream is None and self._current(self.device.index) != self._raw:
            _record_use(self.device, self.k, self.v, self.k_scale, self.v_scale)
        _bs._check(_on_device(self.device, self.stream, self._write, self._ref,
                              _bs.BS_F32 if f32 else _bs.BS_BF16, k.data_ptr(), v.data_ptr(),
                              stride, slots.data_ptr(), n), "bs_kvq_write")

    def read(self, slots, dtype="f32"):
        torch = _t()
        _need(slots, "slots", self.device, torch.int32)
        if slots.dim() != 1 or slots.shape[0] > _MOST or not slots.is_contiguous():
            raise ValueError(f"slots: a contiguous list of at most {_MOST} is needed")
        n = slots.shape[0]
        shape = (2, n, self.heads, self.head_dim)
        if self.stream is None:
            kv = torch.empty(shape, dtype=self._dtypes[dtype], device=self.device)
        else:
            with torch.cuda.stream(self.stream):
                kv = torch.empty(shape, dtype=self._dtypes[dtype], device=self.device)
        k, v = kv.unbind(0)
        if self.stream is None and self._current(self.device.index) != self._raw:
            _record_use(self.device, self.k, self.v, self.k_scale, self.v_scale)
        _bs._check(_on_device(self.device, self.stream, self._read, self._ref, _bs.DTYPES[dtype],
                              slots.data_ptr(), n, k.data_ptr(), v.data_ptr()), "bs_kvq_read")
        return k, v


def bs_kvq_reorder(p: int, caches: Sequence[QuantCache], gen_len: int) -> None:
    """bs_kv_paged_reorder of the paged cache ``p`` for layers of 8-bit caches."""
    arr = (bs_kvq_desc * len(caches))(*[c.desc for c in caches])
    _bs._check(attn_library().bs_kvq_reorder(p, arr, len(caches), gen_len), "bs_kvq_reorder")


class CacheAttention(_Handle):
    """Attention of batch * rows rows over a QuantCache (bs_cache_attn).

    ``att(q, cache, table, lens, prompt_table=None, prompt_lens=None)`` with q
    [batch * rows * q_len, heads, head_dim] returns the output, of q's shape and
    type: the handle's own tensor, written again by the next call, or ``out``.
    ``table`` is a tensor [batch * rows, max_blocks] or a PagedKV. Every call runs
    on the stream given here; without one, on the stream that was current when this was
    made, in order with the stream that is current at the call.
    """

    def __init__(self, batch, rows, heads, kv_heads, head_dim, block_size, max_blocks,
                 max_prompt_blocks=0, q_len=1, dtype="bf16", scale=None, stream=None):
        torch = _t()
        _int32(batch=batch, rows=rows, q_len=q_len, heads=heads, kv_heads=kv_heads,
               head_dim=head_dim, block_size=block_size, max_blocks=max_blocks,
               max_prompt_blocks=max_prompt_blocks)
        cfg = bs_cache_attn_config(batch, rows, q_len, heads, kv_heads, head_dim, block_size,
                                   max_blocks, max_prompt_blocks, _bs.DTYPES[dtype],
                                   head_dim ** -0.5 if scale is None else scale)
        self.cfg, self._lib = cfg, attn_library()
        self._create(self._lib.bs_cache_attn_create, cfg, stream)
        self._rows, self._n = batch * rows, batch * rows * q_len
        with _memory_of(stream):
            self.out = torch.empty((self._n, heads, head_dim), dtype=_torch_dtypes()[dtype],
                                   device=self.device)
        self._i32 = torch.int32

    def __call__(self, q, cache: QuantCache, table, lens, prompt_table=None, prompt_lens=None,
                 out=None):
        c, dev = self.cfg, self.device
        own = self.out
        _need(q, "q", dev, own.dtype)
        stride = _head_rows(q, "q", (self._n,), c.heads, c.head_dim)
        if cache.device != dev:
            raise ValueError(f"cache: on {cache.device}, expected {dev}")
        at, width = _table_arg(table, self._rows, dev, c.block_size)
        if width < c.max_blocks:
            raise ValueError(f"table: {width} entries per row, {c.max_blocks} needed")
        _need(lens, "lens", dev, self._i32, (self._rows,))
        if (prompt_table is None) != (prompt_lens is None):
            raise ValueError("prompt_table and prompt_lens go together")
        pt = pl = None
        if prompt_table is not None:
            _need(prompt_table, "prompt_table", dev, self._i32, (c.batch, c.max_prompt_blocks))
            _need(prompt_lens, "prompt_lens", dev, self._i32, (c.batch,))
            pt, pl = prompt_table.data_ptr(), prompt_lens.data_ptr()
        if out is None:
            out = own
        else:
            _need(out, "out", dev, own.dtype, tuple(own.shape))
        _bs._check(self._call(self._lib.bs_cache_attn, cache._ref, q.data_ptr(), stride, at,
                              width, lens.data_ptr(), pt, pl, out.data_ptr()), "bs_cache_attn")
        return out

    def close(self):
        if getattr(self, "h", None):
            self._lib.bs_cache_attn_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class CrossAttention(_Handle):
    """Attention of an item's rows to its encoder's states (bs_cross_attn).

    ``att(q, k, v, lens=None, mask=None)`` with q [batch, rows, heads, head_dim]
    (rows up to max_rows, evenly spaced), k and v [batch, keys, kv_heads,
    head_dim] (keys up to max_keys, any strides that keep head_dim contiguous),
    lens int32 [batch], mask uint8 or bool [batch, keys] (nonzero: seen) returns
    the output, of q's shape and type, contiguous: the handle's own memory,
    written again by the next call, or ``out``. Every call runs on the stream given
    here; without one, on the stream that was current when this was made, in order with
    the stream that is current at the call.
    """

    def __init__(self, batch, max_rows, heads, kv_heads, head_dim, max_keys, dtype="bf16",
                 scale=None, stream=None):
        torch = _t()
        _int32(batch=batch, max_rows=max_rows, heads=heads, kv_heads=kv_heads, head_dim=head_dim,
               max_keys=max_keys)
        cfg = bs_cross_attn_config(batch, max_rows, heads, kv_heads, head_dim, max_keys,
                                   _bs.DTYPES[dtype], head_dim ** -0.5 if scale is None else scale)
        self.cfg, self._lib = cfg, attn_library()
        self._create(self._lib.bs_cross_attn_create, cfg, stream)
        with _memory_of(stream):
            self._buf = torch.empty(batch * max_rows * heads * head_dim,
                                    dtype=_torch_dtypes()[dtype], device=self.device)
        self._i32, self._mask_types = torch.int32, (torch.uint8, torch.bool)
        self._outs = {}  # the views of _buf by their rows
        self._kv = bs_cross_kv()
        self._kv_ref = ctypes.addressof(self._kv)

    def __call__(self, q, k, v, lens=None, mask=None, out=None):
        c, dev = self.cfg, self.device
        dt = self._buf.dtype
        _need(q, "q", dev, dt)
        _need(k, "k", dev, dt)
        _need(v, "v", dev, dt)
        if q.dim() != 4 or not q.shape[1] <= c.max_rows:
            raise ValueError(f"q: shape {list(q.shape)}, at most {c.max_rows} rows")
        rows = q.shape[1]
        stride = _head_rows(q, "q", (c.batch, rows), c.heads, c.head_dim)
        n = k.shape[1] if k.dim() == 4 else -1
        if k.shape != (c.batch, n, c.kv_heads, c.head_dim) or v.shape != k.shape or \
                n > c.max_keys:
            raise ValueError(f"k, v: shapes {list(k.shape)}, {list(v.shape)}, expected two "
                             f"[{c.batch}, at most {c.max_keys}, {c.kv_heads}, {c.head_dim}]")
        kv = self._kv
        if k.is_contiguous() and v.is_contiguous():
            kv.head_stride = c.head_dim
            kv.pos_stride = c.kv_heads * c.head_dim
            kv.batch_stride = n * kv.pos_stride
        else:
            ks, vs = ([s if size > 1 else 0 for s, size in zip(t.stride()[:3], t.shape)]
                      for t in (k, v))
            if ks != vs or k.stride(3) != 1 or v.stride(3) != 1:
                raise ValueError("k, v: equal strides and a contiguous last dimension are needed")
            kv.batch_stride, kv.pos_stride, kv.head_stride = ks
        kv.k, kv.v = k.data_ptr() or None, v.data_ptr() or None
        lp = mp = None
        ms = n
        if lens is not None:
            _need(lens, "lens", dev, self._i32, (c.batch,))
            lp = lens.data_ptr()
        if mask is not None:
            if mask.device != dev or mask.dtype not in self._mask_types:
                raise ValueError(f"mask: {mask.dtype} on {mask.device}, expected uint8 or bool on {dev}")
            if tuple(mask.shape) != (c.batch, n) or (n > 1 and mask.stride(1) != 1):
                raise ValueError(f"mask: rows of contiguous values [{c.batch}, {n}] are needed")
            ms = mask.stride(0) if c.batch > 1 else n
            mp = mask.data_ptr() or None
        if out is None:
            out = self._outs.get(rows)
            if out is None:
                out = self._outs[rows] = \
                    self._buf[:c.batch * rows * c.heads * c.head_dim].view(q.shape)
        else:
            _need(out, "out", dev, dt, tuple(q.shape))
        _bs._check(self._call(self._lib.bs_cross_attn, q.data_ptr() or None, stride, rows,
                              self._kv_ref, n, lp, mp, ms, out.data_ptr() or None),
                   "bs_cross_attn")
        return out

    def close(self):
        if getattr(self, "h", None):
            self._lib.bs_cross_attn_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
