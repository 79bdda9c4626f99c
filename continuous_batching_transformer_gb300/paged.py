"""Operators on a paged KV cache, over torch tensors (see the paged section of include/cbt.h).

For a model of one's own that keeps its KV cache in the engine's page layout: ``PagedKV`` describes
a pool of pages, ``PageMap`` turns request lengths into block tables and slots, ``RopeAppend``
normalises and rotates q and k and writes k and v into the pages, ``Attention`` reads them.  The
handles check what they are given, borrow the tensors they were made with (which must outlive
them) and queue their work on the current stream of the pool's device; lengths, tables and the
free stack stay on the device, so a step can be captured in a CUDA graph.

The workspace, error words and outputs that a handle makes itself may be used on any stream of the
device, and are kept from reuse while queued work needs them, also where the handle goes before.  A
captured graph holds their addresses alone: its handles have to outlive it.  Order between streams that
use one handle, and the caller's own tensors, are the caller's to keep.  Threads may share a handle.

A step of one layer::

    cache = PagedKV(pool, block_table, kv_lens, page_tokens=128, n_kv_heads=8, head_dim=128)
    pages = PageMap(block_table, kv_lens, free_pages, free_count, page_tokens=128, max_tokens=8)
    rope = Rope(128, theta=1e6)
    append = RopeAppend(cache, rope, n_heads=32)
    attn = Attention(cache, n_heads=32, max_kv=4096)
    pages(new_lens)                                      # kv_lens and the free stack move on
    append(0, qkv, pages.positions, pages.slots, q)      # qkv: [tokens, (32 + 2 * 8) * 128]
    attn(0, q, out)                                      # one token per row
    pages.check()                                        # synchronises; raises on device errors
"""
from __future__ import annotations

import ctypes
import math
import operator
import threading

import torch

from . import binding as B

DEV_ERRORS = {B.DEV_PAGE_ID: "page id outside the pool", B.DEV_PAGES: "too few free pages",
              B.DEV_LENGTH: "row length out of range", B.DEV_TOKENS: "more tokens than max_tokens",
              B.DEV_TIMEOUT: "a kernel's bounded wait ran out"}


def page_bytes(page_tokens: int, n_kv_heads: int, head_dim: int, n_layers: int = 1) -> int:
    """Bytes of one page holding `n_layers` layers."""
    return 4 * n_layers * n_kv_heads * page_tokens * head_dim


def size32(v, what: str) -> int:
    """v, a whole number that a 32-bit field holds (ctypes cuts others without a word)."""
    n = operator.index(v)
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError(f"{what}: {n} does not fit 32 bits")
    return n


def _bad(t, what, dtypes, index, dims=None):
    """Raises what is wrong with t."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise TypeError(f"{what}: a tensor of {' or '.join(map(str, dtypes))} is wanted")
    if t.get_device() < 0 or (index is not None and t.get_device() != index):
        raise ValueError(f"{what}: is on {t.device}, not on {'a GPU' if index is None else f'cuda:{index}'}")
    raise ValueError(f"{what}: a contiguous tensor of {dims} dimensions is wanted, not one of shape "
                     f"{tuple(t.shape)} and strides {t.stride()}")


def _tensor(t, what, dtypes, index=None, dims=None):
    """t, checked: a tensor of one of the types, on GPU `index` (None: any), contiguous with `dims`
    dimensions."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.get_device() < 0 or \
            (index is not None and t.get_device() != index) or \
            (dims is not None and (t.dim() != dims or not t.is_contiguous())):
        _bad(t, what, dtypes, index, dims)
    return t


def _vec(t, what, index, n=None):
    """t's address: a contiguous int32 vector on GPU `index`, of n elements where n is given."""
    if t.dtype is not torch.int32 or t.get_device() != index or t.dim() != 1 or not t.is_contiguous():
        _bad(t, what, _I32, index, 1)
    if n is not None and t.numel() != n:
        raise ValueError(f"{what}: {t.numel()} elements, {n} are wanted")
    return t.data_ptr()


def _rows(t, what, dtypes, index, tokens, width):
    """The row stride of t, [tokens, ...] with rows of `width` contiguous elements."""
    if t.dtype not in dtypes or t.get_device() != index:
        _bad(t, what, dtypes, index)
    shape = t.shape
    if t.is_contiguous() and len(shape) >= 2 and shape[0] == tokens and t.numel() == tokens * width:
        return width
    if len(shape) < 2 or shape[0] != tokens or math.prod(shape[1:]) != width:
        raise ValueError(f"{what}: shape {tuple(shape)} is not {tokens} rows of {width}")
    inner = 1
    for n, s in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if n > 1 and s != inner:
            raise ValueError(f"{what}: rows are not contiguous (strides {t.stride()})")
        inner *= n
    return width if tokens <= 1 else t.stride(0)  # of a single row no stride is used


_I32, _BF16, _ROWS = (torch.int32,), (torch.bfloat16,), (torch.bfloat16, torch.float32)


class _Device:
    """Queues a handle's calls on its device's current stream, with that device current.

    own     device tensors that the handle made.  A stream other than the one they were made on waits
            for that one before its first call, and is made known to torch's allocator, so that
            their memory is not given away under queued work when the handle goes.
    parent  of the handle's cache
    Within a capture neither is done: a graph's first replay follows what the capture waited for, and a
    graph has to be outlived by its handles."""

    def __init__(self, index, own, parent=None):
        self.index, self.own, self.parent = index, own, parent
        with torch.cuda.device(index):
            stream = torch.cuda.current_stream()
            self.ready = None if torch.cuda.is_current_stream_capturing() else stream.record_event()
        self.streams = {stream.cuda_stream}
        if parent is not None:
            parent.join(stream.cuda_stream)

    def join(self, raw):
        if raw in self.streams:
            return
        if self.parent is not None:
            self.parent.join(raw)
        with torch.cuda.device(self.index):
            if torch.cuda.is_current_stream_capturing():
                return
            stream = torch.cuda.current_stream()
            if self.ready is not None:
                stream.wait_event(self.ready)
            for t in self.own:
                t.record_stream(stream)
        self.streams.add(raw)

    def __call__(self, fn, args):
        # the stream's handle alone: torch.cuda.current_stream builds an object around it (1 us)
        raw = torch._C._cuda_getCurrentRawStream(self.index)
        if raw not in self.streams:
            self.join(raw)
        if torch.cuda.current_device() == self.index:
            fn(args, raw)
        else:
            with torch.cuda.device(self.index):
                fn(args, raw)


def _read_err(err: torch.Tensor) -> None:
    code, info = err.tolist()
    if code:
        err.zero_()
        raise B.CbtError(-10, f"paged operator: {DEV_ERRORS.get(code, code)} ({info})")


class Rope:
    """Rotary frequencies (cbt_rope_config).  layout "half" or "interleaved"; scaling "none",
    "linear", "base" or "by_parts"."""

    def __init__(self, head_dim: int, rot_dim: int | None = None, layout: str = "half",
                 theta: float = 1e4, scaling: str = "none", factor: float = 1.0,
                 original_len: int = 0, beta_fast: float = 0.0, beta_slow: float = 0.0,
                 mscale: float = 0.0):
        if layout not in B.ROPE_LAYOUTS or scaling not in B.ROPE_SCALINGS:
            raise ValueError(f"layout {layout!r}, scaling {scaling!r}")
        self.head_dim = size32(head_dim, "head_dim")
        self.config = B.RopeConfig(B.ROPE_LAYOUTS[layout],
                                   head_dim if rot_dim is None else size32(rot_dim, "rot_dim"),
                                   B.ROPE_SCALINGS[scaling], size32(original_len, "original_len"), theta,
                                   factor, beta_fast, beta_slow, mscale)
        self.desc = B.rope_init(self.config, head_dim)


class PagedKV:
    """A pool of pages, each holding K and V of `n_layers` layers for `page_tokens` positions.

    pool         1-D contiguous bf16 or uint8 tensor, 256-byte aligned; its length gives the pages
    block_table  int32 [rows, max_pages], kv_lens int32 [rows]: which pages a row holds and how
                 many positions (both may be None for a cache that is only appended to by slot)
    """

    def __init__(self, pool, block_table, kv_lens, *, page_tokens: int, n_kv_heads: int,
                 head_dim: int, n_layers: int = 1):
        for n, what in ((page_tokens, "page_tokens"), (n_kv_heads, "n_kv_heads"), (head_dim, "head_dim"),
                        (n_layers, "n_layers")):
            size32(n, what)
        _tensor(pool, "pool", (torch.bfloat16, torch.uint8), dims=1)
        self.device = pool.device
        self.index = pool.get_device()
        self.pool, self.block_table, self.kv_lens = pool, block_table, kv_lens
        self.rows = 0
        if block_table is not None or kv_lens is not None:
            _tensor(block_table, "block_table", _I32, self.index, 2)
            _tensor(kv_lens, "kv_lens", _I32, self.index, 1)
            if kv_lens.shape[0] != block_table.shape[0]:
                raise ValueError("block_table and kv_lens have different numbers of rows")
            self.rows = block_table.shape[0]
        self.page_tokens, self.n_kv_heads, self.head_dim = page_tokens, n_kv_heads, head_dim
        if min(page_tokens, n_kv_heads, head_dim, n_layers) <= 0:
            raise ValueError("page_tokens, n_kv_heads, head_dim and n_layers are positive")
        self.n_layers = n_layers
        size = pool.numel() * pool.element_size()
        step = page_bytes(page_tokens, n_kv_heads, head_dim, n_layers)
        self.n_pages = size // step
        if self.n_pages == 0:
            raise ValueError(f"pool: {size} bytes hold no page of {step}")
        block = step // (2 * n_layers)
        self.layers = [B.PagedKvDesc(pool.data_ptr(), size, step, 2 * l * block, (2 * l + 1) * block,
                                     self.n_pages, page_tokens, n_kv_heads, head_dim)
                       for l in range(n_layers)]
        self.err = torch.zeros(2, dtype=torch.int32, device=self.device)
        self.call = _Device(self.index, [self.err])

    def check(self) -> None:
        """Wait for the work queued on the current stream and raise if a kernel found an error."""
        _read_err(self.err)


class PageMap:
    """Block tables and slot maps (cbt_page_map).

    block_table, kv_lens  as in PagedKV; rewritten by every call
    free_pages, free_count  int32 stack of free page ids and its count [1], or None, None: rows
                 find the pages they grow into in their table already
    n_pages      pages in the pool (ids are below it); free_pages' length where that is given
    A call fills cu_q [rows + 1], positions and slots [max_tokens], tensors of the handle (or, at
    construction, the caller's), which later calls overwrite.  Until the first they name no token."""

    def __init__(self, block_table, kv_lens, free_pages, free_count, *, page_tokens: int,
                 max_tokens: int, n_pages: int | None = None, cu_q=None, positions=None, slots=None):
        for n, what in ((page_tokens, "page_tokens"), (max_tokens, "max_tokens"),
                        (0 if n_pages is None else n_pages, "n_pages")):
            size32(n, what)
        _tensor(block_table, "block_table", _I32, dims=2)
        self.index = block_table.get_device()
        rows, max_pages = block_table.shape
        _vec(_tensor(kv_lens, "kv_lens", _I32, self.index), "kv_lens", self.index, rows)
        if (free_pages is None) != (free_count is None):
            raise ValueError("free_pages and free_count go together")
        if free_pages is not None:
            _tensor(free_pages, "free_pages", _I32, self.index, 1)
            _vec(_tensor(free_count, "free_count", _I32, self.index), "free_count", self.index, 1)
            if n_pages is not None and n_pages != free_pages.shape[0]:
                raise ValueError("n_pages is not the length of free_pages")
            n_pages = free_pages.shape[0]
        if n_pages is None:
            raise ValueError("n_pages is wanted where there is no free stack")
        if max_tokens < 0:
            raise ValueError("max_tokens is negative")

        own = []

        def new(t, what, n, none=-1):
            if t is None:
                own.append(torch.full((n,), none, dtype=torch.int32, device=block_table.device))
                return own[-1]
            _vec(_tensor(t, what, _I32, self.index), what, self.index, n)
            return t
        self.cu_q = new(cu_q, "cu_q", rows + 1, 0)
        self.positions = new(positions, "positions", max_tokens)
        self.slots = new(slots, "slots", max_tokens)
        self.err = torch.zeros(2, dtype=torch.int32, device=block_table.device)
        self.rows = rows
        self._keep = (block_table, kv_lens, free_pages, free_count)
        self._lock = threading.Lock()  # a call's arguments are its own until it is queued
        opt = lambda t: None if t is None else t.data_ptr()
        self.args = B.PageMapArgs(block_table.data_ptr(), max_pages, page_tokens, n_pages, rows,
                                  kv_lens.data_ptr(), None, opt(free_pages), opt(free_count),
                                  max_tokens, None, None, self.cu_q.data_ptr(),
                                  self.positions.data_ptr(), self.slots.data_ptr(),
                                  self.err.data_ptr())
        self.call = _Device(self.index, own + [self.err])

    def __call__(self, new_lens, kv_lens_out=None, free_count_out=None) -> None:
        """One step: row b takes new_lens[b] more positions (negative: it retires).  The lengths
        and the count afterwards go to kv_lens and free_count, or to the tensors given."""
        a, dev = self.args, self.index
        with self._lock:
            a.new_lens = _vec(new_lens, "new_lens", dev, self.rows)
            a.kv_lens_out = a.kv_lens if kv_lens_out is None else \
                _vec(kv_lens_out, "kv_lens_out", dev, self.rows)
            a.free_count_out = a.free_count if free_count_out is None else \
                _vec(free_count_out, "free_count_out", dev, 1)
            if self.rows == 0:  # queues nothing; no token is what the outputs say
                self.call(self._none, a)
            self.call(B.page_map, a)

    def _none(self, a, stream):
        self.cu_q.zero_()
        self.positions.fill_(-1)
        self.slots.fill_(-1)

    def check(self) -> None:
        _read_err(self.err)


class RopeAppend:
    """Per-head norm, rotary positions and KV append (cbt_rope_append).  rope None: no rotation."""

    def __init__(self, cache: PagedKV, rope: Rope | None, *, n_heads: int, eps: float = 1e-6):
        if rope is not None and rope.head_dim != cache.head_dim:
            raise ValueError("rope and cache have different head_dim")
        self.cache, self.rope, self.n_heads = cache, rope, size32(n_heads, "n_heads")
        self.width = (n_heads + 2 * cache.n_kv_heads) * cache.head_dim
        self.q_width = n_heads * cache.head_dim
        self._layer = None
        self._lock = threading.Lock()
        self.args = B.RopeAppendArgs()
        self.args.rope = None if rope is None else ctypes.pointer(rope.desc)
        self.args.n_heads = n_heads
        self.args.eps = eps
        self.args.err = cache.err.data_ptr()

    def __call__(self, layer: int, qkv, positions, slots, q_out, q_gain=None, k_gain=None) -> None:
        """qkv [tokens, (n_heads + 2 n_kv_heads) * head_dim] bf16 or fp32, q_out [tokens, n_heads,
        head_dim] (or two dimensions) bf16; rows may be strided.  positions and slots int32, at
        least `tokens` long (the first `tokens` are used); gains bf16 [head_dim] or None."""
        c, a = self.cache, self.args
        dev = c.index
        with self._lock:
            a.tokens = tokens = qkv.shape[0]
            if layer != self._layer:
                a.kv = c.layers[layer]
                self._layer = layer
            a.qkv_stride = _rows(qkv, "qkv", _ROWS, dev, tokens, self.width)
            a.q_stride = _rows(q_out, "q_out", _BF16, dev, tokens, self.q_width)
            a.positions = _vec(positions, "positions", dev)
            a.slots = _vec(slots, "slots", dev)
            if positions.numel() < tokens or slots.numel() < tokens:
                raise ValueError(f"positions and slots: fewer than {tokens} elements")
            a.q_gain = None if q_gain is None else self._gain(q_gain, "q_gain")
            a.k_gain = None if k_gain is None else self._gain(k_gain, "k_gain")
            a.qkv, a.q_out = qkv.data_ptr(), q_out.data_ptr()
            a.qkv_dtype = B.DTYPE_F32 if qkv.dtype is torch.float32 else B.DTYPE_BF16
            c.call(B.rope_append, a)

    def _gain(self, t, what):
        if _tensor(t, what, _BF16, self.cache.index, 1).numel() != self.cache.head_dim:
            raise ValueError(f"{what}: {t.numel()} elements, {self.cache.head_dim} are wanted")
        return t.data_ptr()


class Attention:
    """Attention over the cache's pages (cbt_paged_attention), with a workspace of its own.

    max_kv, max_q  upper bounds of a row's positions and query tokens.  With max_q > 1 they also decide how
                 the work is cut: bounds far above the rows cost time.  Weights are then rounded to
                 bf16, which with max_q == 1 they are not
    max_tokens     most rows of q in a call (default: the cache's rows, one token each)
    window, sinks  0: causal; else position p sees j > p - window and j < sinks
    Calls of one handle share its workspace: they may not overlap on the GPU (two streams, or two
    captured graphs replayed side by side, take a handle each)."""

    def __init__(self, cache: PagedKV, *, n_heads: int, max_kv: int, max_q: int = 1,
                 max_tokens: int | None = None, window: int = 0, sinks: int = 0,
                 scale: float | None = None):
        if cache.block_table is None:
            raise ValueError("the cache has no block table")
        for n, what in ((n_heads, "n_heads"), (max_kv, "max_kv"), (max_q, "max_q"),
                        (0 if max_tokens is None else max_tokens, "max_tokens"), (window, "window"),
                        (sinks, "sinks")):
            size32(n, what)
        self.cache, self.n_heads = cache, n_heads
        self.width = n_heads * cache.head_dim
        self._layer = None
        self._lock = threading.Lock()
        self.max_tokens = cache.rows if max_tokens is None else max_tokens
        a = self.args = B.PagedAttentionArgs()
        a.kv = cache.layers[0]
        a.block_table, a.max_pages, a.rows = (cache.block_table.data_ptr(),
                                              cache.block_table.shape[1], cache.rows)
        a.kv_lens = cache.kv_lens.data_ptr()
        a.tokens, a.max_q, a.max_kv, a.n_heads = self.max_tokens, max_q, max_kv, n_heads
        a.scale = 1 / math.sqrt(cache.head_dim) if scale is None else scale
        a.window, a.sinks = window, sinks
        a.err = cache.err.data_ptr()
        n = B.paged_attention_workspace(a)
        self.workspace = torch.empty(n, dtype=torch.uint8, device=cache.device) if n else None
        a.workspace = self.workspace.data_ptr() if n else None
        a.workspace_bytes = n
        self.call = _Device(cache.index, [self.workspace] if n else [], cache.call)

    def __call__(self, layer: int, q, out, cu_q=None) -> None:
        """q [tokens, n_heads, head_dim] (or two dimensions) bf16, out the same shape in bf16 or
        fp32; rows may be strided.  cu_q int32 [rows + 1]: row b's query tokens; None: one each."""
        c, a = self.cache, self.args
        dev = c.index
        with self._lock:
            tokens = q.shape[0]
            if layer != self._layer:
                a.kv = c.layers[layer]
                self._layer = layer
            a.q_stride = _rows(q, "q", _BF16, dev, tokens, self.width)
            a.out_stride = _rows(out, "out", _ROWS, dev, tokens, self.width)
            if tokens > self.max_tokens:
                raise ValueError(f"q: {tokens} rows, at most {self.max_tokens}")
            if cu_q is None:
                if tokens != c.rows:
                    raise ValueError(f"q: {tokens} rows for {c.rows} sequences and no cu_q")
                if a.max_q != 1:
                    raise ValueError("a handle with max_q > 1 wants cu_q")
                a.cu_q = None
            else:
                a.cu_q = _vec(cu_q, "cu_q", dev, c.rows + 1)
            a.q, a.out, a.tokens = q.data_ptr(), out.data_ptr(), tokens
            a.out_dtype = B.DTYPE_F32 if out.dtype is torch.float32 else B.DTYPE_BF16
            self.call(B.paged_attention, a)
