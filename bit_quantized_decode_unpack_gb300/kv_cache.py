"""Paged 8-bit KV cache: quantising append, attention over it, page operations.

What a decode step needs between its k/v projections and its o projection
(both served by ``quant_linear``).  A value is stored as code * scale with an
8-bit code (int8 or e4m3) and one fp32 scale for each block of 16 tokens and
head; sequences list their pages in an int32 table on the device, so every
call below is asynchronous and none reads anything back.

    cache = KVCache.empty(layers=1, pages=4096, kv_heads=8, head_dim=128, rows=32, row_pages=128)
    base, status = cache.reserve(counts)            # pages for the step's tokens; lens grows
    cache.append(k, v, base, starts)                # per layer: quantise into the pages
    out, lse = cache.attend(q, starts, max_new=5)   # per layer
    cache = cache.truncate(keep)                    # drop rejected draft tokens, free their pages

``starts`` (int32 [rows + 1], on the device) gives each row's tokens in the
ragged q, k and v; without it every row has one token.  ``fork`` makes new
rows from old ones (beams, reordering, freeing) by sharing pages; a shared,
partly filled page is copied when ``reserve`` next extends one of its rows.
``compact`` moves the live pages to the low end of the pool.

Arguments are checked here (type, shape, device, strides) and again, as far as
a host can, by the C entry points of the same names; every step of the
computation runs in the library's kernels.
"""
from __future__ import annotations

import ctypes
import math

from . import DTYPE_BF16, DTYPE_F16, _check, load

BLOCK = 16
FORMATS = {"int8": 1, "e4m3": 2}
torch = None     # bound when the first cache is made: importing the package needs no torch
_device = _raw_stream = None  # the current device's index, a device's current stream
_KINDS = {}      # element types of q, k and v
PAGE_TOKENS = (16, 32, 64, 128, 256)
HEAD_DIMS = (64, 128, 256)
MASK_WORDS = 16  # BQD_TREE_MAX_WORDS


class CacheStruct(ctypes.Structure):
    """bqd_kv_cache (include/bqd.h)."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("refs", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("layers", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_tokens", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("row_pages", ctypes.c_int32), ("format", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def declare(lib):
    """Argument types of the cache's entry points."""
    i64, i32, vp, cp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.POINTER(CacheStruct)
    lib.bqd_kv_append.argtypes = [cp, i32, vp, i64, i64, vp, i64, i64, i32, vp, vp, i64, i64, vp]
    lib.bqd_kv_attend.argtypes = [cp, i32, vp, i64, i64, i32, i32, vp, i64, i64, i64, ctypes.c_float, i64, vp, vp, vp,
                                  i64, vp]
    lib.bqd_kv_attend_masked.argtypes = [cp, i32, vp, i64, i64, i32, i32, vp, i64, i64, i64, ctypes.c_float, i64, vp, i32,
                                         vp, vp, vp, vp, i64, vp]
    lib.bqd_kv_accept.argtypes = [cp, cp, vp, i32, vp, vp]
    for f in (lib.bqd_kv_attend_workspace, lib.bqd_kv_attend_masked_workspace):
        f.argtypes, f.restype = [cp, i32, i64, i64, i64, i64], i64
    lib.bqd_kv_reserve.argtypes = [cp, vp, vp, vp, vp, vp]
    lib.bqd_kv_fork.argtypes = [cp, cp, vp, vp, vp]
    lib.bqd_kv_compact.argtypes = [cp, cp, vp, vp, vp]
    lib.bqd_kv_copy_pages.argtypes = [cp, vp, vp, i64, vp]
    for f in ("append", "attend", "attend_masked", "reserve", "fork", "accept", "compact", "copy_pages"):
        getattr(lib, f"bqd_kv_{f}").restype = i32


def _bind():
    """Binds the module's torch."""
    global torch, _device, _raw_stream
    if torch is None:
        import torch as t
        _KINDS.update({t.float16: DTYPE_F16, t.bfloat16: DTYPE_BF16})
        _device, _raw_stream = t.cuda.current_device, t._C._cuda_getCurrentRawStream
        torch = t


def _dense(t, name, dtype, shape, device):
    """A dense tensor of this type and shape on this device (an integer array that a kernel indexes)."""
    if t is None or t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        got = None if t is None else f"{t.dtype} {tuple(t.shape)} on {t.device}"
        raise ValueError(f"{name}: must be a contiguous {dtype} tensor of shape {shape} on {device}, got {got}")
    return t


class _On:
    """Makes the cache's device current, and allocates on the stream that is used."""

    def __init__(self, device, stream):
        self.device, self.stream = device, stream

    def __enter__(self):
        self.a = torch.cuda.device(self.device)
        self.a.__enter__()
        self.b = torch.cuda.stream(self.stream)
        self.b.__enter__()

    def __exit__(self, *e):
        self.b.__exit__(*e)
        self.a.__exit__(*e)


class KVCache:
    """A cache over the caller's tensors (bqd_kv_cache; nothing is copied).

    k, v: int8 (or uint8) or float8_e4m3fn [layers, pages, kv_heads, page_tokens, head_dim];
    k_scales, v_scales: fp32 [layers, pages, kv_heads, page_tokens / 16];
    table: int32 [rows, row_pages]; lens: int32 [rows]; refs: int32 [pages]."""

    def __init__(self, k, v, k_scales, v_scales, table, lens, refs):
        _bind()
        if getattr(k, "dim", lambda: 0)() != 5 or not k.is_cuda:
            raise ValueError("k must be a CUDA tensor [layers, pages, kv_heads, page_tokens, head_dim]")
        kinds = {torch.int8: "int8", torch.uint8: "int8", torch.float8_e4m3fn: "e4m3"}
        if k.dtype not in kinds:
            raise ValueError(f"k: dtype {k.dtype}, expected int8 or float8_e4m3fn")
        layers, pages, heads, pt, d = k.shape
        if pt not in PAGE_TOKENS or d not in HEAD_DIMS:
            raise ValueError(f"page_tokens must be one of {PAGE_TOKENS} and head_dim one of {HEAD_DIMS}, got {pt} and {d}")
        if min(layers, pages, heads) < 1:
            raise ValueError("layers, pages and kv_heads must be at least 1")
        dev, i32 = k.device, torch.int32
        _dense(k, "k", k.dtype, tuple(k.shape), dev)
        _dense(v, "v", k.dtype, tuple(k.shape), dev)
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            _dense(t, name, torch.float32, (layers, pages, heads, pt // BLOCK), dev)
        if getattr(table, "dim", lambda: 0)() != 2 or table.shape[1] < 1:
            raise ValueError("table must be int32 [rows, row_pages] with row_pages >= 1")
        rows, width = table.shape
        _dense(table, "table", i32, (rows, width), dev)
        _dense(lens, "lens", i32, (rows,), dev)
        _dense(refs, "refs", i32, (pages,), dev)
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.format = kinds[k.dtype]
        self.layers, self.pages, self.kv_heads, self.page_tokens, self.head_dim = layers, pages, heads, pt, d
        self.device, self._index, self._scale = dev, dev.index, 1.0 / math.sqrt(d)
        self._lib = load()
        self._attend, self._append = self._lib.bqd_kv_attend, self._lib.bqd_kv_append
        self._need = (None, 0)  # the last call's sizes and bytes of scratch
        p = lambda t: t.data_ptr() or None
        self._own(table, lens, refs, CacheStruct(p(k), p(v), p(k_scales), p(v_scales), None, None, None, pages, layers,
                                                 heads, d, pt, 0, table.shape[1], FORMATS[self.format], 0))

    def _own(self, table, lens, refs, c):
        """Takes the table, lens and refs, and a struct with the rest filled in."""
        self.table, self.lens, self.refs = table, lens, refs
        self.rows, self.row_pages = table.shape
        c.table, c.lens, c.refs, c.rows = table.data_ptr() or None, lens.data_ptr() or None, refs.data_ptr(), self.rows
        self._c, self._ref = c, ctypes.byref(c)

    @classmethod
    def empty(cls, layers: int, pages: int, kv_heads: int, head_dim: int, rows: int, row_pages: int,
              page_tokens: int = 64, format: str = "int8", device="cuda"):
        """A cache of its own memory with every page free and every row empty."""
        _bind()
        if format not in FORMATS:
            raise ValueError(f"format must be one of {sorted(FORMATS)}, got {format!r}")
        kind = torch.int8 if format == "int8" else torch.float8_e4m3fn
        shape = (layers, pages, kv_heads, page_tokens, head_dim)
        k, v = (torch.empty(shape, dtype=torch.int8, device=device).view(kind) for _ in range(2))
        ks, vs = (torch.empty(shape[:3] + (page_tokens // BLOCK,), dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs, torch.full((rows, row_pages), -1, dtype=torch.int32, device=device),
                   torch.zeros(rows, dtype=torch.int32, device=device),
                   torch.zeros(pages, dtype=torch.int32, device=device))

    def _sibling(self, rows, out):
        """A cache over the same pools with a table, lens and refs of its own."""
        if out is not None:
            same = isinstance(out, KVCache) and out.rows == rows and out.row_pages == self.row_pages and \
                out.k is self.k and out.v is self.v and out.k_scales is self.k_scales and out.v_scales is self.v_scales
            if not same or out is self:
                raise ValueError(f"out: must be another KVCache of {rows} rows over the same pools")
            return out
        new = object.__new__(KVCache)
        new.__dict__.update(self.__dict__)
        new._need = (None, 0)
        i32, dev = torch.int32, self.device
        new._own(torch.empty((rows, self.row_pages), dtype=i32, device=dev), torch.empty(rows, dtype=i32, device=dev),
                 torch.empty(self.pages, dtype=i32, device=dev), CacheStruct.from_buffer_copy(self._c))
        return new

    def _on(self, stream):
        """None, or a context that a call has to run in: another current device, or an explicit stream."""
        if stream is None and _device() == self._index:
            return None
        return _On(self.device, stream)

    def _stream(self):
        return _raw_stream(self._index)

    def _half(self, t, name, heads):
        """Element type of q, k or v: fp16 or bf16 [tokens, heads, head_dim] on the device, head_dim contiguous."""
        shape = getattr(t, "shape", ())
        if len(shape) != 3 or t.device != self.device:
            raise ValueError(f"{name}: must be a 3-D tensor [tokens, heads, head_dim] on {self.device}")
        kind = _KINDS.get(t.dtype)
        if kind is None:
            raise ValueError(f"{name}: dtype {t.dtype}, expected float16 or bfloat16")
        if shape[2] != self.head_dim or (heads and shape[1] != heads):
            raise ValueError(f"{name}: shape {tuple(shape)}, expected [tokens, {heads or 'q_heads'}, {self.head_dim}]")
        if t.stride(2) != 1:
            raise ValueError(f"{name}: head_dim must be contiguous")
        return kind

    def _ragged(self, starts, tokens, max_new):
        """Pointer of starts and the bound of a row's new tokens."""
        if starts is None:
            if tokens != self.rows:
                raise ValueError(f"without starts there is one token for each of {self.rows} rows, got {tokens}")
            return None, 1
        _dense(starts, "starts", torch.int32, (self.rows + 1,), self.device)
        if max_new is None:
            max_new = tokens
        elif max_new < 0:
            raise ValueError(f"max_new must be >= 0, got {max_new}")
        return starts.data_ptr(), max_new

    def _layer(self, layer):
        if not 0 <= layer < self.layers:
            raise ValueError(f"layer must be in [0, {self.layers}), got {layer}")
        return layer

    # ---- tokens ------------------------------------------------------------------

    def append(self, k, v, base, starts=None, *, layer: int = 0, max_new=None, stream=None):
        """Quantise new tokens into the pages (bqd_kv_append).

        k, v: fp16 or bf16 [tokens, kv_heads, head_dim], any strides of token and head;
        row r's tokens go to positions base[r], base[r] + 1, ... (base of ``reserve``;
        negative: skipped).  A row has at most ``max_new`` (default: all of them)."""
        kind = self._half(k, "k", self.kv_heads)
        if self._half(v, "v", self.kv_heads) != kind or v.shape[0] != k.shape[0]:
            raise ValueError("k and v must have the same dtype and number of tokens")
        tokens = k.shape[0]
        at, max_new = self._ragged(starts, tokens, max_new)
        _dense(base, "base", torch.int32, (self.rows,), self.device)
        on = self._on(stream)
        if on is not None:
            with on:
                return self.append(k, v, base, starts, layer=layer, max_new=max_new)
        ks, vs = k.stride(), v.stride()
        _check("bqd_kv_append", self._append(
            self._ref, self._layer(layer), k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], kind,
            base.data_ptr(), at, tokens, max_new, self._stream()))

    def attend(self, q, starts=None, *, layer: int = 0, scale=None, window: int = 0, max_new=None, max_len: int = 0,
               mask=None, depth=None, out=None, lse=None, stream=None):
        """Causal attention of the rows' last tokens over the cache (bqd_kv_attend).

        q: fp16 or bf16 [tokens, q_heads, head_dim], any strides of token and head; the cache
        already holds the queries' own tokens.  ``window`` > 0 keeps the last ``window`` keys
        of each query; ``scale`` defaults to 1 / sqrt(head_dim); ``max_len`` bounds the rows'
        lengths where the caller knows them (only speed depends on it).  With ``starts``, give
        ``max_new``, the most queries of a row: it selects the kernel and sizes the scratch, and
        without it a batch of single tokens is planned as one row of them all.

        ``mask`` (int64 [tokens, words], of ``tree_mask`` or any other) replaces the causal rule
        among a row's last n tokens, the n that starts gives it: every query sees the tokens before
        them, and of the n those whose bit is set in its words (bqd_kv_attend_masked).  With a
        window, ``depth`` (int32 [tokens]) places a query at the length before the n plus its
        depth, and the window hides tokens before the n; the mask alone decides on the n.  Returns
        (out [tokens, q_heads, head_dim], lse fp32 [tokens, q_heads]); tokens that no row has,
        and a row's queries beyond ``max_new``, are not written."""
        kind = self._half(q, "q", None)
        tokens, heads, d = q.shape
        if heads == 0 or heads % self.kv_heads:
            raise ValueError(f"q: {heads} heads are no multiple of {self.kv_heads} KV heads")
        at, max_new = self._ragged(starts, tokens, max_new)
        if window < 0 or max_len < 0:
            raise ValueError("window and max_len must be >= 0")
        if mask is not None or depth is not None:
            self._masks(mask, depth, tokens, window)
        on = self._on(stream)
        if on is not None:
            with on:
                return self.attend(q, starts, layer=layer, scale=scale, window=window, max_new=max_new,
                                   max_len=max_len, mask=mask, depth=depth, out=out, lse=lse)
        if out is None:
            out = torch.empty((tokens, heads, d), dtype=q.dtype, device=self.device)
        else:
            _dense(out, "out", q.dtype, (tokens, heads, d), self.device)
        if lse is None:
            lse = torch.empty((tokens, heads), dtype=torch.float32, device=self.device)
        else:
            _dense(lse, "lse", torch.float32, (tokens, heads), self.device)
        # scratch, from the allocator's pool of this stream: used by this call alone
        sizes = (heads, tokens, max_new, max_len, window, mask is not None)
        if self._need[0] != sizes:
            self._need = (sizes, self.attend_workspace(heads, tokens, max_new, max_len, window, masked=mask is not None))
        need = self._need[1]
        work = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
        qs = q.stride()
        if mask is not None:
            _check("bqd_kv_attend_masked", self._lib.bqd_kv_attend_masked(
                self._ref, self._layer(layer), q.data_ptr(), qs[0], qs[1], kind, heads, at, tokens, max_new, max_len,
                self._scale if scale is None else scale, window, mask.data_ptr(), mask.shape[1],
                None if depth is None else depth.data_ptr(), out.data_ptr(), lse.data_ptr(),
                work.data_ptr() if need else None, need, self._stream()))
            return out, lse
        _check("bqd_kv_attend", self._attend(
            self._ref, self._layer(layer), q.data_ptr(), qs[0], qs[1], kind, heads, at, tokens, max_new, max_len,
            self._scale if scale is None else scale, window, out.data_ptr(), lse.data_ptr(),
            work.data_ptr() if need else None, need, self._stream()))
        return out, lse

    def _masks(self, mask, depth, tokens, window):
        """Checks a masked call's tensors."""
        if mask is None:
            raise ValueError("depth: belongs to a mask")
        words = mask.shape[1] if getattr(mask, "dim", lambda: 0)() == 2 else 0
        if not 1 <= words <= MASK_WORDS:
            raise ValueError(f"mask: must be int64 [tokens, words] with words in [1, {MASK_WORDS}]")
        _dense(mask, "mask", torch.int64, (tokens, words), self.device)
        if depth is not None:
            _dense(depth, "depth", torch.int32, (tokens,), self.device)
        elif window:
            raise ValueError("depth: a window needs the queries' positions")

    def attend_workspace(self, q_heads: int, tokens: int, max_new: int, max_len: int = 0, window: int = 0, *,
                         masked: bool = False) -> int:
        """Bytes of scratch that ``attend`` takes for such a call (bqd_kv_attend_workspace, and
        bqd_kv_attend_masked_workspace for one with a mask)."""
        f = self._lib.bqd_kv_attend_masked_workspace if masked else self._lib.bqd_kv_attend_workspace
        return f(self._ref, q_heads, tokens, max_new, max_len, window)

    # ---- pages -------------------------------------------------------------------

    def reserve(self, counts=None, *, stream=None):
        """Room for counts[r] more tokens in each row (default: one in each row that is not
        empty), copying shared partly filled pages (bqd_kv_reserve).

        Returns (base int32 [rows]: where the new tokens go, -1 where the call failed;
        status int32 [2]: missing pages and rows that outgrow the table, (0, 0) on success)."""
        if counts is not None:
            _dense(counts, "counts", torch.int32, (self.rows,), self.device)
        on = self._on(stream)
        if on is not None:
            with on:
                return self.reserve(counts)
        base = torch.empty(self.rows, dtype=torch.int32, device=self.device)
        status = torch.empty(2, dtype=torch.int32, device=self.device)
        copies = torch.empty((self.rows, 2), dtype=torch.int32, device=self.device)
        _check("bqd_kv_reserve", self._lib.bqd_kv_reserve(
            self._ref, None if counts is None else counts.data_ptr(), base.data_ptr() or None, copies.data_ptr() or None,
            status.data_ptr(), self._stream()))
        return base, status

    def fork(self, parents, keep=None, *, out=None, stream=None):
        """The cache whose row i shares the pages of row parents[i]'s first keep[i] tokens
        (default: all; a parent outside [0, rows) gives an empty row), with the reference
        counts that follow (bqd_kv_fork).  It takes this cache's place: of the two, only one
        may go on.  parents, keep: int32 [new rows]."""
        if getattr(parents, "dim", lambda: 0)() != 1:
            raise ValueError("parents must be an int32 tensor [new rows]")
        rows = parents.shape[0]
        _dense(parents, "parents", torch.int32, (rows,), self.device)
        if keep is not None:
            _dense(keep, "keep", torch.int32, (rows,), self.device)
        on = self._on(stream)
        if on is not None:
            with on:
                return self.fork(parents, keep, out=out)
        new = self._sibling(rows, out)
        _check("bqd_kv_fork", self._lib.bqd_kv_fork(self._ref, new._ref, parents.data_ptr() or None,
                                                    None if keep is None else keep.data_ptr(), self._stream()))
        return new

    def truncate(self, keep, *, out=None, stream=None):
        """Each row cut to its first keep[r] tokens; pages that no row lists any more are free."""
        on = self._on(stream)
        if on is not None:
            with on:
                return self.truncate(keep, out=out)
        return self.fork(torch.arange(self.rows, dtype=torch.int32, device=self.device), keep, out=out)

    def accept(self, path, starts=None, *, out=None, stream=None):
        """Of each row's last tokens (starts[r + 1] - starts[r] of them, or one) keeps those that
        its path names, in every layer: token number path[r, k] of them becomes number k
        (bqd_kv_accept).  path int32 [rows, width] rises and ends before the first entry that does
        not, as ``spec_tree_verify`` returns it.  A row with fewer tokens than nodes has a node for
        each, counted from its first token.  Returns the cache that takes this one's place; pages
        that no row lists any more are free."""
        if getattr(path, "dim", lambda: 0)() != 2 or path.shape[1] < 1:
            raise ValueError("path must be an int32 tensor [rows, width]")
        _dense(path, "path", torch.int32, (self.rows, path.shape[1]), self.device)
        if starts is not None:
            _dense(starts, "starts", torch.int32, (self.rows + 1,), self.device)
        on = self._on(stream)
        if on is not None:
            with on:
                return self.accept(path, starts, out=out)
        new = self._sibling(self.rows, out)
        _check("bqd_kv_accept", self._lib.bqd_kv_accept(self._ref, new._ref, path.data_ptr() or None, path.shape[1],
                                                        None if starts is None else starts.data_ptr(), self._stream()))
        return new

    def compact(self, *, out=None, work=None, stream=None):
        """Moves the live pages to the low end of the pool (bqd_kv_compact).  Returns the cache
        that takes this one's place and an int32 [1] count of the pages that moved.  ``work``
        (int32 [2 * pages], else allocated) holds page q's new index in work[pages + q]
        afterwards: a caller that pins pages (counts of its own in refs) follows them by it."""
        if work is not None:
            _dense(work, "work", torch.int32, (2 * self.pages,), self.device)
        on = self._on(stream)
        if on is not None:
            with on:
                return self.compact(out=out, work=work)
        new = self._sibling(self.rows, out)
        moved = torch.empty(1, dtype=torch.int32, device=self.device)
        if work is None:
            work = torch.empty(2 * self.pages, dtype=torch.int32, device=self.device)
        _check("bqd_kv_compact", self._lib.bqd_kv_compact(self._ref, new._ref, work.data_ptr(), moved.data_ptr(),
                                                          self._stream()))
        return new, moved

    def copy_pages(self, src, dst, *, stream=None):
        """Copies page src[i] to page dst[i] in every layer (bqd_kv_copy_pages); int32 [n] each,
        no page in both nor twice in dst.  table and refs are the caller's to change."""
        if getattr(src, "dim", lambda: 0)() != 1:
            raise ValueError("src must be an int32 tensor [n]")
        n = src.shape[0]
        _dense(src, "src", torch.int32, (n,), self.device)
        _dense(dst, "dst", torch.int32, (n,), self.device)
        on = self._on(stream)
        if on is not None:
            with on:
                return self.copy_pages(src, dst)
        _check("bqd_kv_copy_pages", self._lib.bqd_kv_copy_pages(self._ref, src.data_ptr() or None,
                                                                dst.data_ptr() or None, n, self._stream()))


# the entry points' names, as functions of a cache
kv_append, kv_attend, kv_reserve = KVCache.append, KVCache.attend, KVCache.reserve
kv_attend_workspace = KVCache.attend_workspace
kv_fork, kv_compact, kv_copy_pages = KVCache.fork, KVCache.compact, KVCache.copy_pages
kv_accept = KVCache.accept


def kv_attend_masked(cache: KVCache, q, starts=None, *, mask=None, **how):
    """``attend`` with a mask (bqd_kv_attend_masked); a call without one is refused, not causal."""
    if mask is None:
        raise ValueError("mask: must be int64 [tokens, words] (attend without one is causal)")
    return cache.attend(q, starts, mask=mask, **how)


def kv_attend_masked_workspace(cache: KVCache, q_heads: int, tokens: int, max_new: int, max_len: int = 0, window: int = 0) -> int:
    """Bytes of scratch that ``attend`` takes with a mask (bqd_kv_attend_masked_workspace)."""
    return cache.attend_workspace(q_heads, tokens, max_new, max_len, window, masked=True)
