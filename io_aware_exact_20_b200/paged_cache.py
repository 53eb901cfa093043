"""Paged key / value cache: the tensors of ``fa_cache_t`` (include/fa.h) and its
calls.  Everything the calls decide (which pages are free, which are shared,
what has to be copied) is decided on the device, so none of them waits for it
and all of them can be captured in a CUDA graph."""

from __future__ import annotations

import ctypes

import io_aware_exact_20_b200 as _fa


class PagedCache:
    """Keys and values of up to ``slots`` sequences in pages of a common pool.

    k, v      bf16 [layers, pages, heads_kv, page_size, d], any strides with d
              contiguous (multiples of 8 elements)
    table     int32 [slots, max_pages]: page numbers, -1 where there is none
    lengths   int32 [slots]: tokens of each sequence
    refs      int32 [pages]: slots that hold a page, 0: free

    The tensors stay the caller's (they may be views of one buffer) and are
    changed in place; ``allocate`` makes an empty cache.  The library keeps their
    addresses, so these attributes and the sizes cannot be set: other tensors are
    another PagedCache.  Slots are given as int32 device tensors.  Calls on one
    cache have to be ordered: one stream, or events."""

    _FIXED = frozenset(("k", "v", "table", "lengths", "refs", "layers", "pages", "heads_kv", "page_size",
                        "head_dim", "slots", "max_pages", "device"))

    _sizes = None  # (set last; reading __dict__ here would slow every attribute's load down)

    def __setattr__(self, name, value):
        # (the same tensor comes back from an in-place operator, `cache.lengths += 1`)
        if name in self._FIXED and self._sizes is not None and value is not getattr(self, name):
            raise AttributeError(f"PagedCache.{name} cannot be replaced: its address and sizes are the "
                                 "library's already; make another PagedCache")
        object.__setattr__(self, name, value)

    def __init__(self, k, v, table, lengths, refs):
        import torch
        if k.dim() != 5 or v.shape != k.shape:
            raise ValueError("k, v: [layers, pages, heads_kv, page_size, d] tensors of one shape")
        if table.dim() != 2 or lengths.shape != table.shape[:1] or refs.shape != k.shape[1:2]:
            raise ValueError("table [slots, max_pages], lengths [slots], refs [pages] are expected")
        for name, t in (("k", k), ("v", v)):
            if not t.is_cuda or t.dtype != torch.bfloat16 or t.device != k.device:
                raise ValueError(f"{name}: bfloat16 on one CUDA device is expected")
            if t.stride(4) != 1:
                raise ValueError(f"{name}: the head dimension must be contiguous")
        for name, t in (("table", table), ("lengths", lengths), ("refs", refs)):
            if t.device != k.device or t.dtype != torch.int32 or not t.is_contiguous():
                raise ValueError(f"{name}: contiguous int32 on the device of k is expected")
        self.k, self.v, self.table, self.lengths, self.refs = k, v, table, lengths, refs
        self.layers, self.pages, self.heads_kv, self.page_size, self.head_dim = k.shape
        self.slots, self.max_pages = table.shape
        self.device = k.device
        a = _fa.CacheDesc()
        a.layers, a.pages, a.page_size = self.layers, self.pages, self.page_size
        a.heads_kv, a.head_dim = self.heads_kv, self.head_dim
        a.slots, a.max_pages = self.slots, self.max_pages
        a.k, a.v = k.data_ptr(), v.data_ptr()
        a.k_layer, a.v_layer = k.stride(0), v.stride(0)
        a.ks = _fa.Strides(k.stride(1), k.stride(2), k.stride(3))
        a.vs = _fa.Strides(v.stride(1), v.stride(2), v.stride(3))
        a.table, a.lengths, a.refs = table.data_ptr(), lengths.data_ptr(), refs.data_ptr()
        self._desc, self._ref = a, ctypes.byref(a)
        self._lib, self._torch, self._index = _fa.library(), torch, k.get_device()
        self._i32, self._bf16 = torch.int32, torch.bfloat16
        self._sizes = {}
        if self._lib.fa_cache_workspace_size(self._ref, 0) == 0:
            raise ValueError("the cache's sizes, strides or alignment are not supported (fa.h)")

    @classmethod
    def allocate(cls, layers, pages, page_size, heads_kv, head_dim, slots, max_pages, device="cuda"):
        """An empty cache: every page free, every slot empty."""
        import torch
        shape = (layers, pages, heads_kv, page_size, head_dim)
        kv = [torch.empty(shape, dtype=torch.bfloat16, device=device) for _ in range(2)]
        ints = lambda *s: torch.zeros(s, dtype=torch.int32, device=device)  # noqa: E731
        return cls(*kv, ints(slots, max_pages).fill_(-1), ints(slots), ints(pages))

    def _ints(self, name, t, n):
        if (t.dtype is not self._i32 or t.shape != (n,) or t.get_device() != self._index
                or not t.is_contiguous()):
            raise ValueError(f"{name}: a contiguous 1-D int32 tensor of {n} entries on the cache's "
                             f"device is expected, got {t.dtype} {tuple(t.shape)} on {t.device}")
        return t.data_ptr()

    def _queries(self, name, t, shape):
        """The strides of a tensor of the queries' shape."""
        st = t.stride()
        if (t.dtype is not self._bf16 or t.get_device() != self._index or t.shape != shape
                or st[2] != 1):
            raise ValueError(f"{name}: bfloat16 {tuple(shape)} on the cache's device, d contiguous, "
                             "is expected")
        return st

    def _workspace(self, call, n):
        size = self._sizes.get((call, n))
        if size is None:  # a function of the cache's sizes and n alone
            args = (self._ref,) if n is None else (self._ref, n)
            size = self._sizes[call, n] = getattr(self._lib, f"fa_cache_{call}_workspace_size")(*args)
        return self.lengths.new_empty(size // 4), size

    def _call(self, fn, *args):
        """The C call on the cache's device and that device's current stream."""
        c = self._torch._C
        if c._cuda_getDevice() == self._index:
            code = fn(self._ref, *args, c._cuda_getCurrentRawStream(self._index))
        else:
            with self._torch.cuda.device(self._index):
                code = fn(self._ref, *args, c._cuda_getCurrentRawStream(self._index))
        if code:
            _fa._check(code, fn.__name__)

    @_fa._nvtx("fa.cache.extend")
    def extend(self, slots, tokens):
        """Grows slots[i] by tokens[i]; returns start (int32 [n]), each entry's
        first new position, -1 where it was not granted (fa_cache_extend)."""
        n = slots.numel()
        start = self.lengths.new_empty(n)
        ws, size = self._workspace("extend", n)
        self._call(self._lib.fa_cache_extend, self._ints("slots", slots, n),
                   self._ints("tokens", tokens, n), n, start.data_ptr(), ws.data_ptr(), size)
        return start

    @_fa._nvtx("fa.cache.write")
    def write(self, layer, k, v, slots, start, cu_seqlens=None):
        """Writes k, v (bf16 [T, heads_kv, d]) of one layer to the positions
        start[i], start[i] + 1, ... of slots[i]: one row per entry, or with
        cu_seqlens (int32 [n + 1]) rows cu_seqlens[i] .. cu_seqlens[i + 1] - 1."""
        n, bf16, index = slots.numel(), self._bf16, self._index
        if not 0 <= layer < self.layers:
            layer = -1  # refused by the library (a C int would take 2^32 for 0)
        shape = k.shape
        if (len(shape) != 3 or shape[1] != self.heads_kv or shape[2] != self.head_dim
                or v.shape != shape):
            raise ValueError(f"k, v: [T, {self.heads_kv}, {self.head_dim}] of one shape are expected")
        sk, sv = k.stride(), v.stride()
        if (k.dtype is not bf16 or v.dtype is not bf16 or k.get_device() != index
                or v.get_device() != index or sk[2] != 1 or sv[2] != 1):
            raise ValueError("k, v: bfloat16 on the cache's device, d contiguous, are expected")
        if cu_seqlens is None and shape[0] != n:
            raise ValueError("write: one row per slot is expected without cu_seqlens")
        cu = None if cu_seqlens is None else self._ints("cu_seqlens", cu_seqlens, n + 1)
        self._call(self._lib.fa_cache_write, layer, k.data_ptr(), v.data_ptr(), sk[0], sk[1], sv[0],
                   sv[1], self._ints("slots", slots, n), self._ints("start", start, n), cu, n,
                   shape[0])

    @_fa._nvtx("fa.cache.attend")
    def attend(self, layer, q, slots=None, scale=None, window=0, sinks=0, out=None, lse=None):
        """O, LSE of one query per sequence (q bf16 [B, H, d]) over the keys of
        its slot (slots int32 [B]; None: slot b for query b), with a window and
        first tokens as in forward_general.  The newest token has to be in the
        cache.  LSE: fp32 [B, H]."""
        if not 0 <= layer < self.layers:
            layer = -1  # as in write
        shape = q.shape
        if len(shape) != 3 or shape[2] != self.head_dim:
            raise ValueError(f"q: [B, H, {self.head_dim}] is expected")
        B, H, d = shape
        if H < 1 or H % self.heads_kv:
            raise ValueError("q's heads must be a multiple of the cache's")
        sq = self._queries("q", q, shape)
        if out is None:
            out = self._torch.empty_like(q)
            so = out.stride()
        else:
            so = self._queries("out", out, shape)
        if lse is None:
            lse = q.new_empty((B, H), dtype=self._torch.float32)
        elif (lse.shape != (B, H) or lse.dtype is not self._torch.float32
              or lse.get_device() != self._index or not lse.is_contiguous()):
            raise ValueError(f"lse: contiguous float32 {(B, H)} on the cache's device is expected")
        window, sinks = _fa._window(window, sinks) if window or sinks else (0, 0)
        key = (B, H, window, sinks)
        size = self._sizes.get(key)
        if size is None:  # a function of the cache's sizes and these alone
            size = self._sizes[key] = self._lib.fa_cache_attend_workspace_size(self._ref, *key)
        ws = self.lengths.new_empty((size + 3) // 4) if size else None
        self._call(self._lib.fa_cache_attend, layer, q.data_ptr(), out.data_ptr(), lse.data_ptr(),
                   sq[0], sq[1], so[0], so[1],
                   None if slots is None else self._ints("slots", slots, B), B, H,
                   d ** -0.5 if scale is None else scale, window, sinks,
                   ws.data_ptr() if size else None, size)
        return out, lse

    @_fa._nvtx("fa.cache.fork")
    def fork(self, src, dst):
        """Slot dst[i] lets its pages go and shares src[i]'s (fa_cache_fork)."""
        n = src.numel()
        ws, size = self._workspace("fork", n)
        self._call(self._lib.fa_cache_fork, self._ints("src", src, n), self._ints("dst", dst, n), n,
                   ws.data_ptr(), size)

    @_fa._nvtx("fa.cache.free")
    def free(self, slots):
        """The slots let their pages go and become empty."""
        n = slots.numel()
        self._call(self._lib.fa_cache_free, self._ints("slots", slots, n), n)

    @_fa._nvtx("fa.cache.compact")
    def compact(self):
        """Moves the pages in use into the lowest numbers; returns how many there
        are (int32 [1], on the device)."""
        used = self.lengths.new_empty(1)
        ws, size = self._workspace("compact", None)
        self._call(self._lib.fa_cache_compact, used.data_ptr(), ws.data_ptr(), size)
        return used

    @_fa._nvtx("fa.cache.copy_pages")
    def copy_pages(self, src, dst, source=None):
        """Copies page src[i] (of the cache `source`, default this one) to page
        dst[i], every layer; the book-keeping stays (fa_cache_copy_pages)."""
        if source is not None and source.device != self.device:
            raise ValueError("copy_pages: both caches on one device are expected")
        n = src.numel()
        ws, size = self._workspace("copy_pages", n)
        self._call(self._lib.fa_cache_copy_pages, None if source is None else source._ref,
                   self._ints("src", src, n), self._ints("dst", dst, n), n, ws.data_ptr(), size)
