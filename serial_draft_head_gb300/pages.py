"""Thin ctypes binding of include/dspark_pages.h: the page tables of a paged cache, kept on the GPU.

    pool = Pages(n_pages, page_size, requests, max_pages)
    first, slot, position = pool.grow(length, count, n_rows)     # a round's rows, and pages for them
    q = tree.place(cache, slot, q, k, v, position, rotation)
    out, lse = tree.attend(q, cache, pool.table, length, first)
    pool.trim(length + kept)                                     # pages that are not needed go back

Lengths and counts stay on the device; nothing here waits for it but `status`.  Calls on one pool
are ordered by the caller.  There is no fallback.
"""
import ctypes

import torch

from . import walk
from .tree import _need, _raw_stream
from .walk import WalkError

PAGES_MAX_REQUESTS = 1024

EXPORTS = ["dspark_pages_reset", "dspark_pages_grow", "dspark_pages_trim", "dspark_pages_status"]


class dspark_pages(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("held", ctypes.c_void_p), ("free", ctypes.c_void_p),
                ("n_free", ctypes.c_void_p), ("state", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("requests", ctypes.c_int),
                ("max_pages", ctypes.c_int)]


_int32 = torch.int32
_lib = None


def load():
    """The library with this header's signatures."""
    global _lib
    if _lib is None:
        L = walk.load()
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        L.dspark_pages_reset.argtypes = [vp, vp]
        L.dspark_pages_grow.argtypes = [vp, vp, vp, i32, vp, i64, i32, vp, vp, vp, vp]
        L.dspark_pages_trim.argtypes = [vp, vp, vp]
        L.dspark_pages_status.argtypes = [vp, vp]
        for name in EXPORTS:
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


class Pages:
    """The pages of a cache of n_pages pages and who holds them: `table` int32 [requests, max_pages]
    (-1 where a request holds none; the page table that the tree operators take), `held` int32
    [requests], `free` int32 [n_pages] of which the first `n_free` [1] are free."""

    def __init__(self, n_pages, page_size, requests, max_pages, device=None):
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None \
            else torch.device(device)
        _need(self.device.type == "cuda", "the pool's device is a CUDA device")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        _need(1 <= requests <= PAGES_MAX_REQUESTS, "1 to %d requests" % PAGES_MAX_REQUESTS)
        _need(min(n_pages, page_size, max_pages) >= 1 and max(n_pages, max_pages) * page_size < 2 ** 31,
              "pages and slots are at least 1 and fewer than 2^31 in all")
        self.lib = load()
        self.n_pages, self.page_size, self.requests, self.max_pages = n_pages, page_size, requests, max_pages

        def ints(*shape):
            return torch.empty(shape, dtype=_int32, device=self.device)

        self.table, self.held, self.free, self.n_free = ints(requests, max_pages), ints(requests), ints(n_pages), ints(1)
        self._state = torch.zeros(2, dtype=_int32, device=self.device)
        self._index = self.device.index
        self.c = dspark_pages(self.table.data_ptr(), self.held.data_ptr(), self.free.data_ptr(),
                              self.n_free.data_ptr(), self._state.data_ptr(), max_pages, n_pages, page_size,
                              requests, max_pages)
        self._at = ctypes.addressof(self.c)
        self.reset()
        torch.cuda.current_stream(self.device).synchronize()     # ready for calls on any stream

    def _call(self, what, *args):
        if torch.cuda.current_device() == self._index:
            rc = getattr(self.lib, what)(self._at, *args)
        else:
            with torch.cuda.device(self.device):
                rc = getattr(self.lib, what)(self._at, *args)
        if rc:
            raise WalkError(rc, what)

    def _stream(self, stream):
        return _raw_stream(self._index) if stream is None else walk._stream(stream)

    def _empty(self, n):
        return torch.empty(n, dtype=_int32, device=self.device)

    def _numbers(self, x):
        if not (x.dtype is _int32 and x.get_device() == self._index and x.shape == (self.requests,)
                and (x.stride(0) == 1 or self.requests == 1)):
            raise ValueError("lengths and counts are int32 [requests] on the pool's device")
        return x.data_ptr()

    def reset(self, stream=None):
        """All pages free."""
        self._call("dspark_pages_reset", self._stream(stream))

    def grow(self, length, count, n_rows, mask=None, out=None, stream=None):
        """Pages for count[r] more rows of each request behind its length[r], and (first int32
        [requests + 1], slot int32 [n_rows], position int32 [n_rows]) of the rows: where each goes in
        the cache and its position, with mask int32 [n_rows, words] (see `ancestor_bits`) by its depth
        in the tree.  Rows past the last request's have slot -1.  Free pages go to the requests in
        order: from the first that they do not serve on, those that lack a page get none, also where
        one is left, and slot -1; so do requests that do not fit, and `status` says so."""
        at_length, at_count = self._numbers(length), self._numbers(count)
        if not 0 <= n_rows < 2 ** 31:
            raise ValueError("n_rows is from 0 on and below 2^31")
        m, ms, mw = None, 0, 0
        if mask is not None:
            if not (mask.dtype is _int32 and mask.get_device() == self._index and mask.dim() == 2
                    and mask.shape[0] == n_rows and (mask.shape[1] >= 1 or n_rows == 0)
                    and (mask.shape[1] <= 1 or mask.stride(1) == 1)):
                raise ValueError("mask is int32 [n_rows, words] on the pool's device, words next to each other")
            m, ms, mw = mask.data_ptr(), mask.stride(0), mask.shape[1]
        if out is None:
            if stream is None:
                first, slot, position = self._empty(self.requests + 1), self._empty(n_rows), self._empty(n_rows)
            else:
                s = torch.cuda.ExternalStream(stream, device=self.device) if isinstance(stream, int) else stream
                with torch.cuda.stream(s):           # the blocks belong to the stream that fills them
                    first, slot, position = self._empty(self.requests + 1), self._empty(n_rows), self._empty(n_rows)
        else:
            first, slot, position = out
            for x, n in ((first, self.requests + 1), (slot, n_rows), (position, n_rows)):
                if not (x.dtype is _int32 and x.get_device() == self._index and x.shape == (n,) and x.is_contiguous()):
                    raise ValueError("out is int32 [requests + 1], [n_rows] and [n_rows] on the pool's device")
        self._call("dspark_pages_grow", at_length, at_count, n_rows, m, ms, mw, first.data_ptr(), slot.data_ptr(),
                   position.data_ptr(), self._stream(stream))
        return first, slot, position

    def trim(self, length, stream=None):
        """Each request keeps the pages of its first length[r] rows; the others are free again."""
        self._call("dspark_pages_trim", self._numbers(length), self._stream(stream))

    def status(self, stream=None):
        """Wait for the stream; the device status since the last call (0: all requests were served)."""
        if torch.cuda.current_device() == self._index:
            return self.lib.dspark_pages_status(self._at, self._stream(stream))
        with torch.cuda.device(self.device):
            return self.lib.dspark_pages_status(self._at, self._stream(stream))
