"""Thin ctypes binding of include/dspark_tree.h: the target model's check of
drafted tokens over a paged key/value cache.

    cache = KVCache(k, v)                        # or KVCache(codes_k, codes_v, k_scale, v_scale)
    tree = Tree(q_heads, kv_heads, head_dim, max_requests=B, max_nodes=T)
    tree.write(cache, pages, length, first, k, v)             # the draft's keys and values
    out, lse = tree.attend(q, cache, pages, length, first, mask=ancestor_bits(parent, first))
    tree.keep(cache, pages, length, path, count)              # the accepted path stays

Arguments that the host can see are checked before a launch (ValueError here,
WalkError from the C calls); lengths, row ranges, paths and page tables live on
the device and are checked there (`status`).  As with the walk, calls on one
handle are ordered by the caller, and a call given `stream` works on that
stream: its inputs have to be ready there.  There is no fallback.
"""
import ctypes
import math
import struct
from fractions import Fraction

import torch

from . import walk
from .walk import WalkError, _check

TYPE_BF16 = 0
TYPE_F16 = 1
TYPE_E4M3 = 2
TYPE_E2M1 = 3

TREE_MAX_HEAD_DIM = 128
TREE_MAX_REQUESTS = 1024
TREE_MAX_NODES = 256
TREE_MAX_LENGTH = 2147483392

_TYPES = {torch.bfloat16: TYPE_BF16, torch.float16: TYPE_F16, torch.float8_e4m3fn: TYPE_E4M3,
          torch.uint8: TYPE_E2M1}

EXPORTS = ["dspark_tree_create", "dspark_tree_write", "dspark_tree_read", "dspark_tree_keep",
           "dspark_tree_attend", "dspark_tree_rotate", "dspark_tree_place", "dspark_tree_status",
           "dspark_tree_destroy"]

_i64x3 = ctypes.c_int64 * 3


class dspark_tree_config(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int), ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("type", ctypes.c_int), ("max_requests", ctypes.c_int),
                ("max_nodes", ctypes.c_int)]


class dspark_tree_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("k_stride", _i64x3), ("v_stride", _i64x3),
                ("k_scale_stride", _i64x3), ("v_scale_stride", _i64x3),
                ("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int), ("type", ctypes.c_int)]


class dspark_tree_batch(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("start", ctypes.c_void_p), ("first", ctypes.c_void_p),
                ("pages_stride", ctypes.c_int64), ("max_pages", ctypes.c_int), ("B", ctypes.c_int),
                ("N", ctypes.c_int)]


class dspark_tree_rotation(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int)]


_pack_batch = struct.Struct("@PPPqiii").pack_into      # dspark_tree_batch
_pack_strides = struct.Struct("@qq").pack_into
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") \
    else lambda index: torch.cuda.current_stream(index).cuda_stream
_int32 = torch.int32

_lib = None


def load():
    """The library with this header's signatures (one library holds the walk and these)."""
    global _lib
    if _lib is None:
        L = walk.load()
        vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        # structs and arrays go by address: ctypes converts an int fastest
        L.dspark_tree_create.argtypes = [ctypes.POINTER(dspark_tree_config), ctypes.POINTER(vp)]
        L.dspark_tree_write.argtypes = [vp] * 8
        L.dspark_tree_read.argtypes = [vp] * 6
        L.dspark_tree_keep.argtypes = [vp, vp, vp, vp, i64, i32, vp, vp]
        L.dspark_tree_attend.argtypes = [vp, vp, vp, vp, vp, vp, i64, i32, f32, f32, vp, vp, vp]
        L.dspark_tree_rotate.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp]
        L.dspark_tree_place.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp]
        L.dspark_tree_status.argtypes = [vp, vp]
        L.dspark_tree_destroy.argtypes = [vp]
        for name in EXPORTS:
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _need(ok, what):
    if not ok:
        raise ValueError(what)


class KVCache:
    """A paged cache: k and v [n_pages, page_size, kv_heads, head_dim], bfloat16, float16,
    float8_e4m3fn (then with uint8 scales [n_pages, page_size, kv_heads]), or 4 bits an element:
    uint8 [n_pages, page_size, kv_heads, head_dim / 2], two e2m1 codes a byte, with uint8 scales
    [n_pages, page_size, kv_heads, head_dim / 16].  Any strides that are multiples of 16 bytes
    (scales of e2m1: of the largest power of two in head_dim / 16), the last dimension contiguous.
    Holds the tensors, not copies of them."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        _need(k.is_cuda and v.is_cuda and k.device == v.device, "k and v are on one CUDA device")
        _need(k.dim() == 4 and k.shape == v.shape, "k and v are [n_pages, page_size, heads, dim]")
        _need(k.dtype in _TYPES and v.dtype == k.dtype, "k and v are bf16, f16, e4m3 or uint8 (e2m1)")
        _need(k.stride(3) == 1 and v.stride(3) == 1, "head_dim is contiguous")
        e4m3, e2m1 = k.dtype == torch.float8_e4m3fn, k.dtype == torch.uint8
        _need((k_scale is not None) == (e4m3 or e2m1) and (v_scale is not None) == (e4m3 or e2m1),
              "an e4m3 or e2m1 cache, and no other, has scales")
        c = dspark_tree_cache(k=k.data_ptr(), v=v.data_ptr(), n_pages=k.shape[0],
                              page_size=k.shape[1], type=_TYPES[k.dtype])
        c.k_stride[:] = k.stride()[:3]
        c.v_stride[:] = v.stride()[:3]
        self.kv_heads, self.head_dim = k.shape[2], k.shape[3] * (2 if e2m1 else 1)
        if e4m3 or e2m1:
            shape = k.shape[:3] if e4m3 else k.shape[:3] + (self.head_dim // 16,)
            for s in (k_scale, v_scale):
                _need(s.device == k.device and s.dtype == torch.uint8 and s.shape == shape,
                      "scales are uint8 [n_pages, page_size, heads], of e2m1 [.., head_dim / 16]")
                _need(e4m3 or s.shape[3] <= 1 or s.stride(3) == 1, "a row's scales are contiguous")
            c.k_scale, c.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
            c.k_scale_stride[:] = k_scale.stride()[:3]
            c.v_scale_stride[:] = v_scale.stride()[:3]
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device, self.dtype = k.device, k.dtype
        self.key = (k.get_device(), self.kv_heads, self.head_dim, self.dtype)
        self.c = c
        self.address = ctypes.addressof(c)

    @classmethod
    def zeros(cls, n_pages, page_size, kv_heads, head_dim, dtype, device="cuda"):
        """A cache of zeros; dtype torch.uint8: e2m1.  A page holds the slots of one head next to
        each other, as attention reads them (e2m1: a head's scales of 16 slots are 128 bytes that
        way, and 8 bytes of every 64 with the heads of a slot next to each other)."""
        _need(dtype in _TYPES, "a cache is bf16, f16, e4m3 or uint8 (e2m1)")
        e2m1 = dtype == torch.uint8

        def rows(*last, of=torch.uint8):
            return torch.zeros(n_pages, kv_heads, page_size, *last, dtype=of, device=device).transpose(1, 2)

        x = [rows(head_dim // 2 if e2m1 else head_dim, of=dtype) for _ in range(2)]
        if e2m1:
            return cls(*x, rows(head_dim // 16), rows(head_dim // 16))
        if dtype == torch.float8_e4m3fn:
            return cls(*x, rows(), rows())
        return cls(*x)


def _turn(bits):
    """1 / (2 pi) as a fraction of 2^bits, to half of one: pi by Machin's formula."""
    one = 1 << (bits + 32)

    def arctan_inverse(n):
        total, term, k = 0, one // n, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total

    pi = 4 * (4 * arctan_inverse(5) - arctan_inverse(239))
    return ((one << bits) // pi + 1) >> 1


# enough for the turns of any float, up to 2^1024, to 2^-64
_TURN_BITS = 1152
_TURN_WHOLE = _turn(_TURN_BITS)
_TURN = Fraction(_TURN_WHOLE, 1 << _TURN_BITS)


def _turns(f):
    """The turns of f radians, a float, as a fraction of 2^64; whole ones do not count."""
    n, d = f.as_integer_ratio()                      # d is a power of two
    shift = _TURN_BITS - 64 + d.bit_length() - 1
    return ((n * _TURN_WHOLE + (1 << (shift - 1))) >> shift) % 2 ** 64


class Rotation:
    """How query and key heads are normed and turned (see `Tree.rotate`): `freq` [R / 2], radians a
    position of every pair (any finite numbers, taken as float64), or None: no rotation; q_norm and
    k_norm [head_dim] or None: no norm; pairs are elements i and i + R / 2, or, `interleaved`, 2 i
    and 2 i + 1.  Copies what it is given, on the host where needed: made once, not in a graph."""

    def __init__(self, head_dim, freq=None, q_norm=None, k_norm=None, eps=1e-6, interleaved=False,
                 device=None):
        device = torch.device("cuda", torch.cuda.current_device()) if device is None \
            else torch.device(device)
        _need(device.type == "cuda", "the rotation's device is a CUDA device")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        f = [] if freq is None else torch.as_tensor(freq, dtype=torch.float64).cpu()
        if freq is not None:
            _need(f.dim() == 1 and bool(torch.isfinite(f).all()), "freq is [R / 2], finite")
            f = f.tolist()
        _need(head_dim % 16 == 0 and len(f) % 8 == 0 and 2 * len(f) <= head_dim,
              "head_dim and R are multiples of 16, R at most head_dim")
        _need(eps >= 0.0 and math.isfinite(eps), "eps is a number from 0 on")
        turns = [_turns(x) for x in f]
        self.turns = torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in turns],
                                  dtype=torch.int64).to(device)
        norms = []
        for w in (q_norm, k_norm):
            if w is not None:
                _need(tuple(w.shape) == (head_dim,), "a norm is [head_dim]")
                w = w.detach().to(device=device, dtype=torch.float32, copy=True).contiguous()
            norms.append(w)
        self.q_norm, self.k_norm = norms
        self.head_dim, self.key = head_dim, (device.index, head_dim)
        self.c = dspark_tree_rotation(self.turns.data_ptr() if turns else None,
                                      *(None if w is None else w.data_ptr() for w in norms), eps,
                                      2 * len(f), int(bool(interleaved)))
        self.address = ctypes.addressof(self.c)
        torch.cuda.current_stream(device).synchronize()      # ready for calls on any stream


def ancestor_bits(parent, first):
    """The mask words of trees: parent int32 [N], each node's parent as its place within its own
    request's rows (smaller than the node's own; -1: a root, whose parent is the context), first
    int32 [B + 1].  Returns int32 [N, ceil(T / 32)] with T the most nodes of a request: a node
    sees itself and its ancestors.  Host arithmetic (some ms for 64 trees of 64 nodes), and it
    waits for arrays on the device: not for inside a captured graph.  The result is on parent's
    device."""
    device = parent.device
    parent, first = parent.cpu().long().tolist(), first.cpu().long().tolist()
    T = max([b - a for a, b in zip(first, first[1:])] + [1])
    words = (T + 31) // 32
    rows = [0] * len(parent)
    for a, b in zip(first, first[1:]):
        for i in range(b - a):
            p = parent[a + i]
            _need(-1 <= p < i, "a parent comes before its node")
            rows[a + i] = (1 << i) | (rows[a + p] if p >= 0 else 0)
    out = torch.tensor([[(r >> 32 * w) & 0xffffffff for w in range(words)] for r in rows],
                       dtype=torch.int64).view(len(rows), words)
    return torch.where(out >= 1 << 31, out - (1 << 32), out).to(torch.int32).to(device)


class Tree:
    """Owns one handle: the operators of a target model with q_heads query heads over kv_heads
    cached heads of head_dim elements, rows of `dtype` (bfloat16 or float16)."""

    def __init__(self, q_heads, kv_heads, head_dim, dtype=torch.bfloat16, max_requests=1,
                 max_nodes=64, device=None):
        self.h = None
        _need(dtype in (torch.bfloat16, torch.float16), "rows are bf16 or f16")
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None \
            else torch.device(device)
        _need(self.device.type == "cuda", "the handle's device is a CUDA device")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.q_heads, self.kv_heads, self.head_dim, self.dtype = q_heads, kv_heads, head_dim, dtype
        cfg = dspark_tree_config(q_heads, kv_heads, head_dim, _TYPES[dtype], max_requests,
                                 max_nodes)
        h = ctypes.c_void_p()
        self.lib = load()
        with torch.cuda.device(self.device):
            _check(self.lib.dspark_tree_create(ctypes.byref(cfg), ctypes.byref(h)),
                   "dspark_tree_create")
        self.h = h.value
        self._index = self.device.index
        self._keys = {(self._index, kv_heads, head_dim, t)
                      for t in (dtype, torch.float8_e4m3fn, torch.uint8)}
        self._scale = head_dim ** -0.5
        self._batch = dspark_tree_batch()
        self._batch_mem = (ctypes.c_char * ctypes.sizeof(self._batch)).from_buffer(self._batch)
        self._batch_at = ctypes.addressof(self._batch)
        self._strides = (ctypes.c_char * 48)()       # three rows' {token, head}
        self._s0 = ctypes.addressof(self._strides)
        self._s1 = self._s0 + 16
        self._s2 = self._s0 + 32

    # ---- argument marshalling: a few microseconds a call matter here ----

    def _cache(self, cache):
        if cache.key not in self._keys:
            raise ValueError("the cache has the handle's device, heads, head_dim and type (or e4m3, e2m1)")
        return cache.address

    def _requests(self, pages, start, first, n_rows):
        i = self._index
        try:
            B, width = pages.shape
            row, one = pages.stride()
            n, = start.shape
            step, = start.stride()
        except ValueError:
            n = B = -1
        if not (n == B >= 0 and pages.dtype is _int32 and start.dtype is _int32
                and pages.get_device() == i and start.get_device() == i):
            raise ValueError("pages is int32 [B, P] and lengths int32 [B], on the handle's device")
        if (one != 1 and width > 1) or (step != 1 and B > 1):
            raise ValueError("pages and lengths have one row a request, entries next to each other")
        f = 0
        if first is not None:
            if not (first.dtype is _int32 and first.get_device() == i and first.shape == (B + 1,)
                    and (B == 0 or first.stride(0) == 1)):
                raise ValueError("first is int32 [B + 1] on the handle's device")
            f = first.data_ptr()
        _pack_batch(self._batch_mem, 0, pages.data_ptr(), start.data_ptr(), f, row, width, B, n_rows)
        return self._batch_at

    def _rows(self, t, heads, at, what):
        try:
            n, h, d = t.shape
            s0, s1, s2 = t.stride()
        except ValueError:
            raise ValueError(what) from None
        if not (h == heads and d == self.head_dim and (s2 == 1 or d == 1)
                and t.dtype is self.dtype and t.get_device() == self._index):
            raise ValueError(what)
        _pack_strides(self._strides, at, s0, s1)
        return n

    def _out(self, t, shape, dtype, what):
        if not (t.dtype is dtype and t.get_device() == self._index and t.shape == shape
                and t.is_contiguous()):
            raise ValueError(what)
        return t

    def _stream(self, stream):
        if stream is None:
            return _raw_stream(self._index)
        return walk._stream(stream)

    def _empty(self, shape, dtype, stream):
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        s = torch.cuda.ExternalStream(stream, device=self.device) if isinstance(stream, int) \
            else stream
        with torch.cuda.stream(s):           # the block belongs to the stream that fills it
            return torch.empty(shape, dtype=dtype, device=self.device)

    # ---- the operators ----

    def write(self, cache, pages, start, first, k, v, stream=None):
        """Rows first[b] + i of k and v [N, kv_heads, head_dim] to positions start[b] + i."""
        n = self._rows(k, self.kv_heads, 0, "k is [N, kv_heads, head_dim] of the handle's type")
        if self._rows(v, self.kv_heads, 16,
                      "v is [N, kv_heads, head_dim] of the handle's type") != n:
            raise ValueError("k and v have as many rows")
        rc = self.lib.dspark_tree_write(
            self.h, self._cache(cache), self._requests(pages, start, first, n), k.data_ptr(),
            self._s0, v.data_ptr(), self._s1, self._stream(stream))
        if rc:
            raise WalkError(rc, "dspark_tree_write")

    def read(self, cache, pages, start, first, n_rows, out=None, stream=None):
        """Positions start[b] + i to rows first[b] + i of (k, v) [n_rows, kv_heads, head_dim]."""
        shape = (n_rows, self.kv_heads, self.head_dim)
        if out is None:
            k, v = self._empty(shape, self.dtype, stream), self._empty(shape, self.dtype, stream)
        else:
            k, v = (self._out(t, shape, self.dtype, "out is two contiguous [n_rows, kv_heads, "
                              "head_dim] tensors of the handle's type") for t in out)
        rc = self.lib.dspark_tree_read(
            self.h, self._cache(cache), self._requests(pages, start, first, n_rows), k.data_ptr(),
            v.data_ptr(), self._stream(stream))
        if rc:
            raise WalkError(rc, "dspark_tree_read")
        return k, v

    def keep(self, cache, pages, start, path, count, stream=None):
        """Position start[b] + path[b, i] moves to start[b] + i for i < count[b]; path int32
        [B, P'], strictly ascending in its first count[b] entries."""
        i = self._index
        try:
            n, width = path.shape
            row, one = path.stride()
            m, = count.shape
            step, = count.stride()
        except ValueError:
            n, m = -1, -2
        if not (n >= 0 and path.dtype is _int32 and path.get_device() == i
                and count.dtype is _int32 and count.get_device() == i):
            raise ValueError("path is int32 [B, n] and count int32 [B], on the handle's device")
        batch = self._requests(pages, start, None, 0)
        if not (n == m == len(pages) and (one == 1 or width <= 1) and (step == 1 or n <= 1)):
            raise ValueError("one path and count a request, entries next to each other")
        rc = self.lib.dspark_tree_keep(self.h, self._cache(cache), batch, path.data_ptr(), row, width,
                                       count.data_ptr(), self._stream(stream))
        if rc:
            raise WalkError(rc, "dspark_tree_keep")

    def _turning(self, rotation, position, n):
        if rotation.key != (self._index, self.head_dim):
            raise ValueError("the rotation has the handle's device and head_dim")
        if not (position.dtype is _int32 and position.get_device() == self._index
                and position.shape == (n,) and (n <= 1 or position.stride(0) == 1)):
            raise ValueError("position is int32 [N] on the handle's device, its entries next to each other")
        return rotation.address

    def rotate(self, q, k, position, rotation, out=None, stream=None):
        """Norms and rotation (`Rotation`) of q [N, q_heads, head_dim] and k [N, kv_heads, head_dim]
        by position int32 [N]; returns new (q, k).  fp32 inside, one rounding."""
        n = self._rows(q, self.q_heads, 0, "q is [N, q_heads, head_dim] of the handle's type")
        if self._rows(k, self.kv_heads, 16, "k is [N, kv_heads, head_dim] of the handle's type") != n:
            raise ValueError("q and k have as many rows")
        if out is None:
            out_q, out_k = (self._empty(x.shape, self.dtype, stream) for x in (q, k))
        else:
            out_q, out_k = (self._out(y, x.shape, self.dtype, "out is two contiguous tensors like q and k")
                            for x, y in zip((q, k), out))
        rc = self.lib.dspark_tree_rotate(
            self.h, self._turning(rotation, position, n), position.data_ptr(), n, q.data_ptr(), self._s0,
            k.data_ptr(), self._s1, out_q.data_ptr(), out_k.data_ptr(), self._stream(stream))
        if rc:
            raise WalkError(rc, "dspark_tree_rotate")
        return out_q, out_k

    def place(self, cache, slot, q, k, v, position, rotation, out=None, stream=None):
        """`rotate`, with k and v [N, kv_heads, head_dim] going to the cache at slot int32 [N] (page
        slot // page_size, place slot % page_size; see `Pages.grow`), quantised where it is, as
        rotate and then write leave them.  Returns the new q.  Rows with a slot below 0 are left
        out: the cache and their rows of q stay as they were."""
        n = self._rows(q, self.q_heads, 0, "q is [N, q_heads, head_dim] of the handle's type")
        for x, at in ((k, 16), (v, 32)):
            if self._rows(x, self.kv_heads, at, "k and v are [N, kv_heads, head_dim] of the handle's type") != n:
                raise ValueError("q, k and v have as many rows")
        if not (slot.dtype is _int32 and slot.get_device() == self._index and slot.shape == (n,)
                and (n <= 1 or slot.stride(0) == 1)):
            raise ValueError("slot is int32 [N] on the handle's device, its entries next to each other")
        if out is None:
            out = self._empty(q.shape, self.dtype, stream)
        else:
            self._out(out, q.shape, self.dtype, "out is like q, contiguous")
        rc = self.lib.dspark_tree_place(
            self.h, self._cache(cache), slot.data_ptr(), self._turning(rotation, position, n),
            position.data_ptr(), n, q.data_ptr(), self._s0, k.data_ptr(), self._s1, v.data_ptr(), self._s2,
            out.data_ptr(), self._stream(stream))
        if rc:
            raise WalkError(rc, "dspark_tree_place")
        return out

    def attend(self, q, cache, pages, length, first, mask=None, scale=None, softcap=0.0, out=None,
               lse=None, stream=None):
        """Attention of the drafted rows q [N, q_heads, head_dim] over positions 0 ..
        length[b] + T_b - 1 of their requests.  mask int32 [N, words] (see `ancestor_bits`) or
        None for chains.  scale: 1 / sqrt(head_dim) unless given.  softcap c > 0: scores become
        c tanh(s / c).  Returns (out [N, q_heads, head_dim], lse float32 [N, q_heads])."""
        n = self._rows(q, self.q_heads, 0, "q is [N, q_heads, head_dim] of the handle's type")
        shape = q.shape
        if out is None:
            out = self._empty(shape, self.dtype, stream)
        else:
            self._out(out, shape, self.dtype, "out is like q, contiguous")
        if lse is None:
            lse = self._empty((n, self.q_heads), torch.float32, stream)
        else:
            self._out(lse, (n, self.q_heads), torch.float32, "lse is float32 [N, q_heads]")
        m, ms, mw = None, 0, 0
        if mask is not None:
            if not (mask.dtype is _int32 and mask.get_device() == self._index and mask.dim() == 2
                    and mask.shape[0] == n):
                raise ValueError("mask is int32 [N, words] on the handle's device")
            m, mw = mask.data_ptr(), mask.shape[1]
            if mw < 1 and n > 0:                  # its address would be null: a chain
                raise ValueError("mask has a word a row at least")
            ms, one = mask.stride()
            if one != 1 and mw > 1:
                raise ValueError("a mask row's words lie next to each other")
        rc = self.lib.dspark_tree_attend(
            self.h, self._cache(cache), self._requests(pages, length, first, n), q.data_ptr(),
            self._s0, m, ms, mw, self._scale if scale is None else scale, softcap, out.data_ptr(),
            lse.data_ptr(), self._stream(stream))
        if rc:
            raise WalkError(rc, "dspark_tree_attend")
        return out, lse

    def status(self, stream=None):
        """Wait for the stream; the device status since the last call (0: all requests ran)."""
        return self.lib.dspark_tree_status(self.h, self._stream(stream))

    def close(self):
        if self.h:
            h, self.h = self.h, None
            _check(self.lib.dspark_tree_destroy(h), "dspark_tree_destroy")

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
