"""The paged 4-bit context cache: device buffers and calls over the C ABI.

``PagedCache`` owns a pool of 4-bit pages for some layers, the page tables,
lengths and reference counts of N sequences, and the scratch of its calls.
Calls run on the current stream (or the one given) and read nothing back, so
they can be captured into CUDA graphs.  The scratch is shared by the calls of
one cache: calls on one cache belong on one stream, or ordered after one
another, and so do two graphs captured from it.  The buffers are made and
filled on the stream that is current at construction: calls on another stream
belong after that, and the cache, like any tensor a call is given, is kept until
the calls have run.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _lib
from ._lib import Kv4Pool, Pages


def on_stream(index, stream):
    """The context in which memory comes from the stream that a call launches on (a Stream or a handle)."""
    if isinstance(stream, int):   # (ExternalStream takes no null handle)
        stream = torch.cuda.ExternalStream(stream, device=index) if stream else torch.cuda.default_stream(index)
    return torch.cuda.stream(stream)


class PagedCache:
    """Pool, page tables and scratch for N sequences on one device.

    ``data`` uint8 [layers][num_pages][page bytes]; ``table`` int32
    [N][max_pages] (-1: no page), ``len`` int32 [N], ``ref`` int32
    [num_pages], the three of them views of one buffer ``book`` (a snapshot of
    the bookkeeping is one copy of it).  ``k_exp`` / ``v_exp``: powers of two
    that move the scales' range (2^-9 .. 448) over the data.
    """

    def __init__(self, layers, num_pages, page, Hkv, hd, N, max_pages, k_exp=0, v_exp=0, device="cuda"):
        dev = torch.device(device)
        self.layers, self.num_pages, self.page, self.Hkv, self.hd = layers, num_pages, page, Hkv, hd
        self.N, self.max_pages = N, max_pages
        self.page_bytes = _lib.dfl_kv4_page_bytes(page, Hkv, hd)
        if self.page_bytes == 0:
            raise ValueError(f"no 4-bit pages of {page} tokens, {Hkv} heads of {hd}: the page must be a multiple of 16 "
                             "up to 1024 and the head dim 64 or 128")
        if min(layers, num_pages, N, max_pages) < 1:
            raise ValueError("layers, num_pages, N and max_pages must be positive")
        self.data = torch.zeros((layers, num_pages, self.page_bytes), dtype=torch.uint8, device=dev)
        self.book = torch.zeros((N * max_pages + N + num_pages,), dtype=torch.int32, device=dev)
        self.table = self.book[:N * max_pages].view(N, max_pages)
        self.len = self.book[N * max_pages:N * max_pages + N]
        self.ref = self.book[N * max_pages + N:]
        self._index = self.book.get_device()
        self._lib = _lib.load()
        self.table.fill_(-1)
        self.start = torch.zeros((N,), dtype=torch.int32, device=dev)
        self.map = torch.zeros((num_pages,), dtype=torch.int32, device=dev)
        self.live = torch.zeros((1,), dtype=torch.int32, device=dev)
        self.pool = Kv4Pool(_lib.ptr(self.data), num_pages * self.page_bytes, layers, num_pages, page, Hkv, hd, k_exp,
                            v_exp)
        self.pages = Pages(_lib.ptr(self.table), _lib.ptr(self.len), _lib.ptr(self.ref), N, max_pages)
        self._pool, self._pages = C.byref(self.pool), C.byref(self.pages)
        self.ws_bytes = max(_lib.workspace_size(_lib.DFL_OP_PAGES_RESERVE, N=N, pages=num_pages),
                            _lib.workspace_size(_lib.DFL_OP_PAGES_REMAP, N=N, pages=max_pages),
                            _lib.workspace_size(_lib.DFL_OP_PAGES_COMPACT, pages=num_pages))
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)
        self._start, self._map, self._live, self._ws = (_lib.ptr(x) for x in (self.start, self.map, self.live, self.ws))
        self._attn_ws = {}   # (B, Hq) -> scratch, its address and size
        self._scratch = {}   # bytes -> the same: the sizes are a few, whatever B and Hq

    def _st(self, stream):
        if torch.cuda.current_device() != self._index:
            raise ValueError(f"the cache lives on cuda:{self._index}, which is not the current device")
        if stream is None:   # the current stream's handle, without a Stream object (3 us of a call's 10)
            return torch._C._cuda_getCurrentRawStream(self._index)
        return _lib._stream(stream)

    def _alloc(self, stream, f, *args, **kw):
        """f(*args, **kw) with its memory from the stream that the call launches on."""
        if stream is None:
            return f(*args, **kw)
        with on_stream(self._index, stream):
            return f(*args, **kw)

    def _i32(self, x, what):
        if x.dtype is not torch.int32 or not x.is_contiguous() or x.get_device() != self._index or x.numel() != self.N:
            raise ValueError(f"{what} must be a contiguous int32 tensor of {self.N} elements on {self.book.device}")
        return x.data_ptr()

    def _rows(self, x, what, heads=None, rows=None):
        """Check a bf16 [N, rows, heads, hd] tensor; returns its pointer and rows."""
        shape = x.shape
        if x.dtype is not torch.bfloat16 or not x.is_contiguous() or x.get_device() != self._index or len(shape) != 4 or \
                shape[0] != self.N or shape[3] != self.hd or (heads and shape[2] != heads) or (rows and shape[1] != rows):
            raise ValueError(f"{what} must be a contiguous bf16 tensor [{self.N}, {rows or 'rows'}, {heads or 'heads'}, "
                             f"{self.hd}] on {self.book.device}")
        return x.data_ptr(), shape[1]

    def append(self, layer, K, V, start, n_new, stream=None, rows=None):
        """Rows K[n, i], V[n, i] (i < n_new[n]) to positions start[n] + i; K, V bf16 [N, R, Hkv, hd].

        With ``rows`` int32 [N, R] rows K[n, rows[n, i]], V[n, rows[n, i]]: those of an accepted path.
        """
        k, R = self._rows(K, "K", self.Hkv)
        v, _ = self._rows(V, "V", self.Hkv, R)
        if rows is not None:
            if rows.dtype is not torch.int32 or not rows.is_contiguous() or rows.get_device() != self._index or \
                    rows.shape != (self.N, R):
                raise ValueError(f"rows must be a contiguous int32 tensor [{self.N}, {R}] on {self.book.device}")
            rc = self._lib.dfl_kv4_append_rows(self._pool, layer, self._pages, self._i32(start, "start"),
                                               self._i32(n_new, "n_new"), rows.data_ptr(), R, k, v, self._st(stream))
            if rc:
                _lib._check("dfl_kv4_append_rows", rc)
            return
        rc = self._lib.dfl_kv4_append(self._pool, layer, self._pages, self._i32(start, "start"),
                                      self._i32(n_new, "n_new"), R, k, v, self._st(stream))
        if rc:
            _lib._check("dfl_kv4_append", rc)

    def read(self, layer, start, count, K, V, stream=None):
        """Positions start[n] .. start[n] + count[n] - 1 into K[n, i], V[n, i] (other rows keep what they hold)."""
        k, R = self._rows(K, "K", self.Hkv)
        v, _ = self._rows(V, "V", self.Hkv, R)
        rc = self._lib.dfl_kv4_read(self._pool, layer, self._pages, self._i32(start, "start"),
                                    self._i32(count, "count"), R, k, v, self._st(stream))
        if rc:
            _lib._check("dfl_kv4_read", rc)
        return K, V

    def attn(self, layer, Q, Kb, Vb, out=None, stream=None, mask=None, window=0, sinks=0):
        """Block attention over each sequence's cached tokens and the block's own rows.

        Q bf16 [N, B, Hq, hd], Kb, Vb bf16 [N, B, Hkv, hd]; returns O bf16 [N, B, Hq, hd], allocated on the stream of
        the call unless ``out`` is given.  Own rows count as at most 65,504 units of 2^k_exp and 2^v_exp, and keep
        bf16's 8 bits from 2^-14 of a unit up.

        ``mask`` int64 [N, B]: row i sees the own rows whose bits are set, as ``DraftTree.mask`` has them; a row without a
        bit is no row, its output 0.  ``window``: a row at position q (the cached length + the row's number, or with a
        mask + its bits less one) sees the keys at positions p with q - p < window or p < ``sinks`` (0: all of them).
        """
        q, B = self._rows(Q, "Q")
        Hq = Q.shape[2]
        k, _ = self._rows(Kb, "Kb", self.Hkv, B)
        v, _ = self._rows(Vb, "Vb", self.Hkv, B)
        if out is None:
            out = torch.empty_like(Q) if stream is None else self._alloc(stream, torch.empty_like, Q)
        o, _ = self._rows(out, "out", Hq, B)
        ws = self._attn_ws.get((B, Hq))
        if ws is None:
            need = _lib.workspace_size(_lib.DFL_OP_KV4_ATTN, N=self.N, B=B, Hq=Hq, Hkv=self.Hkv, hd=self.hd)
            ws = self._scratch.get(need)
            if ws is None:
                ws = self._alloc(stream, torch.empty, max(need, 16), dtype=torch.uint8, device=self.book.device)
                ws = self._scratch[need] = (ws, ws.data_ptr(), ws.numel())
            self._attn_ws[(B, Hq)] = ws
        if mask is None and window == 0 and sinks == 0:
            rc = self._lib.dfl_kv4_attn(self._pool, layer, self._pages, q, k, v, B, Hq, o, ws[1], ws[2], self._st(stream))
            if rc:
                _lib._check("dfl_kv4_attn", rc)
            return out
        m = None
        if mask is not None:
            if mask.dtype is not torch.int64 or not mask.is_contiguous() or mask.get_device() != self._index or \
                    mask.shape != (self.N, B):
                raise ValueError(f"mask must be a contiguous int64 tensor [{self.N}, {B}] on {self.book.device}")
            m = mask.data_ptr()
        rc = self._lib.dfl_kv4_attn_masked(self._pool, layer, self._pages, q, k, v, B, Hq, m, window, sinks, o, ws[1], ws[2],
                                           self._st(stream))
        if rc:
            _lib._check("dfl_kv4_attn_masked", rc)
        return out

    def reserve(self, n_new, stream=None):
        """Pages for n_new[n] more tokens; returns ``start`` (a buffer of the cache): the old lengths, -1 where not served."""
        rc = self._lib.dfl_pages_reserve(self._pool, self._pages, self._i32(n_new, "n_new"), self._start, self._ws,
                                         self.ws_bytes, self._st(stream))
        if rc:
            _lib._check("dfl_pages_reserve", rc)
        return self.start

    def remap(self, parent, keep_len=None, stream=None):
        """Sequence n becomes sequence parent[n] cut to keep_len[n] tokens (fork, reorder, roll back, end: -1)."""
        keep = None if keep_len is None else self._i32(keep_len, "keep_len")
        rc = self._lib.dfl_pages_remap(self._pool, self._pages, self._i32(parent, "parent"), keep, self._ws,
                                       self.ws_bytes, self._st(stream))
        if rc:
            _lib._check("dfl_pages_remap", rc)

    def compact(self, stream=None):
        """Used pages to the pool's low end; returns (map, live), buffers of the cache."""
        rc = self._lib.dfl_pages_compact(self._pool, self._pages, self._map, self._live, self._ws, self.ws_bytes,
                                         self._st(stream))
        if rc:
            _lib._check("dfl_pages_compact", rc)
        return self.map, self.live
