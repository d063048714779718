"""Sequences in a paged KV pool of 16, 8 or 4 bits: page operations and attention.

`PagedCache` holds the tensors that libcg's page calls (cg_pages_*) and
cg_attend work on and marshals their arguments; every step runs in libcg's
CUDA kernels.  A context is decoded into a slot's blocks (`decode`, over
cg_decode_paged), continued by other slots that share its full blocks
(`fork`), attended to by a batch of them (`attend`), and given back (`free`,
`compact`).  `QuantCache` is a cache whose pool is held in 4 or 8 bits: tokens
are quantised as they are stored (`write`, cg_quant_write), read back (`read`)
and attended to as they lie.

All calls are asynchronous on `stream` (default: the current one), and errors
found on the device are OR-ed into `status` as in codec.py.  A cache has one
workspace: calls that use it (fork, compact, attend) belong on one stream, or
are ordered by the caller, as calls on another stream are after the cache's
construction.  A captured graph uses the cache's workspace: keep the cache for
as long as the graph.  What a call returns was allocated on the call's stream,
as if that one were current.  The pool's device has to be the current one.  The
pool, tables, lengths and reference counts are plain torch tensors and may be
read and written by the caller's own kernels between calls, e.g. to store a
new token's K and V and advance `lens`.
"""
from __future__ import annotations

import ctypes as ct
import math
import operator
import struct
from typing import Optional, Tuple

import torch

from . import codec
from .codec import CG_BF16, CG_FP16, Config, _check, cg_pages, cg_quant, lib

NO_BLOCK = NO_SLOT = -1  # CG_NO_BLOCK / CG_NO_SLOT as int32

_DTYPES = {torch.float16: CG_FP16, torch.bfloat16: CG_BF16}


_INT32 = (torch.int32, torch.uint32)
# The fields of cg_attention and cg_token_rows as the C compiler lays them out: building the ctypes structures took a
# quarter of a call.
_pack_attention = struct.Struct("4P9I6Qf4x").pack
_pack_rows = struct.Struct("5P4I4Q").pack
# The current stream's handle without building a Stream object around it (3 us of a 7 us call).
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _ids(t: torch.Tensor, device: torch.device, what: str) -> int:
    if t.dtype not in _INT32 or t.dim() != 1 or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{what}: a contiguous 1-D int32 tensor on {device} is wanted, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _stride3(t: torch.Tensor) -> tuple:
    s = t.stride()
    return s if len(s) == 3 else (0, 0, 0)


def _fixed(name: str) -> property:
    """A tensor whose address the library has: another one may not take its
    place (`cache.lens = cache.lens + 1` would leave the calls with the old
    one).  `cache.lens += 1` assigns the tensor that is there, and may."""
    get = operator.attrgetter("_" + name)

    def put(self, value):
        if value is not get(self):
            raise AttributeError(f"PagedCache.{name} cannot be replaced: write into it, in place")

    return property(get, put)


class PagedCache:
    """A pool [L][n_pool][2][block_tokens][C] (fp16 or bf16; any strides with
    the channels contiguous, e.g. a transposed view of [n_pool][L][2][bt][C])
    and its sequences: tables int32 [n_slots][n_blocks] (-1: no block), lens
    int32 [n_slots], refs int32 [n_pool].  The calls read and write the tensors
    given here: change them in place."""

    _POOL = _DTYPES  # types of the pool's elements
    pool, tables, lens, refs, status = map(_fixed, ("pool", "tables", "lens", "refs", "status"))

    def __init__(self, pool: torch.Tensor, tables: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
                 status: Optional[torch.Tensor] = None):
        if pool.dtype not in self._POOL or pool.dim() != 5 or pool.shape[2] != 2 or pool.stride(4) != 1:
            raise ValueError(f"pool: a tensor [L][n_pool][2][block_tokens][C] of {' or '.join(map(str, self._POOL))} "
                             "with contiguous channels is wanted")
        for t, dim, n in ((tables, 2, "tables"), (lens, 1, "lens"), (refs, 1, "refs")):
            if t.dtype != torch.int32 or t.dim() != dim or not t.is_contiguous() or t.device != pool.device:
                raise ValueError(f"{n}: a contiguous {dim}-D int32 tensor on {pool.device} is wanted")
        if lens.shape[0] != tables.shape[0] or refs.shape[0] != pool.shape[1]:
            raise ValueError("lens has one entry per slot, refs one per block of the pool")
        self._pool, self._tables, self._lens, self._refs = pool, tables, lens, refs
        self._status = status if status is not None else codec.new_status(pool.device)
        L, n_pool, _, bt, C = pool.shape
        sl, sb, skv, st, _ = pool.stride()
        self._c = cg_pages(pool.data_ptr(), L, C, n_pool, bt, sl, skv, sb, st, tables.data_ptr(), lens.data_ptr(),
                           refs.data_ptr(), tables.shape[0], tables.shape[1])
        self._ref = ct.byref(self._c)
        n = ct.c_size_t()
        _check(lib().cg_pages_ws_bytes(self._ref, ct.byref(n)), "cg_pages_ws_bytes")
        self._ws = torch.empty(n.value, dtype=torch.uint8, device=pool.device)
        self._outgrown = []  # earlier workspaces: a captured graph may still use them
        self._status_ptr = self.status.data_ptr()
        self._seen = set()  # streams that status and workspace are recorded on
        self._index = pool.device.index if pool.is_cuda else None
        self._device, self._type, self._dtype = pool.device, pool.dtype, _DTYPES.get(pool.dtype)
        self._attn = {}  # workspace bytes of attend by shape

    @classmethod
    def empty(cls, L: int, n_pool: int, block_tokens: int, C: int, n_slots: int, n_blocks: int,
              dtype: torch.dtype = torch.float16, device="cuda") -> "PagedCache":
        """A cache of free blocks and empty slots."""
        i32 = dict(dtype=torch.int32, device=device)
        return cls(torch.zeros((L, n_pool, 2, block_tokens, C), dtype=dtype, device=device),
                   torch.full((n_slots, n_blocks), NO_BLOCK, **i32), torch.zeros(n_slots, **i32),
                   torch.zeros(n_pool, **i32))

    def c(self) -> cg_pages:
        return self._c

    def _stream(self, stream) -> int:
        if self._index is None:
            raise ValueError("the pool is not in GPU memory")
        if _current_device() != self._index:  # the device that libcg launches on
            raise ValueError(f"the pool is on cuda:{self._index}, which is not the current device")
        handle = stream.cuda_stream if stream is not None else _raw_stream(self._index)
        if handle not in self._seen:  # a cache dropped with work in flight: its memory waits for that stream too
            for t in (self._ws, self.status):
                t.record_stream(stream if stream is not None else torch.cuda.current_stream(self._device))
            self._seen.add(handle)
        return handle

    def _new(self, shape, dtype: torch.dtype, stream) -> torch.Tensor:
        """Memory for kernels on `stream`.  Taken on that stream: what the
        allocator has for the current one may still be in use by work queued
        there, which `stream` does not wait for."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self._device)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=self._device)

    @property
    def block_tokens(self) -> int:
        return self.pool.shape[3]

    def check(self) -> None:
        """Wait for the device and raise on any error found there."""
        torch.cuda.synchronize(self.pool.device)
        code = codec.read_status(self.status)
        if code != codec.CG_OK:
            self.status.zero_()
            torch.cuda.synchronize(self.pool.device)  # before any stream's next call may find an error
        _check(code, "paged cache (device)")

    def _workspace(self, n: int, stream, handle: int) -> torch.Tensor:
        if self._ws.numel() < n:
            # at least twice the last one: all that are kept are then at most four times what is needed
            self._outgrown.append(self._ws)
            self._ws = self._new(max(n, 2 * self._ws.numel()), torch.uint8, stream)
            self._seen = {handle}
        return self._ws

    def fork(self, parent: torch.Tensor, child: torch.Tensor, reserve: Optional[torch.Tensor] = None,
             stream=None) -> None:
        """Start sequence child[i] as a continuation of parent[i] (-1: an
        empty one) with blocks for reserve[i] further tokens (cg_pages_fork)."""
        d = self._device
        n = parent.shape[0]
        if child.shape[0] != n or (reserve is not None and reserve.shape[0] != n):
            raise ValueError("fork: parent, child and reserve have one entry per new sequence")
        _check(lib().cg_pages_fork(self._ref, _ids(parent, d, "parent"), _ids(child, d, "child"),
                                   _ids(reserve, d, "reserve") if reserve is not None else None, n,
                                   self._ws.data_ptr(), self._ws.numel(), self._status_ptr,
                                   self._stream(stream)), "cg_pages_fork")

    def free(self, slots: torch.Tensor, stream=None) -> None:
        """End the sequences in `slots` (cg_pages_free)."""
        _check(lib().cg_pages_free(self._ref, _ids(slots, self._device, "slots"), slots.shape[0],
                                   self._status_ptr, self._stream(stream)), "cg_pages_free")

    def compact(self, remap: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Move the blocks in use to the front of the pool; returns each
        block's new number, -1 for a free one (cg_pages_compact)."""
        d = self._device
        if remap is None:
            remap = self._new(self._pool.shape[1], torch.int32, stream)
        if remap.shape[0] != self._pool.shape[1]:
            raise ValueError("remap has one entry per block of the pool")
        _check(lib().cg_pages_compact(self._ref, _ids(remap, d, "remap"), self._ws.data_ptr(),
                                      self._ws.numel(), self._status_ptr, self._stream(stream)),
               "cg_pages_compact")
        return remap

    def copy(self, src: torch.Tensor, dst: torch.Tensor, source: Optional["PagedCache"] = None, stream=None) -> None:
        """Copy whole blocks src[i] of `source` (default: this cache) to
        blocks dst[i] of this cache (cg_pages_copy)."""
        d = self._device
        other = source if source is not None else self
        if src.shape[0] != dst.shape[0]:
            raise ValueError("copy: src and dst have the same number of blocks")
        if other._form() != self._form() or other._device != d:
            raise ValueError("copy: both pools have one type and one device")
        _check(lib().cg_pages_copy(self._ref, other._ref, _ids(src, d, "src"), _ids(dst, d, "dst"),
                                   src.shape[0], self._status_ptr, self._stream(stream)), "cg_pages_copy")

    def decode(self, cfg: Config, enc, slot: int, stream=None) -> None:
        """Decode a context into the blocks that a slot holds
        (cg_decode_paged) and set its length.  The slot needs blocks for all
        cfg.T tokens (fork with parent -1 and reserve T)."""
        self._stream(stream)  # refuses a pool that the decoder could not write to
        if self.pool.dtype != torch.float16:
            raise ValueError("decode writes fp16: the pool is another type")
        L, n_pool, _, bt, C = self.pool.shape
        if (cfg.L, cfg.C) != (L, C):
            raise ValueError(f"the context has {cfg.L} layers x {cfg.C} channels, the pool {L} x {C}")
        sl, sb, skv, st, _ = self.pool.stride()
        # the blocks of the context alone: the decoder takes every entry it is given for a block to write to
        row = self.tables[slot][: -(-cfg.T // bt)]
        codec.cg_decode_paged(cfg, enc, self.pool, row, bt, sl, skv, sb, st, self.status, stream,
                              n_pool_blocks=n_pool)
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
            self.lens[slot] = cfg.T

    def attend(self, layer: int, q: torch.Tensor, slots: Optional[torch.Tensor] = None, shared_slot: int = 0,
               shared_blocks: int = 0, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Attention of the sequences in `slots` (default: slot r for request
        r) at one layer (cg_attend).  q: [R][n_queries][n_q_heads][head_dim],
        the queries of each sequence's last n_queries tokens; the first
        shared_blocks blocks of every sequence are those of shared_slot.
        scale defaults to head_dim ** -0.5.  Returns out (shape and type of
        q); lse, if given, is a fp32 [R][n_queries][n_q_heads]."""
        d, qs = self._device, q.stride()
        if q.dtype != self._type or len(qs) != 4 or q.device != d or qs[3] != 1:
            raise ValueError("q: a tensor [R][n_queries][n_q_heads][head_dim] of the cache's type and device with "
                             "contiguous head channels is wanted")
        R, nq, hq, hd = q.shape
        if out is None:
            out = self._new(q.shape, q.dtype, stream)
        os_ = out.stride()
        if out.shape != q.shape or out.dtype != q.dtype or out.device != d or os_[3] != 1:
            raise ValueError("out: shape, type and device of q, contiguous head channels")
        if lse is not None and (lse.dtype != torch.float32 or lse.shape != q.shape[:3] or not lse.is_contiguous()
                                or lse.device != d):
            raise ValueError("lse: a contiguous fp32 tensor [R][n_queries][n_q_heads] is wanted")
        if slots is not None and slots.shape[0] != R:
            raise ValueError("slots has one entry per request")
        if slots is None and R > self.tables.shape[0]:
            raise ValueError("more requests than slots")
        if min(layer, shared_slot, shared_blocks) < 0:
            raise ValueError("layer, shared_slot and shared_blocks are not negative")
        if R == 0:
            return out
        try:
            a = _pack_attention(q.data_ptr(), out.data_ptr(), lse.data_ptr() if lse is not None else 0,
                                _ids(slots, d, "slots") if slots is not None else 0, self._dtype, R, nq, hq,
                                self._kv_heads(hd), hd, layer, shared_slot, shared_blocks, *qs[:3], *os_[:3],
                                scale if scale is not None else 1.0 / math.sqrt(hd) if hd else 0.0)
        except struct.error:  # a number that its field cannot hold: refused as those that the library refuses
            _check(codec.CG_ERR_INVALID_ARG, "attend")
        key = (R, nq, hq, hd, self._shared_key(shared_blocks))
        ws_bytes = self._attn.get(key)
        if ws_bytes is None:
            n = ct.c_size_t()
            _check(self._attend_ws_bytes(a, n), "attend (workspace)")
            if len(self._attn) >= 1024:  # shapes come and go: those still in use are soon there again
                self._attn.clear()
            ws_bytes = self._attn[key] = n.value
        handle = self._stream(stream)
        ws = self._workspace(ws_bytes, stream, handle)
        _check(self._attend(a, ws, handle), "attend")
        return out

    # what a pool of another format does otherwise

    def _form(self) -> tuple:
        return (self._type,)

    def _kv_heads(self, head_dim: int) -> int:
        return self._pool.shape[4] // head_dim if head_dim else 0

    def _shared_key(self, shared_blocks: int):
        return shared_blocks > 0  # the workspace does not depend on how many

    def _attend_ws_bytes(self, a, n) -> int:
        return lib().cg_attend_ws_bytes(self._ref, a, ct.byref(n))

    def _attend(self, a, ws, handle) -> int:
        return lib().cg_attend(self._ref, a, ws.data_ptr(), ws.numel(), self._status_ptr, handle)


class QuantCache(PagedCache):
    """A cache whose pool holds K and V in 4 or 8 bits: an int16 tensor
    [L][n_pool][2][block_tokens][row], each row the codes of a token's channels
    and a scale and a low value of `dtype` for each `group` of them (cg_quant in
    cg.h; `row_width` gives the row's length).  Tables, lengths, references and
    the page calls are those of PagedCache; `dtype` (fp16 or bf16) is the type of
    what is written, read and attended with.  group defaults to head_dim."""

    _POOL = (torch.int16,)

    def __init__(self, pool: torch.Tensor, tables: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
                 status: Optional[torch.Tensor] = None, *, n_kv_heads: int, head_dim: int, bits: int = 4,
                 group: Optional[int] = None, dtype: torch.dtype = torch.float16):
        row = self.row_width(n_kv_heads, head_dim, bits, group, dtype)
        if pool.dim() == 5 and pool.shape[4] != row:
            raise ValueError(f"pool: rows of {row} words hold {n_kv_heads} x {head_dim} channels in {bits} bits, "
                             f"not {pool.shape[4]}")
        super().__init__(pool, tables, lens, refs, status)
        self._format = self._format_of(n_kv_heads, head_dim, bits, group, dtype)
        self._at, self._format_at = ct.addressof(self._c), ct.addressof(self._format)
        self._cg_write, self._cg_read = codec.packed_call("cg_quant_write", 5), codec.packed_call("cg_quant_read", 5)
        self._cg_attend = codec.packed_call("cg_quant_attend", 7)
        self._type, self._dtype, self._heads, self._hd = dtype, _DTYPES[dtype], n_kv_heads, head_dim
        self._channels, self._n_slots = n_kv_heads * head_dim, tables.shape[0]

    @staticmethod
    def _format_of(n_kv_heads, head_dim, bits, group, dtype) -> cg_quant:
        if dtype not in _DTYPES:
            raise ValueError("dtype: fp16 or bf16 is wanted")
        return cg_quant(_DTYPES[dtype], bits, group if group is not None else head_dim, n_kv_heads, head_dim)

    @classmethod
    def row_width(cls, n_kv_heads: int, head_dim: int, bits: int = 4, group: Optional[int] = None,
                  dtype: torch.dtype = torch.float16) -> int:
        """Words of a row of the pool (cg_quant_row)."""
        n = ct.c_uint32()
        _check(lib().cg_quant_row(ct.byref(cls._format_of(n_kv_heads, head_dim, bits, group, dtype)), ct.byref(n)),
               "cg_quant_row")
        return n.value

    @classmethod
    def empty(cls, L: int, n_pool: int, block_tokens: int, n_kv_heads: int, head_dim: int, n_slots: int, n_blocks: int,
              bits: int = 4, group: Optional[int] = None, dtype: torch.dtype = torch.float16,
              device="cuda") -> "QuantCache":
        """A cache of free blocks and empty slots."""
        i32 = dict(dtype=torch.int32, device=device)
        row = cls.row_width(n_kv_heads, head_dim, bits, group, dtype)
        return cls(torch.zeros((L, n_pool, 2, block_tokens, row), dtype=torch.int16, device=device),
                   torch.full((n_slots, n_blocks), NO_BLOCK, **i32), torch.zeros(n_slots, **i32),
                   torch.zeros(n_pool, **i32), n_kv_heads=n_kv_heads, head_dim=head_dim, bits=bits, group=group,
                   dtype=dtype)

    @property
    def channels(self) -> int:
        return self._channels

    def _rows(self, k, v, layer, slots, offsets, start) -> bytes:
        """A cg_token_rows."""
        d, shape, (k0, k1, k2), (v0, v1, v2) = self._device, k.shape, _stride3(k), _stride3(v)
        n_layers, n_rows, C = shape if len(shape) == 3 else (0, 0, 0)
        if (k.dtype is not self._type or v.dtype is not self._type or shape != v.shape or C != self._channels
                or k2 != 1 or v2 != 1 or k.device != d or v.device != d):
            raise ValueError(f"k and v: two tensors [layers][rows][{self._channels}] of {self._type} on {d} with contiguous "
                             "channels are wanted")
        n, s, o, b = self._n_slots, 0, 0, 0
        if slots is not None:
            n, s = slots.shape[0], _ids(slots, d, "slots")
        if offsets is not None:
            m, o = offsets.shape[0] - 1, _ids(offsets, d, "offsets")
            if m < 0 or (slots is not None and n != m):
                raise ValueError("slots has one entry per sequence, offsets one more")
            n = m
        if start is not None:
            m, b = start.shape[0], _ids(start, d, "start")
            if (slots is not None or offsets is not None) and n != m:
                raise ValueError("start has one entry per sequence")
            n = m
        if layer < 0 or (slots is None and n > self._n_slots):
            raise ValueError("layer is negative, or there are more sequences than slots")
        try:
            return _pack_rows(k.data_ptr(), v.data_ptr(), s, o, b, n, n_rows, layer, n_layers, k0, k1, v0, v1)
        except struct.error:  # as in attend
            _check(codec.CG_ERR_INVALID_ARG, "write, read")

    def write(self, k: torch.Tensor, v: torch.Tensor, layer: int = 0, slots: Optional[torch.Tensor] = None,
              offsets: Optional[torch.Tensor] = None, start: Optional[torch.Tensor] = None, stream=None) -> None:
        """Quantise the rows of k and v, [layers][rows][C], and store them in
        the pool's layers from `layer` on (cg_quant_write).  The sequence in
        slots[r] (default: slot r) has the rows offsets[r] .. offsets[r + 1] - 1
        (default: an even share); they are its last tokens (advance `lens` first)
        or those from start[r] on."""
        rows = self._rows(k, v, layer, slots, offsets, start)
        _check(self._cg_write(self._at, self._format_at, rows, self._status_ptr, self._stream(stream)),
               "cg_quant_write")

    def read(self, layer: int = 0, n_layers: Optional[int] = None, rows: Optional[int] = None,
             slots: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
             start: Optional[torch.Tensor] = None, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
             stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """The values of tokens as k and v, [layers][rows][C], the reverse of
        `write` (cg_quant_read).  Without out, n_layers (default: 1) and `rows`
        give the shape, and rows that belong to no token are zeros."""
        if out is None:
            if rows is None or rows < 0:
                raise ValueError("read: rows or out is wanted")
            shape = (n_layers if n_layers is not None else 1, rows, self._channels)
            with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(self._device)):
                out = tuple(torch.zeros(shape, dtype=self._type, device=self._device) for _ in range(2))
        k, v = out
        if (n_layers is not None and k.shape[0] != n_layers) or (rows is not None and k.shape[1] != rows):
            raise ValueError("read: n_layers and rows are those of out")
        r = self._rows(k, v, layer, slots, offsets, start)
        _check(self._cg_read(self._at, self._format_at, r, self._status_ptr, self._stream(stream)),
               "cg_quant_read")
        return k, v

    def decode(self, cfg: Config, enc, slot: int, stream=None) -> None:
        """Decode a context and quantise it into the blocks that a slot holds,
        and set its length.  The slot needs blocks for all cfg.T tokens (fork
        with parent -1 and reserve T).  The decoded context, fp16, is held until
        the stream has written it."""
        self._stream(stream)
        if self._type != torch.float16:
            raise ValueError("decode writes fp16: the cache is another type")
        L, C = self._pool.shape[0], self._channels
        if (cfg.L, cfg.C) != (L, C):
            raise ValueError(f"the context has {cfg.L} layers x {cfg.C} channels, the pool {L} x {C}")
        if not 0 <= slot < self._tables.shape[0] or cfg.T > self._tables.shape[1] * self.block_tokens:
            raise ValueError("decode: no such slot, or its row is shorter than the context")
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(self._device)):
            i32 = dict(dtype=torch.int32, device=self._device)
            kv = torch.empty((L, 2, cfg.T, C), dtype=torch.float16, device=self._device)
            codec.cg_decode(cfg, enc, kv, self.status, stream)
            self.lens[slot] = cfg.T
            self.write(kv[:, 0], kv[:, 1], slots=torch.full((1,), slot, **i32), stream=stream)

    def _kv_heads(self, head_dim: int) -> int:
        return self._heads

    def _form(self) -> tuple:
        f = self._format
        return (self._type, f.bits, f.group, f.n_kv_heads, f.head_dim)

    def _shared_key(self, shared_blocks: int):
        return shared_blocks

    def _attend_ws_bytes(self, a, n) -> int:
        return lib().cg_quant_attend_ws_bytes(self._ref, ct.byref(self._format), a, ct.byref(n))

    def _attend(self, a, ws, handle) -> int:
        return self._cg_attend(self._at, self._format_at, a, ws.data_ptr(), ws.numel(), self._status_ptr, handle)
