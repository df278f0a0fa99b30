"""Thin ctypes binding of the page cache (ss_cache_* in include/ss_sampler.h).

A PageCache names the planes (a layer's keys, a layer's values, ...) that share
page numbers; BlockTables holds the device arrays that say which request holds
which pages. The pages around a verification step: reserve slots for the draft,
run the model, verify, commit what was accepted. A cache whose pages hold 8-bit
floats with a scale for each block of slots and head also writes a step's keys
and values, attends over them and reads them back. Nothing is read back to the
host; everything is computed in the HIP library.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from .sampler import (_HALF_DTYPES, SS_OK, CacheConfig, CacheScales, CBlockTables, _check, _check_array,
                      _check_block, _check_dev, _check_rows, _empty_rows, _heads, _out_heads, _pack_step,
                      _pack_tables, _require, _stream_on, load_library)


@dataclass
class BlockTables:
    """The pages of the requests, as device tensors that the calls change in place."""
    tables: torch.Tensor  # [rows, >= max_blocks] int32: each row's pages in order, -1 = none
    ref: torch.Tensor     # [num_pages] int32: table entries that hold each page, 0 = free
    lens: torch.Tensor    # [rows] int32: committed slots


class PageCache:
    """Owns one ss_cache handle. planes: a [num_planes, num_pages, page_size,
    heads, dim] tensor, or a list of [num_pages, page_size, heads, dim] tensors
    of one dtype, shape and stride. The last dimension has unit stride, the
    others any (a transposed view of pages that hold heads outside slots is
    fine) as long as no two pieces overlap. The planes are kept referenced.

    scales: a cache held in 8 bits (write, read, attend). The planes are then
    float8_e4m3fn or uint8, plane 2 l the keys and 2 l + 1 the values of layer l,
    and scales a [num_planes, num_pages, page_size / block, heads] uint8 tensor (or
    a list) for blocks of 16, 32 or 64 slots: a byte q under the scale byte s
    stands for q 2^(s - 127). dim is a multiple of 16 up to 256, page_size a
    multiple of the block."""

    def __init__(self, planes, max_batch, max_blocks, scales=None):
        self.handle = None
        self.lib = load_library()
        planes = list(planes.unbind(0)) if isinstance(planes, torch.Tensor) else list(planes)
        _require(len(planes) >= 1, "a cache needs at least one plane")
        p = planes[0]
        _require(isinstance(p, torch.Tensor) and p.is_cuda, "planes must be device tensors")
        _require(p.dim() == 4 and p.numel() > 0,
                 "a plane must be a non-empty [num_pages, page_size, heads, dim] tensor")
        for q in planes:
            _check_dev(q, "planes", (p.dtype,), p.device.index)
            _require(q.shape == p.shape and q.stride() == p.stride(),
                     "all planes must have one shape and one stride")
        _require(p.shape[3] == 1 or p.stride(3) == 1, "planes must have unit stride along dim")
        es = p.element_size()
        cfg = CacheConfig(len(planes), p.shape[0], p.shape[1], p.shape[2], p.shape[3] * es,
                          p.stride(0) * es, p.stride(1) * es, p.stride(2) * es, max_batch,
                          max_blocks, p.device.index)
        ptrs = (ctypes.c_void_p * len(planes))(*[q.data_ptr() for q in planes])
        h = ctypes.c_void_p()
        if scales is None:
            _check("ss_cache_create",
                   self.lib.ss_cache_create(ctypes.byref(cfg), ptrs, ctypes.byref(h)))
        else:
            scales = list(scales.unbind(0)) if isinstance(scales, torch.Tensor) else list(scales)
            _require(p.dtype in (torch.float8_e4m3fn, torch.uint8),
                     "planes with scales must be float8_e4m3fn or uint8")
            _require(len(scales) == len(planes), "scales must be one for each plane")
            x = scales[0]
            for q in scales:
                _check_dev(q, "scales", (torch.uint8,), p.device.index)
                _require(q.dim() == 3 and q.shape == x.shape and q.stride() == x.stride(),
                         "all scales must have one shape and one stride")
            _require(x.shape[0] == p.shape[0] and x.shape[2] == p.shape[2] and x.shape[1] > 0 and
                     p.shape[1] % x.shape[1] == 0,
                     "scales must be [num_planes, num_pages, page_size / block, heads]")
            lay = CacheScales(p.shape[1] // x.shape[1], x.stride(0), x.stride(1), x.stride(2))
            xptrs = (ctypes.c_void_p * len(scales))(*[q.data_ptr() for q in scales])
            _check("ss_cache_create_scaled",
                   self.lib.ss_cache_create_scaled(ctypes.byref(cfg), ptrs, xptrs, ctypes.byref(lay),
                                                   ctypes.byref(h)))
        self.handle = h
        self.planes, self.scales = planes, scales
        self.heads, self.dim = p.shape[2], p.shape[3]
        self.num_pages, self.page_size = p.shape[0], p.shape[1]
        self.max_batch, self.max_blocks = max_batch, max_blocks
        self.device = p.device.index

    def close(self):
        if getattr(self, "handle", None):
            self.lib.ss_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        self.close()

    def workspace_bytes(self):
        return int(self.lib.ss_cache_workspace_bytes(self.handle))

    def new_tables(self, rows=None):
        """Empty block tables: no pages held, all free."""
        rows = self.max_batch if rows is None else rows
        dev = self.planes[0].device
        return BlockTables(torch.full((rows, self.max_blocks), -1, dtype=torch.int32, device=dev),
                           torch.zeros(self.num_pages, dtype=torch.int32, device=dev),
                           torch.zeros(rows, dtype=torch.int32, device=dev))

    def _tables(self, t):
        """The tables as the ABI takes them."""
        return CBlockTables(*self._table_words(t))

    def _table_words(self, t):
        """The tables' fields, checked by what costs least; the messages are formed on
        failure only."""
        dev, tab = self.device, t.tables
        shape = getattr(tab, "shape", ())
        if not (len(shape) == 2 and isinstance(tab, torch.Tensor) and tab.dtype is torch.int32 and
                tab.get_device() == dev and tab.is_contiguous() and
                0 < shape[0] <= self.max_batch and shape[1] >= self.max_blocks):
            _check_rows(tab, "tables", 1, (torch.int32,), dev)
            _require(tab.shape[0] <= self.max_batch and tab.shape[1] >= self.max_blocks,
                     f"tables must be [1 .. {self.max_batch}, >= {self.max_blocks}]")
            _require(tab.shape[0] <= 1 or tab.stride(0) >= self.max_blocks,
                     "tables rows must not overlap")
        rows, cols = shape
        return (tab.data_ptr(), tab.stride(0) if rows > 1 else cols, rows,
                _check_array(t.ref, "ref", self.num_pages, dev),
                _check_array(t.lens, "lens", rows, dev))

    def _count(self, v, name, most):
        """Entries of a contiguous 1-D int32 array of at most `most`, and its address."""
        if not (isinstance(v, torch.Tensor) and v.dtype is torch.int32 and
                v.get_device() == self.device and v.dim() == 1 and v.is_contiguous() and
                v.shape[0] <= most):
            _check_dev(v, name, (torch.int32,), self.device)
            raise ValueError(f"{name} must be a contiguous 1-D array of at most {most} entries")
        return v.shape[0], v.data_ptr()

    def _ok(self, ok, n, like, stream):
        if ok is None:
            return _empty_rows(n, None, like, stream=stream)
        _check_array(ok, "ok", n, self.device)
        return ok

    def _vec(self, v, name, n):
        return _check_block(v, name, (n,), torch.int32, self.device)

    def reserve(self, tables: BlockTables, add, lens=None, ok=None, stream=None):
        """Make slots [lens, lens + add) of rows 0 .. B-1 writable (add [B] int32;
        lens None: tables.lens): fresh pages where none is held, and in place of
        shared ones (copy on write). Rows are served in order: behind one that does
        not fit none is, whatever it needs. Returns ok [B] int32 (0: refused, row
        unchanged); commit takes it as reserved."""
        ct = self._tables(tables)
        B, add_ptr = self._count(add, "add", ct.rows)
        base = _check_array(lens, "lens", B, self.device)
        ok = self._ok(ok, B, add, stream)
        st = self.lib.ss_cache_reserve(self.handle, ctypes.byref(ct), base, add_ptr, B,
                                       ok.data_ptr(), _stream_on(stream, self.device))
        if st != SS_OK:
            _check("ss_cache_reserve", st)
        return ok

    def fork(self, tables: BlockTables, src, dst, ok=None, stream=None):
        """Rows dst become copies of rows src (int32 [n]) that share their pages;
        what dst held is given back. Fork between steps, not between a row's reserve
        and its commit, which would refuse it. Returns ok [n] int32."""
        ct = self._tables(tables)
        n, src_ptr = self._count(src, "src", ct.rows)
        dst_ptr = self._vec(dst, "dst", n)
        ok = self._ok(ok, n, src, stream)
        st = self.lib.ss_cache_fork(self.handle, ctypes.byref(ct), src_ptr, dst_ptr, n,
                                    ok.data_ptr(), _stream_on(stream, self.device))
        if st != SS_OK:
            _check("ss_cache_fork", st)
        return ok

    def commit(self, tables: BlockTables, num_accepted, nodes=None, base=None, release=True,
               ok=None, stream=None, reserved=None):
        """Keep what was accepted of a draft written behind base (None:
        tables.lens): the root and num_accepted [B] drafts; with nodes [B, N] (as
        tree_verify returns them) the accepted nodes' slots are moved together.
        tables.lens becomes base + 1 + num_accepted; release: pages behind it are
        given back. reserved [B] int32: what reserve returned for this draft; rows
        with 0 there are refused. Rows whose slots lie on no page, or on one that
        others hold as well, are refused in any case. Returns ok [B] int32 (0: row
        unchanged)."""
        ct = self._tables(tables)
        B, acc = self._count(num_accepted, "num_accepted", ct.rows)
        base = _check_array(base, "base", B, self.device)
        reserved = _check_array(reserved, "reserved", B, self.device)
        at, stride, N = None, 0, 0
        if nodes is not None:
            if not (isinstance(nodes, torch.Tensor) and nodes.dtype is torch.int32 and
                    nodes.get_device() == self.device and nodes.dim() == 2 and
                    nodes.shape[0] >= B and nodes.is_contiguous()):
                _check_rows(nodes, "nodes", B, (torch.int32,), self.device)
            N = nodes.shape[1]
            stride = nodes.stride(0) if B > 1 else N
            if not 1 <= N <= 64 or stride < N:
                raise ValueError("nodes must be [B, N] with N in 1 .. 64 and rows that do not overlap")
            at = nodes.data_ptr()
        ok = self._ok(ok, B, num_accepted, stream)
        st = self.lib.ss_cache_commit_reserved(self.handle, ctypes.byref(ct), base, at, stride, N,
                                               acc, B, 1 if release else 0, reserved,
                                               ok.data_ptr(), _stream_on(stream, self.device))
        if st != SS_OK:
            _check("ss_cache_commit_reserved", st)
        return ok

    def truncate(self, tables: BlockTables, new_len=None, rows=None, stream=None):
        """Give back the pages of rows (None: 0, 1, ...) behind new_len [n] int32
        (None: all their pages: the requests end)."""
        ct = self._tables(tables)
        n, at, keep = ct.rows, None, None
        if rows is not None:
            n, at = self._count(rows, "rows", ct.rows)
            if new_len is not None:
                keep = self._vec(new_len, "new_len", n)
        elif new_len is not None:
            n, keep = self._count(new_len, "new_len", ct.rows)
        st = self.lib.ss_cache_truncate(self.handle, ctypes.byref(ct), at, keep, n,
                                        _stream_on(stream, self.device))
        if st != SS_OK:
            _check("ss_cache_truncate", st)

    def copy_pages(self, src, dst, src_cache: PageCache | None = None, ok=None, stream=None):
        """Copy pages src (int32 [n]) of src_cache (None: this cache) to pages dst of
        this cache, all planes. Returns ok [n] int32."""
        other = self if src_cache is None else src_cache
        n, src_ptr = self._count(src, "src", 65535)
        dst_ptr = self._vec(dst, "dst", n)
        ok = self._ok(ok, n, src, stream)
        st = self.lib.ss_cache_copy_pages(other.handle, src_ptr, self.handle, dst_ptr, n,
                                          ok.data_ptr(), _stream_on(stream, self.device))
        if st != SS_OK:
            _check("ss_cache_copy_pages", st)
        return ok

    def _step(self, tables, shape, lens, counts, parents, reserved):
        """The tables and a step's tokens [B, N, ...] as the ABI takes them."""
        words = self._table_words(tables)
        B, N = shape[0], shape[1]
        if B > words[2] or not 1 <= N <= self.max_blocks * self.page_size:
            raise ValueError(f"a step has at most {words[2]} rows of 1 .. "
                             f"{self.max_blocks * self.page_size} tokens")
        dev, at = self.device, 0
        if parents is not None:
            if N > 64:
                raise ValueError("a draft tree has at most 64 nodes")
            at = _check_block(parents, "parents", (B, N), torch.int32, dev)
        return _pack_tables(*words), _pack_step(B, N, _check_array(lens, "lens", B, dev) or 0,
                                                _check_array(counts, "counts", B, dev) or 0, at,
                                                _check_array(reserved, "reserved", B, dev) or 0)

    def _layer(self, layer):
        if self.scales is None:
            raise ValueError("the cache has no scales")
        if not 0 <= 2 * layer < len(self.planes) - 1:
            raise ValueError(f"layer must be in 0 .. {len(self.planes) // 2 - 1}")
        return 2 * layer, 2 * layer + 1

    def _dtype(self, t, name):
        code = _HALF_DTYPES.get(getattr(t, "dtype", None))
        if code is None or t.dim() != 4:
            raise ValueError(f"{name} must be a [B, N, heads, dim] array of bfloat16 or float16")
        return code

    def write(self, tables: BlockTables, layer, keys, values, lens=None, counts=None, parents=None,
              reserved=None, rotary=None, positions=None, queries=None, out_queries=None,
              stream=None):
        """Write a step's keys and values [B, N, heads, dim] (bfloat16 or float16) into
        the slots behind lens (None: tables.lens), in 8 bits: token i of row b into
        slot lens[b] + i, the first counts[b] of them (None: all N). reserved: what
        reserve returned; rows with 0 there write nothing.

        rotary (a Rotary whose dim is a multiple of 16 or divides the head's): the keys
        are turned by their positions first: positions [B, N] int32, else lens + i, with
        parents [B, N] (a draft tree as tree_verify takes it) lens + the node's depth.
        queries [B, N, q_heads, dim] are turned along, into out_queries, which is
        returned (None: a new array; queries itself: in place); rows of tokens that
        there are not become 0."""
        k_plane, v_plane = self._layer(layer)
        code = self._dtype(keys, "keys")
        shape = (*keys.shape[:2], self.heads, self.dim)
        ct, step = self._step(tables, shape, lens, counts, parents, reserved)
        k = _heads(keys, "keys", shape, keys.dtype, self.device)
        v = _heads(values, "values", shape, keys.dtype, self.device)
        at = None
        if positions is not None:
            if rotary is None:
                raise ValueError("positions are for a rotary: give one")
            at = _check_block(positions, "positions", shape[:2], torch.int32, self.device)
        r = q = o = None
        q_heads = 0
        if rotary is not None:
            r = rotary.on(self.device)
        if queries is not None:
            if rotary is None:
                raise ValueError("queries are turned along: give a rotary")
            q = _heads(queries, "queries", None, keys.dtype, self.device)
            q_heads = queries.shape[2] if queries.dim() == 4 else 0
            if q_heads < 1 or queries.shape != (*shape[:2], q_heads, self.dim):
                raise ValueError("queries must be [B, N, q_heads, dim]")
            out_queries, o = _out_heads(out_queries, "out_queries", queries.shape, queries, keys.dtype, stream)
        elif out_queries is not None:
            raise ValueError("out_queries needs queries")
        st = self.lib.ss_cache_write(self.handle, ct, step, k_plane, v_plane, code, k, v, r, at, q, o,
                                     q_heads, _stream_on(stream, self.device))
        if st != SS_OK:
            _check("ss_cache_write", st)
        return out_queries if q is not None else None

    def read(self, tables: BlockTables, layer, N, start=None, counts=None, dtype=torch.bfloat16,
             out_keys=None, out_values=None, stream=None):
        """The keys and values of slots start .. start + N - 1 of rows 0 .. B-1 (start
        [B] int32, None: 0 of every row) as two [B, N, heads, dim] arrays of dtype
        (bfloat16: exactly; float16). Entries behind counts[b] (None: N) and of slots
        on no page are 0."""
        k_plane, v_plane = self._layer(layer)
        code = _HALF_DTYPES.get(dtype)
        if code is None:
            raise ValueError("dtype must be bfloat16 or float16")
        words = self._table_words(tables)
        B = words[2]
        if start is not None:
            B, _ = self._count(start, "start", B)
        elif counts is not None:
            B, _ = self._count(counts, "counts", B)
        if not 1 <= N <= self.max_blocks * self.page_size:
            raise ValueError(f"at most {words[2]} rows of 1 .. {self.max_blocks * self.page_size} "
                             f"slots are read")
        first = _check_array(start, "start", B, self.device)
        n = _check_array(counts, "counts", B, self.device)
        shape = (B, N, self.heads, self.dim)
        like = tables.tables
        out_keys, k = _out_heads(out_keys, "out_keys", shape, like, dtype, stream)
        out_values, v = _out_heads(out_values, "out_values", shape, like, dtype, stream)
        st = self.lib.ss_cache_read(self.handle, _pack_tables(*words), first, n, B, N, k_plane, v_plane,
                                    code, k, v, _stream_on(stream, self.device))
        if st != SS_OK:
            _check("ss_cache_read", st)
        return out_keys, out_values

    def attend(self, tables: BlockTables, layer, queries, lens=None, counts=None, parents=None,
               reserved=None, scale=None, out=None, lse=None, stream=None):
        """Attention of a step's queries [B, N, q_heads, dim] (bfloat16 or float16) over
        the cache; q_heads is a multiple of its heads. Token i of row b stands in slot
        lens[b] + i (None: tables.lens) and sees the slots before lens[b] and, of the
        step's, its own and those before it; with parents [B, N] (a draft tree as
        tree_verify takes it) its own and those of the nodes above it. counts and
        reserved as for write. scale: 2^-60 .. 2^60, None is 1 / sqrt(dim). Returns out,
        like queries (None: a new array); a token that sees nothing gets 0. lse: None, or
        a contiguous [B, N, q_heads] float32 array for the logarithms of the sums of
        exponentials."""
        k_plane, v_plane = self._layer(layer)
        code = self._dtype(queries, "queries")
        shape = queries.shape
        ct, step = self._step(tables, shape, lens, counts, parents, reserved)
        q = _heads(queries, "queries", None, queries.dtype, self.device)
        q_heads = shape[2]
        if shape[3] != self.dim or q_heads < 1 or q_heads % self.heads:
            raise ValueError(f"queries must be [B, N, a multiple of {self.heads}, {self.dim}]")
        out, o = _out_heads(out, "out", shape, queries, queries.dtype, stream)
        at = None
        if lse is not None:
            at = _check_block(lse, "lse", shape[:3], torch.float32, self.device)
        st = self.lib.ss_cache_attend(self.handle, ct, step, k_plane, v_plane, code, q, o, q_heads,
                                      self.dim ** -0.5 if scale is None else scale, at,
                                      _stream_on(stream, self.device))
        if st != SS_OK:
            _check("ss_cache_attend", st)
        return out
