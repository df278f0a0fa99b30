"""Thin ctypes binding of the page cache (ss_cache_* in include/ss_sampler.h).

A PageCache names the planes (a layer's keys, a layer's values, ...) that share
page numbers; BlockTables holds the device arrays that say which request holds
which pages. The pages around a verification step: reserve slots for the draft,
run the model, verify, commit what was accepted. Nothing is read back to the
host; everything is computed in the HIP library.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from .sampler import (CacheConfig, CBlockTables, _check, _check_block, _check_dev, _check_rows,
                      _check_vec, _ptr, _require, _stream_on, load_library)


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
    fine) as long as no two pieces overlap. The planes are kept referenced."""

    def __init__(self, planes, max_batch, max_blocks):
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
        _check("ss_cache_create", self.lib.ss_cache_create(ctypes.byref(cfg), ptrs, ctypes.byref(h)))
        self.handle = h
        self.planes = planes
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
        dev = self.device
        _check_rows(t.tables, "tables", 1, (torch.int32,), dev)
        rows, cols = t.tables.shape
        _require(rows <= self.max_batch and cols >= self.max_blocks,
                 f"tables must be [1 .. {self.max_batch}, >= {self.max_blocks}]")
        _require(rows <= 1 or t.tables.stride(0) >= self.max_blocks, "tables rows must not overlap")
        _check_vec(t.ref, "ref", self.num_pages, torch.int32, dev)
        _check_vec(t.lens, "lens", rows, torch.int32, dev)
        stride = t.tables.stride(0) if rows > 1 else cols
        return CBlockTables(t.tables.data_ptr(), stride, rows, t.ref.data_ptr(), t.lens.data_ptr())

    def _ok(self, ok, n):
        if ok is None:
            return torch.empty(n, dtype=torch.int32, device=self.planes[0].device)
        _check_vec(ok, "ok", n, torch.int32, self.device)
        return ok

    def _vec(self, v, name, n):
        _check_block(v, name, (n,), torch.int32, self.device)

    def reserve(self, tables: BlockTables, add, lens=None, ok=None, stream=None):
        """Make slots [lens, lens + add) of rows 0 .. B-1 writable (add [B] int32;
        lens None: tables.lens): fresh pages where none is held, and in place of
        shared ones (copy on write). Returns ok [B] int32 (0: not enough pages,
        row unchanged)."""
        ct = self._tables(tables)
        _check_dev(add, "add", (torch.int32,), self.device)
        _require(add.dim() == 1 and add.shape[0] <= ct.rows, "add must be [B] with B <= rows")
        B = add.shape[0]
        self._vec(add, "add", B)
        _check_vec(lens, "lens", B, torch.int32, self.device)
        ok = self._ok(ok, B)
        _check("ss_cache_reserve", self.lib.ss_cache_reserve(
            self.handle, ctypes.byref(ct), _ptr(lens), _ptr(add), B, _ptr(ok),
            _stream_on(stream, self.device)))
        return ok

    def fork(self, tables: BlockTables, src, dst, ok=None, stream=None):
        """Rows dst become copies of rows src (int32 [n]) that share their pages;
        what dst held is given back. Returns ok [n] int32."""
        ct = self._tables(tables)
        _check_dev(src, "src", (torch.int32,), self.device)
        _require(src.dim() == 1 and src.shape[0] <= ct.rows, "src must be [n] with n <= rows")
        n = src.shape[0]
        self._vec(src, "src", n)
        self._vec(dst, "dst", n)
        ok = self._ok(ok, n)
        _check("ss_cache_fork", self.lib.ss_cache_fork(
            self.handle, ctypes.byref(ct), _ptr(src), _ptr(dst), n, _ptr(ok),
            _stream_on(stream, self.device)))
        return ok

    def commit(self, tables: BlockTables, num_accepted, nodes=None, base=None, release=True,
               ok=None, stream=None):
        """Keep what was accepted of a draft written behind base (None:
        tables.lens): the root and num_accepted [B] drafts; with nodes [B, N] (as
        tree_verify returns them) the accepted nodes' slots are moved together.
        tables.lens becomes base + 1 + num_accepted; release: pages behind it are
        given back. Returns ok [B] int32."""
        ct = self._tables(tables)
        _check_dev(num_accepted, "num_accepted", (torch.int32,), self.device)
        _require(num_accepted.dim() == 1 and num_accepted.shape[0] <= ct.rows,
                 "num_accepted must be [B] with B <= rows")
        B = num_accepted.shape[0]
        self._vec(num_accepted, "num_accepted", B)
        _check_vec(base, "base", B, torch.int32, self.device)
        stride = N = 0
        if nodes is not None:
            _check_rows(nodes, "nodes", B, (torch.int32,), self.device)
            N = nodes.shape[1]
            _require(1 <= N <= 64, "nodes must be [B, N] with N in 1 .. 64")
            stride = nodes.stride(0) if B > 1 else N
            _require(stride >= N, "nodes rows must not overlap")
        ok = self._ok(ok, B)
        _check("ss_cache_commit", self.lib.ss_cache_commit(
            self.handle, ctypes.byref(ct), _ptr(base), _ptr(nodes), stride, N, _ptr(num_accepted),
            B, int(bool(release)), _ptr(ok), _stream_on(stream, self.device)))
        return ok

    def truncate(self, tables: BlockTables, new_len=None, rows=None, stream=None):
        """Give back the pages of rows (None: 0, 1, ...) behind new_len [n] int32
        (None: all their pages: the requests end)."""
        ct = self._tables(tables)
        n = ct.rows
        for name, v in (("rows", rows), ("new_len", new_len)):
            if v is not None:
                _check_dev(v, name, (torch.int32,), self.device)
                _require(v.dim() == 1 and v.shape[0] <= ct.rows, f"{name} must be [n] with n <= rows")
                n = v.shape[0]
        for name, v in (("rows", rows), ("new_len", new_len)):
            if v is not None:
                self._vec(v, name, n)
        _check("ss_cache_truncate", self.lib.ss_cache_truncate(
            self.handle, ctypes.byref(ct), _ptr(rows), _ptr(new_len), n,
            _stream_on(stream, self.device)))

    def copy_pages(self, src, dst, src_cache: PageCache | None = None, ok=None, stream=None):
        """Copy pages src (int32 [n]) of src_cache (None: this cache) to pages dst of
        this cache, all planes. Returns ok [n] int32."""
        other = self if src_cache is None else src_cache
        _check_dev(src, "src", (torch.int32,), self.device)
        _require(src.dim() == 1, "src must be [n]")
        n = src.shape[0]
        self._vec(src, "src", n)
        self._vec(dst, "dst", n)
        ok = self._ok(ok, n)
        _check("ss_cache_copy_pages", self.lib.ss_cache_copy_pages(
            other.handle, _ptr(src), self.handle, _ptr(dst), n, _ptr(ok),
            _stream_on(stream, self.device)))
        return ok
