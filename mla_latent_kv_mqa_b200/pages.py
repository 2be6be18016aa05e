"""The pages of a paged latent cache, kept on the device: which sequence holds which, and how many
hold each (include/mla.h, "Pages of the cache").

    seqs = PagedSequences(page_size, num_seqs, max_blocks, num_blocks)
    moves = seqs.grow(new_lens)                  # pages for new tokens, own copies of shared last pages
    seqs.copy_pages(caches, moves)               # before the new rows are appended
    seqs.fork(parent, child)                     # samples, beams: child holds parent's pages too
    seqs.trim(new_lens)                          # cut or end sequences
    seqs.copy_pages(caches, seqs.compact())      # pages in use to the front of the pool

``block_table``, ``refs`` and ``seq_lens`` are the tensors the other calls take.  One table serves the
caches of all layers.  Calls take the current stream, or ``stream``.
"""
from __future__ import annotations

import torch

from . import native as N
from .layer import _INT32, _MISREAD, Workspace, _current_handle, _on_device, _stream_object, new_on, same_caches, used_on


class PageMoves:
    """Page copies to make, on the device: ``pairs`` [most, 2] of (from, to) and their ``number`` [1].  One buffer
    holds both, of the stream that writes them; unpacks as (pairs, number)."""

    def __init__(self, most: int, device, stream=None, handle=None):
        self.most = most
        if stream is None:
            self._buf = torch.empty((most + 1, 2), dtype=torch.int32, device=device)
        else:
            self._buf, = new_on(stream, lambda: (torch.empty((most + 1, 2), dtype=torch.int32, device=device),))
        self._handle = handle  # of the stream that writes them
        self.pairs_ptr = self._buf.data_ptr()
        self.number_ptr = self.pairs_ptr + 8 * most

    @property
    def pairs(self) -> torch.Tensor:
        return self._buf[:self.most]

    @property
    def number(self) -> torch.Tensor:
        return self._buf[self.most, :1]

    def __iter__(self):
        return iter((self.pairs, self.number))

    def __getitem__(self, i):
        return (self.pairs, self.number)[i]


class PagedSequences:
    def __init__(self, page_size: int, num_seqs: int, max_blocks: int, num_blocks: int, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self._block_table = torch.full((num_seqs, max_blocks), -1, **i32)
        self._refs = torch.zeros(num_blocks, **i32)
        self._seq_lens = torch.zeros(num_seqs, **i32)
        self.num_blocks = int(num_blocks)
        self._table = N.make_page_table(page_size, num_seqs, max_blocks, num_blocks, self._block_table, self._refs,
                                        self._seq_lens)
        self._ws = Workspace(self._block_table.device)
        self._device = self._refs.get_device()

    # Written in place (copy_), not replaced: the calls hold their addresses.
    @property
    def block_table(self) -> torch.Tensor:
        return self._block_table

    @property
    def refs(self) -> torch.Tensor:
        return self._refs

    @property
    def seq_lens(self) -> torch.Tensor:
        return self._seq_lens

    def _look_over(self, stream, *indices):
        """The handle of the call's stream, once its tensors are what the kernels read."""
        here = self._device
        if here < 0 or here != _on_device():
            raise ValueError(_MISREAD)
        for x in indices:
            if x is not None and (x.dtype is not _INT32 or x.get_device() != here or not x.is_contiguous()):
                raise ValueError(_MISREAD)
        if stream is None:
            return _current_handle(here)
        used_on(stream, self._block_table, self._refs, self._seq_lens, *indices)
        return N._stream(stream)

    def _workspace(self, n: int, handle, stream):
        return self._ws.get(n, handle, stream, N.mla_pages_workspace_size, self._table, n)

    def fork(self, parent, child, stream=None):
        """Sequence child[i] becomes a copy of parent[i]; all parents are read before any child changes."""
        if parent.numel() != child.numel():
            raise ValueError("fork: a parent for every child")
        handle = self._look_over(stream, parent, child)
        n = parent.numel()
        with self._ws.lock:
            ws = self._workspace(n, handle, stream)
            N.mla_pages_fork(self._table, n, parent, child, ws, ws.numel(), handle)

    def grow(self, new_lens, seqs=None, stream=None):
        """Sequences ``seqs`` (default: 0, 1, ...) grow to ``new_lens`` tokens; returns the page copies to
        make (PageMoves), for copy_pages."""
        n = new_lens.numel()
        if seqs is not None and seqs.numel() != n:
            raise ValueError("grow: a length for every sequence")
        handle = self._look_over(stream, new_lens, seqs)
        moves = PageMoves(n, self._block_table.device, stream, handle)
        with self._ws.lock:
            ws = self._workspace(n, handle, stream)
            N.mla_pages_grow(self._table, n, seqs, new_lens, moves.pairs_ptr, moves.number_ptr, ws, ws.numel(), handle)
        return moves

    def trim(self, new_lens, seqs=None, stream=None):
        """Sequences are cut to ``new_lens`` tokens (0: the sequence ends); their pages lose a holder."""
        if seqs is not None and seqs.numel() != new_lens.numel():
            raise ValueError("trim: a length for every sequence")
        handle = self._look_over(stream, new_lens, seqs)
        with self._ws.lock:  # not between the kernels of another call
            N.mla_pages_trim(self._table, new_lens.numel(), seqs, new_lens, handle)

    def compact(self, stream=None):
        """The pages in use take the lowest ids; returns the page copies to make (PageMoves), for copy_pages."""
        handle = self._look_over(stream)
        moves = PageMoves(self.num_blocks // 2, self._block_table.device, stream, handle)
        with self._ws.lock:
            ws = self._workspace(0, handle, stream)
            N.mla_pages_compact(self._table, moves.pairs_ptr, moves.number_ptr, ws, ws.numel(), handle)
        return moves

    def copy_pages(self, caches, moves, stream=None):
        """Copy the pages that ``moves`` names (PageMoves, or a pair of tensors like its), in every cache."""
        if not caches:
            return
        dims = same_caches(caches, self.num_blocks)
        if dims.page_size != self._table.page_size:
            raise ValueError("copy_pages: the caches' pages are not the table's")
        handle = self._look_over(stream)
        for c in caches:
            if c.kv_pool.get_device() != self._device:
                raise ValueError(_MISREAD)
        pools = N.make_pools([c.pool() for c in caches])
        if isinstance(moves, PageMoves):
            pairs, number, most = moves.pairs_ptr, moves.number_ptr, moves.most
            if handle != moves._handle:  # their memory is not given back before this stream has read them
                moves._buf.record_stream(_stream_object(handle))
        else:
            pairs, number = moves
            self._look_over(stream, pairs, number)
            if pairs.dim() != 2 or pairs.shape[1] != 2 or (number is not None and number.numel() < 1):
                raise ValueError("copy_pages: moves are pairs [n, 2] and their number [1], or None for all")
            most = pairs.shape[0]
        if stream is not None:
            used_on(stream, *(x for c in caches for x in (c.kv_pool, c.kr_pool, c.kv_scale)))
        N.mla_cache_copy_pages(dims, pools, self.num_blocks, pairs, number, most, handle)
