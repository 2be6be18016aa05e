"""Drafted trees of a batch: which nodes, and the buffers that a step's calls share.

A speculative step of one model::

    trees = DraftTrees(cu_nodes, parent, max_nodes)
    trees.prepare(seq_lens)                                            # once: masks, slots, positions
    for layer, cache in ...:
        layer.tree_append(cache, c_kv, k_r, trees, block_table)        # the nodes' rows
        q_abs = layer.absorb(q_c, q_r, trees.pos)
        o_lat, lse = layer.decode_tree(cache, q_abs, block_table, seq_lens, trees, max_seq_len)
        o = layer.out_proj(o_lat)
    new_lens = trees.keep(caches, block_table, seq_lens, keep, num_keep)   # the accepted path

seq_lens counts the committed tokens and the nodes (include/mla.h, "Drafted trees").
"""
from __future__ import annotations

import torch

from . import native as N
from .layer import _INT32, _MISREAD, _current_handle, _on_device, new_on, same_caches, used_on


def _checked(name: str) -> property:
    """A tensor that is replaced only by one of its shape, type and device (or written in place)."""
    def put(self, x):
        old = getattr(self, name)
        if x.shape != old.shape or x.dtype != old.dtype or x.device != old.device or not x.is_contiguous():
            raise ValueError(f"{name[1:]} must be contiguous {old.dtype} {tuple(old.shape)} on {old.device}")
        setattr(self, name, x)
    return property(lambda self: getattr(self, name), put)


class DraftTrees:
    """The drafted nodes of B sequences, packed: ``cu_nodes`` [B + 1] and ``parent`` [total_nodes],
    int32 on the device, and ``max_nodes``, a host-side bound of a sequence's nodes.

    ``mask`` [total_nodes, mask_words], ``pos``, ``slot`` and ``seq_idx`` [total_nodes] are written by
    prepare(); a caller with masks of its own hands ``mask`` over (int32 words) and writes it after prepare(), which
    fills it with the ancestors."""

    def __init__(self, cu_nodes: torch.Tensor, parent: torch.Tensor, max_nodes: int, mask: torch.Tensor | None = None):
        if not 1 <= max_nodes <= N.MLA_MAX_TREE_NODES:
            raise ValueError(f"max_nodes must be in [1, {N.MLA_MAX_TREE_NODES}]")
        for x in (cu_nodes, parent):
            if x.dtype != torch.int32 or x.dim() != 1 or not x.is_contiguous():
                raise ValueError("cu_nodes and parent must be contiguous int32 vectors")
        if parent.device != cu_nodes.device or (mask is not None and mask.device != cu_nodes.device):
            raise ValueError("cu_nodes, parent and mask must be on one device")
        if mask is not None and mask.dim() != 2:
            raise ValueError("mask must be [total_nodes, words]")
        if cu_nodes.numel() < 1:
            raise ValueError("cu_nodes must have an entry per sequence and one more")
        self._cu_nodes, self._parent, self.max_nodes = cu_nodes, parent, int(max_nodes)
        self.B, self.total_nodes = cu_nodes.numel() - 1, parent.numel()
        self.mask_words = (self.max_nodes + 31) // 32 if mask is None else mask.shape[1]
        if mask is not None and (mask.shape[0] != self.total_nodes or 32 * self.mask_words < self.max_nodes or
                                 mask.dtype != torch.int32 or not mask.is_contiguous()):
            raise ValueError("mask must be contiguous int32 [total_nodes, >= ceil(max_nodes / 32)]")
        dev = cu_nodes.device
        self._mask = torch.empty((self.total_nodes, self.mask_words), dtype=torch.int32, device=dev) if mask is None else mask
        self._pos, self._slot = (torch.empty(self.total_nodes, dtype=torch.int32, device=dev) for _ in range(2))
        self._seq_idx = torch.full((self.total_nodes,), -1, dtype=torch.int32, device=dev)  # an append before prepare() goes nowhere

    # Looked over once, when they come, not in every call.
    cu_nodes, parent, mask = _checked("_cu_nodes"), _checked("_parent"), _checked("_mask")
    pos, slot, seq_idx = _checked("_pos"), _checked("_slot"), _checked("_seq_idx")

    def prepare(self, seq_lens, stream=None):
        if seq_lens.numel() != self.B:
            raise ValueError("prepare: seq_lens has an entry per tree")
        here = seq_lens.get_device()
        if (here < 0 or here != _on_device() or self._cu_nodes.get_device() != here or seq_lens.dtype is not _INT32 or
                not seq_lens.is_contiguous()):
            raise ValueError(_MISREAD)
        if stream is not None:
            used_on(stream, seq_lens, self._cu_nodes, self._parent, self._mask, self._pos, self._slot, self._seq_idx)
        N.mla_tree_prepare(self.B, self._cu_nodes, self.total_nodes, self._parent, seq_lens, self.mask_words, self._mask,
                           self._pos, self._slot, self._seq_idx, _current_handle(here) if stream is None else stream)

    def keep(self, caches, block_table, seq_lens, keep, num_keep, new_lens=None, stream=None):
        """The rows of the accepted nodes ``keep`` [B, max_keep] (each row's first num_keep[b],
        ascending) to behind the committed tokens, in every cache; returns the new lengths."""
        B, max_blocks = block_table.shape
        if B != self.B or seq_lens.numel() != B or keep.dim() != 2 or keep.size(0) != B or num_keep.numel() != B:
            raise ValueError("keep: block_table, seq_lens, keep [trees, max_keep] and num_keep have a row per tree")
        if not caches:
            raise ValueError("keep: no caches")
        here = seq_lens.get_device()
        if (here < 0 or here != _on_device() or self._cu_nodes.get_device() != here or block_table.get_device() != here or
                keep.get_device() != here or num_keep.get_device() != here or
                block_table.dtype is not _INT32 or seq_lens.dtype is not _INT32 or keep.dtype is not _INT32 or
                num_keep.dtype is not _INT32 or
                not (block_table.is_contiguous() and seq_lens.is_contiguous() and keep.is_contiguous() and num_keep.is_contiguous())):
            raise ValueError(_MISREAD)
        for c in caches:
            if c.kv_pool.get_device() != here:
                raise ValueError(_MISREAD)
        if new_lens is None:
            if stream is None:
                new_lens = torch.empty_like(seq_lens)
            else:
                new_lens, = new_on(stream, lambda: (torch.empty_like(seq_lens),))
        elif new_lens.dtype is not _INT32 or new_lens.numel() != B or new_lens.get_device() != here or not new_lens.is_contiguous():
            raise ValueError(_MISREAD)
        dims, pools = same_caches(caches, caches[0].num_blocks), N.make_pools([c.pool() for c in caches])
        if stream is not None:
            used_on(stream, block_table, seq_lens, keep, num_keep, new_lens, self._cu_nodes,
                    *(x for c in caches for x in (c.kv_pool, c.kr_pool, c.kv_scale)))
        N.mla_cache_keep(dims, pools, B, self._cu_nodes, self.total_nodes, block_table, max_blocks,
                         caches[0].num_blocks, seq_lens, keep, num_keep, keep.shape[1], new_lens,
                         _current_handle(here) if stream is None else stream)
        return new_lens
