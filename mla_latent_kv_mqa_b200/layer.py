"""User-facing objects over the C ABI: the paged latent cache and one MLA decode layer.

PyTorch only allocates device memory and supplies streams here; each step of the
decode path runs in libmla's kernels through :mod:`.native`.

A decode step of one layer (itwiki "멀티 헤드 잠재 어텐션", sections 분리 RoPE and
행렬 흡수) is::

    layer.append(cache, c_kv_new, k_r_new, seq_idx, pos, block_table)   # cache rows
    q_abs = layer.absorb(q_c, q_r, pos_q)                                # [W_UK^T q_C ; RoPE(q_R)]
    o_lat, lse = layer.decode(cache, q_abs, block_table, seq_lens, s_q)  # attention over the cache
    o = layer.out_proj(o_lat)                                            # W_UV o_lat
"""
from __future__ import annotations

import threading
import weakref

import torch

from . import native as N

DTYPE = {"f32": N.MLA_DTYPE_F32, "bf16": N.MLA_DTYPE_BF16, "fp8": N.MLA_DTYPE_FP8_E4M3}
TORCH_ACT = {N.MLA_DTYPE_F32: torch.float32, N.MLA_DTYPE_BF16: torch.bfloat16}


def dims_for(n_h, d_h, d_c, d_r, *, act="bf16", kv="bf16", page=64, rope_base=1e4, flags=0):
    return N.make_dims(n_h, d_h, d_c, d_r, page, rope_base, DTYPE[act], DTYPE[kv], flags)


class PagedLatentCache:
    """Device buffers of a paged latent cache with ``num_blocks`` blocks of ``page_size`` tokens.

    bf16 / f32: ``kv_pool`` [num_blocks, page, d_c + d_r] rows [c_kv ; RoPE(k_r)].
    fp8: ``kv_pool`` [num_blocks, page, d_c] e4m3 codes, ``kr_pool`` [num_blocks, page, d_r]
    bf16, ``kv_scale`` [num_blocks, page] fp32.  ``poison`` fills every slot with NaN first."""

    _pool = None  # pool()'s last answer, with the addresses it is for

    def __init__(self, dims: N.mla_dims_t, num_blocks: int, device="cuda", poison: bool = False):
        self.dims = dims
        self.num_blocks = int(num_blocks)
        page = dims.page_size
        self.kr_pool = None
        self.kv_scale = None
        if dims.kv_dtype == N.MLA_DTYPE_FP8_E4M3:
            self.kv_pool = torch.empty((num_blocks, page, dims.d_c), dtype=torch.uint8, device=device)
            self.kr_pool = torch.empty((num_blocks, page, dims.d_r), dtype=torch.bfloat16, device=device)
            self.kv_scale = torch.empty((num_blocks, page), dtype=torch.float32, device=device)
            if poison:
                self.kv_pool.fill_(0x7F)
                self.kr_pool.fill_(float("nan"))
                self.kv_scale.fill_(float("nan"))
        else:
            dt = torch.float32 if dims.kv_dtype == N.MLA_DTYPE_F32 else torch.bfloat16
            self.kv_pool = torch.empty((num_blocks, page, dims.d_c + dims.d_r), dtype=dt, device=device)
            if poison:
                self.kv_pool.fill_(float("nan"))

    @classmethod
    def over(cls, dims: N.mla_dims_t, kv_pool, kr_pool=None, kv_scale=None) -> "PagedLatentCache":
        """A cache over buffers that the caller holds (one layer of a stacked allocation, say)."""
        fp8 = dims.kv_dtype == N.MLA_DTYPE_FP8_E4M3
        row = dims.d_c if fp8 else dims.d_c + dims.d_r
        dt = torch.uint8 if fp8 else torch.float32 if dims.kv_dtype == N.MLA_DTYPE_F32 else torch.bfloat16
        n, page = kv_pool.shape[0], dims.page_size
        want = [(kv_pool, (n, page, row), dt)]
        if fp8:
            want += [(kr_pool, (n, page, dims.d_r), torch.bfloat16), (kv_scale, (n, page), torch.float32)]
        elif kr_pool is not None or kv_scale is not None:
            raise ValueError("kr_pool and kv_scale belong to an FP8 cache")
        for x, shape, dtype in want:
            if x is None or tuple(x.shape) != shape or x.dtype != dtype or not x.is_contiguous() or x.device != kv_pool.device:
                raise ValueError(f"cache buffer must be contiguous {dtype} {shape}, all on one device")
        self = cls.__new__(cls)
        self.dims, self.num_blocks = dims, int(n)
        self.kv_pool, self.kr_pool, self.kv_scale = kv_pool, kr_pool, kv_scale
        return self

    def pool(self) -> N.mla_pool_t:
        """The buffers as mla_cache_keep and mla_cache_copy_pages take them."""
        kr, scale = self.kr_pool, self.kv_scale
        at = self.kv_pool.data_ptr(), None if kr is None else kr.data_ptr(), None if scale is None else scale.data_ptr()
        known = self._pool
        if known is None or known[0] != at:
            known = self._pool = at, N.mla_pool_t(*at)
        return known[1]

    @property
    def nbytes(self) -> int:
        n = self.kv_pool.numel() * self.kv_pool.element_size()
        if self.kr_pool is not None:
            n += self.kr_pool.numel() * self.kr_pool.element_size()
            n += self.kv_scale.numel() * self.kv_scale.element_size()
        return n


# The kernels run on the current device and read rows and indices as they lie: a tensor elsewhere, of another type or
# with strides of its own is refused, not misread.  (Written out where it is called: a helper per tensor costs a
# microsecond a call.)
_INT32 = torch.int32
_on_device = getattr(torch._C, "_cuda_getDevice", None)
_is_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None)
_current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_MISREAD = ("tensors are contiguous and on the current CUDA device; lengths, tables and indices are int32")


def _stream_object(handle: int):
    return torch.cuda.ExternalStream(handle) if handle > 1 else torch.cuda.default_stream()  # 0, 1: the legacy stream


def used_on(stream, *tensors):
    """A call on ``stream``, named by its caller, uses the tensors: their memory is not given back before it has."""
    handle = N._stream(stream)
    if handle != N._stream(None):
        stream = _stream_object(handle)
        for x in tensors:
            if x is not None:
                x.record_stream(stream)


def new_on(stream, make):
    """make()'s tensors, for a call that names its ``stream``.  On another one than the current they are taken from that
    stream's memory (what held it before has run there) and given back once both streams are past them."""
    here, handle = N._stream(None), N._stream(stream)
    if here == handle:
        return make()
    current = torch.cuda.current_stream()
    with torch.cuda.stream(_stream_object(handle)):
        made = make()
    for x in made:
        x.record_stream(current)
    return made


def fits(dims: N.mla_dims_t, of: N.mla_dims_t) -> bool:
    """A cache of ``of`` has the rows that a layer of ``dims`` reads and writes."""
    return of is dims or (of.kv_dtype == dims.kv_dtype and of.d_c == dims.d_c and of.d_r == dims.d_r and
                          of.page_size == dims.page_size)


def same_caches(caches, num_blocks) -> N.mla_dims_t:
    """The dims of caches behind one block table, which are of one shape and have its blocks."""
    dims = caches[0].dims
    for c in caches if len(caches) > 1 or caches[0].num_blocks != num_blocks else ():
        if c.num_blocks != num_blocks or (c.dims is not dims and bytes(c.dims) != bytes(dims)):
            raise ValueError("caches behind one block table are of one shape and have its number of blocks")
    return dims


class Workspace:
    """Device scratch for calls of one kind: a buffer per stream, so that calls on two streams do not meet in one,
    grown by doubling.  A call that is being captured gets a buffer of its own from the graph's memory
    (torch.cuda.graph), so that graphs that replay at the same time do not meet either.
    ``lock``: held from get() until the call's kernels are enqueued, or another thread's would come between them."""

    def __init__(self, device):
        self.device = device
        self.lock = threading.Lock()
        self._by_stream, self._known = {}, {}

    _shared = weakref.WeakValueDictionary()

    @classmethod
    def shared(cls, device) -> "Workspace":
        """The device's one, while a layer is there: layers' calls on a stream run one after the other and can share its
        buffer."""
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        return cls._shared.setdefault(device, cls(device))

    def _new(self, need, stream):
        make = lambda: (torch.empty(need, dtype=torch.uint8, device=self.device),)
        return (make() if stream is None else new_on(stream, make))[0]

    def get(self, key, handle, stream, size, *args):
        """A buffer of at least ``size(*args)`` bytes, which depend on ``key`` alone, for a call on ``stream`` (its handle)."""
        if stream is None:
            capturing = _is_capturing()
        else:
            with torch.cuda.stream(_stream_object(handle)):
                capturing = _is_capturing()
        known = None if capturing else self._known.get((key, handle))
        if known is not None:
            return known
        need = max(256, size(*args))
        if capturing:
            return self._new(need, stream)
        buf = self._by_stream.get(handle)
        if buf is None or buf.numel() < need:
            if buf is not None:
                need = max(need, 2 * buf.numel())
                self._known.clear()
            buf = self._by_stream[handle] = self._new(need, stream)
        if len(self._known) > 1024:  # lengths that change every step
            self._known.clear()
        self._known[key, handle] = buf
        return buf


class MLADecodeLayer:
    """Weights of one MLA layer (W_UK, W_UV as [n_h*d_h, d_c]) plus reusable decode and
    prefill workspaces."""

    def __init__(self, dims: N.mla_dims_t, w_uk: torch.Tensor, w_uv: torch.Tensor):
        self.dims = dims
        self.w_uk = w_uk.contiguous()
        self.w_uv = w_uv.contiguous()
        self.device = w_uk.device
        self._ws = None
        self._ws_key = None
        self._pf_ws = None
        self._tree_ws, self._tree_key = Workspace.shared(self.device), bytes(dims)

    # -- the four calls ----------------------------------------------------------------------
    def append(self, cache: PagedLatentCache, c_kv, k_r, seq_idx, pos, block_table, stream=None):
        T = c_kv.shape[0]
        B, max_blocks = block_table.shape
        N.mla_cache_append(self.dims, T, c_kv, k_r, seq_idx, pos, block_table, B, max_blocks,
                           cache.num_blocks, cache.kv_pool, cache.kr_pool, cache.kv_scale, stream)

    def absorb(self, q_c, q_r, pos, out=None, stream=None):
        T = q_c.shape[0]
        d = self.dims
        if out is None:
            out = torch.empty((T, d.n_h, d.d_c + d.d_r), dtype=TORCH_ACT[d.act_dtype], device=self.device)
        N.mla_absorb_q(d, T, q_c, q_r, pos, self.w_uk, out, stream)
        return out

    def append_absorb(self, cache: PagedLatentCache, c_kv, k_r, seq_idx, pos_new, block_table, q_c, q_r, pos,
                      out=None, stream=None):
        """append then absorb in one library call; returns q_abs."""
        T_new = c_kv.shape[0]
        B, max_blocks = block_table.shape
        T = q_c.shape[0]
        d = self.dims
        if out is None:
            out = torch.empty((T, d.n_h, d.d_c + d.d_r), dtype=TORCH_ACT[d.act_dtype], device=self.device)
        N.mla_append_absorb(d, T_new, c_kv, k_r, seq_idx, pos_new, block_table, B, max_blocks, cache.num_blocks,
                            cache.kv_pool, cache.kr_pool, cache.kv_scale, T, q_c, q_r, pos, self.w_uk, out, stream)
        return out

    def workspace(self, B, s_q, max_seq_len):
        key = (B, s_q, max_seq_len)
        if self._ws_key != key:
            n = N.mla_decode_workspace_size(self.dims, B, s_q, max_seq_len)
            if self._ws is None or self._ws.numel() < n:
                self._ws = torch.empty(max(n, 256), dtype=torch.uint8, device=self.device)
            self._ws_key = key
        return self._ws

    def decode(self, cache: PagedLatentCache, q_abs, block_table, seq_lens, s_q, max_seq_len,
               o_lat=None, lse=None, stream=None):
        d = self.dims
        B, max_blocks = block_table.shape
        rows = B * s_q
        if o_lat is None:
            o_lat = torch.empty((rows, d.n_h, d.d_c), dtype=torch.float32, device=self.device)
        if lse is None:
            lse = torch.empty((rows, d.n_h), dtype=torch.float32, device=self.device)
        ws = self.workspace(B, s_q, max_seq_len)
        N.mla_decode(d, B, s_q, q_abs, cache.kv_pool, cache.kr_pool, cache.kv_scale, block_table,
                     max_blocks, cache.num_blocks, seq_lens, max_seq_len, ws, ws.numel(), o_lat,
                     lse, stream)
        return o_lat, lse

    def decode_project(self, cache: PagedLatentCache, q_abs, block_table, seq_lens, s_q, max_seq_len,
                       out_dtype="f32", o=None, o_lat=None, lse=None, stream=None):
        """decode followed by out_proj in one library call; returns (o, o_lat, lse)."""
        d = self.dims
        B, max_blocks = block_table.shape
        rows = B * s_q
        dt = DTYPE[out_dtype]
        if o is None:
            o = torch.empty((rows, d.n_h, d.d_h), dtype=TORCH_ACT[dt], device=self.device)
        if o_lat is None:
            o_lat = torch.empty((rows, d.n_h, d.d_c), dtype=torch.float32, device=self.device)
        if lse is None:
            lse = torch.empty((rows, d.n_h), dtype=torch.float32, device=self.device)
        ws = self.workspace(B, s_q, max_seq_len)
        N.mla_decode_project(d, B, s_q, q_abs, cache.kv_pool, cache.kr_pool, cache.kv_scale, block_table,
                             max_blocks, cache.num_blocks, seq_lens, max_seq_len, ws, ws.numel(), self.w_uv,
                             o, dt, o_lat, lse, stream)
        return o, o_lat, lse

    def prefill(self, q_c, q_r, c_kv, k_r, cu_seqlens, max_seq_len, o=None, lse=None, stream=None):
        """Causal MHA-mode attention over packed prompts (cu_seqlens [B + 1] int32 on the
        device); returns (o [T, n_h, d_h] bf16, lse [T, n_h])."""
        d = self.dims
        T = q_c.shape[0]
        B = cu_seqlens.numel() - 1
        if o is None:
            o = torch.empty((T, d.n_h, d.d_h), dtype=torch.bfloat16, device=self.device)
        if lse is None:
            lse = torch.empty((T, d.n_h), dtype=torch.float32, device=self.device)
        n = N.mla_prefill_workspace_size(d, T)
        if self._pf_ws is None or self._pf_ws.numel() < n:
            self._pf_ws = torch.empty(max(n, 256), dtype=torch.uint8, device=self.device)
        N.mla_prefill(d, B, cu_seqlens, T, max_seq_len, q_c, q_r, c_kv, k_r, self.w_uk, self.w_uv, self._pf_ws,
                      self._pf_ws.numel(), o, lse, stream)
        return o, lse

    # -- drafted trees (see tree.DraftTrees) ---------------------------------------------------
    def tree_append(self, cache: PagedLatentCache, c_kv, k_r, trees, block_table, stream=None):
        """The drafted nodes' rows into their slots (trees.prepare first)."""
        B, max_blocks = block_table.shape
        T, here = trees.total_nodes, c_kv.get_device()
        d = self.dims
        act = TORCH_ACT[d.act_dtype]
        if (c_kv.size(0) != T or k_r.size(0) != T or c_kv.numel() != T * d.d_c or k_r.numel() != T * d.d_r or
                c_kv.dtype is not act or k_r.dtype is not act or B != trees.B):
            raise ValueError("tree_append: c_kv [nodes, d_c] and k_r [nodes, d_r] of the layer's type, block_table a row per tree")
        if not fits(d, cache.dims):
            raise ValueError("tree_append: the cache's rows are not the layer's")
        if (here < 0 or here != _on_device() or k_r.get_device() != here or block_table.get_device() != here or
                trees._slot.get_device() != here or cache.kv_pool.get_device() != here or block_table.dtype is not _INT32 or
                not (c_kv.is_contiguous() and k_r.is_contiguous() and block_table.is_contiguous())):
            raise ValueError(_MISREAD)
        if stream is not None:
            used_on(stream, c_kv, k_r, block_table, trees._seq_idx, trees._slot, trees._pos, cache.kv_pool, cache.kr_pool,
                    cache.kv_scale)
        N.mla_tree_append(d, T, c_kv, k_r, trees._seq_idx, trees._slot, trees._pos, block_table, B, max_blocks,
                          cache.num_blocks, cache.kv_pool, cache.kr_pool, cache.kv_scale,
                          _current_handle(here) if stream is None else stream)

    def decode_tree(self, cache: PagedLatentCache, q_abs, block_table, seq_lens, trees, max_seq_len,
                    out_dtype="f32", o_lat=None, lse=None, stream=None, workspace=None):
        """Every drafted node over the committed tokens and the nodes its mask names; returns
        (o_lat [nodes, n_h, d_c], lse [nodes, n_h]).  Without ``workspace`` (a tensor's bytes) the stream's is used, which
        the layers of a device share, or one of the graph that is being captured; calls that may run at the same
        time take no ``workspace`` in common."""
        d = self.dims
        B, max_blocks = block_table.shape
        T = trees.total_nodes
        dt = DTYPE[out_dtype]
        if (q_abs.size(0) != T or q_abs.numel() != T * d.n_h * (d.d_c + d.d_r) or q_abs.dtype is not TORCH_ACT[d.act_dtype] or
                B != trees.B or seq_lens.numel() != B):
            raise ValueError("decode_tree: q_abs is [nodes, n_h, d_c + d_r] of the layer's type, block_table and seq_lens have a row per tree")
        if not fits(d, cache.dims):
            raise ValueError("decode_tree: the cache's rows are not the layer's")
        here = q_abs.get_device()
        if (here < 0 or here != _on_device() or block_table.get_device() != here or seq_lens.get_device() != here or
                trees._cu_nodes.get_device() != here or cache.kv_pool.get_device() != here or
                block_table.dtype is not _INT32 or seq_lens.dtype is not _INT32 or
                not (q_abs.is_contiguous() and block_table.is_contiguous() and seq_lens.is_contiguous())):
            raise ValueError(_MISREAD)
        if o_lat is None:
            shape = (T, d.n_h, d.d_c)
            if stream is None:
                o_lat = q_abs.new_empty(shape, dtype=TORCH_ACT[dt])
            else:
                o_lat, = new_on(stream, lambda: (q_abs.new_empty(shape, dtype=TORCH_ACT[dt]),))
        elif (o_lat.dtype != TORCH_ACT[dt] or o_lat.shape != (T, d.n_h, d.d_c) or not o_lat.is_contiguous() or
              o_lat.get_device() != here):
            raise ValueError("decode_tree: o_lat is contiguous [nodes, n_h, d_c] of out_dtype, where q_abs is")
        if lse is None:
            if stream is None:
                lse = q_abs.new_empty((T, d.n_h), dtype=torch.float32)
            else:
                lse, = new_on(stream, lambda: (q_abs.new_empty((T, d.n_h), dtype=torch.float32),))
        elif lse.dtype != torch.float32 or lse.shape != (T, d.n_h) or not lse.is_contiguous() or lse.get_device() != here:
            raise ValueError("decode_tree: lse is contiguous [nodes, n_h] fp32, where q_abs is")
        if workspace is not None and (not workspace.is_contiguous() or workspace.get_device() != here):
            raise ValueError("decode_tree: workspace is contiguous, where q_abs is")
        if stream is None:
            handle = _current_handle(here)
        else:
            handle = N._stream(stream)
            used_on(stream, q_abs, block_table, seq_lens, trees._cu_nodes, trees._mask, cache.kv_pool, cache.kr_pool, cache.kv_scale,
                    o_lat, lse, workspace)
        shared = self._tree_ws
        with shared.lock:
            if workspace is None:
                workspace = shared.get((self._tree_key, B, T, max_seq_len), handle, stream,
                                       N.mla_decode_tree_workspace_size, d, B, T, max_seq_len)
            N.mla_decode_tree(d, B, trees._cu_nodes, T, trees.max_nodes, q_abs, cache.kv_pool, cache.kr_pool,
                              cache.kv_scale, block_table, max_blocks, cache.num_blocks, seq_lens, max_seq_len,
                              trees._mask, trees.mask_words, workspace, workspace.nbytes, o_lat, dt, lse, handle)
        return o_lat, lse

    def out_proj(self, o_lat, out_dtype="f32", out=None, stream=None):
        d = self.dims
        T = o_lat.shape[0]
        dt = DTYPE[out_dtype]
        if out is None:
            out = torch.empty((T, d.n_h, d.d_h), dtype=TORCH_ACT[dt], device=self.device)
        N.mla_out_proj(d, T, o_lat, self.w_uv, out, dt, stream)
        return out
