"""ctypes binding of libmla (include/mla.h): same names, argument marshalling only.

Every function takes torch CUDA tensors (or raw device addresses as ints) and the
stream to enqueue on (default: torch's current stream), passes their device
pointers to the C ABI and raises :class:`MLAError` on a non-OK status.  All
computation happens in libmla's CUDA kernels; there is no fallback: if the
library is not built, importing this module fails.
"""
from __future__ import annotations

import ctypes
import os
import re

_PKG = os.path.dirname(os.path.abspath(__file__))
# MLA_LIBRARY may point at another build of the same library (e.g. an instrumented one).
LIB_PATH = os.environ.get("MLA_LIBRARY") or os.path.join(_PKG, "libmla.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "mla.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run `python -m mla_latent_kv_mqa_b200.build`")

_lib = ctypes.CDLL(LIB_PATH)

# mla_status_t
MLA_OK = 0
MLA_ERR_INVALID_ARG = 1
MLA_ERR_UNSUPPORTED = 2
MLA_ERR_WORKSPACE_TOO_SMALL = 3
MLA_ERR_BAD_BLOCK_TABLE = 4
MLA_ERR_BAD_SEQ_LEN = 5
MLA_ERR_DEVICE_TIMEOUT = 6
MLA_ERR_CUDA = 7
MLA_ERR_BAD_TREE = 8
MLA_ERR_OUT_OF_PAGES = 9
MLA_ERR_BAD_SEQ_INDEX = 10
MLA_MAX_TREE_NODES = 1024
# mla_dtype_t
MLA_DTYPE_F32 = 0
MLA_DTYPE_BF16 = 1
MLA_DTYPE_FP8_E4M3 = 2
MLA_FLAG_SIMT_DECODE = 1
MLA_FLAG_SIMT_PROJ = 2
MLA_FLAG_TEST_GIVE_UP = 4
MLA_FLAG_FP8_MMA = 8


class MLAError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call} -> {status_string(status)}")


class mla_dims_t(ctypes.Structure):
    _fields_ = [("n_h", ctypes.c_int), ("d_h", ctypes.c_int), ("d_c", ctypes.c_int),
                ("d_r", ctypes.c_int), ("page_size", ctypes.c_int), ("rope_base", ctypes.c_float),
                ("act_dtype", ctypes.c_int), ("kv_dtype", ctypes.c_int), ("flags", ctypes.c_uint)]


def make_dims(n_h, d_h, d_c, d_r, page_size=64, rope_base=1e4, act_dtype=MLA_DTYPE_BF16,
              kv_dtype=MLA_DTYPE_BF16, flags=0) -> mla_dims_t:
    return mla_dims_t(n_h, d_h, d_c, d_r, page_size, rope_base, act_dtype, kv_dtype, flags)


class mla_pool_t(ctypes.Structure):
    _fields_ = [("kv_pool", ctypes.c_void_p), ("kr_pool", ctypes.c_void_p), ("kv_scale", ctypes.c_void_p)]


class mla_page_table_t(ctypes.Structure):
    _fields_ = [("page_size", ctypes.c_int), ("num_seqs", ctypes.c_int), ("max_blocks", ctypes.c_int),
                ("num_blocks", ctypes.c_int), ("block_table", ctypes.c_void_p), ("refs", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p)]


_vp, _i, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_dp = ctypes.POINTER(mla_dims_t)
_lib.mla_absorb_q.argtypes = [_dp, _i, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.mla_cache_append.argtypes = [_dp, _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp]
_lib.mla_decode_workspace_size.argtypes = [_dp, _i, _i, _i]
_lib.mla_decode_workspace_size.restype = _sz
_lib.mla_decode.argtypes = [_dp, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _vp, _i, _vp, _sz, _vp,
                            _vp, _vp]
_lib.mla_decode_fixed_scratch.argtypes = [_dp, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _vp, _i,
                                          _vp, _vp, _vp]
_lib.mla_out_proj.argtypes = [_dp, _i, _vp, _vp, _vp, _i, _vp]
_lib.mla_append_absorb.argtypes = [_dp, _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _i, _vp, _vp, _vp,
                                   _vp, _vp, _vp]
_lib.mla_decode_project.argtypes = [_dp, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _vp, _i, _vp, _sz,
                                    _vp, _vp, _i, _vp, _vp, _vp]
_lib.mla_prefill_workspace_size.argtypes = [_dp, _i]
_lib.mla_prefill_workspace_size.restype = _sz
_lib.mla_prefill.argtypes = [_dp, _i, _vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp, _vp]
_lib.mla_lse_merge_prepare.argtypes = [_i, _i, _i, _vp, _vp, _vp, _vp, _vp]
_lib.mla_lse_merge_finish.argtypes = [_i, _i, _i, _vp, _vp, _vp, _vp, _vp]
_pp, _tp = ctypes.POINTER(mla_pool_t), ctypes.POINTER(mla_page_table_t)
_lib.mla_tree_prepare.argtypes = [_i, _vp, _i, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp]
_lib.mla_tree_append.argtypes = [_dp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp]
_lib.mla_decode_tree_workspace_size.argtypes = [_dp, _i, _i, _i]
_lib.mla_decode_tree_workspace_size.restype = _sz
_lib.mla_decode_tree.argtypes = [_dp, _i, _vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _vp, _i, _vp, _i, _vp, _sz,
                                 _vp, _i, _vp, _vp]
_lib.mla_cache_keep.argtypes = [_dp, _i, _pp, _i, _vp, _i, _vp, _i, _i, _vp, _vp, _vp, _i, _vp, _vp]
_lib.mla_pages_workspace_size.argtypes = [_tp, _i]
_lib.mla_pages_workspace_size.restype = _sz
_lib.mla_pages_fork.argtypes = [_tp, _i, _vp, _vp, _vp, _sz, _vp]
_lib.mla_pages_grow.argtypes = [_tp, _i, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.mla_pages_trim.argtypes = [_tp, _i, _vp, _vp, _vp]
_lib.mla_pages_compact.argtypes = [_tp, _vp, _vp, _vp, _sz, _vp]
_lib.mla_cache_copy_pages.argtypes = [_dp, _i, _pp, _i, _vp, _vp, _i, _vp]
_lib.mla_get_last_device_error.argtypes = []
_lib.mla_status_string.argtypes = [_i]
_lib.mla_status_string.restype = ctypes.c_char_p
_lib.mla_version.restype = _i
for _f in ("mla_absorb_q", "mla_cache_append", "mla_decode", "mla_decode_fixed_scratch", "mla_out_proj",
           "mla_decode_project", "mla_prefill", "mla_append_absorb", "mla_get_last_device_error",
           "mla_lse_merge_prepare",
           "mla_lse_merge_finish", "mla_tree_prepare", "mla_tree_append", "mla_decode_tree", "mla_cache_keep",
           "mla_pages_fork", "mla_pages_grow", "mla_pages_trim", "mla_pages_compact", "mla_cache_copy_pages"):
    getattr(_lib, _f).restype = _i


def declared_functions() -> list[str]:
    """Names of the functions include/mla.h declares."""
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(mla_[a-z_0-9]+)\s*\(", src)))


def library() -> ctypes.CDLL:
    return _lib


def _ptr(x):
    if x is None or type(x) is int:
        return x
    return x.data_ptr()


_torch = None


def _stream(stream):
    if stream is None:  # torch's current stream, its handle without a Stream object (a call's largest host cost)
        global _torch
        if _torch is None:
            import torch
            torch.cuda.current_stream()  # CUDA is up
            _torch = torch
        return _torch._C._cuda_getCurrentRawStream(_torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, call: str):
    if rc != MLA_OK:
        raise MLAError(rc, call)


def status_string(status: int) -> str:
    return _lib.mla_status_string(status).decode()


def version() -> int:
    return _lib.mla_version()


def mla_absorb_q(dims, T, q_c, q_r, pos, w_uk, q_abs, stream=None):
    _check(_lib.mla_absorb_q(ctypes.byref(dims), T, _ptr(q_c), _ptr(q_r), _ptr(pos), _ptr(w_uk),
                             _ptr(q_abs), _stream(stream)), "mla_absorb_q")


def mla_cache_append(dims, T, c_kv, k_r, seq_idx, pos, block_table, num_seqs, max_blocks_per_seq,
                     num_blocks, kv_pool, kr_pool=None, kv_scale=None, stream=None):
    _check(_lib.mla_cache_append(ctypes.byref(dims), T, _ptr(c_kv), _ptr(k_r), _ptr(seq_idx),
                                 _ptr(pos), _ptr(block_table), num_seqs, max_blocks_per_seq,
                                 num_blocks, _ptr(kv_pool), _ptr(kr_pool), _ptr(kv_scale),
                                 _stream(stream)), "mla_cache_append")


def mla_append_absorb(dims, T_new, c_kv, k_r, seq_idx, pos_new, block_table, num_seqs, max_blocks_per_seq,
                      num_blocks, kv_pool, kr_pool, kv_scale, T, q_c, q_r, pos, w_uk, q_abs, stream=None):
    """mla_cache_append then mla_absorb_q (one launch where the tensor-core absorption applies)."""
    _check(_lib.mla_append_absorb(ctypes.byref(dims), T_new, _ptr(c_kv), _ptr(k_r), _ptr(seq_idx), _ptr(pos_new),
                                  _ptr(block_table), num_seqs, max_blocks_per_seq, num_blocks, _ptr(kv_pool),
                                  _ptr(kr_pool), _ptr(kv_scale), T, _ptr(q_c), _ptr(q_r), _ptr(pos), _ptr(w_uk),
                                  _ptr(q_abs), _stream(stream)), "mla_append_absorb")


def mla_decode_workspace_size(dims, B, s_q, max_seq_len) -> int:
    return int(_lib.mla_decode_workspace_size(ctypes.byref(dims), B, s_q, max_seq_len))


def mla_decode(dims, B, s_q, q_abs, kv_pool, kr_pool, kv_scale, block_table, max_blocks_per_seq,
               num_blocks, seq_lens, max_seq_len, workspace, workspace_bytes, o_lat, lse=None,
               stream=None):
    _check(_lib.mla_decode(ctypes.byref(dims), B, s_q, _ptr(q_abs), _ptr(kv_pool), _ptr(kr_pool),
                           _ptr(kv_scale), _ptr(block_table), max_blocks_per_seq, num_blocks,
                           _ptr(seq_lens), max_seq_len, _ptr(workspace), workspace_bytes,
                           _ptr(o_lat), _ptr(lse), _stream(stream)), "mla_decode")


def mla_decode_fixed_scratch(dims, B, s_q, q_abs, kv_pool, kr_pool, kv_scale, block_table,
                             max_blocks_per_seq, num_blocks, seq_lens, max_seq_len, o_lat, lse=None,
                             stream=None):
    """mla_decode on the library's static scratch array (no workspace argument)."""
    _check(_lib.mla_decode_fixed_scratch(ctypes.byref(dims), B, s_q, _ptr(q_abs), _ptr(kv_pool),
                                         _ptr(kr_pool), _ptr(kv_scale), _ptr(block_table),
                                         max_blocks_per_seq, num_blocks, _ptr(seq_lens), max_seq_len,
                                         _ptr(o_lat), _ptr(lse), _stream(stream)),
           "mla_decode_fixed_scratch")


def mla_out_proj(dims, T, o_lat, w_uv, o, out_dtype=MLA_DTYPE_F32, stream=None):
    _check(_lib.mla_out_proj(ctypes.byref(dims), T, _ptr(o_lat), _ptr(w_uv), _ptr(o), out_dtype,
                             _stream(stream)), "mla_out_proj")


def mla_decode_project(dims, B, s_q, q_abs, kv_pool, kr_pool, kv_scale, block_table, max_blocks_per_seq,
                       num_blocks, seq_lens, max_seq_len, workspace, workspace_bytes, w_uv, o, out_dtype,
                       o_lat, lse=None, stream=None):
    """mla_decode followed by mla_out_proj (one fused merge + projection kernel where it applies)."""
    _check(_lib.mla_decode_project(ctypes.byref(dims), B, s_q, _ptr(q_abs), _ptr(kv_pool), _ptr(kr_pool),
                                   _ptr(kv_scale), _ptr(block_table), max_blocks_per_seq, num_blocks,
                                   _ptr(seq_lens), max_seq_len, _ptr(workspace), workspace_bytes, _ptr(w_uv),
                                   _ptr(o), out_dtype, _ptr(o_lat), _ptr(lse), _stream(stream)),
           "mla_decode_project")


def mla_prefill_workspace_size(dims, total_tokens) -> int:
    return int(_lib.mla_prefill_workspace_size(ctypes.byref(dims), total_tokens))


def mla_prefill(dims, B, cu_seqlens, total_tokens, max_seq_len, q_c, q_r, c_kv, k_r, w_uk, w_uv, workspace,
                workspace_bytes, o, lse=None, stream=None):
    _check(_lib.mla_prefill(ctypes.byref(dims), B, _ptr(cu_seqlens), total_tokens, max_seq_len, _ptr(q_c), _ptr(q_r),
                            _ptr(c_kv), _ptr(k_r), _ptr(w_uk), _ptr(w_uv), _ptr(workspace), workspace_bytes, _ptr(o),
                            _ptr(lse), _stream(stream)), "mla_prefill")


def mla_lse_merge_prepare(rows, n_h, d_c, o_lat, lse, lse_max, acc, stream=None):
    _check(_lib.mla_lse_merge_prepare(rows, n_h, d_c, _ptr(o_lat), _ptr(lse), _ptr(lse_max), _ptr(acc),
                                      _stream(stream)), "mla_lse_merge_prepare")


def mla_lse_merge_finish(rows, n_h, d_c, acc, lse_max, o_lat, lse=None, stream=None):
    _check(_lib.mla_lse_merge_finish(rows, n_h, d_c, _ptr(acc), _ptr(lse_max), _ptr(o_lat), _ptr(lse),
                                     _stream(stream)), "mla_lse_merge_finish")


def mla_tree_prepare(B, cu_nodes, total_nodes, parent, seq_lens, mask_words, mask, pos, slot, seq_idx, stream=None):
    _check(_lib.mla_tree_prepare(B, _ptr(cu_nodes), total_nodes, _ptr(parent), _ptr(seq_lens), mask_words, _ptr(mask),
                                 _ptr(pos), _ptr(slot), _ptr(seq_idx), _stream(stream)), "mla_tree_prepare")


def mla_tree_append(dims, T, c_kv, k_r, seq_idx, slot, pos, block_table, num_seqs, max_blocks_per_seq, num_blocks,
                    kv_pool, kr_pool=None, kv_scale=None, stream=None):
    _check(_lib.mla_tree_append(ctypes.byref(dims), T, _ptr(c_kv), _ptr(k_r), _ptr(seq_idx), _ptr(slot), _ptr(pos),
                                _ptr(block_table), num_seqs, max_blocks_per_seq, num_blocks, _ptr(kv_pool),
                                _ptr(kr_pool), _ptr(kv_scale), _stream(stream)), "mla_tree_append")


def mla_decode_tree_workspace_size(dims, B, total_nodes, max_seq_len) -> int:
    return int(_lib.mla_decode_tree_workspace_size(ctypes.byref(dims), B, total_nodes, max_seq_len))


def mla_decode_tree(dims, B, cu_nodes, total_nodes, max_nodes, q_abs, kv_pool, kr_pool, kv_scale, block_table,
                    max_blocks_per_seq, num_blocks, seq_lens, max_seq_len, mask, mask_words, workspace,
                    workspace_bytes, o_lat, out_dtype=MLA_DTYPE_F32, lse=None, stream=None):
    _check(_lib.mla_decode_tree(ctypes.byref(dims), B, _ptr(cu_nodes), total_nodes, max_nodes, _ptr(q_abs),
                                _ptr(kv_pool), _ptr(kr_pool), _ptr(kv_scale), _ptr(block_table), max_blocks_per_seq,
                                num_blocks, _ptr(seq_lens), max_seq_len, _ptr(mask), mask_words, _ptr(workspace),
                                workspace_bytes, _ptr(o_lat), out_dtype, _ptr(lse), _stream(stream)),
           "mla_decode_tree")


def make_pool(kv_pool, kr_pool=None, kv_scale=None) -> mla_pool_t:
    return mla_pool_t(_ptr(kv_pool), _ptr(kr_pool), _ptr(kv_scale))


def make_pools(pools):
    """Array of mla_pool_t from mla_pool_t's or (kv_pool, kr_pool, kv_scale) triples (tensors, addresses or None)."""
    return (mla_pool_t * len(pools))(*[p if isinstance(p, mla_pool_t) else make_pool(*p) for p in pools])


def mla_cache_keep(dims, pools, B, cu_nodes, total_nodes, block_table, max_blocks_per_seq, num_blocks, seq_lens, keep,
                   num_keep, max_keep, new_lens=None, stream=None):
    """``pools``: make_pools(...)."""
    _check(_lib.mla_cache_keep(ctypes.byref(dims), len(pools), pools, B, _ptr(cu_nodes), total_nodes,
                               _ptr(block_table), max_blocks_per_seq, num_blocks, _ptr(seq_lens), _ptr(keep),
                               _ptr(num_keep), max_keep, _ptr(new_lens), _stream(stream)), "mla_cache_keep")


def make_page_table(page_size, num_seqs, max_blocks, num_blocks, block_table, refs, seq_lens) -> mla_page_table_t:
    return mla_page_table_t(page_size, num_seqs, max_blocks, num_blocks, _ptr(block_table), _ptr(refs), _ptr(seq_lens))


def mla_pages_workspace_size(table, n) -> int:
    return int(_lib.mla_pages_workspace_size(ctypes.byref(table), n))


def mla_pages_fork(table, n, parent, child, workspace, workspace_bytes, stream=None):
    _check(_lib.mla_pages_fork(ctypes.byref(table), n, _ptr(parent), _ptr(child), _ptr(workspace), workspace_bytes,
                               _stream(stream)), "mla_pages_fork")


def mla_pages_grow(table, n, seqs, new_lens, moves, num_moves, workspace, workspace_bytes, stream=None):
    _check(_lib.mla_pages_grow(ctypes.byref(table), n, _ptr(seqs), _ptr(new_lens), _ptr(moves), _ptr(num_moves),
                               _ptr(workspace), workspace_bytes, _stream(stream)), "mla_pages_grow")


def mla_pages_trim(table, n, seqs, new_lens, stream=None):
    _check(_lib.mla_pages_trim(ctypes.byref(table), n, _ptr(seqs), _ptr(new_lens), _stream(stream)), "mla_pages_trim")


def mla_pages_compact(table, moves, num_moves, workspace, workspace_bytes, stream=None):
    _check(_lib.mla_pages_compact(ctypes.byref(table), _ptr(moves), _ptr(num_moves), _ptr(workspace), workspace_bytes,
                                  _stream(stream)), "mla_pages_compact")


def mla_cache_copy_pages(dims, pools, num_blocks, moves, num_moves, max_moves, stream=None):
    """``pools``: make_pools(...); ``num_moves``: device int32 [1], or None for all max_moves."""
    _check(_lib.mla_cache_copy_pages(ctypes.byref(dims), len(pools), pools, num_blocks, _ptr(moves), _ptr(num_moves),
                                     max_moves, _stream(stream)), "mla_cache_copy_pages")


def mla_get_last_device_error() -> int:
    return int(_lib.mla_get_last_device_error())
