"""Drafted trees and pages without a GPU: what the library refuses on the host, its workspace sizes, and
the plain forms that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

from mla_latent_kv_mqa_b200 import build as B
from tests import tree_ref as R


@pytest.fixture(scope="module")
def N():
    B.build()
    from mla_latent_kv_mqa_b200 import native
    return native


def _v3(N, **kw):
    return N.make_dims(128, 128, 512, 64, **kw)


def test_tree_calls_refuse_bad_arguments(N):
    L, bad = N.library(), N.MLA_ERR_INVALID_ARG
    dp = ctypes.byref(_v3(N))

    def prep(B=2, cu=16, T=4, parent=16, lens=16, words=1, mask=16):
        return L.mla_tree_prepare(B, cu, T, parent, lens, words, mask, 16, 16, 16, None)
    assert prep(B=-1) == bad and prep(T=-1) == bad and prep(words=0) == bad and prep(words=33) == bad
    assert prep(cu=None) == bad and prep(parent=None) == bad and prep(lens=None) == bad and prep(mask=None) == bad
    assert prep(T=0, cu=None, parent=None) == N.MLA_OK

    def app(d=dp, T=4, slot=16, kr=None, blocks=4):
        return L.mla_tree_append(d, T, 16, 16, 16, slot, 16, 16, 2, blocks, 8, 16, kr, None, None)
    assert app(slot=None) == bad and app(T=-1) == bad and app(kr=16) == bad and app(blocks=1 << 26) == bad
    assert app(T=0, slot=None) == N.MLA_OK

    def dec(B=2, T=6, most=4, q=16, blocks=4, max_len=256, mask=16, words=1, ws=256, nbytes=1 << 50, o=16, out=0,
            kr=None, cu=16, flags=N.MLA_FLAG_SIMT_DECODE):
        d = _v3(N, flags=flags)
        return L.mla_decode_tree(ctypes.byref(d), B, cu, T, most, q, 16, kr, None, 16, blocks, 8, 16, max_len, mask,
                                 words, ws, nbytes, o, out, None, None)
    assert dec(B=-1) == bad and dec(T=-1) == bad and dec(most=0) == bad and dec(most=1025, words=64) == bad
    assert dec(most=33) == bad and dec(words=0) == bad                      # a word for every 32 nodes
    assert dec(max_len=257) == bad and dec(max_len=0) == bad and dec(blocks=1 << 26) == bad
    assert dec(T=1 << 25) == bad                                            # node rows times heads in int
    for k in ("q", "mask", "ws", "o", "cu"):
        assert dec(**{k: None}) == bad, k
    assert dec(ws=16) == bad and dec(kr=16) == bad
    assert dec(out=N.MLA_DTYPE_FP8_E4M3) == N.MLA_ERR_UNSUPPORTED
    assert dec(nbytes=255) == N.MLA_ERR_WORKSPACE_TOO_SMALL
    assert dec(B=0, q=None) == N.MLA_OK and dec(T=0, q=None) == N.MLA_OK
    s = _v3(N, flags=N.MLA_FLAG_SIMT_DECODE)
    few = N.make_dims(2, 64, 128, 32)                                       # one block a segment: more than a cluster joins
    assert N.mla_decode_tree_workspace_size(few, 1, 1, 1 << 18) > 1 << 14
    assert 0 < N.mla_decode_tree_workspace_size(s, 2, 6, 256)
    assert N.mla_decode_tree_workspace_size(s, 2, -1, 256) == 0 and N.mla_decode_tree_workspace_size(s, 2, 6, 0) == 0
    assert N.mla_decode_tree_workspace_size(s, 2, 6, 2 ** 31 - 1) == 0 and dec(blocks=(1 << 25) - 1, max_len=2 ** 31 - 64) == bad

    pools = N.make_pools([(16, None, None)] * 2)

    def keep(n=2, p=pools, B=2, most=4, lens=16, keep=16, new=32, blocks=4):
        return L.mla_cache_keep(dp, n, p, B, 16, 6, 16, blocks, 8, lens, keep, 16, most, new, None)
    assert keep(n=-1) == bad and keep(p=None) == bad and keep(most=0) == bad and keep(most=1025) == bad
    assert keep(keep=None) == bad and keep(new=16) == bad and keep(blocks=1 << 26) == bad
    assert keep(p=N.make_pools([(16, 16, None)] * 2)) == bad and keep(p=N.make_pools([(None, None, None)] * 2)) == bad
    assert keep(B=0) == N.MLA_OK and keep(n=0, p=None) == N.MLA_OK


def test_page_calls_refuse_bad_arguments(N):
    L, bad = N.library(), N.MLA_ERR_INVALID_ARG

    def table(page=64, seqs=4, width=8, blocks=20, bt=16, refs=16, lens=16):
        return N.make_page_table(page, seqs, width, blocks, bt, refs, lens)
    for kw in (dict(page=0), dict(seqs=0), dict(width=0), dict(blocks=0), dict(bt=None), dict(refs=None), dict(lens=None),
               dict(width=1 << 26), dict(seqs=1 << 30)):
        t = ctypes.byref(table(**kw))
        assert N.mla_pages_workspace_size(table(**kw), 2) == 0
        assert L.mla_pages_fork(t, 2, 16, 16, 256, 1 << 40, None) == bad
        assert L.mla_pages_grow(t, 2, None, 16, 16, 16, 256, 1 << 40, None) == bad
        assert L.mla_pages_trim(t, 2, None, 16, None) == bad
        assert L.mla_pages_compact(t, 16, 16, 256, 1 << 40, None) == bad
    t = ctypes.byref(table())
    assert L.mla_pages_fork(t, -1, 16, 16, 256, 1 << 40, None) == bad
    assert L.mla_pages_fork(t, 2, None, 16, 256, 1 << 40, None) == bad
    assert L.mla_pages_fork(t, 2, 16, 16, 16, 1 << 40, None) == bad
    assert L.mla_pages_fork(t, 2, 16, 16, 256, 16, None) == N.MLA_ERR_WORKSPACE_TOO_SMALL
    assert L.mla_pages_fork(t, 0, None, None, None, 0, None) == N.MLA_OK
    assert L.mla_pages_grow(t, 5, None, 16, 16, 16, 256, 1 << 40, None) == bad      # more lengths than sequences
    assert L.mla_pages_grow(t, 2, None, 16, 16, None, 256, 1 << 40, None) == bad
    assert L.mla_pages_grow(t, 2, None, 16, 16, 16, 256, 16, None) == N.MLA_ERR_WORKSPACE_TOO_SMALL
    assert L.mla_pages_trim(t, 5, None, 16, None) == bad and L.mla_pages_trim(t, 2, None, None, None) == bad
    assert L.mla_pages_trim(t, 0, None, None, None) == N.MLA_OK
    assert L.mla_pages_compact(t, None, 16, 256, 1 << 40, None) == bad
    assert L.mla_pages_compact(t, 16, 16, 256, 16, None) == N.MLA_ERR_WORKSPACE_TOO_SMALL
    assert N.mla_pages_workspace_size(table(), 2) <= N.mla_pages_workspace_size(table(), 200)
    dp, pools = ctypes.byref(_v3(N)), N.make_pools([(16, None, None)])
    assert L.mla_cache_copy_pages(dp, 1, pools, 0, 16, None, 1, None) == bad
    assert L.mla_cache_copy_pages(dp, 1, pools, 8, None, None, 1, None) == bad
    assert L.mla_cache_copy_pages(dp, 1, pools, 8, 16, None, -1, None) == bad
    assert L.mla_cache_copy_pages(dp, 1, None, 8, 16, None, 1, None) == bad
    assert L.mla_cache_copy_pages(dp, 1, pools, 8, None, None, 0, None) == N.MLA_OK
    f8 = ctypes.byref(_v3(N, kv_dtype=N.MLA_DTYPE_FP8_E4M3))
    assert L.mla_cache_copy_pages(f8, 1, pools, 8, 16, None, 1, None) == bad


def test_status_names(N):
    assert N.status_string(N.MLA_ERR_BAD_TREE) == "MLA_ERR_BAD_TREE"
    assert N.status_string(N.MLA_ERR_OUT_OF_PAGES) == "MLA_ERR_OUT_OF_PAGES"
    assert N.status_string(N.MLA_ERR_BAD_SEQ_INDEX) == "MLA_ERR_BAD_SEQ_INDEX"


def test_plain_tree_masks():
    see, depth = R.sees(np.array([-1, 0, 0, 1, -1, 4, 3]))
    assert [list(np.nonzero(r)[0]) for r in see] == [[0], [0, 1], [0, 2], [0, 1, 3], [4], [4, 5], [0, 1, 3, 6]]
    assert list(depth) == [0, 1, 1, 2, 0, 1, 3]
    words = R.bits(see, 2)
    assert list(words[6]) == [1 + 2 + 8 + 64, 0]


def test_plain_pages_count_every_holder():
    rng = np.random.default_rng(0)
    p = R.Pages(4, np.full((5, 6), -1), np.zeros(20, dtype=np.int64), np.zeros(5, dtype=np.int64))
    assert p.grow([9, 3], [0, 1]) == []
    for _ in range(50):
        kind = rng.integers(4)
        if kind == 0:
            p.fork([int(rng.integers(5))], [int(rng.integers(5))])
        elif kind == 1:
            p.grow([int(min(24, p.lens[s] + rng.integers(0, 5))) for s in range(5)])
        elif kind == 2:
            p.trim([int(rng.integers(0, 24))], [int(rng.integers(5))])
        else:
            p.compact()
        held = np.bincount(p.table[p.table >= 0], minlength=20)
        assert np.array_equal(held, p.refs)


def test_the_python_calls_refuse_what_the_kernels_would_misread(N):
    """Shapes, types and places of tensors, checked before any address is handed on."""
    import torch
    from mla_latent_kv_mqa_b200 import layer as L, pages as P, tree as T
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    dims = L.dims_for(2, 8, 16, 4, act="f32", kv="f32", page=4)
    trees = T.DraftTrees(i32(0, 2), i32(-1, 0), 2)
    for cu, parent in ((torch.tensor([0, 2]), i32(-1, 0)), (i32(0, 2), torch.tensor([-1, 0])), (i32(0, 9, 2, 9)[::2], i32(-1, 0)),
                       (i32(), i32())):
        with pytest.raises(ValueError):
            T.DraftTrees(cu, parent, 2)
    for mask in (torch.zeros(2, 1), torch.zeros(3, 1, dtype=torch.int32), torch.zeros(2, 0, dtype=torch.int32)):
        with pytest.raises(ValueError):
            T.DraftTrees(i32(0, 2), i32(-1, 0), 2, mask=mask)
    cache = L.PagedLatentCache(dims, 3, device="cpu")
    other = L.PagedLatentCache(dims, 4, device="cpu")
    lay = L.MLADecodeLayer.__new__(L.MLADecodeLayer)
    lay.dims = dims
    table, lens = torch.zeros(1, 2, dtype=torch.int32), i32(5)
    q = torch.zeros(2, 2, 20)
    for bad in (dict(q_abs=torch.zeros(3, 2, 20)), dict(q_abs=torch.zeros(2, 20, 2).transpose(1, 2)), dict(seq_lens=i32(5, 5)),
                dict(block_table=torch.zeros(2, 2, dtype=torch.int32)), {}):     # the last: host tensors
        with pytest.raises(ValueError):
            lay.decode_tree(**{**dict(cache=cache, q_abs=q, block_table=table, seq_lens=lens, trees=trees, max_seq_len=8), **bad})
    with pytest.raises(ValueError):
        lay.tree_append(cache, torch.zeros(3, 16), torch.zeros(3, 4), trees, table)
    with pytest.raises(ValueError):
        trees.prepare(i32(5, 5))
    with pytest.raises(ValueError):
        trees.keep([cache], table, lens, torch.zeros(2, 1, dtype=torch.int32), i32(1))
    with pytest.raises(ValueError):
        L.same_caches([cache, other], 3)
    with pytest.raises(ValueError):
        L.same_caches([cache, L.PagedLatentCache(L.dims_for(2, 8, 16, 4, act="f32", kv="bf16", page=4), 3, device="cpu")], 3)
    seqs = P.PagedSequences(4, 2, 3, 3, device="cpu")
    for call in (lambda: seqs.fork(i32(0), i32(1)), lambda: seqs.fork(i32(0), i32(0, 1)), lambda: seqs.grow(torch.tensor([4])),
                 lambda: seqs.trim(i32(0, 0), i32(1)), lambda: seqs.compact(), lambda: seqs.copy_pages([other], None),
                 lambda: seqs.copy_pages([L.PagedLatentCache(L.dims_for(2, 8, 16, 4, act="f32", kv="f32", page=8), 3, device="cpu")], None)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(AttributeError):
        seqs.seq_lens = i32(0, 0)
