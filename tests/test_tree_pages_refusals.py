"""What the Python calls for drafted trees and pages refuse before any address reaches a kernel: types, widths, places
and caches that are not the layer's.  Host tensors do: these checks come before the one for the device."""
import pytest
import torch

from mla_latent_kv_mqa_b200 import build as B


@pytest.fixture(scope="module")
def M():
    B.build()
    from types import SimpleNamespace

    from mla_latent_kv_mqa_b200 import layer, pages, tree
    return SimpleNamespace(L=layer, P=pages, T=tree)


def test_rows_wider_than_a_block_s_memory_are_unsupported(M):
    """1452 columns are the most that eight queries and 32 rows fit the shared memory with."""
    import ctypes

    from mla_latent_kv_mqa_b200 import native as N
    for d_c, d_r, holds in ((1024, 428, True), (1024, 430, False), (1024, 1024, False), (600, 900, False), (16, 1436, True)):
        assert (4 * (8 * (d_c + d_r) + 32 * (d_c + d_r + 1)) <= 227 * 1024) == holds
        dims = N.make_dims(4, 8, d_c, d_r, 64)
        assert (N.mla_decode_tree_workspace_size(dims, 1, 4, 100) > 0) == holds
        if not holds:
            rc = N.library().mla_decode_tree(ctypes.byref(dims), 1, 16, 4, 4, 16, 16, None, None, 16, 4, 8, 16, 100, 16, 1, 256, 1 << 40,
                                             16, 0, None, None)
            assert rc == N.MLA_ERR_UNSUPPORTED


def i32(*x, device="cpu"):
    return torch.tensor(x, dtype=torch.int32, device=device)


def setup(M, act="f32", kv="f32"):
    dims = M.L.dims_for(2, 8, 16, 4, act=act, kv=kv, page=4)
    lay = M.L.MLADecodeLayer.__new__(M.L.MLADecodeLayer)
    lay.dims = dims
    return dims, lay, M.L.PagedLatentCache(dims, 3, device="cpu"), M.T.DraftTrees(i32(0, 2), i32(-1, 0), 2)


def test_decode_tree_queries_and_caches(M):
    dims, lay, cache, trees = setup(M)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), i32(5)
    other = {k: M.L.PagedLatentCache(M.L.dims_for(2, 8, c, r, act="f32", kv=kv, page=p), 3, device="cpu")
             for k, (c, r, kv, p) in dict(kind=(16, 4, "bf16", 4), width=(32, 4, "f32", 4), rope=(16, 8, "f32", 4), page=(16, 4, "f32", 8)).items()}

    def call(match, **kw):
        with pytest.raises(ValueError, match=match):
            lay.decode_tree(**{**dict(cache=cache, q_abs=torch.zeros(2, 2, 20), block_table=table, seq_lens=lens, trees=trees,
                                      max_seq_len=8), **kw})
    for q in (torch.zeros(2, 1, 20), torch.zeros(2, 2, 16), torch.zeros(4, 20), torch.zeros(2, 2, 20, dtype=torch.bfloat16),
              torch.zeros(2, 2, 20, dtype=torch.float64)):
        call("q_abs is", q_abs=q)
    for c in other.values():
        call("cache's rows", cache=c)
    call("contiguous and on the current")                                # host tensors
    call("contiguous and on the current", q_abs=torch.zeros(2, 40))


def test_tree_append_rows(M):
    dims, lay, cache, trees = setup(M)
    table = torch.zeros(1, 2, dtype=torch.int32)
    for c, k in ((torch.zeros(2, 8), torch.zeros(2, 4)), (torch.zeros(2, 16), torch.zeros(2, 2)), (torch.zeros(32), torch.zeros(2, 4)),
                 (torch.zeros(2, 16, dtype=torch.bfloat16), torch.zeros(2, 4)), (torch.zeros(2, 16), torch.zeros(2, 4, dtype=torch.bfloat16))):
        with pytest.raises(ValueError, match="c_kv"):
            lay.tree_append(cache, c, k, trees, table)
    wrong = M.L.PagedLatentCache(M.L.dims_for(2, 8, 16, 4, act="f32", kv="bf16", page=4), 3, device="cpu")
    with pytest.raises(ValueError, match="cache's rows"):
        lay.tree_append(wrong, torch.zeros(2, 16), torch.zeros(2, 4), trees, table)
    with pytest.raises(ValueError, match="contiguous and on"):             # a head axis of one is a row all the same
        lay.tree_append(cache, torch.zeros(2, 16), torch.zeros(2, 1, 4), trees, table)


def test_trees_are_on_one_device_and_stay_as_looked_over(M):
    cu, parent, mask = i32(0, 2), i32(-1, 0), torch.zeros(2, 1, dtype=torch.int32)
    for args in ((cu, parent.to("meta"), 2), (cu.to("meta"), parent, 2), (cu, parent, 2, mask.to("meta"))):
        with pytest.raises(ValueError, match="one device"):
            M.T.DraftTrees(*args)
    with pytest.raises(ValueError):
        M.T.DraftTrees(cu, parent, 2, mask.view(-1))
    trees = M.T.DraftTrees(cu, parent, 2, mask)
    assert trees.mask is mask
    for name in ("cu_nodes", "parent", "mask", "pos", "slot", "seq_idx"):
        old = getattr(trees, name)
        for bad in (torch.zeros(1, dtype=torch.int32), old.long(), old.to("meta"), old.repeat_interleave(2, 0)[::2]):
            with pytest.raises(ValueError, match=name):
                setattr(trees, name, bad)
        new = old.clone()
        setattr(trees, name, new)
        assert getattr(trees, name) is new


def test_keep_lists_and_caches(M):
    dims, lay, cache, trees = setup(M)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), i32(5)
    for keep in (i32(0), torch.zeros(1, 1, 1, dtype=torch.int32)):
        with pytest.raises(ValueError, match="max_keep"):
            trees.keep([cache], table, lens, keep, i32(1))
    with pytest.raises(ValueError, match="no caches"):
        trees.keep([], table, lens, torch.zeros(1, 1, dtype=torch.int32), i32(1))


def test_a_pool_is_where_its_tensors_are_now(M):
    """A buffer whose storage is swapped in place is taken at its new address by every call."""
    dims = M.L.dims_for(2, 8, 16, 4, kv="fp8", page=4)
    cache = M.L.PagedLatentCache(dims, 3, device="cpu")
    assert (cache.pool().kv_pool, cache.pool().kv_scale) == (cache.kv_pool.data_ptr(), cache.kv_scale.data_ptr())
    other = [torch.empty_like(x) for x in (cache.kv_pool, cache.kr_pool, cache.kv_scale)]
    for x, y in zip((cache.kv_pool, cache.kr_pool, cache.kv_scale), other):
        x.set_(y)
    p = cache.pool()
    assert (p.kv_pool, p.kr_pool, p.kv_scale) == tuple(x.data_ptr() for x in other)


def test_cache_buffers_are_on_one_device(M):
    dims = M.L.dims_for(2, 8, 16, 4, kv="fp8", page=4)
    kv, kr, s = torch.zeros(3, 4, 16, dtype=torch.uint8), torch.zeros(3, 4, 4, dtype=torch.bfloat16), torch.zeros(3, 4)
    M.L.PagedLatentCache.over(dims, kv, kr, s)
    for a, b in ((kr.to("meta"), s), (kr, s.to("meta"))):
        with pytest.raises(ValueError, match="one device"):
            M.L.PagedLatentCache.over(dims, kv, a, b)
