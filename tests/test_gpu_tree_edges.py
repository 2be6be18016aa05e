"""Drafted trees and pages at the edges of what the calls allow: values at the ends of their types, infinities, scales
far from one, streams, graphs and threads."""
import numpy as np
import pytest
import torch

from tests import tree_ref as R
from tests.test_gpu_tree import Batch, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_mqa_b200 import build
    build.build()


# ---- lengths at the ends of their type ---------------------------------------------------------------

LOWEST = [-2 ** 31, -2 ** 31 + 1, -2 ** 31 + 5, 2 ** 31 - 1]


@pytest.mark.parametrize("L", LOWEST)
@pytest.mark.parametrize("kv,flags", [("bf16", 0), ("fp8", 0), ("bf16", 1)])
def test_a_length_whose_difference_to_the_nodes_passes_the_type(kv, flags, L):
    from mla_latent_kv_mqa_b200 import native as N
    b = Batch([100, 300, 90], [6, 4, 3], kv=kv, flags=flags, heads=16)
    good, good_lse = b.decode()
    b.lens[1] = L
    o, lse = b.decode()
    assert N.mla_get_last_device_error() == N.MLA_ERR_BAD_SEQ_LEN
    others = [0, 1, 2, 3, 4, 5, 10, 11, 12]
    assert torch.equal(o[others], good[others]) and torch.equal(lse[others], good_lse[others])
    assert (o[6:10] == 0).all() and (lse[6:10] == float("-inf")).all()


@pytest.mark.parametrize("L", LOWEST[:3])
def test_prepare_and_keep_refuse_such_a_length(L):
    from mla_latent_kv_mqa_b200 import native as N
    b = Batch([100, 300, 90], [6, 7, 3], heads=1)
    b.lens[1] = L
    b.trees.seq_idx.fill_(1)
    b.trees.prepare(b.lens)
    assert N.mla_get_last_device_error() == N.MLA_ERR_BAD_SEQ_LEN
    assert b.trees.seq_idx.tolist() == [0] * 6 + [-1] * 7 + [2] * 3
    before = b.cache.kv_pool.clone()
    new = b.trees.keep([b.cache], b.table, b.lens, dev([[0, 1], [1, 3], [0, 1]]), dev([2, 2, 1]))
    assert N.mla_get_last_device_error() == N.MLA_ERR_BAD_SEQ_LEN
    assert new.tolist() == [102, L, 91]
    assert torch.equal(b.cache.kv_pool.view(torch.int16), before.view(torch.int16))


# ---- refusals that need a device ---------------------------------------------------------------------

def test_host_tensors_among_device_ones_are_refused():
    from mla_latent_kv_mqa_b200 import layer as L, pages as P
    b = Batch([100, 30], [6, 4], heads=4)
    with pytest.raises(ValueError):
        b.decode(o_lat=torch.zeros(10, 4, 512))
    with pytest.raises(ValueError):
        b.decode(lse=torch.zeros(10, 4))
    for ws in (torch.zeros(1 << 26, dtype=torch.uint8), torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            b.decode(workspace=ws)
    want = b.decode()
    got = b.decode(workspace=torch.empty(1 << 24, device="cuda"))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got = b.layer.decode_tree(b.cache, b.q.view(10, -1), b.table, b.lens, b.trees, b.max_len)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    keep, num = dev([[0], [0]]), dev([1, 1])
    other = L.PagedLatentCache(b.dims, b.cache.num_blocks, device="cpu")
    with pytest.raises(ValueError):
        b.trees.keep([b.cache, other], b.table, b.lens, keep, num)
    seqs = P.PagedSequences(64, 2, 4, b.cache.num_blocks)
    for moves in ((dev([0, 1]), dev([1])), (dev([[0, 1, 2]]), dev([1])), (dev([[0, 1]]), dev([])), (torch.zeros(1, 2, dtype=torch.int32), None)):
        with pytest.raises(ValueError):
            seqs.copy_pages([b.cache], moves)
    b.check(b.decode())


# ---- calls on a stream that is not the current one ----------------------------------------------------

def _sleep(stream, ms=30):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(int(ms * 1.9e6))


def _moved_pool(seqs, cache, blocks):
    """Three sequences over a pool of `blocks` pages, the first ended: pages to move."""
    seqs.grow(dev([64 * 5, 64 * 6, 64 * 4]))
    seqs.trim(dev([0, 64 * 6, 64 * 4]))
    cache.kv_pool.copy_(torch.arange(blocks, device="cuda")[:, None, None].expand_as(cache.kv_pool).to(cache.kv_pool.dtype))
    torch.cuda.synchronize()


@pytest.mark.parametrize("second", [False, True])
def test_moves_that_are_dropped_while_another_stream_reads_them(second):
    """seqs.copy_pages(caches, seqs.compact(stream=s), stream=s): nobody holds the moves when s comes to them."""
    from mla_latent_kv_mqa_b200 import layer as L, pages as P
    cache = L.PagedLatentCache(L.dims_for(2, 128, 512, 64), 40)
    seqs = P.PagedSequences(64, 3, 8, 40)
    s, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        seqs.trim(dev([0, 0, 0]))
        _moved_pool(seqs, cache, 40)
        _sleep(s)
        moves = seqs.compact(stream=s)
        reader = s
        if second:
            s2.wait_stream(s)
            reader = s2
        seqs.copy_pages([cache], moves, stream=reader)
        del moves
        junk = [torch.full((n, 2), 1, dtype=torch.int32, device="cuda") for n in (21, 20, 21, 22) for _ in range(8)]
        with torch.cuda.stream(s):
            junk += [torch.full((21, 2), 1, dtype=torch.int32, device="cuda") for _ in range(8)] if second else []
        torch.cuda.synchronize()
        del junk
        # pages 5..10 and 11..14 were in use, the last five of them move to 0..4
        want = torch.arange(40.0)
        want[:5] = torch.arange(10.0, 15.0)
        assert torch.equal(cache.kv_pool[:, 0, 0].float().cpu(), want)
        seqs.trim(dev([0, 0, 0]))


def test_grow_on_another_stream_and_its_copies():
    from mla_latent_kv_mqa_b200 import layer as L, pages as P
    cache = L.PagedLatentCache(L.dims_for(2, 128, 512, 64), 40)
    seqs = P.PagedSequences(64, 4, 8, 40)
    s = torch.cuda.Stream()
    seqs.grow(dev([100, 0, 0, 0]))
    seqs.fork(dev([0, 0, 0]), dev([1, 2, 3]))
    cache.kv_pool.copy_(torch.arange(40, device="cuda")[:, None, None].expand_as(cache.kv_pool).to(cache.kv_pool.dtype))
    lens = dev([101, 102, 103, 104])
    torch.cuda.synchronize()
    _sleep(s)
    seqs.copy_pages([cache], seqs.grow(lens, stream=s), stream=s)
    junk = [torch.full((5, 2), 30, dtype=torch.int32, device="cuda") for _ in range(16)]
    torch.cuda.synchronize()
    del junk
    assert sorted(seqs.block_table[:, 1].tolist()) == [1, 2, 3, 4]
    want = torch.arange(40.0)
    want[2:5] = 1
    assert torch.equal(cache.kv_pool[:, 0, 0].float().cpu(), want)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("flags", [0, 1])
def test_outputs_and_workspaces_of_another_stream(flags, raw):
    """Memory that pending work of the current stream still writes is not handed to a call on another stream."""
    from mla_latent_kv_mqa_b200 import layer as L
    b = Batch([900, 300, 31], [6, 4, 9], heads=32, seed=65, flags=flags)
    want, want_lse = b.decode()
    keep, num = dev([[0], [0], [0]]), dev([1, 1, 1])
    s = torch.cuda.Stream()
    stream = s.cuda_stream if raw else s
    b.layer._tree_ws = L.Workspace(b.layer.device)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    mem = [torch.empty_like(want), torch.empty_like(want_lse), torch.empty(1 << 26, dtype=torch.uint8, device="cuda"), torch.empty_like(b.lens)]
    torch.cuda._sleep(int(30 * 1.9e6))
    for x in mem:
        x.fill_(7)
    del mem, x
    o, lse = b.layer.decode_tree(b.cache, b.q, b.table, b.lens, b.trees, b.max_len, stream=stream)
    new = b.trees.keep([b.cache], b.table, b.lens, keep, num, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    assert new.tolist() == [901, 301, 32]
    del o, lse, new                                                  # freed with the current stream past them
    again = b.layer.decode_tree(b.cache, b.q, b.table, b.lens, b.trees, b.max_len, stream=stream)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(again[0], want) and torch.equal(again[1], want_lse)


# ---- the widest rows --------------------------------------------------------------------------------------

@pytest.mark.parametrize("kv,act,shape", [("f32", "f32", (16, 1024, 428)), ("fp8", "bf16", (8, 16, 1436))])
def test_the_widest_rows(kv, act, shape):
    b = Batch([129, 33], [5, 3], kv=kv, act=act, shape=shape, page=16, heads=3, seed=7)
    b.check(b.decode())
    b = Batch([3000, 700], [5, 3], kv=kv, act=act, shape=shape, page=16, heads=3, seed=8)   # a cluster of them joins
    b.check(b.decode())


# ---- rows before they have places ---------------------------------------------------------------------------

def test_an_append_before_prepare_goes_nowhere():
    from mla_latent_kv_mqa_b200 import native as N, tree as T
    b = Batch([100, 30], [6, 4], heads=2)
    junk = [torch.full((10,), 1, dtype=torch.int32, device="cuda") for _ in range(32)]
    del junk                                                         # memory that new tensors find
    trees = T.DraftTrees(b.trees.cu_nodes, b.trees.parent, 6)
    before = b.cache.kv_pool.clone()
    b.layer.tree_append(b.cache, torch.ones(10, 512, device="cuda").bfloat16(), torch.ones(10, 64, device="cuda").bfloat16(), trees, b.table)
    torch.cuda.synchronize()
    assert torch.equal(before.view(torch.int16), b.cache.kv_pool.view(torch.int16))
    assert N.mla_get_last_device_error() == N.MLA_OK


# ---- workspaces -----------------------------------------------------------------------------------------

def test_two_graphs_of_a_layer_that_replay_at_the_same_time():
    """Captured one after the other on the same capture stream, replayed on two streams at once."""
    a = Batch([3000, 2500], [20, 9], heads=32, seed=71)
    c = Batch([9000, 700, 41], [6, 4, 30], heads=32, seed=72)
    c.layer = a.layer
    want = [tuple(x.clone() for x in y.decode()) for y in (a, c)]
    graphs, outs = [], []
    for x in (a, c):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(x.layer.decode_tree(x.cache, x.q, x.table, x.lens, x.trees, x.max_len))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for o, lse in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                for _ in range(5):
                    g.replay()
        torch.cuda.synchronize()
        for got, ref in zip(outs, want):
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_a_graph_captured_on_a_stream_that_is_passed():
    b = Batch([900, 300], [6, 4], heads=32, seed=73)
    want, want_lse = (x.clone() for x in b.decode())
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        o, lse = b.layer.decode_tree(b.cache, b.q, b.table, b.lens, b.trees, b.max_len, stream=s.cuda_stream)
    b.decode()
    junk = [torch.full((1 << 22,), float("nan"), device="cuda") for _ in range(16)]
    g.replay()
    torch.cuda.synchronize()
    del junk
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


def test_the_layers_of_a_model_share_a_stream_s_workspace():
    b = Batch([900, 300], [6, 4], heads=32, seed=74)
    from mla_latent_kv_mqa_b200 import layer as L
    want, want_lse = b.decode()
    w = torch.zeros(32 * 128, 512, device="cuda", dtype=torch.bfloat16)
    layers = [L.MLADecodeLayer(b.dims, w, w) for _ in range(61)]
    before = torch.cuda.memory_allocated()
    for lay in layers:
        o, lse = lay.decode_tree(b.cache, b.q, b.table, b.lens, b.trees, b.max_len)
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
    assert torch.cuda.memory_allocated() - before < 8 << 20


def test_two_threads_on_one_stream():
    """Main kernel and join of a call stay together, so do the kernels of the page calls."""
    import threading

    from mla_latent_kv_mqa_b200 import pages as P
    a = Batch([3000, 2500], [20, 9], heads=32, seed=75)
    c = Batch([9000, 700, 41], [6, 4, 30], heads=32, seed=76)
    want = [tuple(x.clone() for x in y.decode()) for y in (a, c)]
    seqs = P.PagedSequences(4, 40, 6, 400)
    seqs.grow(dev(np.full(40, 11)))
    table, refs = seqs.block_table.clone(), seqs.refs.clone()
    wrong = []

    def work(k):
        x = (a, c)[k]
        own = torch.arange(20 * k, 20 * k + 20, device="cuda", dtype=torch.int32)
        got = []
        for _ in range(60):
            got.append(x.layer.decode_tree(x.cache, x.q, x.table, x.lens, x.trees, x.max_len))
            seqs.fork(own, own)                                      # each thread's own sequences, onto themselves
        torch.cuda.synchronize()
        wrong.append(sum(not (torch.equal(o, want[k][0]) and torch.equal(lse, want[k][1])) for o, lse in got))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert wrong == [0, 0]
    assert torch.equal(seqs.block_table, table) and torch.equal(seqs.refs, refs)


# ---- rows that are not finite ---------------------------------------------------------------------------

@pytest.mark.parametrize("kv,flags", [("bf16", 0), ("fp8", 0), ("bf16", 1), ("fp8", 1)])
@pytest.mark.parametrize("ctx", [200, 3000])                         # in one run, and joined from several
@pytest.mark.parametrize("drafted", [False, True])
def test_an_infinite_row_and_queries_of_both_signs(kv, flags, ctx, drafted):
    """Score +inf: NaN.  Score -inf: the token is no part of the sums; a committed one is NaN in the infinite column over
    a bf16 cache on the tensor cores.  (FP8: an infinite scale makes the row's every column infinite.)"""
    b = Batch([ctx, 64], [5, 3], kv=kv, flags=flags, seed=81, heads=16)
    slot, column = (ctx + 1 if drafted else 70), 7
    b.see[0][:, 1] = True                                            # every node sees the drafted row
    b.trees.mask.copy_(dev(np.concatenate([R.bits(s, b.trees.mask_words) for s in b.see])))
    minus = torch.arange(16, device="cuda") % 2 == 1                 # heads whose score is -inf
    at = b.owned[0][slot // 64], slot % 64
    if kv == "fp8":
        b.cache.kv_pool[at] = 0x38                                   # ones: the score's sign is the sum's
        b.cache.kr_pool[at] = 0
        b.q[:, :, :512] = b.q[:, :, :512].abs() * torch.where(minus, -1.0, 1.0)[:, None].to(b.q.dtype)
    else:
        b.q[:, :, column] = torch.where(minus, -1.0, 1.0).to(b.q.dtype)
    n0 = 5
    if kv == "fp8":
        b.cache.kv_scale[at] = float("inf")
    else:
        b.cache.kv_pool[at[0], at[1], column] = float("inf")
    o, lse = b.decode()
    assert torch.isnan(o[:n0, ~minus]).all() and not torch.isfinite(lse[:n0, ~minus]).any()
    rows = R.cache_rows(b.cache.kv_pool, b.cache.kr_pool, b.cache.kv_scale, b.table[0], ctx + 5, 64)
    sees = np.concatenate([np.ones((5, ctx), dtype=bool), b.see[0]], 1)
    sees[:, slot] = False
    sees = torch.from_numpy(sees).cuda()
    ro, rl, size, reach = R.attend(b.q[:n0], rows, sees, 512, b.scale)
    bound = R.o_bound(ro, size, reach, b.row, False, b.tensor_core())
    lb = R.lse_bound(rl, reach, b.row)
    if kv == "fp8" and b.tensor_core():
        j = torch.arange(ctx + 5, device="cuda")
        where = b.owned[0][j // 64], j % 64
        w = torch.where(torch.isfinite(b.cache.kv_scale[where]), b.cache.kv_scale[where], 0)
        ds, da = R.fp8_terms(b.q[:n0], b.cache.kv_pool[where], w, sees, 512, b.scale)
        bound, lb = bound + 2 * size * ds[..., None] + da * float(w.max()), lb + ds
    right = (o[:n0].double() - ro).abs() <= bound
    if kv == "bf16" and flags == 0 and not drafted:
        assert torch.isnan(o[:n0, minus, column]).all()
        right[:, :, column] = True
    assert right[:, minus].all()
    assert ((lse[:n0].double() - rl).abs() <= lb)[:, minus].all()
    assert torch.isfinite(o[n0:]).all() and torch.isfinite(lse[n0:]).all()


# ---- pages ----------------------------------------------------------------------------------------------

def test_compact_reports_an_entry_of_a_page_that_nobody_holds_wherever_it_lies():
    """Also among the lowest ids, where a page in use moves to it; entries of pages in use follow."""
    from mla_latent_kv_mqa_b200 import native as N, pages as P
    seqs = P.PagedSequences(4, 4, 3, 12)
    seqs.grow(dev([8, 8, 8, 0]))                                     # pages 0,1 / 2,3 / 4,5
    seqs.trim(dev([0]), dev([0]))
    seqs.block_table[3, 1] = 1
    moves, number = seqs.compact()
    assert N.mla_get_last_device_error() == N.MLA_ERR_BAD_BLOCK_TABLE
    assert moves[:int(number)].tolist() == [[4, 0], [5, 1]]
    assert seqs.block_table.tolist() == [[-1] * 3, [2, 3, -1], [0, 1, -1], [-1, 1, -1]]
    assert seqs.refs.tolist() == [1] * 4 + [0] * 8
    seqs.block_table[3, 1] = -1
    moves, number = seqs.compact()
    assert int(number) == 0 and N.mla_get_last_device_error() == N.MLA_OK


@pytest.mark.parametrize("width", [4, 60])                           # few pages, and many a sequence
def test_grow_refuses_to_write_a_reserved_page_that_another_sequence_holds(width):
    from mla_latent_kv_mqa_b200 import native as N, pages as P
    seqs = P.PagedSequences(4, 3, width, 200)
    seqs.grow(dev([4 * width, 3, 0]))
    seqs.fork(dev([0]), dev([2]))
    seqs.seq_lens[2] = 6                                             # cut without a trim: its pages behind are shared
    before = [x.clone() for x in (seqs.block_table, seqs.refs, seqs.seq_lens)]
    for new in (4 * width, 9):
        _, number = seqs.grow(dev([new, 5]), dev([2, 1]))
        assert int(number) == 0 and N.mla_get_last_device_error() == N.MLA_ERR_BAD_BLOCK_TABLE
        assert all(torch.equal(x, y) for x, y in zip(before, (seqs.block_table, seqs.refs, seqs.seq_lens)))
    seqs.trim(seqs.seq_lens.clone())
    moves, number = seqs.grow(dev([4 * width, 5]), dev([2, 1]))
    assert N.mla_get_last_device_error() == N.MLA_OK and int(number) == 1
    assert (seqs.refs[seqs.block_table[seqs.block_table >= 0].long()] >= 1).all()
    held = torch.bincount(seqs.block_table[seqs.block_table >= 0].long(), minlength=200)
    assert torch.equal(held.int(), seqs.refs)
    shared = set(seqs.block_table[0].tolist()) & set(seqs.block_table[2].tolist())
    assert shared - {-1} == {int(before[0][0, 0])}                   # the full page alone
    # its own pages behind a lowered length stay
    seqs.seq_lens[0] = 5
    seqs.trim(dev([0]), dev([2]))
    row = seqs.block_table[0].clone()
    seqs.grow(dev([4 * width]))
    assert torch.equal(seqs.block_table[0], row) and N.mla_get_last_device_error() == N.MLA_OK
    # an entry that names a page nobody holds
    seqs.seq_lens[1] = 6
    seqs.refs[seqs.block_table[1, 1].long()] = 0
    seqs.grow(dev([7]), dev([1]))
    assert N.mla_get_last_device_error() == N.MLA_ERR_BAD_BLOCK_TABLE


def test_what_a_call_on_another_stream_uses_may_be_dropped():
    """Lists, trees, queries and tables that nobody holds any more when the stream comes to them."""
    from mla_latent_kv_mqa_b200 import layer as L, pages as P, tree as T
    b = Batch([900, 300, 31], [6, 4, 9], heads=32, seed=67)
    want, want_lse = (x.clone() for x in b.decode())
    s = torch.cuda.Stream()
    ones = lambda n: torch.full((n,), 1, dtype=torch.int32, device="cuda")
    cu, parent, lens = b.trees.cu_nodes.clone(), b.trees.parent.clone(), b.lens.clone()
    trees = T.DraftTrees(cu, parent, b.most)
    q, table = b.q.clone(), b.table.clone()
    seqs = P.PagedSequences(64, 3, 8, 40)
    rows = torch.randn(19, 512, device="cuda").bfloat16(), torch.randn(19, 64, device="cuda").bfloat16()
    other = L.PagedLatentCache(b.dims, b.cache.num_blocks)
    held = L.PagedLatentCache(b.dims, b.cache.num_blocks)
    for c in (other, held):
        c.kv_pool.zero_()
    b.trees.prepare(lens)
    b.layer.tree_append(held, *rows, b.trees, table)
    new_lens, seq = dev([100, 30, 200]), dev([0, 1, 2])
    torch.cuda.synchronize()
    _sleep(s)
    trees.prepare(lens, stream=s)
    o, lse = b.layer.decode_tree(b.cache, q, table, lens, trees, b.max_len, stream=s)
    b.layer.tree_append(other, *rows, trees, table, stream=s)
    seqs.grow(new_lens, seq, stream=s)
    del cu, parent, lens, trees, q, table, rows, new_lens, seq
    junk = [ones(n) for n in (3, 4, 19, 20, 2, 38) for _ in range(8)] + [torch.full_like(b.q, 9.0) for _ in range(2)]
    junk += [torch.full_like(b.table, 0) for _ in range(4)] + [torch.full((19, k), 5.0, device="cuda").bfloat16() for k in (512, 64) for _ in range(2)]
    torch.cuda.synchronize()
    del junk
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    assert torch.equal(other.kv_pool, held.kv_pool)
    assert seqs.seq_lens.tolist() == [100, 30, 200]
