"""The cache's pages on the GPU: fork, grow, trim, compact and the copies, against a model that applies the
entries one after the other (tests/tree_ref.Pages), and a speculative step with all calls together."""
import numpy as np
import pytest
import torch

from tests import tree_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_mqa_b200 import build
    build.build()


def dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def error():
    from mla_latent_kv_mqa_b200 import native as N
    return N.mla_get_last_device_error()


def caches(kv, shape, page, blocks, layers, seed=0):
    from mla_latent_kv_mqa_b200 import layer as L
    torch.manual_seed(seed)
    dims = L.dims_for(2, shape[0], shape[1], shape[2], act="bf16", kv=kv, page=page)
    out = []
    for _ in range(layers):
        c = L.PagedLatentCache(dims, blocks)
        for x in parts(c):
            x.copy_(torch.randint(0, 120, x.shape, device="cuda").to(x.dtype))
        out.append(c)
    return out


def parts(c):
    return [x for x in (c.kv_pool, c.kr_pool, c.kv_scale) if x is not None]


def same(seqs, model):
    torch.cuda.synchronize()
    assert np.array_equal(seqs.block_table.cpu().numpy(), model.table)
    assert np.array_equal(seqs.refs.cpu().numpy(), model.refs)
    assert np.array_equal(seqs.seq_lens.cpu().numpy(), model.lens)


def pairs(moves):
    n = int(moves[1])
    return [tuple(r) for r in moves[0][:n].cpu().numpy().tolist()]


@pytest.mark.parametrize("num_seqs,width,blocks,page", [(1, 1, 1, 1), (5, 6, 40, 4), (40, 9, 300, 64), (1200, 4, 5000, 16), (3, 2500, 7000, 2)])
def test_random_calls_against_the_model(num_seqs, width, blocks, page):
    from mla_latent_kv_mqa_b200 import native as N, pages as P
    rng = np.random.default_rng(num_seqs + blocks)
    seqs = P.PagedSequences(page, num_seqs, width, blocks)
    model = R.Pages(page, seqs.block_table.cpu().numpy(), seqs.refs.cpu().numpy(), seqs.seq_lens.cpu().numpy())
    most, refused = width * page, 0
    for step in range(40):
        kind = rng.integers(5)
        k = int(rng.integers(1, num_seqs + 1))
        some = rng.permutation(num_seqs)[:k]
        if kind <= 1:
            new = np.minimum(most, model.lens[some] + rng.integers(0, max(2, most // 3), k))
            want = model.grow(new, some)
            got = seqs.grow(dev(new), dev(some))
            if want is None:
                refused += 1
                assert error() == N.MLA_ERR_OUT_OF_PAGES and pairs(got) == []
            else:
                assert pairs(got) == want and error() == N.MLA_OK
        elif kind == 2:
            parent = rng.integers(0, num_seqs, k)
            model.fork(parent, some)
            seqs.fork(dev(parent), dev(some))
        elif kind == 3:
            seq = rng.integers(0, num_seqs, k)                     # the same one more than once
            new = rng.integers(0, most + 1, k)
            model.trim(new, seq)
            seqs.trim(dev(new), dev(seq))
        else:
            want = model.compact()
            assert pairs(seqs.compact()) == want
        same(seqs, model)
        held = np.bincount(model.table[model.table >= 0], minlength=blocks)
        assert np.array_equal(held, model.refs)
    assert error() == N.MLA_OK


def test_the_last_sharer_keeps_the_page():
    from mla_latent_kv_mqa_b200 import pages as P
    seqs = P.PagedSequences(4, 4, 3, 12)
    assert pairs(seqs.grow(dev([6, 0, 0, 0]))) == []
    seqs.fork(dev([0, 0, 0]), dev([1, 2, 3]))
    assert list(seqs.refs.cpu()[:2]) == [4, 4]
    assert pairs(seqs.grow(dev([7, 7, 6, 7]))) == [(1, 2), (1, 3), (1, 4)]      # sequence 2 still holds it: all copy
    assert pairs(seqs.grow(dev([7, 7, 7, 7]))) == []                            # alone by now
    seqs.trim(dev([0, 0, 0]), dev([1, 2, 3]))
    seqs.fork(dev([0, 0]), dev([1, 2]))
    assert pairs(seqs.grow(dev([8, 8, 8]), dev([2, 0, 1]))) == [(2, 1), (2, 3)]  # in the call's order; 1 keeps page 2
    assert seqs.block_table[:, 1].tolist() == [3, 2, 1, -1]


def test_reordering_beams():
    """new[i] = old[parent[i]] for all i at once."""
    from mla_latent_kv_mqa_b200 import pages as P
    seqs = P.PagedSequences(4, 4, 2, 20)
    seqs.grow(dev([5, 6, 7, 8]))
    old, lens = seqs.block_table.clone(), seqs.seq_lens.clone()
    parent = dev([2, 2, 0, 3])
    seqs.fork(parent, dev([0, 1, 2, 3]))
    assert torch.equal(seqs.block_table, old[parent.long()]) and torch.equal(seqs.seq_lens, lens[parent.long()])
    held = torch.bincount(seqs.block_table.flatten().long(), minlength=20)
    assert torch.equal(held.int(), seqs.refs)


def test_bad_entries():
    from mla_latent_kv_mqa_b200 import native as N, pages as P

    def fresh():
        s = P.PagedSequences(4, 4, 2, 6)
        s.grow(dev([5, 3, 0, 0]))
        return s

    def state(s):
        return [x.clone() for x in (s.block_table, s.refs, s.seq_lens)]
    for parent, child, code in [([9], [2], N.MLA_ERR_BAD_SEQ_INDEX), ([0], [-1], N.MLA_ERR_BAD_SEQ_INDEX), ([0, 1], [2, 2], N.MLA_ERR_BAD_SEQ_INDEX)]:
        s = fresh()
        before = state(s)
        s.fork(dev(parent), dev(child))
        assert error() == code and all(torch.equal(a, b) for a, b in zip(before, state(s)))
    for new, seq, code in [([6, 6], [0, 0], N.MLA_ERR_BAD_SEQ_INDEX), ([6, 6], [0, 4], N.MLA_ERR_BAD_SEQ_INDEX), ([6, 9], [0, 1], N.MLA_ERR_BAD_SEQ_LEN),
                           ([-1, 6], [0, 1], N.MLA_ERR_BAD_SEQ_LEN), ([8, 8, 8, 8], [0, 1, 2, 3], N.MLA_ERR_OUT_OF_PAGES)]:
        s = fresh()
        before = state(s)
        moves = s.grow(dev(new), dev(seq))
        assert error() == code and pairs(moves) == [] and all(torch.equal(a, b) for a, b in zip(before, state(s)))
    s = fresh()
    before = state(s)
    s.trim(dev([-1, 3]), dev([0, 7]))
    assert error() in (N.MLA_ERR_BAD_SEQ_LEN, N.MLA_ERR_BAD_SEQ_INDEX) and all(torch.equal(a, b) for a, b in zip(before, state(s)))
    s = fresh()
    s.block_table[3, 0] = 5                                         # a page that nobody holds
    assert pairs(s.compact()) == [] and error() == N.MLA_ERR_BAD_BLOCK_TABLE
    assert int(s.block_table[3, 0]) == 5
    s.block_table[3, 0] = 77
    s.compact()
    assert error() == N.MLA_ERR_BAD_BLOCK_TABLE


@pytest.mark.parametrize("kv,shape,page,layers", [("bf16", (128, 512, 64), 64, 2), ("fp8", (128, 512, 64), 64, 3), ("f32", (64, 128, 32), 64, 1),
                                                  ("bf16", (8, 25, 6), 3, 1), ("fp8", (8, 33, 2), 5, 70)])
def test_copy_pages(kv, shape, page, layers):
    from mla_latent_kv_mqa_b200 import native as N, pages as P
    blocks = 41
    cs = caches(kv, shape, page, blocks, layers)
    ids = np.random.default_rng(0).permutation(blocks)
    mv = np.stack([ids[:13], ids[13:26]], 1)
    mv[5] = mv[4][0], mv[5][1]                                      # one source, two targets
    mv[7] = blocks, 3                                               # no page: skipped
    mv[8] = mv[8][0], mv[8][0]                                      # onto itself
    seqs = P.PagedSequences(page, 1, 1, blocks)
    for count in (13, 0, 9):
        want = [x.clone() for c in cs for x in parts(c)]
        for s, d in mv[:count]:
            if s < blocks:
                for w in want:
                    w[d] = w[s].clone()
        seqs.copy_pages(cs, (dev(mv), dev([count])))
        assert error() == (N.MLA_ERR_BAD_BLOCK_TABLE if count > 7 else N.MLA_OK)
        for x, w in zip([x for c in cs for x in parts(c)], want):
            assert torch.equal(x.view(torch.uint8), w.view(torch.uint8))
    seqs.copy_pages(cs, (dev(mv[:4]), dev([50])))                   # more than the list holds: the list's


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_speculative_step_with_forked_sequences(kv):
    """Prompts, forks, drafted trees, the accepted path kept, ended sequences, a compacted pool: afterwards
    every sequence's rows are, bit for bit, those of its tokens appended one after the other, and
    mla_decode on the two caches gives the same bits."""
    from mla_latent_kv_mqa_b200 import layer as L, pages as P, tree as T
    heads, d_h, d_c, d_r, page = 128, 128, 512, 64, 64
    rng = np.random.default_rng(3)
    torch.manual_seed(3)
    bf = dict(device="cuda", dtype=torch.bfloat16)
    dims = L.dims_for(heads, d_h, d_c, d_r, kv=kv, page=page)
    layer = L.MLADecodeLayer(dims, torch.randn(heads * d_h, d_c, **bf) / d_c ** 0.5, torch.randn(heads * d_h, d_c, **bf) / d_c ** 0.5)
    S, blocks = 6, 60
    cs = [L.PagedLatentCache(dims, blocks, poison=True) for _ in range(2)]
    seqs = P.PagedSequences(page, S, 8, blocks)
    toks = [[] for _ in range(S)]                                   # the committed tokens' (c, k) by layer

    def new_rows(n):
        return [(torch.randn(n, d_c, **bf), torch.randn(n, d_r, **bf)) for _ in cs]
    prompt = [100, 70, 64]
    moves = seqs.grow(dev(prompt + [0] * 3))
    seqs.copy_pages(cs, moves)
    for s, n in enumerate(prompt):
        rows = new_rows(n)
        for c, (ckv, kr) in zip(cs, rows):
            layer.append(c, ckv, kr, dev(np.full(n, s)), dev(np.arange(n)), seqs.block_table)
        toks[s] = [[(ckv[i], kr[i]) for ckv, kr in rows] for i in range(n)]
    seqs.fork(dev([0, 0, 2]), dev([3, 4, 5]))
    for p, c in zip([0, 0, 2], [3, 4, 5]):
        toks[c] = list(toks[p])
    for step in range(3):
        n = rng.integers(1, 20, S)
        cu, parent = R.trees(rng, n)
        ctx = seqs.seq_lens.cpu().numpy()
        seqs.copy_pages(cs, seqs.grow(dev(ctx + n)))
        trees = T.DraftTrees(dev(cu), dev(parent), int(n.max()))
        trees.prepare(seqs.seq_lens)
        rows = new_rows(int(cu[-1]))
        for c, (ckv, kr) in zip(cs, rows):
            layer.tree_append(c, ckv, kr, trees, seqs.block_table)
        q_abs = layer.absorb(torch.randn(int(cu[-1]), heads, d_h, **bf), torch.randn(int(cu[-1]), heads, d_r, **bf), trees.pos)
        o_lat, lse = layer.decode_tree(cs[1], q_abs, seqs.block_table, seqs.seq_lens, trees, 8 * page)
        assert torch.isfinite(layer.out_proj(o_lat)).all() and torch.isfinite(lse).all()
        for s in range(S):                                          # the step's attention, node by node, on a sample
            see, depth = R.sees(parent[cu[s]:cu[s + 1]])
            nodes = np.unique([0, n[s] - 1])
            c = cs[1]
            full = R.cache_rows(c.kv_pool, c.kr_pool, c.kv_scale, seqs.block_table[s], int(ctx[s] + n[s]), page)
            vis = torch.from_numpy(np.concatenate([np.ones((len(nodes), ctx[s]), dtype=bool), see[nodes]], 1)).cuda()
            t = torch.from_numpy(cu[s] + nodes).cuda()
            ro, rl, size, reach = R.attend(q_abs[t], full, vis, d_c, (d_h + d_r) ** -0.5)
            assert ((o_lat[t].double() - ro).abs() <= R.o_bound(ro, size, reach, 576, False, True)).all()
            assert ((lse[t].double() - rl).abs() <= R.lse_bound(rl, reach, 576)).all()
        keep, num = np.zeros((S, int(n.max())), dtype=np.int64), np.zeros(S, dtype=np.int64)
        for s in range(S):
            see, _ = R.sees(parent[cu[s]:cu[s + 1]])
            path = np.nonzero(see[rng.integers(n[s])])[0]
            num[s] = rng.integers(0, len(path) + 1)
            keep[s, :num[s]] = path[:num[s]]
            toks[s] += [[(ckv[cu[s] + k], kr[cu[s] + k]) for ckv, kr in rows] for k in path[:num[s]]]
        new = trees.keep(cs, seqs.block_table, seqs.seq_lens, dev(keep), dev(num))
        seqs.trim(new)
        if step == 1:
            seqs.trim(dev([0]), dev([1]))
            toks[1] = []
            seqs.copy_pages(cs, seqs.compact())
            seqs.fork(dev([3]), dev([1]))
            toks[1] = list(toks[3])
    lens = seqs.seq_lens.cpu().numpy()
    assert [len(t) for t in toks] == list(lens)
    held = torch.bincount(seqs.block_table[seqs.block_table >= 0].long(), minlength=blocks)
    assert torch.equal(held.int(), seqs.refs)
    plain = L.PagedLatentCache(dims, S * 8, poison=True)
    table = dev(np.arange(S * 8).reshape(S, 8))
    for i, c in enumerate(cs):
        for s in range(S):
            ckv, kr = torch.stack([t[i][0] for t in toks[s]]), torch.stack([t[i][1] for t in toks[s]])
            layer.append(plain, ckv, kr, dev(np.full(len(toks[s]), s)), dev(np.arange(len(toks[s]))), table)
            j = torch.arange(len(toks[s]), device="cuda")
            for x, y in zip(parts(c), parts(plain)):
                a, b = x[seqs.block_table[s].long()[j // page], j % page], y[table[s].long()[j // page], j % page]
                assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
        q = layer.absorb(torch.randn(S, heads, d_h, **bf), torch.randn(S, heads, d_r, **bf), dev(lens - 1))
        a = layer.decode(c, q, seqs.block_table, seqs.seq_lens, 1, 8 * page)
        b = layer.decode(plain, q, table, seqs.seq_lens, 1, 8 * page)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert error() == 0


def test_a_captured_step_of_page_calls():
    from mla_latent_kv_mqa_b200 import pages as P
    seqs = P.PagedSequences(4, 4, 5, 30)
    cs = caches("bf16", (8, 24, 8), 4, 30, 2)
    new, parent, child = dev([5, 9, 0, 0]), dev([0, 1]), dev([2, 3])
    seqs.copy_pages(cs, seqs.grow(new))
    seqs.fork(parent, child)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moves = seqs.grow(new)
        seqs.copy_pages(cs, moves)
    model = R.Pages(4, seqs.block_table.cpu().numpy(), seqs.refs.cpu().numpy(), seqs.seq_lens.cpu().numpy())
    for length in (6, 7, 12, 20):
        new.fill_(length)
        want = model.grow([length] * 4)
        before = [x.clone() for c in cs for x in parts(c)]
        g.replay()
        same(seqs, model)
        assert pairs(moves) == want
        for x, w in zip([x for c in cs for x in parts(c)], before):
            for s, d in want:
                w[d] = w[s]
            assert torch.equal(x, w)
