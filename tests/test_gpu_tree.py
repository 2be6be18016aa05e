"""Drafted trees on the GPU: masks and positions, rows into and along the cache, and the attention,
against plain forms in 64 bits (tests/tree_ref.py)."""
import numpy as np
import pytest
import torch

from tests import tree_ref as R

pytestmark = pytest.mark.gpu

V3 = (128, 512, 64)      # d_h, d_c, d_r
TOY = (64, 128, 32)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_latent_kv_mqa_b200 import build
    build.build()


def dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def no_error():
    from mla_latent_kv_mqa_b200 import native as N
    assert N.mla_get_last_device_error() == N.MLA_OK


class Batch:
    """A filled cache, trees with their masks, queries, and the layer: sequence b has ctx[b] committed
    tokens and n[b] nodes; slots that belong to nobody hold NaN."""

    def __init__(self, ctx, n, *, heads=128, shape=V3, kv="bf16", act="bf16", page=64, seed=0, chain=False, flags=0,
                 pad=0, extra_words=0, spread=1.0, num_blocks=None):
        from mla_latent_kv_mqa_b200 import layer as L, tree as T
        d_h, d_c, d_r = shape
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.ctx, self.n, self.page, self.kv = np.asarray(ctx), np.asarray(n), page, kv
        self.B, self.heads, self.d_c, self.row = len(ctx), heads, d_c, d_c + d_r
        self.dims = L.dims_for(heads, d_h, d_c, d_r, act=act, kv=kv, page=page, flags=flags)
        self.scale = (d_h + d_r) ** -0.5
        lens = self.ctx + self.n
        cu, parent = R.trees(rng, self.n, chain)
        T_nodes = int(cu[-1])
        self.most = int(max(1, self.n.max()))
        pages = -(-lens // page)
        blocks = num_blocks or int(pages.sum()) + 3
        ids = (blocks - 1 - np.arange(blocks) if num_blocks else rng.permutation(blocks)).astype(np.int32)
        table = np.full((self.B, int(max(1, pages.max()))), -1, dtype=np.int32)
        k = 0
        for b in range(self.B):
            table[b, :pages[b]] = ids[k:k + pages[b]]
            k += pages[b]
        self.table, self.lens, self.max_len = dev(table), dev(lens), int(max(1, lens.max()))
        self.cache = L.PagedLatentCache(self.dims, blocks, poison=True)
        self.owned = [torch.from_numpy(table[b, :pages[b]].astype(np.int64)).cuda() for b in range(self.B)]
        for b in range(self.B):
            j = torch.arange(int(lens[b]), device="cuda")
            blk, off = self.owned[b][j // page] if len(j) else j, j % page
            x = torch.randn(len(j), self.row, generator=g, device="cuda")
            if kv == "fp8":
                s = x[:, :d_c].abs().amax(-1) / 448
                self.cache.kv_pool[blk, off] = (x[:, :d_c] / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
                self.cache.kv_scale[blk, off] = s
                self.cache.kr_pool[blk, off] = x[:, d_c:].bfloat16()
            else:
                self.cache.kv_pool[blk, off] = x.to(self.cache.kv_pool.dtype)
        words = (self.most + 31) // 32 + extra_words
        self.see = [R.sees(parent[cu[b]:cu[b + 1]])[0] for b in range(self.B)]
        mask = np.concatenate([R.bits(s, words) for s in self.see] + [np.full((pad, words), -1, dtype=np.int32)])
        self.cu = cu
        self.trees = T.DraftTrees(dev(cu), dev(np.concatenate([parent, np.zeros(pad, dtype=np.int32)])), self.most,
                                  mask=dev(mask))
        q = torch.randn(T_nodes + pad, heads, self.row, generator=g, device="cuda") * spread
        self.q = q.to(torch.float32 if act == "f32" else torch.bfloat16)
        w = torch.zeros(heads * d_h, d_c, device="cuda", dtype=self.q.dtype)
        self.layer = L.MLADecodeLayer(self.dims, w, w)
        self.T = T_nodes

    def tensor_core(self):
        d = self.dims
        return (d.d_c, d.d_r, d.page_size, d.flags) == (512, 64, 64, 0) and self.q.dtype == torch.bfloat16 and self.kv != "f32"

    def decode(self, out="f32", **kw):
        got = self.layer.decode_tree(self.cache, self.q, self.table, self.lens, self.trees, self.max_len, out_dtype=out, **kw)
        torch.cuda.synchronize()
        return got

    def reference(self, b, nodes=None):
        c, L = self.cache, int(self.ctx[b] + self.n[b])
        rows = R.cache_rows(c.kv_pool, c.kr_pool, c.kv_scale, self.table[b], L, self.page)
        nodes = np.arange(self.n[b]) if nodes is None else np.asarray(nodes)
        see = np.concatenate([np.ones((len(nodes), self.ctx[b]), dtype=bool), self.see[b][nodes]], 1)
        t, see = torch.from_numpy(self.cu[b] + nodes).cuda(), torch.from_numpy(see).cuda()
        self.extra = (0, 0)
        if self.kv == "fp8" and self.tensor_core():
            # every weight is 1 at most, so the row's largest weight times scale is the largest scale at most
            at = self.owned[b][torch.arange(L, device="cuda") // self.page], torch.arange(L, device="cuda") % self.page
            ds, da = R.fp8_terms(self.q[t], c.kv_pool[at], c.kv_scale[at], see, self.d_c, self.scale)
            w = torch.where(torch.isfinite(c.kv_scale[at]), c.kv_scale[at], 0).abs()
            largest = torch.stack([w[m].amax() if m.any() else w.new_zeros(()) for m in see]).double()
            self.extra = (ds, da * largest[:, None, None])
        return t, R.attend(self.q[t], rows, see, self.d_c, self.scale)

    def check(self, got, out="f32", sample=None):
        o, lse = got
        for b in range(self.B):
            if self.n[b] == 0:
                continue
            nodes = None if sample is None or self.n[b] <= sample else np.unique(np.linspace(0, self.n[b] - 1, sample).astype(int))
            t, (ro, rl, size, reach) = self.reference(b, nodes)
            eo = (o[t].double() - ro).abs()
            bound = R.o_bound(ro, size, reach, self.row, out == "bf16", self.tensor_core())
            if self.kv == "fp8" and self.tensor_core():
                bound = bound + 2 * size * self.extra[0][..., None] + self.extra[1]
            assert (eo <= bound).all(), (b, float((eo / bound).max()))
            seen = torch.isfinite(rl)
            assert torch.equal(torch.isfinite(lse[t]), seen)
            el = (lse[t].double() - rl).abs()[seen]
            lb = (R.lse_bound(rl, reach, self.row) + self.extra[0])[seen]
            assert (el <= lb).all(), (b, float((el / lb).max()))
            assert (o[t][~seen] == 0).all() and (lse[t][~seen] == float("-inf")).all()
        no_error()


# ---- masks, slots, positions ---------------------------------------------------------------------

@pytest.mark.parametrize("sizes,chain", [([1], False), ([5, 0, 1, 33], False), ([32, 31, 64, 2], False), ([200, 7], False),
                                         ([1024, 3], True), ([1024], False), ([0, 0], False)])
@pytest.mark.parametrize("pad", [0, 5])
def test_prepare(sizes, chain, pad):
    from mla_latent_kv_mqa_b200 import tree as T
    rng = np.random.default_rng(sum(sizes) + pad)
    cu, parent = R.trees(rng, sizes, chain)
    ctx = rng.integers(0, 1000, len(sizes))
    total = int(cu[-1]) + pad
    if total == 0:
        return
    trees = T.DraftTrees(dev(cu), dev(np.concatenate([parent, np.full(pad, -1, dtype=np.int32)])), max(1, max(sizes)))
    for x in (trees.mask, trees.pos, trees.slot, trees.seq_idx):
        x.fill_(77)
    trees.prepare(dev(ctx + np.asarray(sizes)))
    torch.cuda.synchronize()
    for b, n in enumerate(sizes):
        see, depth = R.sees(parent[cu[b]:cu[b + 1]])
        at = slice(int(cu[b]), int(cu[b + 1]))
        assert np.array_equal(trees.mask[at].cpu().numpy(), R.bits(see, trees.mask_words))
        assert np.array_equal(trees.pos[at].cpu().numpy(), ctx[b] + depth)
        assert np.array_equal(trees.slot[at].cpu().numpy(), ctx[b] + np.arange(n))
        assert (trees.seq_idx[at] == b).all()
    assert (trees.seq_idx[int(cu[-1]):] == -1).all() and (trees.mask[int(cu[-1]):] == 0).all()
    no_error()


def test_prepare_reports_what_is_no_tree():
    from mla_latent_kv_mqa_b200 import native as N, tree as T
    for cu, parent, lens, code in [([0, 3], [-1, 1, 0], [10], N.MLA_ERR_BAD_TREE), ([0, 3], [-1, -2, 0], [10], N.MLA_ERR_BAD_TREE),
                                   ([0, 4], [-1, 0, 0], [10], N.MLA_ERR_BAD_TREE), ([1, 3], [-1, 0, 0], [10], N.MLA_ERR_BAD_TREE),
                                   ([0, 3], [-1, 0, 0], [2], N.MLA_ERR_BAD_SEQ_LEN)]:
        trees = T.DraftTrees(dev(cu), dev(parent), 4)
        trees.seq_idx.fill_(-1)
        trees.prepare(dev(lens))
        assert N.mla_get_last_device_error() == code
        if code == N.MLA_ERR_BAD_SEQ_LEN:
            assert (trees.seq_idx == -1).all()
    trees = T.DraftTrees(dev([0, 40]), dev([-1] * 40), 20)       # more nodes than the mask has bits
    trees.prepare(dev([50]))
    assert N.mla_get_last_device_error() == N.MLA_ERR_BAD_TREE


# ---- rows ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("kv,act,shape", [("bf16", "bf16", V3), ("fp8", "bf16", V3), ("f32", "f32", TOY), ("bf16", "f32", V3),
                                          ("fp8", "f32", (64, 600, 130))])
def test_append_puts_the_position_s_row_into_the_slot(kv, act, shape):
    """Bit for bit the row that mla_cache_append writes at the position, in the slot instead; nothing else
    of the pool changes."""
    b = Batch([130, 0, 63], [7, 3, 2], kv=kv, act=act, shape=shape, heads=2, seed=3, pad=2)
    d_h, d_c, d_r = shape
    dt = torch.float32 if act == "f32" else torch.bfloat16
    c, k = torch.randn(b.T + 2, d_c, device="cuda").to(dt), torch.randn(b.T + 2, d_r, device="cuda").to(dt)
    b.trees.prepare(b.lens)
    pos, slot, seq = (x.cpu().numpy() for x in (b.trees.pos, b.trees.slot, b.trees.seq_idx))
    assert (pos != slot).any()
    parts = [x for x in (b.cache.kv_pool, b.cache.kr_pool, b.cache.kv_scale) if x is not None]
    want = [x.clone() for x in parts]
    for t in range(b.T):                                            # one token at a time at its position, row taken from there
        b.layer.append(b.cache, c[t:t + 1], k[t:t + 1], dev(seq[t:t + 1]), dev(pos[t:t + 1]), b.table)
        s = int(seq[t])
        for x, w in zip(parts, want):
            w[b.owned[s][slot[t] // 64], slot[t] % 64] = x[b.owned[s][pos[t] // 64], pos[t] % 64]
    for x in parts:
        x.copy_(x.new_full((), 0).expand_as(x))
    before = [w.clone() for w in want]
    for x, w in zip(parts, before):
        x.copy_(w)
        for t in range(b.T):
            x[b.owned[int(seq[t])][slot[t] // 64], slot[t] % 64] = 0
    b.layer.tree_append(b.cache, c, k, b.trees, b.table)
    torch.cuda.synchronize()
    for x, w in zip(parts, want):
        assert torch.equal(x.view(torch.uint8), w.view(torch.uint8))
    no_error()


def test_append_reports_a_slot_outside_the_table():
    from mla_latent_kv_mqa_b200 import native as N
    b = Batch([60], [3], heads=1)
    c, k = torch.zeros(3, 512, device="cuda", dtype=torch.bfloat16), torch.zeros(3, 64, device="cuda", dtype=torch.bfloat16)
    b.trees.prepare(b.lens)
    for slot in (-1, 64, 1 << 30):
        before = b.cache.kv_pool.clone()
        b.trees.slot[1] = slot
        b.trees.seq_idx[0] = b.trees.seq_idx[2] = -1
        b.layer.tree_append(b.cache, c, k, b.trees, b.table)
        assert N.mla_get_last_device_error() == N.MLA_ERR_BAD_BLOCK_TABLE
        assert torch.equal(before.view(torch.int16), b.cache.kv_pool.view(torch.int16))


@pytest.mark.parametrize("kv,shape,layers", [("bf16", V3, 1), ("fp8", V3, 3), ("f32", TOY, 2), ("bf16", (64, 25, 6), 1), ("fp8", (8, 33, 2), 66)])
def test_keep(kv, shape, layers):
    from mla_latent_kv_mqa_b200 import layer as L
    b = Batch([61, 0, 640, 5, 127], [6, 4, 90, 0, 1], kv=kv, act="f32" if kv == "f32" else "bf16", shape=shape, heads=1, seed=5)
    keep = np.full((5, 40), 99, dtype=np.int32)
    rows = [[0, 2, 5], [3], sorted(np.random.default_rng(1).permutation(90)[:40]), [], [0]]
    for i, r in enumerate(rows):
        keep[i, :len(r)] = r
    caches = [b.cache]
    for i in range(layers - 1):
        c = L.PagedLatentCache(b.dims, b.cache.num_blocks)
        for x, y in zip((c.kv_pool, c.kr_pool, c.kv_scale), (b.cache.kv_pool, b.cache.kr_pool, b.cache.kv_scale)):
            if x is not None:
                x.copy_(y.roll(i + 1, -1))
        caches.append(c)
    want = []
    for c in caches:
        for x in (c.kv_pool, c.kr_pool, c.kv_scale):
            if x is None:
                continue
            w = x.clone()
            for s, r in enumerate(rows):
                for i, k in enumerate(r):
                    src, dst = int(b.ctx[s]) + int(k), int(b.ctx[s]) + i
                    w[b.owned[s][dst // 64], dst % 64] = x[b.owned[s][src // 64], src % 64]
            want.append((x, w))
    new = b.trees.keep(caches, b.table, b.lens, dev(keep), dev([len(r) for r in rows]))
    torch.cuda.synchronize()
    for x, w in want:
        assert torch.equal(x.view(torch.uint8), w.view(torch.uint8))
    assert list(new.cpu().numpy()) == [int(c) + len(r) for c, r in zip(b.ctx, rows)]
    no_error()


def test_keep_leaves_a_sequence_whose_path_is_none():
    from mla_latent_kv_mqa_b200 import native as N
    b = Batch([61, 10], [6, 4], heads=1)
    for keep, num, code in [([[2, 2, 0], [1, 3, 0]], [2, 2], N.MLA_ERR_BAD_TREE), ([[4, 6, 0], [1, 3, 0]], [2, 2], N.MLA_ERR_BAD_TREE),
                            ([[-1, 0, 0], [1, 3, 0]], [2, 2], N.MLA_ERR_BAD_TREE), ([[0, 1, 2], [1, 3, 0]], [4, 2], N.MLA_ERR_BAD_TREE),
                            ([[0, 1, 2], [1, 3, 0]], [-1, 2], N.MLA_ERR_BAD_TREE)]:
        before = b.cache.kv_pool.clone()
        new = b.trees.keep([b.cache], b.table, b.lens, dev(keep), dev(num))
        assert N.mla_get_last_device_error() == code
        assert list(new.cpu().numpy()) == [67, 12]
        after = b.cache.kv_pool
        assert torch.equal(after[b.owned[0]].view(torch.int16), before[b.owned[0]].view(torch.int16))
        assert torch.equal(after[b.owned[1][0], 10:12], before[b.owned[1][0], [11, 13]])
        after.copy_(before)


# ---- attention -------------------------------------------------------------------------------------

@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("ctx,n,heads", [
    ([0], [1], 128), ([1], [1], 1), ([250], [5], 128), ([255, 256, 257], [1, 1, 1], 128), ([64, 0, 700, 63], [3, 9, 1, 64], 16),
    ([1000, 130], [33, 2], 20), ([5, 300, 0], [0, 4, 0], 64), ([2000], [7], 128), ([511, 3000], [130, 1], 8), ([190], [300], 3)])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_decode(ctx, n, heads, kv, out):
    b = Batch(ctx, n, heads=heads, kv=kv, seed=len(ctx) + heads)
    b.check(b.decode(out), out, sample=9)


@pytest.mark.parametrize("kv,act,shape,page,heads,flags", [
    ("f32", "f32", TOY, 64, 8, 0), ("bf16", "f32", TOY, 16, 8, 0), ("fp8", "f32", V3, 64, 4, 0), ("bf16", "bf16", V3, 64, 128, 1),
    ("fp8", "bf16", V3, 64, 128, 1), ("f32", "bf16", (32, 96, 10), 7, 5, 0), ("bf16", "bf16", (128, 512, 64), 128, 9, 0),
    ("f32", "f32", (16, 1024, 2), 1, 2, 0)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_decode_other_shapes(kv, act, shape, page, heads, flags, out):
    b = Batch([129, 0, 33], [5, 3, 40], kv=kv, act=act, shape=shape, page=page, heads=heads, flags=flags, seed=7)
    b.check(b.decode(out), out)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_decode_large_scores(kv):
    """Scores of tens: the running maximum moves and the output is rescaled."""
    b = Batch([900, 70], [9, 4], kv=kv, spread=12.0, seed=2)
    b.check(b.decode())


def _break_rows(b, seq, slots, value):
    for s in slots:
        blk, off = b.owned[seq][s // b.page], s % b.page
        if b.kv == "fp8":
            b.cache.kv_pool[blk, off] = 0x7F
            b.cache.kr_pool[blk, off] = value
        else:
            b.cache.kv_pool[blk, off] = value


@pytest.mark.parametrize("kv,flags", [("bf16", 0), ("fp8", 0), ("bf16", 1), ("fp8", 1)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_masked_row_s_content_does_not_matter(kv, flags, value):
    """A drafted row of NaN or infinities reaches the nodes that see it and no other."""
    b = Batch([200, 64], [12, 5], kv=kv, flags=flags, seed=11, heads=16)
    good, good_lse = b.decode()
    _break_rows(b, 0, [203], value)
    o, lse = b.decode()
    sees = np.concatenate([b.see[0][:, 3], np.zeros(5, dtype=bool)])
    assert sees.any() and not sees[:12].all()
    sees = torch.from_numpy(sees).cuda()
    assert torch.equal(o[~sees], good[~sees]) and torch.equal(lse[~sees], good_lse[~sees])
    if value != value:
        assert torch.isnan(o[sees]).all() and torch.isnan(lse[sees]).all()
    no_error()


@pytest.mark.parametrize("kv,flags", [("bf16", 0), ("fp8", 0), ("bf16", 1)])
def test_any_mask_and_rows_that_see_nothing(kv, flags):
    b = Batch([0, 300, 0], [70, 65, 3], kv=kv, flags=flags, heads=12, seed=4, extra_words=1)
    rng = np.random.default_rng(8)
    b.see = [rng.random((n, n)) < 0.3 for n in b.n]
    b.see[0][5] = b.see[0][69] = False
    b.see[2][:] = False
    b.trees.mask.copy_(dev(np.concatenate([R.bits(s, b.trees.mask_words) for s in b.see])))
    b.check(b.decode())


@pytest.mark.parametrize("flags", [0, 1])
def test_padding_rows_stay_and_nothing_depends_on_the_workspace(flags):
    b = Batch([100, 0, 700], [6, 0, 3], flags=flags, pad=4, seed=9, heads=32)
    first = b.decode()
    for fill in (0, 0xFF):
        b.layer._tree_ws._by_stream[torch.cuda.current_stream().cuda_stream].fill_(fill)
        o = torch.full_like(first[0], 3.0)
        lse = torch.full_like(first[1], 4.0)
        b.decode(o_lat=o, lse=lse)
        assert torch.equal(o[:9], first[0][:9]) and torch.equal(lse[:9], first[1][:9])
        assert (o[9:] == 3).all() and (lse[9:] == 4).all()
    b.check(first)


@pytest.mark.parametrize("flags", [0, 1])
def test_bad_lengths_pages_and_trees_are_reported(flags):
    from mla_latent_kv_mqa_b200 import native as N
    b = Batch([100, 300], [6, 4], flags=flags, heads=16)
    good, good_lse = b.decode()
    for L in (3, b.max_len + 1, -5, 1 << 30):                       # of the second sequence
        b.lens[1] = L
        o, lse = b.decode()
        assert N.mla_get_last_device_error() == N.MLA_ERR_BAD_SEQ_LEN
        assert torch.equal(o[:6], good[:6]) and (o[6:] == 0).all() and (lse[6:] == float("-inf")).all()
    b.lens[1] = 304
    keep = int(b.table[1, 2])
    for blk in (-1, b.cache.num_blocks, 1 << 30):
        b.table[1, 2] = blk
        o, lse = b.decode()
        assert N.mla_get_last_device_error() == N.MLA_ERR_BAD_BLOCK_TABLE
        assert torch.equal(o[:6], good[:6])
    b.table[1, 2] = keep
    for cu in ([0, 6, 60], [0, 8, 6], [2, 6, 10], [0, -3, 10]):
        b.trees.cu_nodes.copy_(dev(cu))
        b.decode()
        assert N.mla_get_last_device_error() == N.MLA_ERR_BAD_TREE
    b.trees.cu_nodes.copy_(dev([0, 6, 10]))
    o, lse = b.decode()
    assert torch.equal(o, good) and torch.equal(lse, good_lse)
    no_error()


def test_pages_beyond_2_31_elements():
    """Block ids whose byte and element offsets pass 32 bits."""
    b = Batch([70, 500], [3, 4], heads=16, num_blocks=60000, seed=13)
    assert int(b.table[b.table >= 0].min()) * 64 * 576 > 2 ** 31
    b.check(b.decode())


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_equal_logical_caches_give_equal_bits(kv):
    a = Batch([700, 65], [9, 30], kv=kv, seed=21, heads=40)
    o, lse = a.decode()
    for _ in range(3):
        again = a.decode()
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    perm = torch.from_numpy(np.random.default_rng(0).permutation(a.cache.num_blocks)).cuda()
    for x in (a.cache.kv_pool, a.cache.kr_pool, a.cache.kv_scale):
        if x is not None:
            x[perm] = x.clone()
    a.table.copy_(torch.where(a.table >= 0, perm.int()[a.table.clamp(min=0).long()], a.table))
    again = a.decode()
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


def test_a_chain_is_what_mla_decode_computes():
    """A chain of nodes is mla_decode's causal queries; both kernels' own bounds between them."""
    b = Batch([333, 1000], [2, 2], chain=True, seed=6)
    o, lse = b.decode()
    o2, lse2 = b.layer.decode(b.cache, b.q, b.table, b.lens, 2, b.max_len)
    for s in range(2):
        t, (ro, rl, size, reach) = b.reference(s)
        bound = 2 * R.o_bound(ro, size, reach, b.row, False, True)
        assert ((o[t].double() - o2[t].double()).abs() <= bound).all()
        assert ((lse[t] - lse2[t]).abs() <= 2 * R.lse_bound(rl, reach, b.row)).all()


def test_other_streams_and_a_captured_step():
    """The calls run on the stream that they are given, and a captured step replays on new inputs."""
    b = Batch([100, 640, 31], [6, 4, 9], heads=32, seed=15)
    want, want_lse = b.decode()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    with torch.cuda.stream(s):
        b.layer.decode_tree(b.cache, b.q, b.table, b.lens, b.trees, b.max_len, o_lat=o, lse=lse)
    s.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    g = torch.cuda.CUDAGraph()
    q = b.q.clone()
    b.trees.prepare(b.lens)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        b.trees.prepare(b.lens)
        b.layer.decode_tree(b.cache, q, b.table, b.lens, b.trees, b.max_len, o_lat=o, lse=lse)
    o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    q.copy_(b.q.flip(0))
    b.lens.copy_(dev([90, 644, 40]))                                # fewer committed tokens too
    g.replay()
    torch.cuda.synchronize()
    b.q, b.ctx = q, np.array([84, 640, 31])
    b.check((o, lse))


@pytest.mark.parametrize("flags", [0, 1])
def test_every_fp8_code(flags):
    """All 256 codes, denormals among them, exactly; a NaN code reaches who sees it."""
    b = Batch([250], [6], kv="fp8", flags=flags, heads=24, seed=31)
    codes = torch.arange(256, device="cuda", dtype=torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0
    rows = torch.stack([codes.roll(7 * i) for i in range(256)])
    j = torch.arange(256, device="cuda")
    b.cache.kv_pool[b.owned[0][j // 64], j % 64] = torch.cat([rows, rows.flip(1)], 1)
    b.cache.kv_scale[b.owned[0][j // 64], j % 64] = torch.rand(256, device="cuda") * 0.02 + 1e-4
    b.check(b.decode())
    b.cache.kv_pool[b.owned[0][0], 5, 77] = 0xFF
    o, lse = b.decode()
    assert torch.isnan(o).all() and torch.isnan(lse).all()
    b.cache.kv_pool[b.owned[0][0], 5, 77] = 3
    for bad in (float("nan"), float("inf")):
        b.cache.kv_scale[b.owned[0][252 // 64], 252 % 64] = bad          # node 2: its descendants alone
        o, lse = b.decode()
        sees = torch.from_numpy(b.see[0][:, 2]).cuda()
        assert torch.isfinite(o[~sees]).all()
        # an infinite scale makes the score +inf or -inf, by the sign of q . code: weight NaN, or 0 and no part of o
        assert not torch.isfinite(lse[sees]).any() if bad != bad else not torch.isfinite(lse[sees]).all()
    no_error()


# ---- FP8 on the tensor cores: query parts and fp16 weights -----------------------------------------

def test_fp8_scales_far_apart():
    """Tokens' scales over 2^40 within a page, some of them 0, under flat weights; the largest float in
    the scale of drafted tokens reaches only the nodes that see them."""
    b = Batch([500, 90], [9, 4], kv="fp8", heads=24, seed=41)
    b.q[:, ::2, :512] = 0                                            # weights by the RoPE part alone
    b.q[:, 1::2] *= 2.0 ** -12
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    for s in range(2):
        j = torch.arange(int(b.ctx[s] + b.n[s]), device="cuda")
        at = b.owned[s][j // 64], j % 64
        b.cache.kv_scale[at] *= 2.0 ** torch.randint(-20, 21, (len(j),), generator=g, device="cuda").float()
        b.cache.kv_scale[at[0][::7], at[1][::7]] = 0
    o, lse = b.decode()
    b.check((o, lse))
    # in each segment the error is counted against the row's own largest weight times scale
    for s in range(2):
        L = int(b.ctx[s] + b.n[s])
        at = b.owned[s][torch.arange(L, device="cuda") // 64], torch.arange(L, device="cuda") % 64
        rows = R.cache_rows(b.cache.kv_pool, b.cache.kr_pool, b.cache.kv_scale, b.table[s], L, 64)
        t, (ro, rl, size, reach) = b.reference(s)
        see = np.concatenate([np.ones((b.n[s], b.ctx[s]), dtype=bool), b.see[s]], 1)
        ds, da = R.fp8_terms(b.q[t], b.cache.kv_pool[at], b.cache.kv_scale[at], torch.from_numpy(see).cuda(), 512, b.scale)
        for i in range(int(b.n[s])):
            m = torch.from_numpy(see[i]).cuda()
            p = torch.softmax(b.q[t[i]].double() @ rows[m].T * b.scale, -1)
            largest = (p * b.cache.kv_scale[at][m].double()).amax(-1)
            bound = R.o_bound(ro[i], size[i], reach[i], b.row, False, True) + 2 * size[i] * ds[i][:, None] + da[i] * largest[:, None]
            assert ((o[t[i]].double() - ro[i]).abs() <= bound).all()
    slot = int(b.ctx[0]) + 3
    b.cache.kv_scale[b.owned[0][slot // 64], slot % 64] = torch.finfo(torch.float32).max
    o2, lse2 = b.decode()
    sees = torch.from_numpy(np.concatenate([b.see[0][:, 3], np.zeros(4, dtype=bool)])).cuda()
    assert torch.equal(o2[~sees], o[~sees]) and torch.equal(lse2[~sees], lse[~sees])
    no_error()


def test_fp8_queries_with_one_large_element():
    b = Batch([700, 3], [5, 8], kv="fp8", heads=40, seed=43)
    b.q[:, :, 17] *= 1000
    b.q[0, 3, :512] = 0
    b.q[1, :, :512] *= 2.0 ** -40                                    # content far below the RoPE part, and far above
    b.q[2, :, :512] *= 2.0 ** 10
    b.q[3, :, 512:] = 0
    b.check(b.decode())


@pytest.mark.parametrize("kv,flags", [("bf16", 0), ("fp8", 0), ("bf16", 1), ("fp8", 1)])
@pytest.mark.parametrize("ctx", [40, 2000])                          # in one run, and joined from several
@pytest.mark.parametrize("column", [5, 530])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite_stays_in_its_row(kv, flags, ctx, column, value):
    b = Batch([ctx], [4], kv=kv, heads=16, flags=flags, seed=47)
    good, good_lse = b.decode()
    b.q[2, 7, column] = value
    o, lse = b.decode()
    assert torch.isnan(o[2, 7]).all() and not torch.isfinite(lse[2, 7])
    others = torch.ones(4, 16, dtype=torch.bool, device="cuda")
    others[2, 7] = False
    assert torch.equal(o[others], good[others]) and torch.equal(lse[others], good_lse[others])
    no_error()


# ---- larger work: several tiles and runs a pair, many sequences, many segments ----------------------

@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("ctx,n,heads", [([3000, 2100, 700, 2900], [40, 17, 33, 64], 128), ([4000] * 6, [5, 9, 2, 7, 1, 3], 128),
                                         ([20000, 5], [3, 200], 16), ([33000, 17001, 16500], [4, 1, 6], 128),
                                           ([65535], [2], 64)])
def test_many_units_a_pair(kv, ctx, n, heads):
    b = Batch(ctx, n, heads=heads, kv=kv, seed=51)
    first = b.decode("bf16")
    b.check(first, "bf16", sample=3)
    for _ in range(3):
        again = b.decode("bf16")
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


@pytest.mark.parametrize("kv,flags", [("bf16", 0), ("fp8", 0), ("bf16", 1)])
def test_more_sequences_than_a_block_has_threads(kv, flags):
    """1100 sequences, some without nodes, one with a bad length."""
    from mla_latent_kv_mqa_b200 import native as N
    rng = np.random.default_rng(5)
    n = rng.integers(0, 4, 1100)
    n[[0, 511, 512, 1099]] = [1, 0, 2, 3]
    b = Batch(rng.integers(0, 130, 1100), n, heads=3, kv=kv, flags=flags, seed=53)
    o, lse = b.decode()
    keep_B, b.B = b.B, 40                                            # the whole batch against the plain form takes minutes
    b.check((o, lse))
    b.B = keep_B
    for s in (511, 512, 513, 700, 1098, 1099):
        if b.n[s]:
            t, (ro, rl, size, reach) = b.reference(s)
            bound = R.o_bound(ro, size, reach, b.row, False, b.tensor_core())
            if kv == "fp8":
                bound = bound + 2 * size * b.extra[0][..., None] + b.extra[1]
            assert ((o[t].double() - ro).abs() <= bound).all()
    b.lens[600] = -1
    n600 = slice(int(b.cu[600]), int(b.cu[601]))
    o2, lse2 = b.decode()
    if b.n[600]:
        assert N.mla_get_last_device_error() == N.MLA_ERR_BAD_SEQ_LEN
        o[n600], lse[n600] = 0, float("-inf")
    assert torch.equal(o2, o) and torch.equal(lse2, lse)


@pytest.mark.parametrize("kv,act,shape,L", [("f32", "f32", TOY, 4000), ("bf16", "bf16", (128, 256, 32), 3100)])
def test_a_long_context_of_other_shapes(kv, act, shape, L):
    """More segments than a cluster joins."""
    b = Batch([L], [1], kv=kv, act=act, shape=shape, heads=2, seed=57)
    b.check(b.decode())


def test_two_streams_at_once_and_a_workspace_that_grows():
    """Calls of one layer on two streams have a workspace each; a captured graph keeps the one it was captured with."""
    a = Batch([900, 300], [6, 4], heads=32, seed=61)
    c = Batch([3000, 2000, 1000], [30, 20, 10], heads=32, seed=62)
    c.layer = a.layer
    want_a, want_c = a.decode(), c.decode()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for k in range(6):
        with torch.cuda.stream(streams[k & 1]):
            x = (a, c)[k & 1]
            got.append((x, x.layer.decode_tree(x.cache, x.q, x.table, x.lens, x.trees, x.max_len)))
    torch.cuda.synchronize()
    for x, (o, lse) in got:
        want = want_a if x is a else want_c
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    s = torch.cuda.Stream()
    o, lse = torch.zeros_like(want_a[0]), torch.zeros_like(want_a[1])
    with torch.cuda.stream(s):
        a.layer.decode_tree(a.cache, a.q, a.table, a.lens, a.trees, a.max_len, o_lat=o, lse=lse)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            a.layer.decode_tree(a.cache, a.q, a.table, a.lens, a.trees, a.max_len, o_lat=o, lse=lse)
        c.layer.decode_tree(c.cache, c.q, c.table, c.lens, c.trees, c.max_len)   # a larger workspace on the same stream
        junk = [torch.full((1 << 22,), float("nan"), device="cuda") for _ in range(8)]
        o.zero_()
        g.replay()
    s.synchronize()
    del junk
    assert torch.equal(o, want_a[0]) and torch.equal(lse, want_a[1])
    no_error()


@pytest.mark.parametrize("cu,rows", [([0, 40, 43], range(0, 40)), ([3, 5, 43], range(0, 5)), ([0, 2, 60], range(2, 43))])
def test_prepare_leaves_no_place_in_the_rows_of_what_is_no_tree(cu, rows):
    """More nodes than the mask has bits, rows before the first, rows behind the last: the rows' sequence is none,
    whatever an earlier step left there, so that an append goes nowhere."""
    from mla_latent_kv_mqa_b200 import native as N, tree as T
    trees = T.DraftTrees(dev(cu), dev(np.full(43, -1)), 32)
    for x in (trees.seq_idx, trees.slot, trees.pos):
        x.fill_(1)
    trees.prepare(dev([100, 100]))
    torch.cuda.synchronize()
    assert N.mla_get_last_device_error() == N.MLA_ERR_BAD_TREE
    assert (trees.seq_idx.cpu().numpy()[list(rows)] == -1).all()
