"""Speculative decoding with drafted trees, and the pages of the latent cache: what is measured, and the plain forms.

Four passes over the paged latent cache, each as a serving loop makes it:

  decode   absorbed attention of every node of a drafted tree over the cache: all committed tokens, and of the drafted ones the
           node's ancestors and itself
  verify   the tree's masks, slots and positions from its parents, its rows into the cache, and after verification the accepted
           path's rows moved up behind the committed ones
  fork     sequences that share their parents' pages, grown by a few tokens: pages allotted, shared last pages copied
  compact  sequences cut short, their pages freed, and the pages in use moved to the front of the pool
"""
import numpy as np
import torch

own = False

PAGE = 64
V3 = {"d_h": 128, "d_c": 512, "d_r": 64}
TOY = {"d_h": 64, "d_c": 128, "d_r": 32}
BASE = 1e4


# ---- the cases -----------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # The toy layer in fp32, one short sequence, five drafted tokens: the smallest call, where latency counts.
        {"name": "decode toy f32", "op": "decode", "kv": "f32", "heads": 8, "B": 1, "lo": 251, "hi": 251, "n_lo": 5, "n_hi": 5},
        # A tensor-parallel rank of eight (16 of 128 heads), a few sequences of chat length.
        {"name": "decode 16 heads", "op": "decode", "kv": "bf16", "heads": 16, "B": 8, "lo": 300, "hi": 2500, "n_lo": 7, "n_hi": 16},
        # The variable-length batch, each sequence with a tree of its own size.
        {"name": "decode ragged", "op": "decode", "kv": "bf16", "heads": 128, "B": 24, "lo": 1024, "hi": 8190, "n_lo": 3, "n_hi": 24},
        # The FP8 cache at the speculative-decoding workload's context.
        {"name": "decode fp8", "op": "decode", "kv": "fp8", "heads": 128, "B": 32, "lo": 4097, "hi": 8192, "n_lo": 2, "n_hi": 12},
        # The long-context workload: few sequences, the work split along the context.
        {"name": "decode long", "op": "decode", "kv": "bf16", "heads": 128, "B": 4, "lo": 131072, "hi": 131072, "n_lo": 4, "n_hi": 4},
        # Large trees for a full batch: compute-bound.
        {"name": "decode 64 nodes", "op": "decode", "kv": "bf16", "heads": 128, "B": 16, "lo": 6000, "hi": 8192, "n_lo": 64, "n_hi": 64},
        # One layer's rows of a batch's drafted trees.
        {"name": "verify bf16", "op": "verify", "kv": "bf16", "layers": 1, "B": 16, "lo": 200, "hi": 1500, "n_lo": 9, "n_hi": 32},
        # The FP8 cache, several layers behind one table, large batch.
        {"name": "verify fp8", "op": "verify", "kv": "fp8", "layers": 4, "B": 128, "lo": 100, "hi": 1000, "n_lo": 4, "n_hi": 16},
        # Parallel samples of a few prompts: each prompt's pages shared by its samples.
        {"name": "fork few", "op": "fork", "kv": "bf16", "layers": 2, "B": 6, "width": 3, "lo": 90, "hi": 1800, "spare": 60},
        # Beams of a large batch, the next tokens' pages allotted in every layer.
        {"name": "fork beams", "op": "fork", "kv": "bf16", "layers": 12, "B": 64, "width": 4, "lo": 130, "hi": 2050, "spare": 700},
        # A small pool with an FP8 cache after some sequences ended.
        {"name": "compact fp8", "op": "compact", "kv": "fp8", "layers": 2, "B": 12, "lo": 60, "hi": 1500, "spare": 33},
        # A large pool: half of its sequences ended or were cut, the rest is moved together.
        {"name": "compact large", "op": "compact", "kv": "bf16", "layers": 8, "B": 96, "lo": 700, "hi": 4100, "spare": 200},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["decode", "decode", "decode", "verify", "fork", "compact"])
    if op == "decode":
        kv = rng.choice(["bf16", "bf16", "fp8", "f32"])
        if kv == "f32":
            lo = log(1, 500)
            return {"op": op, "kv": kv, "heads": 8, "B": log(1, 8), "lo": lo, "hi": lo + log(1, 500), "n_lo": 1, "n_hi": log(1, 32)}
        heads = rng.choice([8, 16, 20, 32, 64, 128, 128])
        B, n_hi = log(1, 48), log(1, 64)
        most = min(40000, int(0.9e9 / (B * n_hi * heads)))
        hi = log(40, max(80, most))
        return {"op": op, "kv": kv, "heads": heads, "B": B, "lo": max(1, int(hi * rng.random())), "hi": hi, "n_lo": max(1, n_hi // 3), "n_hi": n_hi}
    kv = rng.choice(["bf16", "bf16", "fp8"])
    if op == "verify":
        n_hi = log(2, 64)
        lo = log(1, 800)
        return {"op": op, "kv": kv, "layers": rng.randint(1, 4), "B": log(1, 128), "lo": lo, "hi": lo + log(1, 800), "n_lo": max(1, n_hi // 4), "n_hi": n_hi}
    B, lo = log(1, 64), log(1, 1500)
    case = {"op": op, "kv": kv, "layers": rng.randint(1, 6), "B": B, "lo": lo, "hi": lo + log(1, 1500)}
    if op == "fork":
        case["width"] = rng.randint(1, 4)
        case["spare"] = 3 * B * (case["width"] + 1) + log(1, 100)
    else:
        case["spare"] = log(1, 200)
    return case


def _spread(B, lo, hi, step):
    """B whole numbers from lo to hi, hi first, the others spread evenly over the range in no order."""
    b = np.arange(B)
    v = lo + np.floor((hi - lo + 1) * ((b * step) % 1.0)).astype(np.int64)
    return np.where(b == 0, hi, np.minimum(v, hi))


def _sizes(case):
    """(committed tokens, drafted nodes) of every sequence, from the case alone."""
    B = case["B"]
    ctx = _spread(B, case["lo"], case["hi"], 0.6180339887498949)
    n = _spread(B, case["n_lo"], case["n_hi"], 0.4142135623730950) if "n_lo" in case else np.zeros(B, dtype=np.int64)
    return ctx, n


def _dims(case):
    return TOY if case["kv"] == "f32" else V3


def _row_bytes(case):
    d = _dims(case)
    return d["d_c"] + 2 * d["d_r"] + 4 if case["kv"] == "fp8" else (d["d_c"] + d["d_r"]) * (4 if case["kv"] == "f32" else 2)


# ---- inputs --------------------------------------------------------------------------------------------------------------------

def _pool(g, layers, blocks, kv, d):
    """A cache's pages in `layers` layers, every slot filled: FP8 as codes, keys and scales, each [layers, blocks, page, ...]."""
    if kv != "fp8":
        dt = torch.float32 if kv == "f32" else torch.bfloat16
        return {"kv": torch.randn(layers, blocks, PAGE, d["d_c"] + d["d_r"], generator=g, device="cuda", dtype=dt), "kr": None, "scale": None}
    c = torch.randn(layers, blocks, PAGE, d["d_c"], generator=g, device="cuda")
    s = c.abs().amax(-1) / 448
    return {"kv": (c / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8),
            "kr": torch.randn(layers, blocks, PAGE, d["d_r"], generator=g, device="cuda", dtype=torch.bfloat16), "scale": s}


def _table(rng, lens, blocks, rows, width):
    """A block table of `rows` rows: pages of a shuffled pool for the first len(lens) of them, -1 elsewhere."""
    pages = -(-lens // PAGE)
    ids = rng.permutation(blocks).astype(np.int32)
    bt = np.full((rows, width), -1, dtype=np.int32)
    at = np.arange(width)[None, :] < pages[:, None]
    bt[:len(lens)][at] = ids[:int(pages.sum())]
    return bt


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    d, op = _dims(case), case["op"]
    st = {"op": op, "kv": case["kv"], "d": d, "layers": case.get("layers", 1)}
    ctx, n = _sizes(case)
    B = case["B"]
    act = torch.float32 if case["kv"] == "f32" else torch.bfloat16
    if op in ("decode", "verify"):
        lens = ctx + n
        T = int(n.sum())
        cu = np.concatenate([[0], np.cumsum(n)])
        within = np.arange(T) - np.repeat(cu[:-1], n)
        parent = np.floor(rng.random(T) * (within + 1)).astype(np.int64) - 1  # any earlier node, or -1: a child of the last committed token
        blocks = int((-(-lens // PAGE)).sum()) + 3
        st.update(table=_i32(_table(rng, lens, blocks, B, int(-(-lens.max() // PAGE)))), lens=_i32(lens), cu=_i32(cu), parent=_i32(parent),
                  max_len=int(lens.max()), max_nodes=int(n.max()), nodes=T, B=B, pool=_pool(g, st["layers"], blocks, case["kv"], d))
        path = [[] for _ in range(B)]
        mask = np.zeros((T, -(-st["max_nodes"] // 32)), dtype=np.uint32)
        for b in range(B):
            p = parent[cu[b]:cu[b + 1]]
            see = np.zeros((n[b], n[b]), dtype=bool)
            for i in range(n[b]):
                if p[i] >= 0:
                    see[i] = see[p[i]]
                see[i, i] = True
            path[b] = np.nonzero(see[rng.integers(n[b])])[0]
            bits = np.zeros((n[b], 32 * mask.shape[1]), dtype=np.uint32)
            bits[:, :n[b]] = see
            mask[cu[b]:cu[b + 1]] = (bits.reshape(n[b], -1, 32) << np.arange(32, dtype=np.uint32)).sum(-1, dtype=np.uint32)
        if op == "decode":
            H = st["heads"] = case["heads"]
            q = torch.randn(T, H, d["d_c"] + d["d_r"], generator=g, device="cuda")
            q[..., :d["d_c"]] *= (d["d_h"] / d["d_c"]) ** 0.5  # W_UK ~ N(0, 1/d_c) on q_c ~ N(0, 1)
            st.update(q=q.to(act), mask=torch.from_numpy(mask.view(np.int32)).cuda())
        else:
            keep = np.zeros((B, max(len(p) for p in path)), dtype=np.int64)
            for b in range(B):
                keep[b, :len(path[b])] = path[b]
            st.update(keep=_i32(keep), num_keep=_i32([len(p) for p in path]),
                      c=torch.randn(st["layers"], T, d["d_c"], generator=g, device="cuda", dtype=act),
                      k=torch.randn(st["layers"], T, d["d_r"], generator=g, device="cuda", dtype=act))
        return st
    pages = -(-ctx // PAGE)
    blocks = int(pages.sum()) + case["spare"]
    width = int(pages.max()) + 2
    if op == "fork":
        W = case["width"]
        rows = B * (W + 1)
        parent = np.repeat(np.arange(B), W)
        child = B + rng.permutation(B * W)
        lens = np.zeros(rows, dtype=np.int64)
        lens[:B] = ctx
        new = lens.copy()
        new[:B] = np.where(rng.random(B) < 0.3, ctx, ctx + rng.integers(1, 40, B))  # a parent that stays as it is keeps its last page: every child copies
        new[child] = ctx[parent] + rng.integers(1, 40, B * W)
        st.update(parent=_i32(parent), child=_i32(child), new=_i32(new))
    else:
        rows = B
        lens = ctx
        kind = rng.random(B)
        new = np.where(kind < 0.4, 0, np.where(kind < 0.6, np.floor(lens * rng.random(B)).astype(np.int64), lens))
        st.update(new=_i32(new))
    table = _table(rng, ctx, blocks, rows, width)
    refs = np.zeros(blocks, dtype=np.int64)
    refs[table[table >= 0]] = 1
    st.update(table=_i32(table), refs=_i32(refs), lens=_i32(lens), rows=rows, blocks=blocks, width=width, pool=_pool(g, st["layers"], blocks, case["kv"], d))
    return st


# ---- the framework's own operators -----------------------------------------------------------------------------------------------

def _handles(st):
    """What a user's program keeps: the layer, its caches over the pool's tensors, the trees or the page table."""
    from mla_latent_kv_mqa_b200 import layer as L, pages as P, tree as R
    d, pool = st["d"], st["pool"]
    kv = st["kv"]
    dims = L.dims_for(st.get("heads", 128), d["d_h"], d["d_c"], d["d_r"], act="f32" if kv == "f32" else "bf16", kv=kv, page=PAGE, rope_base=BASE)
    w = torch.zeros(dims.n_h * dims.d_h, dims.d_c, dtype=torch.float32 if kv == "f32" else torch.bfloat16, device="cuda")
    caches = [L.PagedLatentCache.over(dims, pool["kv"][i], None if pool["kr"] is None else pool["kr"][i],
                                      None if pool["scale"] is None else pool["scale"][i]) for i in range(st["layers"])]
    h = {"layer": L.MLADecodeLayer(dims, w, w), "caches": caches}
    if st["op"] in ("decode", "verify"):
        h["trees"] = R.DraftTrees(st["cu"], st["parent"], st["max_nodes"], mask=st.get("mask"))
    else:
        h["seqs"] = P.PagedSequences(PAGE, st["rows"], st["width"], st["blocks"])
    return h


def _own(st):
    if "h" not in st:
        st["h"] = _handles(st)
    h = st["h"]
    if st["op"] == "decode":
        out = "f32" if st["kv"] == "f32" else "bf16"
        return h["layer"].decode_tree(h["caches"][0], st["q"], st["table"], st["lens"], h["trees"], st["max_len"], out_dtype=out)
    if st["op"] == "verify":
        trees, layer = h["trees"], h["layer"]
        trees.prepare(st["lens"])
        [layer.tree_append(cache, c, k, trees, st["table"]) for cache, c, k in zip(h["caches"], st["c"], st["k"])]
        new = trees.keep(h["caches"], st["table"], st["lens"], st["keep"], st["num_keep"])
        return {"mask": trees.mask, "pos": trees.pos, "slot": trees.slot, "new": new, **_whole(st)}
    seqs = h["seqs"]
    seqs.block_table.copy_(st["table"])
    seqs.refs.copy_(st["refs"])
    seqs.seq_lens.copy_(st["lens"])
    if st["op"] == "fork":
        seqs.fork(st["parent"], st["child"])
        moves = seqs.grow(st["new"])
    else:
        seqs.trim(st["new"])
        moves = seqs.compact()
    seqs.copy_pages(h["caches"], moves)
    return {"table": seqs.block_table, "refs": seqs.refs, "lens": seqs.seq_lens, **_whole(st)}


def _whole(st):
    p = st["pool"]
    if st["kv"] != "fp8":
        return {"kv": p["kv"]}
    return {"kv": p["kv"].view(torch.float8_e4m3fn), "kr": p["kr"], "scale": p["scale"]}


# ---- the plain forms -------------------------------------------------------------------------------------------------------------

def _decode(st):
    d, dc = st["d"], st["d"]["d_c"]
    pool, table, lens, cu = st["pool"], st["table"].long(), st["lens"].long(), st["cu"].long()
    dev = table.device
    n = cu[1:] - cu[:-1]
    ctx = lens - n
    j = torch.arange(st["max_len"], device=dev)
    at = table.clamp(min=0)[:, j // PAGE]                                     # page of every token [B, L]
    rows = pool["kv"][0][at, j % PAGE].float() if st["kv"] != "fp8" else torch.cat(
        [pool["kv"][0].view(torch.float8_e4m3fn)[at, j % PAGE].float() * pool["scale"][0][at, j % PAGE][..., None], pool["kr"][0][at, j % PAGE].float()], -1)
    rows = rows * (j < lens[:, None])[..., None]
    i = torch.arange(st["max_nodes"], device=dev)
    t = (cu[:-1, None] + i).clamp(max=st["nodes"] - 1)                        # row of every node [B, n]
    node = j - ctx[:, None]                                                    # the drafted node a token is, negative: committed [B, L]
    word = st["mask"].long()[t]                                                # [B, n, words]
    bit = torch.gather(word, 2, (node.clamp(min=0) // 32).clamp(max=word.shape[2] - 1)[:, None].expand(-1, st["max_nodes"], -1))
    see = ((bit >> (node.clamp(min=0) % 32)[:, None]) & 1).bool()
    see = ((node < 0)[:, None] | see) & (j < lens[:, None])[:, None]           # [B, n, L]
    B, H = table.shape[0], st["heads"]
    q = st["q"][t].float().reshape(B, -1, d["d_c"] + d["d_r"])                 # [B, n H, row]
    s = torch.bmm(q, rows.transpose(1, 2)).mul_((d["d_h"] + d["d_r"]) ** -0.5).view(B, st["max_nodes"], H, -1)
    s.masked_fill_(~see[:, :, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(B, -1, p.shape[-1]), rows[..., :dc]).view(B, st["max_nodes"], H, dc)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (total.log() + top)[..., 0]
    own_row = i < n[:, None]
    return o[own_row].to(torch.float32 if st["kv"] == "f32" else torch.bfloat16), lse[own_row]


def _tree(parent, within, first, words, most):
    """Ancestors and itself as bits, and the number of ancestors, of every node: the parents' links followed at most `most` times."""
    T = parent.shape[0]
    up = torch.where(parent >= 0, first + parent, torch.full_like(parent, T))
    up = torch.cat([up, up.new_full((1,), T)])                                 # T: above the roots
    reach = torch.zeros(T + 1, 32 * words, dtype=torch.bool, device=parent.device)
    reach[torch.arange(T, device=parent.device), within] = True
    hops = max(1, (most - 1).bit_length())
    depth = (up < T).long()
    jump = up
    for _ in range(hops):                                                      # doubled links: 1, 2, 4, ... steps at a time
        reach = reach | (reach[jump] & (jump < T)[:, None])
        depth = depth + torch.where(jump < T, depth[jump], torch.zeros_like(depth))
        jump = jump[jump]
    bits = reach[:T].view(T, words, 32).long() << torch.arange(32, device=parent.device)
    word = bits.sum(-1)
    return torch.where(word >= 2 ** 31, word - 2 ** 32, word).int(), depth[:T]


def _rope(k, pos, d_r):
    """Half-split rotation of k [..., T, d_r] by angles pos * BASE^(-2i/d_r), in 64 bits."""
    half = d_r // 2
    a = pos.double()[:, None] * BASE ** (-2.0 * torch.arange(half, device=k.device, dtype=torch.float64) / d_r)
    x, y = k[..., :half].double(), k[..., half:].double()
    return torch.cat([x * a.cos() - y * a.sin(), y * a.cos() + x * a.sin()], -1).float()


def _verify(st):
    d, pool, table, lens, cu = st["d"], st["pool"], st["table"].long(), st["lens"].long(), st["cu"].long()
    dev = table.device
    n = cu[1:] - cu[:-1]
    ctx = lens - n
    seq = torch.repeat_interleave(torch.arange(st["B"], device=dev), n, output_size=st["nodes"])
    first = cu[:-1][seq]
    within = torch.arange(st["nodes"], device=dev) - first
    mask, depth = _tree(st["parent"].long(), within, first, -(-st["max_nodes"] // 32), st["max_nodes"])
    slot, pos = ctx[seq] + within, ctx[seq] + depth
    page, off = table[seq, slot // PAGE], slot % PAGE
    k = _rope(st["k"], pos, d["d_r"])
    if st["kv"] == "fp8":
        c = st["c"].float()
        top = c.abs().amax(-1)
        scale = torch.where(top > 0, (top / 448).clamp(min=torch.finfo(torch.float32).tiny), torch.ones_like(top))
        code = (c / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        pool["kv"][:, page, off] = code
        pool["kr"][:, page, off] = k.to(torch.bfloat16)
        pool["scale"][:, page, off] = scale
    else:
        pool["kv"][:, page, off] = torch.cat([st["c"].float(), k], -1).to(pool["kv"].dtype)
    keep, num = st["keep"].long(), st["num_keep"].long()
    i = torch.arange(keep.shape[1], device=dev)
    row, col = torch.nonzero(i < num[:, None], as_tuple=True)
    src, dst = ctx[row] + keep[row, col], ctx[row] + col
    sp, so, dp, do = table[row, src // PAGE], src % PAGE, table[row, dst // PAGE], dst % PAGE
    pool["kv"][:, dp, do] = pool["kv"][:, sp, so]
    if st["kv"] == "fp8":
        pool["kr"][:, dp, do] = pool["kr"][:, sp, so]
        pool["scale"][:, dp, do] = pool["scale"][:, sp, so]
    return {"mask": mask, "pos": pos.int(), "slot": slot.int(), "new": (ctx + num).int(), **_whole(st)}


def _copy(st, src, dst):
    p = st["pool"]
    p["kv"][:, dst] = p["kv"][:, src]
    if st["kv"] == "fp8":
        p["kr"][:, dst] = p["kr"][:, src]
        p["scale"][:, dst] = p["scale"][:, src]


def _fork(st):
    table, refs, lens = st["table"].long(), st["refs"].long(), st["lens"].long()
    parent, child, new = st["parent"].long(), st["child"].long(), st["new"].long()
    dev = table.device
    p = torch.arange(st["width"], device=dev)
    # every parent's row is read before any child's is written
    rows = torch.where(p < -(-lens[parent] // PAGE)[:, None], table[parent], torch.full_like(table[parent], -1))
    old = table[child]
    refs = refs + torch.bincount(rows[rows >= 0], minlength=st["blocks"]) - torch.bincount(old[old >= 0], minlength=st["blocks"])
    table[child] = rows
    lens[child] = lens[parent]
    # grow: a last page that is not full and shared is replaced by a copy, except for the last of its sharers
    grows = new > lens
    slot = lens // PAGE
    part = grows & (lens % PAGE != 0)
    page = table[torch.arange(st["rows"], device=dev), slot.clamp(max=st["width"] - 1)].clamp(min=0)
    here = torch.bincount(page[part], minlength=st["blocks"])
    last = torch.full((st["blocks"],), -1, device=dev).scatter_reduce(0, page, torch.where(part, torch.arange(st["rows"], device=dev), -1), "amax")
    copies = part & ((here[page] < refs[page]) | (last[page] != torch.arange(st["rows"], device=dev)))
    need = (grows[:, None] & (p >= -(-lens // PAGE)[:, None]) & (p < -(-new // PAGE)[:, None])) | (copies[:, None] & (p == slot[:, None]))
    r, c = torch.nonzero(need, as_tuple=True)
    got = torch.nonzero(refs == 0)[:r.shape[0], 0]
    was = table[r, c]
    table[r, c] = got
    refs = refs - torch.bincount(was[was >= 0], minlength=st["blocks"])
    refs[got] = 1
    _copy(st, was[was >= 0], got[was >= 0])
    return {"table": table.int(), "refs": refs.int(), "lens": torch.maximum(new, lens).int(), **_whole(st)}


def _compact(st):
    table, refs, lens, new = st["table"].long(), st["refs"].long(), st["lens"].long(), st["new"].long()
    p = torch.arange(st["width"], device=table.device)
    goes = (p >= -(-new // PAGE)[:, None]) & (table >= 0)
    refs = refs - torch.bincount(table[goes], minlength=st["blocks"])
    table = torch.where(goes, torch.full_like(table, -1), table)
    used = refs > 0
    front = torch.arange(st["blocks"], device=table.device) < used.sum()
    src, dst = torch.nonzero(used & ~front)[:, 0], torch.nonzero(~used & front)[:, 0]
    to = torch.arange(st["blocks"], device=table.device)
    to[src] = dst
    table = torch.where(table >= 0, to[table.clamp(min=0)], table)
    refs[dst] = refs[src]
    refs[src] = 0
    _copy(st, src, dst)
    return {"table": table.int(), "refs": refs.int(), "lens": torch.minimum(lens, new).int(), **_whole(st)}


def run(st):
    if own:
        return _own(st)
    return {"decode": _decode, "verify": _verify, "fork": _fork, "compact": _compact}[st["op"]](st)


# ---- work, and the definition in 64 bits -----------------------------------------------------------------------------------------

def work(case):
    d, (ctx, n) = _dims(case), _sizes(case)
    row, layers = _row_bytes(case), case.get("layers", 1)
    if case["op"] == "decode":
        H, T, es = case["heads"], int(n.sum()), 4 if case["kv"] == "f32" else 2
        seen = int((n * ctx).sum()) + T  # committed tokens and itself: a tree's ancestors are few
        return {"bytes": int((ctx + n).sum()) * row + T * H * ((d["d_c"] + d["d_r"]) * es + d["d_c"] * es + 4), "flops": 2 * H * seen * (2 * d["d_c"] + d["d_r"])}
    if case["op"] == "verify":
        T = int(n.sum())  # activations read, rows written; a path of about ln n + 1 nodes read and written
        path = int((np.log(n) + 1).sum())
        return {"bytes": layers * (T * ((d["d_c"] + d["d_r"]) * 2 + row) + 2 * path * row) + T * 4 * (4 + -(-int(n.max()) // 32)), "flops": 0}
    pages = -(-ctx // PAGE)
    if case["op"] == "fork":  # a child's last page copied, a page's worth at most for each; the tables and counts
        W = case["width"]
        moved = int((W * (ctx % PAGE != 0)).sum())
        small = 4 * (int(pages.sum()) * (2 * W + 1) + int(pages.sum()) + case["spare"])
    else:  # of the pages in use half lie behind the front part
        moved = int(pages.sum()) // 4
        small = 4 * (3 * int(pages.sum()) + case["spare"])
    return {"bytes": 2 * moved * PAGE * row * layers + small, "flops": 0}


def exact(case, seed):
    st = prepare(case, seed)
    h = {k: v.cpu().numpy().astype(np.int64) for k, v in st.items() if isinstance(v, torch.Tensor) and v.dtype == torch.int32}
    d, pool, op = st["d"], st["pool"], st["op"]
    table, lens = h["table"], h["lens"]
    if op == "decode":
        outs, sums = [], []
        for b in range(case["B"]):
            L = int(lens[b])
            nodes = range(h["cu"][b], h["cu"][b + 1])
            pages = torch.from_numpy(table[b, :-(-L // PAGE)]).cuda()
            c = pool["kv"][0][pages]
            if st["kv"] == "fp8":
                c = torch.cat([c.view(torch.float8_e4m3fn).double() * pool["scale"][0][pages][..., None].double(), pool["kr"][0][pages].double()], -1)
            c = c.double().reshape(-1, d["d_c"] + d["d_r"])[:L]
            first = L - len(nodes)
            for part in range(0, len(nodes), 8):
                rows = list(nodes)[part:part + 8]
                s = torch.einsum("thr,lr->thl", st["q"][rows[0]:rows[-1] + 1].double(), c) / (d["d_h"] + d["d_r"]) ** 0.5
                hide = np.zeros((len(rows), L), dtype=bool)
                for x, t in enumerate(rows):
                    for k in range(len(nodes)):
                        hide[x, first + k] = not (int(h["mask"][t, k // 32]) >> (k % 32)) & 1
                s.masked_fill_(torch.from_numpy(hide).cuda()[:, None], float("-inf"))
                w = torch.logsumexp(s, -1)
                outs.append(torch.einsum("thl,lr->thr", torch.exp(s - w[..., None]), c[:, :d["d_c"]]))
                sums.append(w)
        return torch.cat(outs), torch.cat(sums)
    if op == "verify":
        T = st["nodes"]
        mask, pos, slot = np.zeros((T, -(-st["max_nodes"] // 32)), dtype=np.int64), np.zeros(T, dtype=np.int64), np.zeros(T, dtype=np.int64)
        page = np.zeros(T, dtype=np.int64)
        moves = []
        new = np.zeros(case["B"], dtype=np.int64)
        for b in range(case["B"]):
            lo, hi = h["cu"][b], h["cu"][b + 1]
            first = lens[b] - (hi - lo)
            for t in range(lo, hi):
                k, depth = t - lo, 0
                mask[t, k // 32] |= 1 << (k % 32)
                while h["parent"][lo + k] >= 0:
                    k = h["parent"][lo + k]
                    depth += 1
                    mask[t, k // 32] |= 1 << (k % 32)
                pos[t], slot[t] = first + depth, first + t - lo
                page[t] = table[b, slot[t] // PAGE]
            for k in range(h["num_keep"][b]):
                s, e = first + h["keep"][b, k], first + k
                moves.append((table[b, s // PAGE], s % PAGE, table[b, e // PAGE], e % PAGE))
            new[b] = first + h["num_keep"][b]
        half = d["d_r"] // 2
        a = pos[:, None] * BASE ** (-2.0 * np.arange(half) / d["d_r"])
        cs, sn = torch.from_numpy(np.cos(a)).cuda(), torch.from_numpy(np.sin(a)).cuda()
        x, y = st["k"].double()[..., :half], st["k"].double()[..., half:]
        k = torch.cat([x * cs - y * sn, x * sn + y * cs], -1)
        page, slot_t = torch.from_numpy(page).cuda(), torch.from_numpy(slot % PAGE).cuda()
        m = torch.from_numpy(np.array(moves, dtype=np.int64)).cuda().T
        if st["kv"] == "fp8":  # the codes are a decision that the definition takes in 32 bits, scale = amax / 448
            c = st["c"].float()
            scale = c.abs().amax(-1) / 448
            kv, kr, sc = pool["kv"].view(torch.float8_e4m3fn).double(), pool["kr"].double(), pool["scale"].double()
            kv[:, page, slot_t] = (c / scale[..., None]).to(torch.float8_e4m3fn).double()
            kr[:, page, slot_t], sc[:, page, slot_t] = k, scale.double()
            got = {"kv": kv, "kr": kr, "scale": sc}
        else:
            kv = pool["kv"].double()
            kv[:, page, slot_t] = torch.cat([st["c"].double(), k], -1)
            got = {"kv": kv}
        for v in got.values():
            v[:, m[2], m[3]] = v[:, m[0], m[1]]
        return {"mask": torch.from_numpy(mask.astype(np.uint32).view(np.int32)), "pos": torch.from_numpy(pos).int(), "slot": torch.from_numpy(slot).int(),
                "new": torch.from_numpy(new).int(), **got}
    refs, new = h["refs"], h["new"]
    src, dst = [], []
    if op == "fork":
        was, was_lens = table.copy(), lens.copy()
        for i, c in zip(h["parent"], h["child"]):
            table[c], lens[c] = was[i], was_lens[i]
            for p in was[i][was[i] >= 0]:
                refs[p] += 1
        grows = [s for s in range(st["rows"]) if new[s] > lens[s]]
        free = list(np.nonzero(refs == 0)[0])
        for s in grows:
            if lens[s] % PAGE and refs[p := table[s, lens[s] // PAGE]] > 1:
                to = free.pop(0)
                refs[p] -= 1
                refs[to] = 1
                table[s, lens[s] // PAGE] = to
                src.append(p)
                dst.append(to)
            for k in range(-(-lens[s] // PAGE), -(-new[s] // PAGE)):
                table[s, k] = free.pop(0)
                refs[table[s, k]] = 1
            lens[s] = new[s]
    else:
        for s in range(st["rows"]):
            for k in range(-(-new[s] // PAGE), st["width"]):
                if table[s, k] >= 0:
                    refs[table[s, k]] -= 1
                    table[s, k] = -1
            lens[s] = min(lens[s], new[s])
        total = int((refs > 0).sum())
        src = [p for p in range(total, st["blocks"]) if refs[p]]
        dst = [p for p in range(total) if not refs[p]]
        for p, q in zip(src, dst):
            table[table == p] = q
            refs[q], refs[p] = refs[p], 0
    _copy(st, torch.tensor(src, dtype=torch.long, device="cuda"), torch.tensor(dst, dtype=torch.long, device="cuda"))
    return {"table": torch.from_numpy(table).int(), "refs": torch.from_numpy(refs).int(), "lens": torch.from_numpy(lens).int(), **_whole(st)}
