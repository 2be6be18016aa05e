"""Plain forms of the drafted-tree and page operators, in 64 bits and in Python integers, and the
bounds that the arithmetic of the kernels gives."""
from __future__ import annotations

import numpy as np
import torch

EPS_BF16, EPS_F32 = 2.0 ** -8, 2.0 ** -24      # half a step, relative


def trees(rng, sizes, chain=False):
    """(cu, parent) of trees with the given node counts: random parents, or chains."""
    cu = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    parent = [np.arange(n) - 1 if chain else np.array([rng.integers(-1, i) if i else -1 for i in range(n)]) for n in sizes]
    return cu, np.concatenate(parent + [np.zeros(0)]).astype(np.int32)


def sees(parent):
    """[n, n] booleans: node i sees node k (its ancestors and itself); and the depths."""
    n = len(parent)
    see, depth = np.zeros((n, n), dtype=bool), np.zeros(n, dtype=np.int64)
    for i in range(n):
        if parent[i] >= 0:
            see[i] = see[parent[i]]
            depth[i] = depth[parent[i]] + 1
        see[i, i] = True
    return see, depth


def bits(see, words):
    out = np.zeros((see.shape[0], 32 * words), dtype=np.uint32)
    out[:, :see.shape[1]] = see
    return (out.reshape(see.shape[0], words, 32) << np.arange(32, dtype=np.uint32)).sum(-1, dtype=np.uint32).view(np.int32)


def cache_rows(kv, kr, scale, table_row, L, page):
    """Rows 0 .. L-1 of one sequence in float64 [L, d_c + d_r]."""
    j = torch.arange(L, device=kv.device)
    blk = table_row.long()[j // page]
    if kr is None:
        return kv[blk, j % page].double()
    return torch.cat([kv.view(torch.float8_e4m3fn)[blk, j % page].double() * scale[blk, j % page].double()[:, None],
                      kr[blk, j % page].double()], 1)


def attend(q, rows, see, d_c, scale):
    """Attention of q [n, H, row] over rows [L, row] with see [n, L]: (o, lse, sum p |c|, largest
    sum |q c| scale over the tokens seen), masked rows left out whatever they hold."""
    n, H, _ = q.shape
    o = torch.zeros(n, H, d_c, dtype=torch.float64, device=q.device)
    lse = torch.full((n, H), float("-inf"), dtype=torch.float64, device=q.device)
    size, reach = torch.zeros_like(o), torch.zeros_like(lse)
    for i in range(n):
        r = rows[see[i]]
        if not len(r):
            continue
        s = q[i].double() @ r.T * scale
        lse[i] = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[i][:, None])
        o[i], size[i] = p @ r[:, :d_c], p @ r[:, :d_c].abs()
        reach[i] = (q[i].double().abs() @ r.abs().T).amax(-1) * scale
    return o, lse, size, reach


def o_bound(o, size, reach, row, out_bf16, tensor_core, segments=True):
    """|error| of o_lat, element by element.  fp32 products and sums in a score: row + 1 roundings (twice
    that where the tensor core truncates) of terms whose sum of sizes is `reach`, which moves every
    weight by that much, and 2^-21 for each of exp2's approximations; on the tensor core a weight is
    rounded to bf16 once and a segment's sum once more; the output once.  (FP8 there: fp8_terms too.)"""
    ds = (row + 1) * EPS_F32 * 2 * reach
    rel = 2 * ds[..., None] + 2.0 ** -20 + 64 * EPS_F32 + (EPS_BF16 * (2 if segments else 1) if tensor_core else 0)
    return size * rel + (EPS_BF16 if out_bf16 else EPS_F32) * o.abs() + 1e-30


def fp8_terms(q, kv, scale_t, see, d_c, scale):
    """What the tensor-core kernel's formats add over an FP8 cache: (error of a score, absolute error of
    o).  q [n, H, row]; kv, scale_t: codes [L, d_c] and scales [L]; see [n, L].  A query's content element
    is off by 2^-10 where its row's largest is at least 2^7.  A weight times its scale is off by 2^-25 at
    most where fp16 has no 11 bits for it, and the row's largest is 2^2 at least."""
    codes = kv.view(torch.float8_e4m3fn).double()[:, :d_c].abs()
    s = torch.where(torch.isfinite(scale_t), scale_t, 0).double().abs()
    dq = q[..., :d_c].double().abs().amax(-1) * 2.0 ** -17 * scale
    n, H, _ = q.shape
    ds, da = torch.zeros(n, H, dtype=torch.float64, device=q.device), torch.zeros(n, H, d_c, dtype=torch.float64, device=q.device)
    for i in range(n):
        if see[i].any():
            ds[i] = dq[i] * (codes[see[i]].sum(-1) * s[see[i]]).max()
            da[i] = 2.0 ** -27 * codes[see[i]].sum(0)
    return ds, da


def lse_bound(lse, reach, row):
    return (row + 1) * EPS_F32 * 2 * reach + 2.0 ** -19 + 4 * EPS_F32 * lse.abs()


class Pages:
    """mla_pages_* as the header words them, one entry after the other."""

    def __init__(self, page, table, refs, lens):
        self.page, self.table, self.refs, self.lens = page, table.copy(), refs.copy(), lens.copy()

    def n(self, length):
        return -(-int(length) // self.page)

    def fork(self, parent, child):
        table, lens = self.table.copy(), self.lens.copy()
        for s, c in zip(parent, child):
            row = np.full(table.shape[1], -1)
            row[:self.n(lens[s])] = table[s, :self.n(lens[s])]
            for v in row[row >= 0]:
                self.refs[v] += 1
            for v in table[c][table[c] >= 0]:
                self.refs[v] -= 1
            self.table[c], self.lens[c] = row, lens[s]

    def grow(self, new, seqs=None):
        seqs = range(len(new)) if seqs is None else seqs
        keep = self.table.copy(), self.refs.copy(), self.lens.copy()
        moves, free = [], list(np.nonzero(self.refs == 0)[0])
        for s, length in zip(seqs, new):
            cur = int(self.lens[s])
            if length <= cur:
                continue
            want = []
            if cur % self.page and self.refs[self.table[s, cur // self.page]] > 1:
                want.append(cur // self.page)
            want += [k for k in range(self.n(cur), self.n(length)) if self.table[s, k] < 0]
            if len(want) > len(free):
                self.table, self.refs, self.lens = keep
                return None
            for k in want:
                to = free.pop(0)
                if self.table[s, k] >= 0:
                    moves.append((self.table[s, k], to))
                    self.refs[self.table[s, k]] -= 1
                self.table[s, k], self.refs[to] = to, 1
            self.lens[s] = length
        return moves

    def trim(self, new, seqs=None):
        for s, length in zip(range(len(new)) if seqs is None else seqs, new):
            for k in range(self.n(length), self.table.shape[1]):
                if self.table[s, k] >= 0:
                    self.refs[self.table[s, k]] -= 1
                    self.table[s, k] = -1
            self.lens[s] = min(self.lens[s], length)

    def compact(self):
        used = int((self.refs > 0).sum())
        src = [v for v in range(used, len(self.refs)) if self.refs[v] > 0]
        dst = [v for v in range(used) if self.refs[v] == 0]
        for s, d in zip(src, dst):
            self.table[self.table == s] = d
            self.refs[d], self.refs[s] = self.refs[s], 0
        return list(zip(src, dst))
