"""CPU model of the barriers between the MMA threads and the softmax warps of the tensor-core tree attention:
two CTAs whose warps run at random speeds, mbarriers with an arrival count and a phase that waits tell by
its parity, commits that arrive late and at different times in the two CTAs.  Every run must end, and no
operand may be read before it is written nor overwritten before it is read.  Mistakes planted in
the model fail.  bufs: buffers of S, two over a bf16 cache and one over an FP8 cache, where a segment's
queries also leave the unit of their scores to the softmax, in two places by segment parity."""
import random

import pytest

CTAS, PAGES = 2, 4
WARPS = [(cta, pg, h) for cta in range(CTAS) for pg in range(PAGES) for h in range(2)]


class Bar:
    def __init__(self, count):
        self.count = self.pending = count
        self.phase = 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0
        if self.pending == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def passed(self, parity):
        return (self.phase & 1) != (parity & 1)


class Deadlock(Exception):
    pass


def run(seed, units, planted=None, bufs=2):
    """units: (first, last, pages, rescale) per step."""
    rng = random.Random(seed)
    pair = lambda count: [Bar(count) for _ in range(CTAS)]
    s_full, s_free = [pair(1), pair(1)], [Bar(16), Bar(16)]
    p_full, p_free = [Bar(4) for _ in range(PAGES)], [pair(1) for _ in range(PAGES)]
    o_ok = [Bar(16), Bar(16)]
    pv_done = [pair(1), pair(1)]
    votes = [{"n": 0, "gen": 0} for _ in range(CTAS)]
    S = [None, None]                       # unit whose scores a buffer holds
    read_s = {}                            # unit -> warps that have read it
    P = {}                                 # (cta, page, half) -> unit
    q_empty, q_full = [Bar(1) for _ in range(CTAS)], Bar(CTAS)
    unit = {}                              # (cta, segment parity) -> segment whose scores' unit it is
    read_q = {}                            # (cta, segment) -> warps that have read it
    ok_for = {}                            # unit -> warps past their O duties
    done = set()                           # units whose PV has run
    started = set()
    tensor = {"qk": [], "pv": []}          # per issuing thread: queued MMAs and commits, in order
    commits = []                           # arrivals under way, in order per thread and CTA

    def qk():
        seg = 0
        for u, (first, last, _, _) in enumerate(units):
            while first and not q_full.passed(seg):
                yield
            seg += first
            while not s_free[u % bufs].passed((u // bufs) ^ 1):
                yield
            if u >= bufs:
                assert len(read_s.get(u - bufs, ())) == 16, "S overwritten before it was read"
            tensor["qk"] += [("S", u), ("c", s_full[u % bufs])]
            if last:
                tensor["qk"] += [("c", q_empty)]
            yield

    def queries(cta):
        for seg in range(sum(first for first, _, _, _ in units)):
            while not q_empty[cta].passed(seg ^ 1):
                yield
            at = cta, 0 if planted == "one place for the units" else seg & 1
            if at in unit and bufs == 1:
                assert len(read_q.get((cta, unit[at]), ())) == 8, "unit overwritten before it was read"
            unit[at] = seg
            q_full.arrive()
            yield

    def pv():
        ph = [0] * PAGES
        for u, (first, last, pages, _) in enumerate(units):
            while not o_ok[u & 1].passed(u >> 1):
                yield
            assert len(ok_for.get(u, ())) == 16, "PV before every warp was past O"
            for p in range(pages):
                while not p_full[p].passed(ph[p]):
                    yield
                ph[p] ^= 1
                assert all(P.get((c, p, h)) == u for c in range(CTAS) for h in range(2)), "P not written"
                tensor["pv"] += [("O", u, p), ("c", p_free[p])]
                yield
            tensor["pv"] += [("end", u), ("c", pv_done[u & 1])]

    def softmax(cta, pg, h):
        before, seg, me, vote = 0, 0, (cta, pg, h), votes[cta]

        def ballot():
            gen = vote["gen"]
            vote["n"] += 1
            if vote["n"] == 8:
                vote["n"], vote["gen"] = 0, gen + 1
            while vote["gen"] == gen:
                yield
        for u, (first, last, pages, rescale) in enumerate(units):
            sb = u & 1
            while not s_full[u % bufs][cta].passed(u // bufs):
                yield
            assert S[u % bufs] == u, "S read too early"
            if first:
                assert planted or bufs == 2 or unit[cta, seg & 1] == seg, "unit of another segment"
                read_q.setdefault((cta, seg), set()).add(me)
                seg += 1
            read_s.setdefault(u, set()).add(me)
            s_free[u % bufs].arrive()
            yield
            yield from ballot()
            if u >= 2:
                while not pv_done[sb][cta].passed((u >> 1) ^ 1):
                    yield
            if not first and rescale and planted != 'rescale at once':
                while not pv_done[sb ^ 1][cta].passed((u - 1) >> 1):
                    yield
            if not first and rescale:
                assert u - 1 in done, "O rescaled while the step before runs"
            ok_for.setdefault(u, set()).add(me)
            o_ok[u & 1].arrive()
            yield
            if pg < pages:
                while not first and planted != 'no wait for P' and not p_free[pg][cta].passed(before - 1):
                    yield
                P[cta, pg, h] = u
                p_full[pg].arrive()
                yield
            before += pg < pages
            if last:
                while not pv_done[sb][cta].passed(u >> 1):
                    yield
                yield from ballot()
                assert u in done, "O read before its MMAs were done"
                yield

    def units_run():                       # the tensor cores: each thread's operations in order
        while True:
            q = tensor[rng.choice(["qk", "pv"])]
            if q:
                op = q.pop(0)
                if op[0] == "S":
                    S[op[1] % bufs] = op[1]
                elif op[0] == "O":
                    started.add(op[1])
                    assert all(P.get((c, op[2], h)) == op[1] for c in range(CTAS) for h in range(2)), "P overwritten before it was read"
                elif op[0] == "end":
                    done.add(op[1])
                else:
                    commits.append([(b, rng.randrange(6)) for b in op[1]])
            for c in commits[:]:
                c[:] = [(b, d - 1) if d else (b.arrive(), None) for b, d in c]
                c[:] = [x for x in c if x[1] is not None]
                if not c:
                    commits.remove(c)
            yield

    roles = [qk(), pv()] + [queries(c) for c in range(CTAS)] + [softmax(*w) for w in WARPS]
    weights = [rng.choice([1, 1, 4, 12]) for _ in roles]
    live, hw = dict(enumerate(roles)), units_run()
    for _ in range(4000 * len(units)):
        if rng.random() < 0.3:
            next(hw)
        if not live:
            return
        k = rng.choices(list(live), [weights[i] for i in live])[0]
        try:
            next(live[k])
        except StopIteration:
            del live[k]
    raise Deadlock


def batch(seed, n=14):
    rng = random.Random(seed)
    units, left = [], 0
    for _ in range(n):
        first = left == 0
        if first:
            left = rng.randint(1, 4)
        left -= 1
        # a tile's steps go around, so the one with fewer pages may be any of them
        units.append((first, left == 0, rng.randint(1, 4) if rng.random() < 0.3 else 4, rng.random() < 0.3))
    units[-1] = (units[-1][0], True) + units[-1][2:]
    return units


@pytest.mark.parametrize("bufs", [1, 2])
@pytest.mark.parametrize("seed", range(60))
def test_every_schedule_ends_and_keeps_the_order(seed, bufs):
    run(seed, batch(seed), bufs=bufs)


@pytest.mark.parametrize("planted", ["no wait for P", "rescale at once", "one place for the units"])
def test_planted_mistakes_fail(planted):
    bad = 0
    for seed in range(40):
        try:
            run(seed, batch(seed), planted, bufs=1 if planted == "one place for the units" else 2)
        except (AssertionError, Deadlock):
            bad += 1
    assert bad > (5 if planted == "one place for the units" else 30)
