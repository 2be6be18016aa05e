"""CPU model of a give-up among the four warps of the tensor-core tree attention that convert an FP8 cache's
values (and split a segment's queries): copies land at random times, a wait gives up at a random one, and
what was on its way lands all the same.  A warp that gives up leaves its loop by itself, so no other warp may
wait for it at a barrier among the four: that wait would have no bound."""
import random

import pytest

from tests.test_tree_split_model import CASES, pair_of_unit, shapes, unit_start

WARPS, RAW = 4, 2


def run(seed, votes):
    """True if all four warps leave.  votes: the queries' warps vote at a barrier instead of arriving one by one."""
    rng = random.Random(seed)
    segments = [rng.randint(1, 3) for _ in range(4)]         # stages a segment
    stages = sum(segments)
    q_landed, landed = set(), set()
    emptied = [0] * stages                                   # warps done with a stage
    state = {"abort": False, "voters": 0, "gen": 0}

    def wait(there):
        while not there():
            if state["abort"]:
                return False
            yield
        return True

    def warp():
        i = 0
        for k, n in enumerate(segments):
            good = yield from wait(lambda: k in q_landed)
            if votes:
                gen = state["gen"]
                state["voters"] += 1
                if state["voters"] == WARPS:
                    state["voters"], state["gen"] = 0, gen + 1
                while state["gen"] == gen:
                    yield
                good = not state["abort"]
            if not good:
                return
            for _ in range(n):
                if not (yield from wait(lambda: i in landed)):
                    return
                emptied[i] += 1
                i += 1
                yield

    live = {w: warp() for w in range(WARPS)}
    give_up, flying = rng.randrange(60), []
    sent = sent_q = 0
    for step in range(4000):
        if step == give_up:
            state["abort"] = True
        if not state["abort"]:                               # the loader: a code stage may be overwritten once all are done with it
            if sent < stages and (sent < RAW or emptied[sent - RAW] == WARPS):
                flying.append((landed, sent))
                sent += 1
            if sent_q < len(segments) and (sent_q == 0 or sent >= sum(segments[:sent_q])):
                flying.append((q_landed, sent_q))
                sent_q += 1
        if flying and rng.random() < 0.3:
            where, what = flying.pop(0)
            where.add(what)
        if not live:
            return True
        k = rng.choice(list(live))
        try:
            next(live[k])
        except StopIteration:
            del live[k]
    return False


def test_every_warp_leaves_after_a_give_up():
    assert all(run(seed, votes=False) for seed in range(400))


def test_a_vote_among_them_would_wait_without_bound():
    assert any(not run(seed, votes=True) for seed in range(400))


# ---- the join's records ------------------------------------------------------------------------------

def records(tiles, steps, pair, pairs):
    """(tile of the batch, first pair, its pairs, head) that a pair writes before it waits for anything."""
    U = sum(t * s for t, s in zip(tiles, steps))
    s0, s1 = unit_start(pair, U, pairs), unit_start(pair + 1, U, pairs)
    out, u0, t0 = [], 0, 0
    for t, s in zip(tiles, steps):
        u1 = u0 + t * s
        if u1 > u0 and u0 < s1 and s0 < u1:
            k = (s0 - u0 + s - 1) // s if s0 > u0 else 0
            while k < t and u0 + k * s < s1:
                v = u0 + k * s
                last = v + s - 1
                out.append((t0 + k, pair, 1 if last < s1 else pair_of_unit(last, U, pairs) - pair + 1, v == s0))
                k += 1
        u0, t0 = u1, t0 + t
    return out


@pytest.mark.parametrize("pairs", [1, 2, 74])
@pytest.mark.parametrize("n,lens,heads", CASES + [([9], [70000], 128), ([4] * 4, [131072] * 4, 128)])
def test_every_tile_has_one_record(n, lens, heads, pairs):
    tiles, steps = shapes(n, lens, heads)
    U = sum(t * s for t, s in zip(tiles, steps))
    got = [r for c in range(pairs) for r in records(tiles, steps, c, pairs)]
    want, u0, t0 = [], 0, 0
    for t, s in zip(tiles, steps):
        for k in range(t if s else 0):
            c0, c1 = pair_of_unit(u0, U, pairs), pair_of_unit(u0 + s - 1, U, pairs)
            want.append((t0 + k, c0, c1 - c0 + 1, unit_start(c0, U, pairs) == u0))
            u0 += s
        t0 += t
    assert got == want
