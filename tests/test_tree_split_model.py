"""CPU model of the tensor-core tree attention's work division: every (tile, step) unit is walked once, in
order, and partial results take slots of their own, which the join finds again."""
import numpy as np
import pytest

TILE, STEP = 128, 256


def unit_start(c, U, pairs):
    return c * U // pairs


def pair_of_unit(u, U, pairs):
    c = u * pairs // U
    while c + 1 < pairs and unit_start(c + 1, U, pairs) <= u:
        c += 1
    while c > 0 and unit_start(c, U, pairs) > u:
        c -= 1
    return c


def shapes(n, lens, heads):
    return [-(-k * heads // TILE) for k in n], [-(-L // STEP) for L in lens]


def walk(n, lens, heads, pair, pairs):
    """The pair's units as (sequence, tile, step, first, last, segment's first step, head)."""
    tiles, steps = shapes(n, lens, heads)
    units = [t * s for t, s in zip(tiles, steps)]
    U = sum(units)
    s0, s1 = unit_start(pair, U, pairs), unit_start(pair + 1, U, pairs)
    left = s1 - s0
    if left == 0:
        return []
    b, at = 0, s0
    while at >= units[b]:
        at -= units[b]
        b += 1
    tile, step = divmod(at, steps[b])
    out, first, head, seg0 = [], True, True, step
    while left > 0:
        last = left == 1 or step == steps[b] - 1
        out.append((b, tile, step, first, last, seg0, head))
        first = last
        if first:
            head = False
        left -= 1
        step += 1
        if step == steps[b]:
            step, tile = 0, tile + 1
            if tile == tiles[b]:
                tile, b = 0, b + 1
                while left > 0 and b < len(units) and units[b] == 0:
                    b += 1
        if first:
            seg0 = step
    return out


CASES = [([1], [1], 1), ([5], [250], 128), ([3, 0, 1, 64], [67, 9, 701, 127], 16), ([300], [490], 3), ([64] * 16, [8000] * 16, 128),
         ([1] * 200, list(range(1, 201)), 8), ([7, 2], [131072, 3], 128), ([0, 0, 2], [5, 5, 5], 64)]


@pytest.mark.parametrize("pairs", [1, 2, 74])
@pytest.mark.parametrize("n,lens,heads", CASES)
def test_units_slots_and_the_join(n, lens, heads, pairs):
    tiles, steps = shapes(n, lens, heads)
    want = [(b, t, s) for b in range(len(n)) for t in range(tiles[b]) for s in range(steps[b])]
    runs = [walk(n, lens, heads, c, pairs) for c in range(pairs)]
    assert [x[:3] for r in runs for x in r] == want
    U = len(want)
    slots = {}                                                    # (tile, segment steps) by slot
    for c, run in enumerate(runs):
        for b, t, s, first, last, seg0, head in run:
            if last and not (seg0 == 0 and s == steps[b] - 1):
                slot = 2 * c + (0 if head else 1)
                assert slot not in slots
                slots[slot] = (b, t, seg0, s)
    u0 = 0
    for b in range(len(n)):
        for t in range(tiles[b]):
            c0, c1 = pair_of_unit(u0, U, pairs), pair_of_unit(u0 + steps[b] - 1, U, pairs)
            if c0 != c1:
                got = []
                for c in range(c0, c1 + 1):
                    if unit_start(c, U, pairs) == unit_start(c + 1, U, pairs):
                        continue
                    got.append(slots.pop(2 * c + (1 if c == c0 and unit_start(c0, U, pairs) != u0 else 0)))
                assert all(g[:2] == (b, t) for g in got)
                assert [s for g in got for s in range(g[2], g[3] + 1)] == list(range(steps[b]))
            u0 += steps[b]
    assert not slots


def sees32(bits, j, ctx, L):
    rem, k = L - j, j - ctx
    if rem <= 0:
        return 0
    v = 0xffffffff
    if k > -32:
        word = lambda w: (bits >> (32 * w)) & 0xffffffff if w < 4 else 0
        if k < 0:
            v = (0xffffffff >> (32 + k)) | (word(0) << -k) & 0xffffffff
        else:
            v = ((word((k >> 5) + 1) << 32 | word(k >> 5)) >> (k & 31)) & 0xffffffff
    return v & (0xffffffff >> (32 - rem)) if rem < 32 else v


def test_mask_words():
    rng = np.random.default_rng(0)
    for _ in range(2000):
        ctx, n = int(rng.integers(0, 200)), int(rng.integers(1, 129))
        bits = int.from_bytes(rng.bytes(16), "little")
        j = 32 * int(rng.integers(0, 12))
        want = sum(1 << i for i in range(32) if j + i < ctx + n and (j + i < ctx or (bits >> (j + i - ctx)) & 1))
        assert sees32(bits, j, ctx, ctx + n) == want


@pytest.mark.parametrize("n,lens,heads", [([4] * 4, [131072] * 4, 128), ([4, 1, 6], [33004, 17002, 16506], 128), ([3], [20003], 16), ([9], [70000], 128)])
def test_turned_tiles(n, lens, heads):
    """A tile's steps go around from its turn; the first whole run of every long tile starts at the sequence's first step."""
    pairs = 74
    tiles, steps = shapes(n, lens, heads)
    U = sum(t * s for t, s in zip(tiles, steps))
    u0 = 0
    for t, s in zip(tiles, steps):
        for _ in range(t):
            c, turn = pair_of_unit(u0, U, pairs), 0
            if s * pairs > U + pairs and unit_start(c, U, pairs) != u0:
                turn = s - (unit_start(c + 1, U, pairs) - u0)
                assert 0 < turn < s
                assert (unit_start(c + 1, U, pairs) - u0 + turn) % s == 0
            assert sorted(k + turn if k + turn < s else k + turn - s for k in range(s)) == list(range(s))
            u0 += s
