"""How the paged kernel shares out its work, restated on the host: the places of all units cut into
equal shares, what each CTA finds in its share, and what the joins take for the parts of a unit.
Every tile of every unit has to be taken once, a CTA has to leave at most two parts, and each unit's
parts have to be the ones that its join reads, in order."""
import numpy as np
import pytest


def shares(total, G):
    q, r = divmod(total, G)
    start = lambda i: i * q + min(i, r)  # noqa: E731

    def owner(place):
        big = r * (q + 1)
        return place // (q + 1) if place < big else r + (place - big) // q

    return start, owner


def plan(tiles, per, ctas, cost):
    """Places of units in order: (first place, tiles) of each, the total, and the CTAs with work."""
    units, at = [], 0
    for n in tiles:
        for _ in range(per):
            units.append((at, n))
            at += n + cost
    return units, at, min(ctas, at)


def walk(units, total, G, cost, cta):
    """(unit, first tile, last tile + 1) that a CTA computes, as the kernel's loop goes."""
    start, _ = shares(total, G)
    place = start(cta)
    u = max(i for i, (a, _) in enumerate(units) if a <= place)
    t = place - units[u][0]
    left = start(cta + 1) - place
    if t >= units[u][1]:
        left -= units[u][0] + units[u][1] + cost - place
        if left <= 0:
            return []
        u, t = u + 1, 0
    done = []
    while left > 0:
        n = units[u][1]
        end = min(n, t + left)
        done.append((u, t, end))
        left -= end - t + (cost if end == n else 0)
        u, t = u + 1, 0
    return done


def join(units, total, G, cost, x, by_unit):
    """The (CTA, part) list that block x merges, for its unit; None where it has nothing to do."""
    start, owner = shares(total, G)
    if by_unit:
        u = x
    else:
        if x >= G:
            return None
        place = start(x)
        u = max(i for i, (a, _) in enumerate(units) if a <= place)
        t = place - units[u][0]
        if not (0 < t < units[u][1] and owner(units[u][0] + units[u][1] - 1) == x):
            return None
    first, n = units[u]
    i0, last = owner(first), owner(first + n - 1)
    if i0 == last:
        return None
    second = 1 if start(i0) < first - cost else 0
    return u, [(i, second if i == i0 else 0) for i in range(i0, last + 1)]


@pytest.mark.parametrize("cost", [0, 1, 2])
@pytest.mark.parametrize("seed", range(40))
def test_every_tile_once_and_joins_find_their_parts(seed, cost):
    r = np.random.default_rng(seed)
    B, per = int(r.integers(1, 40)), int(r.integers(1, 9))
    top = int(r.choice([1, 3, 20, 300]))
    tiles = [max(1, int(n)) for n in r.integers(0, top + 1, B)]
    ctas = int(r.choice([1, 2, 7, 152, 304, 456, 608]))
    units, total, G = plan(tiles, per, ctas, cost)
    taken = [np.zeros(n, dtype=int) for _, n in units]
    parts = {}
    for cta in range(G):
        left_parts = 0
        for seg, (u, a, b) in enumerate(walk(units, total, G, cost, cta)):
            assert a < b
            taken[u][a:b] += 1
            if (a, b) != (0, units[u][1]):
                parts.setdefault(u, []).append((cta, 0 if seg == 0 else 1, a, b))
                left_parts += 1
        assert left_parts <= 2
    assert all((t == 1).all() for t in taken)
    for by_unit in (True, False):
        found = {}
        for x in range(len(units) if by_unit else ctas):
            j = join(units, total, G, cost, x, by_unit)
            if j is not None:
                assert j[0] not in found
                found[j[0]] = j[1]
        assert found == {u: [(c, s) for c, s, _, _ in p] for u, p in parts.items()}
        for u, p in parts.items():  # in order and touching
            assert p[0][2] == 0 and p[-1][3] == units[u][1]
            assert all(x[3] == y[2] for x, y in zip(p, p[1:]))


def test_shares_are_even():
    for total, G in ((1, 1), (7, 3), (100, 608), (12345, 304)):
        G = min(G, total)
        start, owner = shares(total, G)
        sizes = [start(i + 1) - start(i) for i in range(G)]
        assert sum(sizes) == total and max(sizes) - min(sizes) <= 1
        assert [owner(p) for p in range(total)] == [i for i in range(G) for _ in range(sizes[i])]
