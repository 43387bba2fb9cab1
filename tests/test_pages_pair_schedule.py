"""Where the two softmax warps of a row meet in the kernel for many new tokens (attn_chunk_kernel.cuh), restated on the host:
their barriers have no limit, so whichever waits of either give up, neither may be left at one.  Every pattern of waits
that give up is gone through, a warp as a generator that stops where it meets the other."""
import itertools

import pytest


def warp(chance, units):
    """units: (key tiles, whether the warp has rows).  chance: whether each wait in turn gives up, and whether a later tile's
    sum asks for the maximum."""
    chance = iter(chance)

    def hit():
        return next(chance, False)

    def exchange(x):
        theirs = yield ("value", x)
        yield ("read", None)
        return theirs

    meet = 1
    for tiles, rows in units:
        if hit():                                        # the next unit is not told in time
            break
        ok = True
        for j in range(tiles):
            if hit():                                    # nor are a tile's scores there
                ok, meet = False, 2 if rows and j > 0 else 1
                break
            if not rows:
                continue
            need = j == 0 or hit()
            if j == 0 or (yield ("or", need)):
                yield from exchange(0.0)                 # the maximum
                if (yield from exchange(float(need))) == 2.0:
                    ok, meet = False, 0
                    break
                if j > 0 and hit():                      # the product before, whose O is to be rescaled, is not done
                    ok, meet = False, 2 if j + 1 < tiles else 1
                    break
        if not ok:
            break
    if meet == 2:
        yield ("or", True)
    for _ in range(2 if meet else 0):
        yield from exchange(2.0)


def met(pair):
    """Both to their ends, or whether one is left at a barrier."""
    at = [next(w, None) for w in pair]
    while at[0] and at[1]:
        assert at[0][0] == at[1][0], at                  # and they are at the same one
        both = [at[0][1] or at[1][1]] * 2 if at[0][0] == "or" else [at[1][1], at[0][1]]
        for i, w in enumerate(pair):
            try:
                at[i] = w.send(both[i])
            except StopIteration:
                at[i] = None
    return at == [None, None]


@pytest.mark.parametrize("units", [[(1, True)], [(3, True)], [(2, True), (2, True)], [(1, True), (2, False), (2, True)],
                                   [(2, False), (1, True)], []])
def test_neither_warp_of_a_row_is_left_at_a_barrier(units):
    patterns = list(itertools.product((False, True), repeat=8))
    for a in patterns:
        for b in patterns:
            assert met((warp(a, units), warp(b, units))), (a, b)
