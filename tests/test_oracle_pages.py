"""Pins of the oracle of work over pages: attention of several new tokens against plain attention of the whole
sequence's last rows, attention behind a prefix against the same over one sequence, empty rows."""
import numpy as np
import pytest

from oracle import attention as orc
from oracle import pages

D, P, SCALE = 8, 4, 0.3


def setup(lens, KV, seed):
    r = np.random.default_rng(seed)
    need = [-(-n // P) for n in lens]
    order = iter(r.permutation(sum(need) + 3))
    table = np.full((len(lens), max(need + [1])), -1)
    for s, n in enumerate(need):
        table[s, :n] = [next(order) for _ in range(n)]
    k, v = r.standard_normal((2, sum(need) + 3, KV, P, D))
    return r, k, v, table


def by_hand(x, table, n, h):
    return np.array([x[table[i // P], h, i % P] for i in range(n)]).reshape(n, D)


def softmax_rows(q, k, v, seen):
    s = np.where(np.arange(len(k)) < np.asarray(seen)[:, None], SCALE * q @ k.T, -np.inf)
    lse = np.logaddexp.reduce(s, axis=1)
    return np.exp(s - lse[:, None]) @ v, lse


@pytest.mark.parametrize("causal", [True, False])
def test_several_new_tokens_are_the_last_rows(causal):
    new, lens, H, KV = [3, 0, 5, 1], [9, 4, 5, 17], 4, 2
    r, k, v, table = setup(lens, KV, 1)
    cu = np.concatenate([[0], np.cumsum(new)])
    q = r.standard_normal((H, sum(new), D))
    got = pages.varlen(q, k, v, table, lens, cu, causal, SCALE)
    assert [t for t, *_ in got] == list(range(sum(new)))
    for t, o, lse, a, z, w in got:
        s = int(np.searchsorted(cu, t, side="right")) - 1
        seen = lens[s] - new[s] + t - cu[s] + 1 if causal else lens[s]
        for h in range(H):
            kk, vv = by_hand(k, table[s], lens[s], h // 2), by_hand(v, table[s], lens[s], h // 2)
            ro, rl = softmax_rows(q[h, t:t + 1], kk, vv, [seen])
            assert np.allclose(o[h], ro[0], atol=1e-13) and np.isclose(lse[h], rl[0], atol=1e-13)
            assert (a[h] >= np.abs(o[h]) - 1e-13).all() and w[h] >= z[h] - 1e-13
            assert z[h] >= SCALE * np.abs(kk[:seen] @ q[h, t]).max() - 1e-13


def test_one_request_without_old_rows_is_plain_causal_attention():
    r, k, v, table = setup([7], 1, 2)
    q = r.standard_normal((1, 7, D))
    got = pages.varlen(q, k, v, table, [7], [0, 7], True, SCALE)
    k1, v1 = by_hand(k, table[0], 7, 0), by_hand(v, table[0], 7, 0)
    o, lse = orc.attention_dense(q[None], k1[None, None], v1[None, None], True, SCALE)
    for t, x, y, *_ in got:
        assert np.allclose(x[0], o[0, 0, t], atol=1e-13) and np.isclose(y[0], lse[0, 0, t], atol=1e-13)


def test_tokens_before_the_first_row_see_nothing():
    r, k, v, table = setup([2, 0], 1, 3)
    got = pages.varlen(r.standard_normal((1, 6, D)), k, v, table, [2, 0], [0, 4, 6], True, SCALE)
    for t, o, lse, a, z, w in got:
        empty = t not in (2, 3)
        assert np.isneginf(lse[0]) == empty and (o[0] == 0).all() == empty


def test_behind_a_prefix_is_one_sequence():
    lens, own, cu, H, KV = [6, 0, 9], [3, 0, 2, 5, 0], [0, 2, 4, 5], 2, 1
    r, k, v, table = setup(lens + own, KV, 4)
    q = r.standard_normal((5, H, D))
    o, lse, *_ = pages.shared(q, k, v, table[:3], lens, cu, table[3:], own, SCALE)
    for s, g in enumerate([0, 0, 1, 1, 2]):
        kk, vv = (np.concatenate([by_hand(x, table[g], lens[g], 0), by_hand(x, table[3 + s], own[s], 0)]) for x in (k, v))
        for h in range(H):
            ro, rl = softmax_rows(q[s, h:h + 1], kk, vv, [len(kk)])
            assert np.allclose(o[s, h], ro[0], atol=1e-13) and np.isclose(lse[s, h], rl[0], atol=1e-13)
