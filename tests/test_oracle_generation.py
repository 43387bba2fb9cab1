"""Pins of the generation oracle: properties of the rotation and the norm, gradients against
differences, attention over pages against attention over a plain sequence, invariants of slots."""
import numpy as np
import pytest

from oracle import attention as orc
from oracle import generation as gen

RNG = np.random.default_rng


def freqs(rot, base=10000.0):
    return base ** (-np.arange(0, rot, 2) / max(rot, 1))


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_keeps_norms_and_depends_on_distance(inter):
    r = RNG(1)
    q, k = r.standard_normal((1, 32)), r.standard_normal((1, 32))
    f = freqs(32)
    dots = []
    for p in (0, 7, 1000):
        a, b = gen.rotate(q, [p + 5], f, inter), gen.rotate(k, [p], f, inter)
        assert np.allclose(np.linalg.norm(a), np.linalg.norm(q), rtol=1e-13)
        dots.append(float(a[0] @ b[0]))
    assert np.ptp(dots) < 1e-10


def test_rotation_by_hand():
    x = np.array([[1.0, 2.0, 3.0, 4.0, 5.0]])
    t = np.array([0.5, 0.25]) * 3
    y = gen.rotate(x, [3], [0.5, 0.25], False)[0]
    assert np.allclose(y, [np.cos(t[0]) - 3 * np.sin(t[0]), 2 * np.cos(t[1]) - 4 * np.sin(t[1]),
                           3 * np.cos(t[0]) + np.sin(t[0]), 4 * np.cos(t[1]) + 2 * np.sin(t[1]), 5.0])
    y = gen.rotate(x, [3], [0.5, 0.25], True)[0]
    assert np.allclose(y, [np.cos(t[0]) - 2 * np.sin(t[0]), 2 * np.cos(t[0]) + np.sin(t[0]),
                           3 * np.cos(t[1]) - 4 * np.sin(t[1]), 4 * np.cos(t[1]) + 3 * np.sin(t[1]), 5.0])


def test_the_two_layouts_are_one_permutation_apart():
    r = RNG(2)
    x, f, pos = r.standard_normal((4, 24)), freqs(16), [0, 3, 9, 100]
    perm = np.concatenate([np.arange(0, 16, 2), np.arange(1, 16, 2), np.arange(16, 24)])
    assert np.allclose(gen.rotate(x[:, perm], pos, f, False), gen.rotate(x, pos, f, True)[:, perm])


@pytest.mark.parametrize("inter,normed", [(False, True), (True, True), (False, False)])
def test_gradients_against_differences(inter, normed):
    r = RNG(3)
    H, KV, d, T = 2, 1, 6, 3
    x = r.standard_normal((T, (H + 2 * KV) * d))
    wq, wk = (r.standard_normal(d), r.standard_normal(d)) if normed else (None, None)
    dq, dk, dv = r.standard_normal((H, T, d)), r.standard_normal((KV, T, d)), r.standard_normal((KV, T, d))
    pos, f = [0, 4, 11], freqs(4)

    def loss(x, wq, wk):
        q, k, v = gen.qkv_rope(x, H, KV, d, pos, f, inter, wq, wk, 1e-3, 1.1)
        return np.sum(q * dq) + np.sum(k * dk) + np.sum(v * dv)

    dx, dwq, dwk = gen.qkv_rope_bwd(dq, dk, dv, x, H, KV, d, pos, f, inter, wq, wk, 1e-3, 1.1)
    h = 1e-6
    for arr, grad, at in ((x, dx, 0), (wq, dwq, 1), (wk, dwk, 2)):
        if arr is None:
            assert grad is None
            continue
        num = np.empty(arr.size)
        for i in range(arr.size):
            args = [x, wq, wk]
            hi, lo = arr.copy(), arr.copy()
            hi.flat[i] += h
            lo.flat[i] -= h
            args[at] = hi
            up = loss(*args)
            args[at] = lo
            num[i] = (up - loss(*args)) / (2 * h)
        assert np.allclose(num, grad.ravel(), atol=2e-8 * max(1, np.abs(grad).max()))


def test_paged_attention_is_attention_of_the_last_row():
    r = RNG(4)
    H, KV, d, P, n = 4, 2, 8, 4, 11
    k, v = r.standard_normal((5, KV, P, d)), r.standard_normal((5, KV, P, d))
    table, q = [[3, 0, 4]], r.standard_normal((1, H, d))
    o, lse, _, _ = gen.paged_attention(q, k, v, table, [n], 0.3)
    for h in range(H):
        kk = np.concatenate([k[p, h // 2] for p in table[0]])[:n]
        vv = np.concatenate([v[p, h // 2] for p in table[0]])[:n]
        qq = np.zeros((n, d))
        qq[-1] = q[0, h]
        p = orc.probabilities(qq, kk, True, 0.3)[-1]
        assert np.allclose(o[0, h], p @ vv)
        assert np.isclose(lse[0, h], np.log(np.sum(np.exp(0.3 * kk @ q[0, h]))))
    o, lse, _, _ = gen.paged_attention(q, k, v, table, [0], 0.3)
    assert (o == 0).all() and (lse == -np.inf).all()


def test_slots_by_hand():
    table = [[7, -1, -1], [-1, -1, -1], [4, 5, -1]]
    slots, pos, t, lens, head = gen.kv_slots([3, 0, 8], [0, 2, 2, 5], table, [9, 8, 6, 2], 1, 4)
    assert slots == [7 * 4 + 3, 8 * 4, 6 * 4, 6 * 4 + 1, 6 * 4 + 2] and pos == [3, 4, 8, 9, 10]
    assert t == [[7, 8, -1], [-1, -1, -1], [4, 5, 6]] and lens == [5, 0, 11] and head == 3


def test_slots_run_out():
    slots, _, t, _, head = gen.kv_slots([0, 0], [0, 3, 5], [[-1], [-1]], [1], 0, 2)
    assert slots == [2, 3, -1, -1, -1] and t == [[1], [-1]] and head == 2
