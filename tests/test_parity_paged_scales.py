"""GPU parity of attention over an E4M3 cache against the float64 oracle where the scales of a request's
V rows differ in size and sign.

Tolerance, from the arithmetic: P s is rounded to f16 for the product (2^-11 of the value), or, below
f16's normal range, by 2^-25 where the largest P s of a row with a code other than zero is 2^6 or
more: n 2^-31 x 448 max(P s) over n keys; P's own relative error e_s = 2^-16 Z + 2^-20, Z = scale max
sum |q k| (the score's fp32 sum, a truncation a term, and exp2), counts twice against A = P|V|; then
bf16.  No term holds the scale of a row whose weight or whose codes are zero.
"""
import math

import numpy as np
import pytest
import torch

from io_aware_attention_attn_gb300 import attn
from oracle import fp8 as ofp8
from oracle import generation as gen

from test_parity_generation import _gpu, bf16_tol, check_paged, f64, normal, paged_inputs, within  # noqa: F401

pytestmark = pytest.mark.gpu
ROWS = [(64, 4), (64, 16), (64, 32), (128, 4), (128, 16), (128, 32)]  # d, query rows a K/V head


@pytest.mark.parametrize("d,rows", ROWS)
@pytest.mark.parametrize("share", [0.5, 1.0])
def test_negative_scales(d, rows, share):
    lens = [300, 17, 1]
    q, cache, table, n, vals = paged_inputs(40 + rows, lens, 2 * rows, 2, d, 16, "e4m3")
    r = np.random.default_rng(rows)
    signs = [np.where(r.random(t.shape) < share, -1.0, 1.0) for t in (cache.k_scale, cache.v_scale)]
    scales = [t * torch.from_numpy(s).float().cuda() for t, s in zip(cache[2:], signs)]
    vals = [v * s[..., None] for v, s in zip(vals, signs)]
    o, lse = attn.attn_fwd_paged(q, attn.KVCache(cache.k, cache.v, *scales), table, n)
    check_paged(o, lse, q, vals, table, lens, 1 / math.sqrt(d), "e4m3", f"paged negative scales d{d} {rows}")


def check_weights(q, cache, table, lens, what, scale):
    """attn_fwd_paged on the values that an E4M3 cache holds, to the tolerance above."""
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    o, lse = attn.attn_fwd_paged(q, cache, table, n, scale)
    codes = [ofp8.e4m3_value(c.view(torch.uint8).cpu().numpy()) for c in cache[:2]]
    sc = [f64(s) for s in cache[2:]]
    vals = [c * s[..., None] for c, s in zip(codes, sc)]
    ids = table.cpu().numpy()
    ro, rl, a, z = gen.paged_attention(f64(q)[:, :, 0], *vals, ids, lens, scale)
    weight = np.where((codes[1] != 0).any(-1), np.abs(sc[1]), 0.0)
    low = np.zeros(rl.shape)
    group = q.shape[1] // cache.k.shape[1]
    for s, length in enumerate(lens):
        at = ids[s, :-(-length // cache.k.shape[2])]
        for h in range(q.shape[1]):
            k = np.concatenate([vals[0][p, h // group] for p in at])[:length]
            w = np.concatenate([weight[p, h // group] for p in at])[:length]
            low[s, h] = length * 2.0 ** -31 * 448 * (np.exp(scale * (k @ f64(q)[s, h, 0]) - rl[s, h]) * w).max()
    es = 2.0 ** -16 * z + 2.0 ** -20
    e = (2.0 ** -11 + 2 * es)[..., None] * a + low[..., None]
    within(f64(o)[:, :, 0], ro, bf16_tol(ro, e), what + " O")
    within(lse.cpu().numpy().astype(np.float64)[:, :, 0], rl, es + 2.0 ** -20 * (1 + np.abs(rl)), what + " lse")


def written(seed, lens, H, KV, d, sigma, empty, page=16):
    """q and an E4M3 cache that attn.qkv_rope wrote: V of deviation sigma, zero rows at the positions
    `empty` of every request."""
    T = sum(lens)
    rows = normal(seed, T, H + 2 * KV, d)
    rows[:, H + KV:] = sigma * rows[:, H + KV:].float()
    used = [-(-n // page) for n in lens]
    cache = attn.kv_cache(sum(used), KV, page, d, torch.float8_e4m3fn)
    table = torch.full((len(lens), max(used)), -1, dtype=torch.int32, device="cuda")
    slots, at, first = [], 0, 0
    for s, n in enumerate(lens):
        table[s, :used[s]] = torch.arange(at, at + used[s], dtype=torch.int32)
        slots += [at * page + i for i in range(n)]
        for i in empty:
            if i < n:
                rows[first + i, H + KV:] = 0
        at += used[s]
        first += n
    attn.qkv_rope(rows.view(T, -1), H, KV, cache=cache, slots=torch.tensor(slots, device="cuda"))
    return normal(seed + 1, len(lens), H, 1, d), cache, table


@pytest.mark.parametrize("d,rows", ROWS)
@pytest.mark.parametrize("sigma", [1.0, 1e-2, 1e-3, 1e-5, 1e-30, 1e36])
def test_rows_of_zeros_among_written_rows(d, rows, sigma):
    # the writer gives a row of zeros scale 1
    lens = [1000, 70]
    q, cache, table = written(rows, lens, 2 * rows, 2, d, sigma, (0, 5, 64, 333))
    assert (cache.v_scale[0, :, 5] == 1).all()
    check_weights(q, cache, table, lens, f"paged zero rows d{d} {rows} sigma {sigma}", 1 / math.sqrt(d))


@pytest.mark.parametrize("d,rows", ROWS)
@pytest.mark.parametrize("peak", [1.0, 20.0])
def test_scales_of_any_size(d, rows, peak):
    lens = [700, 33]
    q, cache, table = written(7 + rows, lens, 2 * rows, 2, d, 1.0, (3, 100))
    r = np.random.default_rng(d + rows)
    cache.v_scale.mul_(torch.from_numpy(np.exp2(r.integers(-20, 21, cache.v_scale.shape))).float().cuda())
    check_weights(q, cache, table, lens, f"paged scales d{d} {rows} peak {peak}", peak / math.sqrt(d))


@pytest.mark.parametrize("d,rows", ROWS)
def test_large_row_without_weight_and_weight_without_values(d, rows):
    lens = [500, 129]
    H = 2 * rows
    q, cache, table = written(9 + rows, lens, H, 2, d, 1.0, (17,))
    # q's rows nearly alike, so that keys along them have a score far from all others
    along = normal(3, 1, 1, 1, d)
    q = (along + 0.1 * q.float()).to(torch.bfloat16)
    unit = (along / along.float().norm()).reshape(d)
    for row, score in ((33, -60.0), (17, 60.0)):  # a row without weight, large; one of zeros with all of it
        for s in range(2):
            p, i = int(table[s, row // 16]), row % 16
            cache.k.view(torch.uint8)[p, :, i] = (unit * 448).to(torch.float8_e4m3fn).view(torch.uint8)
            cache.k_scale[p, :, i] = score / 448
            if score < 0:
                cache.v_scale[p, :, i] *= 2.0 ** 14
    check_weights(q, cache, table, lens, f"paged weights d{d} {rows}", 1 / math.sqrt(d))


@pytest.mark.parametrize("d,rows", ROWS)
def test_values_all_zero_and_scales_that_are_not_finite(d, rows):
    lens = [200, 90, 90]
    q, cache, table = written(5 + rows, lens, 2 * rows, 2, d, 1.0, ())
    cache.v.view(torch.uint8)[table[0, :13].long()] = 0x80  # zeros with a sign
    cache.v_scale[int(table[1, 2]), 0, 3] = float("nan")
    cache.v_scale[int(table[2, 2]), 1, 3] = float("inf")
    o, lse = attn.attn_fwd_paged(q, cache, table, torch.tensor(lens, dtype=torch.int32).cuda())
    assert (o[0] == 0).all() and torch.isfinite(lse).all()
    assert torch.isnan(o[1, :rows]).all() and torch.isfinite(o[1, rows:]).all()
    assert not torch.isfinite(o[2, rows:]).any() and torch.isfinite(o[2, :rows]).all()


@pytest.mark.parametrize("d,rows", ROWS)
def test_rows_with_one_code(d, rows):
    # rows that are zero but for one element each, at every position of a row
    lens = [d + 40, 50]
    q, cache, table = written(11 + rows, lens, 2 * rows, 2, d, 1.0, ())
    for i in range(d):
        p, at = int(table[0, (i + 20) // 16]), (i + 20) % 16
        cache.v.view(torch.uint8)[p, :, at] = 0
        cache.v.view(torch.uint8)[p, :, at, i] = 0x81  # -2^-9
        cache.v_scale[p, :, at] = 2.0 ** (9 + i % 12)
    check_weights(q, cache, table, lens, f"paged one code d{d} {rows}", 1 / math.sqrt(d))


@pytest.mark.parametrize("d,rows", ROWS)
@pytest.mark.parametrize("gap", [0, 15, 100, 600])
def test_weight_on_values_of_zero_apart_from_large_values(d, rows, gap):
    # the keys with values lie in one warp's share, in one tile or (by the gap) one CTA's, and their scales
    # are large; all other keys have codes of zero and, from key to key, as much weight
    lens = [2048, 200]
    q, cache, table = written(13 + rows, lens, 2 * rows, 2, d, 1.0, range(2048))
    r = np.random.default_rng(rows + gap)
    v = torch.from_numpy(r.integers(0x30, 0x78, (2, 3, d), dtype=np.uint8)).cuda()
    for s in range(2):
        for i in range(3):
            at = min(gap + i, lens[s] - 1)
            p, at = int(table[s, at // 16]), at % 16
            cache.v.view(torch.uint8)[p, :, at] = v[:, i]
            cache.v_scale[p, :, at] = 2.0 ** (55 + 10 * i)
    check_weights(q, cache, table, lens, f"paged apart d{d} {rows} gap {gap}", 1 / math.sqrt(d))
