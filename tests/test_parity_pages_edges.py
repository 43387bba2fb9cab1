"""Edges of work over a paged cache beyond one new token a request: every E4M3 code of a value, scales far from one,
batches whose requests go to both kernels, padding and bad tables where requests share prefixes, far pages with few rows.

Tolerances as in test_parity_pages.py.  Where K scales carry a power of two that q does not, or V scales one in the
kernel for many rows, the outcome is that without it, bit for bit: each step (products, sums, roundings to bf16 and
E4M3) differs by the same factor, away from the types' limits.  In the kernel for few rows the reference that is taken off a
score in log2 units follows the V scales: up to 128 more, so the difference is off by 2^-18 and a weight by as much
of itself, which the tolerance of O (2 e_s A, e_s above 2^-16 Z, and here Z > 1 for the largest rows; 2^-8 A of P's
own rounding where it is kept to 2^-11) has room for."""
import math

import numpy as np
import pytest
import torch

from io_aware_attention_attn_gb300 import attn
from oracle import fp8 as ofp8
from test_parity_generation import _gpu, f64, i32, normal, paged_inputs  # noqa: F401
from test_parity_pages import check_shared, check_varlen, shared_inputs, sums

pytestmark = pytest.mark.gpu


def same(a, b):
    return torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("n", [128, 16])  # tokens: the kernel for many rows, and the one for few
@pytest.mark.parametrize("d", [64, 128])
def test_every_value_code(n, d):
    # token i's key beats the others by over 1000 (their weights are 0): O is row i of V, here a code times 1.5 2^j, which
    # bf16 holds exactly
    page = 16
    cache = attn.kv_cache(n // page, 1, page, d, torch.float8_e4m3fn)
    cache.k.view(torch.uint8).zero_()
    cache.k_scale.fill_(64.0)
    cache.v_scale.copy_((1.5 * torch.exp2((torch.arange(n, device="cuda") % 7 - 3).float())).view(n // page, 1, page))
    cache.v_scale[:, :, ::3] *= -1
    codes = (torch.arange(n * d, device="cuda") * 5 % 256).to(torch.uint8)  # every code, in every row of four or two
    codes = torch.where(codes % 128 == 127, codes - 1, codes)               # but the two that are no number
    cache.v.view(torch.uint8).copy_(codes.view(n // page, 1, page, d))
    bits = 7 if n == 128 else 4                                            # the row's number in signs of K
    j = torch.arange(n, device="cuda")
    sign = torch.stack([1 - 2 * (j >> b & 1) for b in range(bits)], 1)     # [n, bits]
    k = torch.zeros(n, d, dtype=torch.uint8, device="cuda")
    k[:, :bits] = torch.where(sign > 0, 0x38, 0xB8).to(torch.uint8)        # 1 and -1
    cache.k.view(torch.uint8).copy_(k.view(n // page, 1, page, d))
    q = torch.zeros(1, n, d, dtype=torch.bfloat16, device="cuda")
    q[0, :, :bits] = 16 * sign.to(torch.bfloat16)
    table = torch.arange(n // page, dtype=torch.int32, device="cuda").view(1, -1)
    o, lse = attn.attn_fwd_paged_varlen(q, cache, table, i32(n), i32(0, n), causal=False, scale=1.0)
    want = ofp8.e4m3_value(cache.v.view(torch.uint8).cpu().numpy()) * f64(cache.v_scale)[..., None]
    assert np.array_equal(f64(o)[0], want.transpose(1, 0, 2, 3).reshape(n, d))
    assert ((lse - bits * 1024).abs() <= bits * 1024 * 2.0 ** -16 + 2.0 ** -20).all()


@pytest.mark.parametrize("new", [[200, 70], [3, 5], [1]])
@pytest.mark.parametrize("d", [64, 128])
def test_scales_far_from_one(new, d):
    lens = [n + 150 * i + 90 for i, n in enumerate(new)]
    _, cache, table, n, vals = paged_inputs(3, lens, 8, 2, d, 16, "e4m3")
    q, cu = normal(4, 8, sum(new), d), sums(new)
    o, lse = attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu))
    check_varlen(o, lse, q, vals, table, lens, cu, True, 1 / math.sqrt(d), "e4m3", "varlen scales")
    for by in (2.0 ** 60, 2.0 ** -60, -2.0 ** 90):
        c = cache._replace(k_scale=cache.k_scale * by)
        assert same(attn.attn_fwd_paged_varlen((q.float() / by).to(torch.bfloat16), c, table, n, i32(*cu)), (o, lse))
        c = cache._replace(v_scale=cache.v_scale * by)
        got = attn.attn_fwd_paged_varlen(q, c, table, n, i32(*cu))
        back = (got[0].float() / by).to(torch.bfloat16), got[1]
        if len(new) == 2 and new[0] > 32:
            assert same(back, (o, lse))
        check_varlen(*back, q, vals, table, lens, cu, True, 1 / math.sqrt(d), "e4m3", f"varlen scales {by:g}")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_rows_of_zeros(kind):
    # a query row of zeros weighs all keys alike; a cache row of zeros counts with its weight
    _, cache, table, n, vals = paged_inputs(3, [70, 300], 4, 2, 128, 16, kind)
    for new in ([50, 60], [2, 3]):
        q, cu = normal(4, 4, sum(new), 128), sums(new)
        q[:, 1::2] = 0
        o, lse = attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu))
        check_varlen(o, lse, q, vals, table, [70, 300], cu, True, 1 / math.sqrt(128), kind, f"varlen {kind} zeros")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("B", [33, 300, 700])
def test_many_requests_of_few_and_many_rows(B, kind, causal):
    # both kernels, each with its own requests, more of them than a warp or a block looks at in one step
    new = [(7 * i) % 4 for i in range(B)]
    new[5], new[B // 2], new[B - 1] = 40, 33, 130
    lens = [n + (61 * i) % 90 for i, n in enumerate(new)]
    _, cache, table, n, vals = paged_inputs(3, lens, 4, 2, 64, 16, kind)
    q, cu = normal(4, 4, sum(new), 64), sums(new)
    o, lse = attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu), causal=causal)
    check_varlen(o, lse, q, vals, table, lens, cu, causal, 1 / 8, kind, f"varlen {kind} {B} mixed")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows", [0, 1, 2, 70])
def test_one_short_request_with_padding(rows, kind):
    # one CTA a unit, no join; tokens behind the request's two are padding
    _, cache, table, n, vals = paged_inputs(3, [rows], 6, 2, 64, 16, kind)
    q = normal(4, 6, 5, 64)
    for new in (2, 0):
        out = torch.full((6, 5, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((6, 5), 7.0, device="cuda")
        attn.attn_fwd_paged_varlen(q, cache, table, n, i32(0, new), out=out, lse=lse)
        assert (out[:, new:] == 7).all() and (lse[:, new:] == 7).all()
        if new:
            check_varlen(out[:, :new].contiguous(), lse[:, :new].contiguous(), q[:, :new], vals, table, [rows], [0, new], True,
                         1 / 8, kind, f"varlen {kind} one short")
    assert attn.last_device_error() == 0


SHARES = [([3, 2], 4, 2), ([30, 3], 16, 2)]  # each group's requests, heads, K/V heads: few rows, many rows


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("each,H,KV", SHARES)
def test_shared_tables_outside_the_cache(each, H, KV, kind):
    args, own, vals = shared_inputs(each, [200, 90], H, KV, 64, 16, 31, 60, kind)
    q, cache, pt, pl, cu, table, lens = args
    lens = torch.full_like(lens, 50)
    pages = cache.k.shape[0]
    pt, table = pt.clone(), table.clone()
    table[:, :4] = torch.arange(table.shape[0] * 4, device="cuda").view(-1, 4) % pages  # (pages of others: real rows or NaN)
    cache = attn.KVCache(*(torch.nan_to_num(t.float(), 0.5).to(t.dtype) if t is not None and t.dtype != torch.uint8 else t
                           for t in cache))
    if kind == "bf16":
        vals = f64(cache.k), f64(cache.v)
    else:
        vals = [ofp8.e4m3_value(c.view(torch.uint8).cpu().numpy()) * f64(s)[..., None]
                for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    attn.attn_fwd_paged_shared(q, cache, pt, pl, cu, table, lens)
    assert attn.last_device_error() == 0
    pt[0, 3], pt[1, 5], table[1, 0], table[4, 3] = -1, pages, 2 ** 31 - 1, pages
    o, lse = attn.attn_fwd_paged_shared(q, cache, pt, pl, cu, table, lens)
    assert attn.decode_status(attn.last_device_error())["kind"] == 5
    vals = [np.concatenate([x, np.zeros_like(x[:1])]) for x in vals]
    pt[0, 3] = pt[1, 5] = table[1, 0] = table[4, 3] = pages
    check_shared(o, lse, (q, cache, pt, pl, cu, table, lens), vals, 1 / 8, kind, f"shared {kind} bad pages")


@pytest.mark.parametrize("each,H,KV", SHARES)
def test_shared_bad_prefix_sums_are_reported(each, H, KV):
    args, own, vals = shared_inputs(each, [200, 90], H, KV, 64, 16, 32, 60, "bf16")
    B = sum(each)
    for cu in ((1, 2, B), (0, 4, 2), (0, 2, B + 1)):
        attn.attn_fwd_paged_shared(*args[:4], i32(*cu), *args[5:])
        assert attn.decode_status(attn.last_device_error())["kind"] == 2


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("each,H,KV", SHARES)
def test_shared_padding_and_lengths_past_the_table(each, H, KV, kind):
    args, own, vals = shared_inputs(each, [64, 33], H, KV, 128, 32, 33, 90, kind)
    q, cache, pt, pl, cu, table, lens = args
    B = sum(each)
    ref = attn.attn_fwd_paged_shared(q, cache, pt[:, :2].contiguous(), i32(64, 33), cu, table, lens)
    got = attn.attn_fwd_paged_shared(q, cache, pt[:, :2].contiguous(), i32(10 ** 6, 33), cu, table, lens)
    assert same(ref, got)
    cut = cu.clone()
    cut[2] = B - 1
    out, lse = torch.full_like(ref[0], 7.0), torch.full_like(ref[1], 7.0)
    neg = lens.clone()
    neg[0] = -3  # as 0
    attn.attn_fwd_paged_shared(q, cache, pt, pl, cut, table, neg, out=out, lse=lse)
    assert (out[B - 1:] == 7).all() and (lse[B - 1:] == 7).all()
    neg[0] = 0
    check_shared(out[:-1], lse[:-1], (q[:-1], cache, pt, pl, cut, table[:-1], neg[:-1]), vals, 1 / math.sqrt(128), kind,
                 f"shared {kind} padded {B}")


@pytest.mark.parametrize("each,H,KV", SHARES)
def test_shared_nan_stays_in_its_group(each, H, KV):
    args, own, vals = shared_inputs(each, [200, 90], H, KV, 64, 16, 34, 60, "bf16")
    q, cache, pt, pl, cu, table, lens = args
    clean, _ = attn.attn_fwd_paged_shared(*args)
    cache.v[pt[0, 2].long(), 0, 3, 5] = float("nan")       # the first group's prefix: its requests' first heads
    q[sum(each) - 1, H - 1, 0, 7] = float("inf")
    o, _ = attn.attn_fwd_paged_shared(*args)
    bad = torch.isnan(o[:, :, 0])
    n, g = each[0], H // KV
    assert bad[:n, :g, 5].all() and bad[-1, H - 1].all() and int(bad.sum()) == n * g + 64
    keep = ~bad
    assert torch.equal(o[:, :, 0][keep], clean[:, :, 0][keep])


def test_far_pages_with_few_rows():
    d, KV, page, H = 128, 8, 128, 16
    pages = (1 << 33) // (2 * KV * page * d * 2) + 50
    both = torch.empty(pages, 2, KV, page, d, dtype=torch.bfloat16, device="cuda")
    args, own, vals = shared_inputs([2, 1], [300, 77], H, KV, d, page, 35, 200, "bf16")
    q, small, pt, pl, cu, table, lens = args
    m = small.k.shape[0]
    both[pages - m:, 0], both[pages - m:, 1] = small.k, small.v
    cache = attn.KVCache(both[:, 0], both[:, 1])
    o, lse = attn.attn_fwd_paged_shared(q, cache, pt + (pages - m), pl, cu, table + (pages - m), lens)
    check_shared(o, lse, args, vals, 1 / math.sqrt(d), "bf16", "shared far")
    qv = normal(3, H, 4, d)
    o, lse = attn.attn_fwd_paged_varlen(qv, cache, pt + (pages - m), pl, i32(0, 3, 4))
    check_varlen(o, lse, qv, vals, pt, [300, 77], [0, 3, 4], True, 1 / math.sqrt(d), "bf16", "varlen far, few rows")


def test_shared_two_streams_at_once():
    work = []
    for i, (each, H, KV) in enumerate(SHARES):
        args, _, _ = shared_inputs(each, [2000, 900], H, KV, 64, 16, 36 + i, 300, "e4m3")
        work.append(args)
    alone = [attn.attn_fwd_paged_shared(*w) for w in work]
    streams = [torch.cuda.Stream() for _ in work]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        got = [attn.attn_fwd_paged_shared(*w, stream=s) for w, s in zip(work, streams)]
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(alone, got))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_two_graphs_replayed_in_turn(kind):
    """Calls captured with workspaces of their own: neither leaves anything that the other reads."""
    lens, new = [500, 70, 900], [40, 3, 100]
    _, cache, table, n, vals = paged_inputs(37, lens, 8, 2, 128, 64, kind)
    q, cu = normal(38, 8, sum(new), 128), sums(new)
    attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu))
    graphs, outs = [], []
    for t in (cu, [0, 1, 2, 3]):
        x, c = q[:, :t[-1]].contiguous(), i32(*t)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((*attn.attn_fwd_paged_varlen(x, cache, table, n, c), x, c))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (o, lse, x, c), t in zip(outs, (cu, [0, 1, 2, 3])):
        check_varlen(o, lse, x, vals, table, lens, t, True, 1 / math.sqrt(128), kind, f"varlen {kind} graphs")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_read_back_and_written_again_is_the_same(kind):
    """Pages to rows to other pages: bf16 rows bit for bit; E4M3 rows within a step of their largest element's code."""
    lens, KV, d = [100, 0, 37, 1], 2, 128
    _, cache, table, n, vals = paged_inputs(39, lens, 4, KV, d, 16, kind)
    cu = i32(*sums(lens))
    k, v = attn.kv_read(cache, table, cu, sum(lens))
    other = attn.kv_cache(9, KV, 32, d, torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn)
    slots = torch.randperm(9 * 32, generator=torch.Generator().manual_seed(1))[:sum(lens)].cuda()
    attn.kv_write(k, v, other, slots)
    flat = torch.arange(9, dtype=torch.int32, device="cuda").view(1, 9)
    k2, v2 = attn.kv_read(other, flat, i32(0, 9 * 32), 9 * 32)
    for a, b in ((k, k2[:, slots]), (v, v2[:, slots])):
        if kind == "bf16":
            assert torch.equal(a, b)
        else:  # an E4M3 step at the row's largest element is 2^-4 of it or less, below it smaller, then bf16's
            top = a.float().abs().amax(-1, keepdim=True)
            assert ((a.float() - b.float()).abs() <= a.float().abs() * (2.0 ** -4 + 2.0 ** -7) + top * 2.0 ** -17).all()
