"""GPU checks of the generation path at its edges, against the float64 oracle or in exact numbers: rows of
zeros and of the smallest values through the step before attention, tokens that belong to no request,
and batches of which every thread of a block looks at several requests (tolerances as in
test_parity_generation.py)."""
import math

import numpy as np
import pytest
import torch

from io_aware_attention_attn_gb300 import attn
from oracle import generation as gen
from test_parity_generation import _gpu, EPS, bf16_tol, check_paged, f64, i32, normal, paged_inputs, within  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------ the step before attention
@pytest.mark.parametrize("d,H,KV,rot", [(64, 2, 1, 0), (128, 3, 3, 128), (64, 12, 4, 32)])
def test_rows_below_the_normal_range_of_a_scale(d, H, KV, rot):
    # amax / 448 below 2^-126, fp32's normal range: scale 1 and codes 0, in key and value rows
    w = H + 2 * KV
    rows = normal(7, 4, w, d)
    rows[1, H:] = 2.0 ** -120 * torch.sign(rows[1, H:].float())
    rows[2, H:] = 0
    rows[3, H:] = 2.0 ** -110 * rows[3, H:].float().sign()   # above it: amax / 448 as ever
    cache = attn.kv_cache(1, KV, 16, d, torch.float8_e4m3fn)
    cache.k.view(torch.uint8).fill_(0x3A)
    cache.v.view(torch.uint8).fill_(0x3A)
    pos, f = torch.zeros(4, dtype=torch.int32, device="cuda"), attn.rope_inv_freq(rot) if rot else None
    attn.qkv_rope(rows.view(4, -1), H, KV, pos if rot else None, f, cache=cache,
                  slots=torch.tensor([9, 0, 15, 4], device="cuda"))
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        raw = codes.view(torch.uint8)[0]
        assert (scale[0, :, [0, 15]] == 1).all() and ((raw[:, [0, 15]] & 0x7F) == 0).all()
        got = scale[0, :, 4].double()
        assert ((got - 2.0 ** -110 / 448).abs() <= 2.0 ** -24 * got).all()
        assert ((raw[:, 4] & 0x7F) == 0x7E).all()             # +-448
        assert (scale[0, :, [1, 2, 3, 5, 8, 10, 14]] == 0).all() and (raw[:, [1, 3, 5, 14]] == 0x3A).all()


@pytest.mark.parametrize("kind", ["none", "bf16", "e4m3"])
@pytest.mark.parametrize("d,H,KV", [(64, 4, 2), (128, 5, 1)])
def test_norm_of_rows_of_zeros(d, H, KV, kind):
    # divides by sqrt(eps): zeros forward; backward dx = R^T g w / sqrt(eps) and no share of dw
    T = 5
    rows = normal(3, T, H + 2 * KV, d)
    rows[2] = 0
    wq, wk = (1 + 0.3 * normal(4, 2, d)).unbind(0)
    pos, f = torch.arange(T, dtype=torch.int32, device="cuda"), attn.rope_inv_freq(d)
    cache = slots = None
    if kind != "none":
        cache = attn.kv_cache(1, KV, 16, d, torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn)
        slots = torch.arange(T, device="cuda")
    q, k, v = attn.qkv_rope(rows.view(T, -1), H, KV, pos, f, wq=wq, wk=wk, eps=EPS, cache=cache, slots=slots)
    for t in (q, k, v):
        assert (t[:, 2] == 0).all() and torch.isfinite(t).all() and (t[:, 1] != 0).any()
    if kind == "e4m3":
        assert (cache.k_scale[0, :, 2] == 1).all() and (cache.k.float()[0, :, 2] == 0).all()
    dq, dk, dv = normal(5, H, T, d), normal(6, KV, T, d), normal(8, KV, T, d)
    dx, dwq, dwk = attn.qkv_rope_bwd(dq, dk, dv, rows.view(T, -1), pos, f, wq=wq, wk=wk, eps=EPS)
    keep = [0, 1, 3, 4]
    rest = attn.qkv_rope_bwd(dq[:, keep].contiguous(), dk[:, keep].contiguous(), dv[:, keep].contiguous(),
                             rows[keep].reshape(4, -1), pos[keep].contiguous(), f, wq=wq, wk=wk, eps=EPS)
    g = [f64(t) for t in (dq, dk, dv)]
    rdx, rq, rk = gen.qkv_rope_bwd(*g, f64(rows).reshape(T, -1), H, KV, d, np.arange(T), f64(f), False, f64(wq),
                                   f64(wk), EPS)
    # 2^-18 of r |g| |w|, |g| at most the sum of a pair's; r = 1 / sqrt(eps) in the row of zeros
    pairs = np.concatenate([np.abs(t[:, 2]).reshape(len(t), 2, d // 2).sum(1).repeat(2, 0).reshape(len(t), d)
                            for t in g])
    ww = np.concatenate([np.tile(np.abs(f64(w)), (n, 1)) for w, n in ((wq, H), (wk, KV))] + [np.ones((KV, d))])
    e = 2.0 ** -18 * pairs * ww / math.sqrt(EPS)
    e[H + KV:] = 0
    within(f64(dx)[2].reshape(-1, d), rdx[2].reshape(-1, d), bf16_tol(rdx[2].reshape(-1, d), e), f"zero row dx {d}")
    assert torch.equal(dx[keep], rest[0])
    for got, ref, t, x in ((dwq, rq, g[0], f64(rows)[:, :H]), (dwk, rk, g[1], f64(rows)[:, H:H + KV])):
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
        ga = np.abs(t).transpose(1, 0, 2).reshape(T, -1, 2, d // 2).sum(2)
        within(f64(got), ref, 2.0 ** -16 * (np.concatenate([ga, ga], -1) * np.abs(x) * r).sum((0, 1)), f"zero row dw {d}")


@pytest.mark.parametrize("batched", [False, True])
def test_rows_past_2_32_elements(batched):
    # the last rows of projection rows of over 2^32 elements, against a call on those rows alone
    H, KV, d, n = 16, 8, 128, 64
    width = (H + 2 * KV) * d
    T = (1 << 32) // width + 4096 + n
    assert T % 2 == 0
    rows = torch.zeros(T, width, dtype=torch.bfloat16, device="cuda")
    assert (T - n) * width > 1 << 32
    rows[-n:] = normal(70, n, width)
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    pos[-n:] = torch.arange(n)
    f = attn.rope_inv_freq(d)
    wq, wk = (1 + 0.2 * normal(71, 2, d)).unbind(0)
    kw = dict(inv_freq=f, wq=wq, wk=wk, eps=EPS)
    lead = (lambda t: t.view(2, T // 2, *t.shape[1:])) if batched else (lambda t: t)
    tail = (lambda t: t[1, :, -n:]) if batched else (lambda t: t[:, -n:])
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    slots[-n:] = torch.arange(n)
    caches = [attn.kv_cache(n // 16, KV, 16, d, torch.float8_e4m3fn) for _ in range(2)]
    got = attn.qkv_rope(lead(rows), H, KV, lead(pos), cache=caches[0], slots=lead(slots), **kw)
    want = attn.qkv_rope(rows[-n:], H, KV, pos[-n:].contiguous(), cache=caches[1], slots=slots[-n:].contiguous(), **kw)
    for a, b in zip(got, want):
        assert torch.equal(tail(a), b)
    for a, b in zip(*caches):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and (a.view(torch.uint8) != 0).any()
    del got
    dy = [torch.zeros(*((2, h, T // 2, d) if batched else (h, T, d)), dtype=torch.bfloat16, device="cuda")
          for h in (H, KV, KV)]
    small = [normal(72 + i, h, n, d) for i, h in enumerate((H, KV, KV))]
    for t, g in zip(dy, small):
        tail(t).copy_(g)
    dx, dwq, dwk = attn.qkv_rope_bwd(*dy, lead(rows), lead(pos), **kw)
    rx, rq, rk = attn.qkv_rope_bwd(*small, rows[-n:], pos[-n:].contiguous(), **kw)
    assert torch.equal(dx.view(T, width)[-n:], rx) and not dx.view(T, width)[0].any()
    # dw: the same terms g x r in another order, n H <= 2^10 of them, each sum within 2^10 u of sum |g x r|,
    # |g| at most the sum of a pair's |dy|
    x = rows[-n:].view(n, H + 2 * KV, d)[:, :H + KV].double()
    x = (x.abs() / (x.square().mean(-1, keepdim=True) + EPS).sqrt()).transpose(0, 1)
    for a, b, dyh, xh in ((dwq, rq, small[0], x[:H]), (dwk, rk, small[1], x[H:])):
        pair = dyh.double().abs().view(-1, n, 2, d // 2).sum(2).repeat(1, 1, 2)
        assert ((a - b).abs() <= 2 * 2.0 ** -14 * (pair * xh).sum((0, 1))).all() and b.any()


# ------------------------------------------------------------------------------------------- slots
@pytest.mark.parametrize("cu,T", [((0, 2, 4), 6), ((1, 2, 6), 6), ((3, 3, 3), 5), ((0, 9, 4), 6), ((0, 4, 2, 6), 6),
                                  ((-2, 3, 300), 290), ((0, 0, 0), 300)])
def test_prefix_sums_that_leave_tokens_out(cu, T):
    # clamped into [0, T]; a token of no request: slot -1, position 0; the status word says so
    B, page = len(cu) - 1, 16
    table = torch.full((B, 20), -1, dtype=torch.int32, device="cuda")
    table[:, 0] = torch.arange(50, 50 + B)
    free = torch.arange(100, 160, dtype=torch.int32, device="cuda")
    slots, pos, t, lens, head = attn.kv_slots(i32(*[3] * B), i32(*cu), T, table, free, i32(2), page)
    assert attn.decode_status(attn.last_device_error())["kind"] == 2
    c = [min(max(x, 0), T) for x in cu]
    new = [max(b - a, 0) for a, b in zip(c, c[1:])]
    assert lens.tolist() == [3 + n for n in new]
    need = [-(-(3 + n) // page) - 1 for n in new]
    assert head.tolist() == [2 + sum(need)]
    want = []
    for i in range(T):  # where the sums fall again, the request is the one that a search by halves finds
        a, b = 0, B
        while b - a > 1:
            m = (a + b) // 2
            a, b = (m, b) if c[m] <= i else (a, m)
        if not c[a] <= i < c[a + 1]:
            want.append((-1, 0))
            continue
        at = 3 + i - c[a]
        j = at // page
        entry = 50 + a if j == 0 else 100 + 2 + sum(need[:a]) + j - 1
        want.append((entry * page + at % page, at))
    assert list(zip(slots.tolist(), pos.tolist())) == want
    assert attn.last_device_error() == 0


# -------------------------------------------------------------------------- attention over pages
LARGE = [  # more than 256 requests: a block looks at them together, each thread at several
    ([53 * i % 97 for i in range(2000)], 4, 2, 64, 16),
    ([29 * i % 70 for i in range(1201)], 16, 1, 128, 32),
    ([5] * 1000 + [3000] + [0] * 500 + [200] * 7, 32, 1, 64, 64),
    ([1] * 2500, 2, 2, 128, 16),
    ([0] * 700 + [1] + [0] * 300, 24, 1, 128, 64),
    ([9000] + [0] * 600 + [4000, 63, 64, 65], 8, 2, 128, 128),
    ([17 * i % 300 for i in range(513)], 12, 1, 64, 256),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,H,KV,d,page", LARGE)
def test_large_batches(lens, H, KV, d, page, kind):
    q, cache, table, n, vals = paged_inputs(len(lens) + H, lens, H, KV, d, page, kind)
    o, lse = attn.attn_fwd_paged(q, cache, table, n)
    again = attn.attn_fwd_paged(q, cache, table, n)
    assert torch.equal(o.view(torch.int16), again[0].view(torch.int16)) and torch.equal(lse, again[1])
    check_paged(o, lse, q, vals, table, lens, 1 / math.sqrt(d), kind, f"paged {kind} {len(lens)} requests H{H}")
