"""Work over a paged cache at the limits of what its entry points promise: more requests than a block looks at in one
step, prefix sums that are not sums, values that are not finite, scales at the ends of their range, groups without requests.

Tolerances as in test_parity_pages.py unless a test derives its own."""
import math

import numpy as np
import pytest
import torch

from io_aware_attention_attn_gb300 import attn
from oracle import fp8 as ofp8
from test_parity_generation import _gpu, i32, normal, paged_inputs  # noqa: F401
from test_parity_pages import check_shared, check_varlen, shared_inputs, sums

pytestmark = pytest.mark.gpu


def same(a, b):
    return torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_many_short_requests_of_many_rows(kind):
    # the first shares end after a tile or two, while other warps may still look for where theirs begin
    B, d = 520, 64
    new = [17 + i % 5 for i in range(B)]
    lens = [n + i % 3 for i, n in enumerate(new)]
    _, cache, table, n, vals = paged_inputs(3, lens, 4, 1, d, 16, kind)
    q, cu = normal(4, 4, sum(new), d), sums(new)
    first = attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu))
    for _ in range(50):
        assert same(first, attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu)))
    tokens = set(range(0, cu[-1], 53)) | {cu[-1] - 1}
    check_varlen(*first, q, vals, table, lens, cu, True, 1 / math.sqrt(d), kind, f"varlen {kind} many short", tokens)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("B", [5, 40, 300])
@pytest.mark.parametrize("T", [12, 60, 2000])
def test_nothing_is_computed_for_sums_that_fall(T, B, kind):
    # each of the requests behind a fall would be as many tokens as there are, together more than the host's check of sizes
    # counts: both kernels leave O and lse alone, with either way of adding the requests up
    _, cache, table, n, _ = paged_inputs(3, [40] * B, 4, 2, 64, 16, kind)
    q = normal(2, 4, T, 64)
    for cu in ([0] + [T if i % 2 else 0 for i in range(B)], [0] * (B - 1) + [T, T - 1], [0] * B + [-1]):
        o = torch.full((4, T, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((4, T), 7.0, device="cuda")
        attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu), out=o, lse=lse)
        assert attn.decode_status(attn.last_device_error())["kind"] == 2
        assert (o == 7).all() and (lse == 7).all()
    cu = [0] * B + [T]
    o, lse = attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu))
    assert torch.isfinite(o.float()[:, -40:]).all() and attn.last_device_error() == 0


def wide(table, pages):
    """The table in rows of `pages` entries: what lies behind a request's own is never read."""
    out = torch.full((table.shape[0], pages), -7, dtype=torch.int32, device="cuda")
    out[:, :table.shape[1]] = table
    return out


def test_batch_padded_to_a_long_context():
    # 32768 tokens' room over a table for 2^20 keys, of which one request uses little
    T, H, KV, d, new, L = 32768, 32, 8, 64, 700, 3000
    _, cache, table, n, vals = paged_inputs(3, [L], H, KV, d, 64, "bf16")
    q = normal(4, H, T, d)
    out = torch.full((H, T, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, T), 7.0, device="cuda")
    attn.attn_fwd_paged_varlen(q, cache, wide(table, 1 << 14), n, i32(0, new), out=out, lse=lse)
    assert attn.last_device_error() == 0 and (out[:, new:] == 7).all() and (lse[:, new:] == 7).all()
    check_varlen(out[:, :new], lse[:, :new], q[:, :new], vals, table, [L], [0, new], True, 1 / 8, "bf16", "varlen long context",
                 set(range(0, new, 23)) | {new - 1})


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,old,H,KV,d", [([5], [295], 16, 4, 64), ([2] * 4, [900, 1, 0, 500], 32, 8, 128),
                                            ([8], [4000], 32, 8, 128), ([1, 3, 60], [100, 0, 40], 8, 2, 64)])
def test_tables_wider_than_the_lengths(new, old, H, KV, d, kind):
    # as a server keeps them, for its longest context: other shares, joins where the narrow table has none
    lens = [a + b for a, b in zip(new, old)]
    _, cache, table, n, vals = paged_inputs(5, lens, H, KV, d, 16, kind)
    q, cu = normal(6, H, sum(new), d), sums(new)
    for pages in (table.shape[1], 4 * table.shape[1], 2048):
        o, lse = attn.attn_fwd_paged_varlen(q, cache, wide(table, pages), n, i32(*cu))
        check_varlen(o, lse, q, vals, table, lens, cu, True, 1 / math.sqrt(d), kind, f"varlen {kind} table of {pages}")
    assert attn.last_device_error() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("each,H,KV", [([4], 16, 16), ([4] * 12, 16, 4), ([40, 1], 16, 2)])
def test_shared_tables_wider_than_the_lengths(each, H, KV, kind):
    args, own, vals = shared_inputs(each, [90 * (i + 1) for i in range(len(each))], H, KV, 64, 16, 7, 30, kind)
    q, cache, pt, pl, cu, table, lens = args
    for a, b in ((pt.shape[1], 2048), (2048, table.shape[1]), (2048, 2048)):
        o, lse = attn.attn_fwd_paged_shared(q, cache, wide(pt, a), pl, cu, wide(table, b), lens)
        check_shared(o, lse, args, vals, 1 / 8, kind, f"shared {kind} tables of {a}, {b}")
    assert attn.last_device_error() == 0


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,L,H,KV", [(10, 4, 4, 2), (10, 4, 8, 1), (20, 7, 1, 1), (60, 9, 1, 1), (200, 130, 4, 2)])
def test_tokens_that_see_nothing_beside_values_that_are_not_finite(new, L, H, KV, kind, bad):
    # more tokens than rows: O = 0 and lse = -inf for the first ones, whatever the rows hold that others of their unit see
    _, cache, table, n, vals = paged_inputs(3, [L], H, KV, 64, 16, kind, junk=False)
    page = table[0, 0].long()
    if kind == "bf16":
        cache.v[page, :, 2, 5] = bad
    else:
        cache.v_scale[page, :, 2] = bad
    q = normal(4, H, new, 64)
    o, lse = attn.attn_fwd_paged_varlen(q, cache, table, n, i32(0, new))
    blind = new - L
    assert (o[:, :blind] == 0).all() and torch.isneginf(lse[:, :blind]).all()
    assert not torch.isfinite(o[:, blind + 2:, 5].float()).any() and torch.isfinite(lse[:, blind:]).all()


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("new,H,KV", [([3, 3], 2, 1), ([4, 2], 4, 1), ([6, 5], 4, 1), ([9, 12], 4, 1), ([40, 70], 4, 2)])
def test_query_rows_with_an_infinity(new, H, KV, sign):
    # over E4M3 pages such a row gives NaN, also where all its products have one sign; the other rows are as without it
    lens = [n + 150 for n in new]
    _, cache, table, n, _ = paged_inputs(3, lens, H, KV, 64, 16, "e4m3", junk=False)
    codes = cache.k.view(torch.uint8)
    codes[..., 7] = 0x80 | codes[..., 7].clamp(1, 0x7E)    # negative, none of them zero
    q, cu = normal(4, H, sum(new), 64), sums(new)
    clean = attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu))
    q[H - 1, 1, 7] = sign * math.inf
    o, lse = attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu))
    assert torch.isnan(o[H - 1, 1]).all() and torch.isnan(lse[H - 1, 1])
    o[H - 1, 1], lse[H - 1, 1] = clean[0][H - 1, 1], clean[1][H - 1, 1]
    assert same((o, lse), clean)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("each,H,KV", [([2, 1], 2, 1), ([4, 3], 4, 1), ([40, 30], 4, 2)])
def test_shared_query_rows_with_an_infinity(each, H, KV, sign):
    args, own, _ = shared_inputs(each, [200, 90], H, KV, 64, 16, 31, 60, "e4m3")
    q, cache, *rest = args
    cache = attn.KVCache(*(torch.nan_to_num(t.float(), 0.5).to(t.dtype) if t.dtype == torch.float32 else t for t in cache))
    codes = cache.k.view(torch.uint8)
    codes[..., 7] = 0x80 | codes[..., 7].clamp(1, 0x7E)
    clean = attn.attn_fwd_paged_shared(q, cache, *rest)
    q[1, H - 1, 0, 7] = sign * math.inf
    o, lse = attn.attn_fwd_paged_shared(q, cache, *rest)
    assert torch.isnan(o[1, H - 1]).all() and torch.isnan(lse[1, H - 1]).all()
    o[1, H - 1], lse[1, H - 1] = clean[0][1, H - 1], clean[1][1, H - 1]
    assert same((o, lse), clean)


@pytest.mark.parametrize("new", [[200, 70], [3, 5], [1]])
@pytest.mark.parametrize("d", [64, 128])
def test_key_scales_at_their_limit(new, d):
    # a power of two that K's scales have and the query does not changes no bit, up to 2^100 and far down
    lens = [n + 150 * i + 90 for i, n in enumerate(new)]
    _, cache, table, n, _ = paged_inputs(3, lens, 8, 2, d, 16, "e4m3", junk=False)
    top = math.floor(math.log2(100.0 * float(cache.k_scale.abs().max()))) - 6
    q, cu = normal(4, 8, sum(new), d), sums(new)
    clean = attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu))
    for by in (2.0 ** (99 - top), -2.0 ** (99 - top), 2.0 ** -100):
        c = cache._replace(k_scale=cache.k_scale * by)
        assert float(c.k_scale.abs().max()) <= 2.0 ** 100
        assert same(attn.attn_fwd_paged_varlen((q.float() / by).to(torch.bfloat16), c, table, n, i32(*cu)), clean)


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("at", [0, 60, -1])
@pytest.mark.parametrize("new", [[3, 5, 2], [16, 12, 9], [8, 300, 33], [256, 256, 1]])
def test_values_that_are_not_finite_stay_in_their_request_and_column(new, at, kind, bad):
    # a row of V that some or none of its request's other new tokens see: what it reaches is not finite, and nothing else
    # changes a bit; a row of K reaches the tokens that see it, all of them and only those
    H, KV, d = 8, 2, 64
    lens = [n + 64 * (i % 2) for i, n in enumerate(new)]
    _, cache, table, n, _ = paged_inputs(3, lens, H, KV, d, 16, kind, junk=False)
    q, cu = normal(4, H, sum(new), d), sums(new)
    clean = attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu))
    row = min(at % lens[1], lens[1] - 1) if at >= 0 else lens[1] - 1
    page = table[1, row // 16].long()
    mine = slice(cu[1], cu[2])
    sees = torch.arange(new[1], device="cuda") + lens[1] - new[1] >= row
    assert sees.any()

    def with_bad(side):
        x = getattr(cache, side).clone()
        if kind == "bf16":
            x[page, 0, row % 16, 5] = bad
        else:
            x.view(torch.uint8)[page, 0, row % 16, 5] = 0x7F
        return attn.attn_fwd_paged_varlen(q, cache._replace(**{side: x}), table, n, i32(*cu))

    o, lse = with_bad("v")
    part = o[:H // KV, mine, 5]
    assert not torch.isfinite(part[:, sees].float()).any()
    kept = torch.isfinite(part.float())
    assert torch.equal(part[kept], clean[0][:H // KV, mine, 5][kept])
    part.copy_(clean[0][:H // KV, mine, 5])
    assert same((o, lse), clean)

    o, lse = with_bad("k")
    part = o[:H // KV, mine]
    assert torch.isnan(part[:, sees].float()).all() if bad != bad else not torch.isfinite(lse[:H // KV, mine][:, sees]).all()
    part[:, sees], lse[:H // KV, mine][:, sees] = clean[0][:H // KV, mine][:, sees], clean[1][:H // KV, mine][:, sees]
    assert same((o, lse), clean)


def bf16_of(x):
    """float64 values rounded once to bf16, as float64."""
    m, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e, -125) - 8)
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.where(np.isfinite(x), np.rint(x / step) * step, x)
        return np.where(np.abs(y) >= 2.0 ** 128, np.copysign(np.inf, y), y)


@pytest.mark.parametrize("d", [64, 128])
def test_rows_read_are_rounded_once(d):
    # every code against scales whose products lie beside the middle of two bf16 numbers, where a rounding to fp32 on the way
    # would be seen, and the ends of the range
    r = np.random.default_rng(5)
    sig = []
    for s in (9, 11, 13, 15, 8):                            # significands of codes
        middle = (2 * r.integers(1 << 7, 1 << 8, 300) + 1) * 2.0 ** r.integers(18, 20, 300)
        sig += [np.floor(middle / s), np.floor(middle / s) + 1]
    sig = np.concatenate(sig)
    m, _ = np.frexp(sig)
    scale = np.concatenate([m, -m * 2.0 ** 20, m * 2.0 ** -120, m * 2.0 ** -130, m * 2.0 ** -140, m * 2.0 ** 127, m * 2.0 ** 119,
                            [0.0, -0.0, np.inf, -np.inf, np.nan, 1.0, 2.0 ** -149]]).astype(np.float32)
    rows = 256 // d                                        # of one scale, so that it meets every code
    n = len(scale) * rows
    page, KV = 16, 2
    pages = -(-n // page)
    cache = attn.kv_cache(pages, KV, page, d, torch.float8_e4m3fn)
    flat = torch.zeros(pages * page, dtype=torch.float32)
    flat[:n] = torch.from_numpy(np.repeat(scale, rows))
    codes = torch.arange(256, dtype=torch.uint8).view(rows, d).repeat(-(-pages * page // rows), 1)[:pages * page]
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        c.view(torch.uint8).copy_(codes.view(pages, 1, page, d).expand(-1, KV, -1, -1))
        s.copy_(flat.view(pages, 1, page).expand(-1, KV, -1))
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1)
    k, v = attn.kv_read(cache, table, i32(0, n), n)
    with np.errstate(invalid="ignore", over="ignore"):
        exact = ofp8.e4m3_value(codes.numpy())[:n] * flat[:n].numpy().astype(np.float64)[:, None]  # 28 bits: exact
    want = bf16_of(exact)
    twice = torch.from_numpy(exact).float().to(torch.bfloat16).double().numpy()
    assert (twice != want).sum() > 100 + np.isnan(want).sum()        # (the inputs do tell the two apart)
    for x in (k, v):
        for h in range(KV):
            got = x[h].double().cpu().numpy()
            assert np.array_equal(got, want, equal_nan=True)
            assert np.array_equal(np.signbit(got[~np.isnan(want)]), np.signbit(want[~np.isnan(want)]))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("each,H,KV", [([64] + [0] * 31, 32, 8), ([0] * 7 + [40, 3], 8, 2), ([30] + [1] * 7, 16, 4), ([1] * 40 + [90], 4, 1)])
def test_shared_groups_much_unlike(each, H, KV, kind):
    # which kernel and how many rows at once go by the mean over the groups, also those without requests
    args, own, vals = shared_inputs(each, [300 + 41 * (i % 5) for i in range(len(each))], H, KV, 64, 16, 41, 30, kind)
    o, lse = attn.attn_fwd_paged_shared(*args)
    check_shared(o, lse, args, vals, 1 / 8, kind, f"shared {kind} {each[:1]}x{len(each)} unlike")
    assert attn.last_device_error() == 0


def test_rows_written_with_values_that_are_not_finite():
    # a row's scale is of its numbers; with an infinity the numbers' codes are 0 (x / inf) and the infinity's that of NaN
    KV, d, T = 2, 64, 6
    k = normal(1, KV, T, d)
    k[:, 1, 3] = math.nan
    k[:, 2, 5] = -math.inf
    k[:, 3] = math.nan
    k[:, 4, :9] = math.inf
    cache = attn.kv_cache(1, KV, 16, d, torch.float8_e4m3fn)
    both = attn.kv_cache(1, KV, 16, d, torch.float8_e4m3fn)
    slots = torch.arange(T, device="cuda")
    attn.kv_write(k, k, cache, slots)
    x = torch.cat([k, k, k]).transpose(0, 1).reshape(T, -1).contiguous()
    attn.qkv_rope(x, KV, KV, cache=both, slots=slots)
    for a, b in ((cache.k, both.k), (cache.v, both.v)):
        va, vb = (ofp8.e4m3_value(c.view(torch.uint8).cpu().numpy())[:, :, :T] for c in (a, b))
        assert np.array_equal(va, vb, equal_nan=True) and np.isnan(va).sum() == KV * (1 + 1 + d + 9)
    for a, b in ((cache.k_scale, both.k_scale), (cache.v_scale, both.v_scale)):
        assert torch.equal(a[:, :, :T], b[:, :, :T]) and not torch.isnan(a[:, :, :T]).any()
