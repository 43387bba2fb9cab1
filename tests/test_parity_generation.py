"""GPU parity of the generation path against the float64 oracle: the step before attention and its
backward, slots of new tokens, attention over the paged cache, and a run of them together.

Tolerances, from the arithmetic (u = 2^-24, half a step of fp32; half a step of bf16 is 2^-8 of the
value, of E4M3 2^-4, below its normal range 2^-10 in code units):

* q, k: sum of squares of d <= 128 terms: 16 fused adds in a lane and 3 across lanes, halved by the
  root: 10 u; root 4 u, two products 2 u; sin and cos 4 u + pi u from the rounded angle, rope_scale 1 u,
  product and add 2 u: at most 28 u < 2^-19 of (|n_a| + |n_b|) rope_scale; then one rounding to bf16.
* dx = r (g w - x r^2 mean(g w x)): g as above (11 u), the sum 128 products in 22 u: 2^-18 of
  r |g||w| + |x| r^3 mean|g w x|, with |g| the rotation of absolute values; then bf16.
* dw: terms within 28 u, and fewer than 200 adds one after another: 2^-16 of sum |g x r|.
* O: P to bf16 (2^-8) or f16 (2^-11, and 2^-25 of the largest V scale x 448 a key below f16's normal
  range, relative to a row sum of at least 1); P's own relative error e_s: the score's 128-term fp32 sum
  may be truncated a term (2^-23 each) and exp2 adds 2^-21: e_s = 2^-16 Z + 2^-20, Z = scale max
  sum |q k|; so |dO| <= (P rounding + 2 e_s) A with A = P|V|, then bf16.  lse: e_s + 2^-20 (1 + |lse|).
"""
import math

import numpy as np
import pytest
import torch

from io_aware_attention_attn_gb300 import accounting as acc
from io_aware_attention_attn_gb300 import attn
from oracle import attention as orc
from oracle import fp8 as ofp8
from oracle import generation as gen

from parity_util import record

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from io_aware_attention_attn_gb300 import build
    build.build()
    yield
    assert attn.last_device_error() == 0


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64) if t.dtype != torch.float64 \
        else t.cpu().numpy()


def normal(seed, *shape, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    return (sigma * torch.randn(*shape, generator=g)).to(torch.bfloat16).cuda()


def within(got, ref, tol, what):
    assert np.isfinite(got).all(), f"{what}: not finite"
    err = np.abs(got - ref)
    record("gen", what, {"max_abs": float(err.max(initial=0.0)),
                         "max_err_over_tol": float((err / np.maximum(tol, 1e-300)).max(initial=0.0))})
    assert (err <= tol).all(), f"{what}: {int((err > tol).sum())} of {err.size} over the bound, " \
                               f"worst {float((err / tol).max()):.3g} of it"


def bf16_tol(ref, e):
    return e + acc.bf16_half_ulp(np.abs(ref) + e)


def rope_err(qkv, H, KV, d, pos, f, inter, wq, wk, scale):
    """2^-19 of (|n_a| + |n_b|) scale, laid out like q and k."""
    x = qkv.reshape(len(qkv), H + 2 * KV, d)
    nf, out = len(f), []
    for h in range(H + KV):
        n = np.abs(gen.norm(x[:, h], wq if h < H else wk, EPS))
        s = n.copy()
        a, b = (np.arange(0, 2 * nf, 2), np.arange(1, 2 * nf, 2)) if inter else \
            (np.arange(nf), np.arange(nf, 2 * nf))
        s[:, a] = s[:, b] = (n[:, a] + n[:, b]) * abs(scale)
        out.append(s * 2.0 ** -19)
    return np.stack(out[:H]), np.stack(out[H:])


# ------------------------------------------------------------------------ the step before attention
ROPE = [
    # B, N, H, KV, d, rot, inter, norm, far, rope_scale, pad (elements between rows)
    (1, 1, 1, 1, 64, 64, False, True, 0, 1.0, 0),
    (1, 7, 3, 1, 128, 128, False, True, 0, 1.0, 0),
    (2, 5, 4, 2, 128, 128, True, True, 0, 1.25, 8),
    (1, 33, 8, 8, 64, 48, True, False, 0, 1.0, 64),
    (3, 17, 6, 3, 128, 112, False, True, 0, 0.5, 0),
    (1, 9, 5, 5, 64, 16, False, False, 0, 1.0, 24),
    (4, 1, 32, 8, 128, 128, False, True, 1 << 20, 1.0, 0),
    (2, 1, 16, 1, 64, 32, True, True, (1 << 31) - 1, 1.0, 0),
    (1, 12, 2, 2, 128, 0, False, True, 0, 1.0, 0),
    (2, 1300, 6, 2, 64, 64, False, True, 0, 1.0, 0),     # four tokens a CTA, a ragged end
    (1, 2435, 2, 1, 128, 96, True, True, 0, 1.0, 0),
]


def rope_inputs(seed, B, N, H, KV, d, rot, norm, far, pad):
    width = (H + 2 * KV) * d
    store = normal(seed, B, N, width + pad)
    qkv = store[..., :width]
    g = torch.Generator().manual_seed(seed + 1)
    pos = torch.randint(max(far - 4096, 0), far, (B, N), generator=g) if far else \
        torch.arange(N).repeat(B, 1)
    pos = pos.to(torch.int32).cuda()
    f = attn.rope_inv_freq(rot, 500000.0) if rot else None
    wq, wk = (1 + 0.3 * normal(seed + 2, 2, d)).unbind(0) if norm else (None, None)
    return qkv, pos, f, wq, wk


@pytest.mark.parametrize("kind", ["none", "bf16", "e4m3"])
@pytest.mark.parametrize("B,N,H,KV,d,rot,inter,norm,far,rs,pad", ROPE)
def test_qkv_rope(B, N, H, KV, d, rot, inter, norm, far, rs, pad, kind):
    qkv, pos, f, wq, wk = rope_inputs(11 * N + H, B, N, H, KV, d, rot, norm, far, pad)
    T, page = B * N, 16
    cache = slots = None
    if kind != "none":
        pages = -(-T // page) + 3
        cache = attn.kv_cache(pages, KV, page, d,
                              torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn)
        for t in cache:
            if t is not None:
                t.view(torch.uint8).fill_(0x3A)
        order = torch.randperm(pages * page, generator=torch.Generator().manual_seed(N))[:T]
        slots = order.to(torch.int64).reshape(B, N).cuda()
        slots.view(-1)[::5] = -1
    q, k, v = attn.qkv_rope(qkv, H, KV, pos if rot else None, f, inter, wq, wk, EPS, rs, cache, slots)
    only = attn.qkv_rope(qkv, H, KV, pos if rot else None, f, inter, wq, wk, EPS, rs, with_kv=False)
    torch.cuda.synchronize()
    assert only[1] is None and torch.equal(only[0].view(torch.int16), q.view(torch.int16))
    x = f64(qkv).reshape(T, -1)
    ff = f64(f) if rot else np.zeros(0)
    ww = [None if w is None else f64(w) for w in (wq, wk)]
    pp = pos.cpu().numpy().reshape(-1)
    rq, rk, rv = gen.qkv_rope(x, H, KV, d, pp, ff, inter, *ww, EPS, rs)
    eq, ek = rope_err(x, H, KV, d, pp, ff, inter, *ww, rs)
    what = f"rope B{B} N{N} H{H} KV{KV} d{d} rot{rot}"

    def rows(t):  # [B, heads, N, d] -> [heads, T, d]
        return f64(t).transpose(1, 0, 2, 3).reshape(t.shape[1], T, d)

    within(rows(q), rq, bf16_tol(rq, eq), what + " q")
    within(rows(k), rk, bf16_tol(rk, ek), what + " k")
    assert np.array_equal(rows(v), rv)
    if kind == "none":
        return
    at = slots.cpu().numpy().reshape(-1)
    kept = at >= 0
    untouched = np.ones(cache.k.shape[0] * page, dtype=bool)
    untouched[at[kept]] = False
    for codes, scale, ref, e in ((cache.k, cache.k_scale, rk, ek), (cache.v, cache.v_scale, rv, 0 * rv)):
        raw = codes.view(torch.uint8).cpu().numpy().reshape(-1, KV, page, codes.view(torch.uint8).shape[-1])
        raw = raw.transpose(0, 2, 1, 3).reshape(len(untouched), -1)
        assert (raw[untouched] == 0x3A).all()
        ref, e = ref[:, kept].transpose(1, 0, 2), e[:, kept].transpose(1, 0, 2)
        if kind == "bf16":
            got = f64(codes).transpose(0, 2, 1, 3).reshape(-1, KV, d)[at[kept]]
            within(got, ref, bf16_tol(ref, e), what + " bf16 cache")
            continue
        vals = ofp8.e4m3_value(codes.view(torch.uint8).cpu().numpy()).transpose(0, 2, 1, 3)
        sc = f64(scale).transpose(0, 2, 1).reshape(-1, KV)[at[kept]]
        ref_sc = np.abs(ref).max(-1) / 448
        within(sc, ref_sc, ref_sc * 2.0 ** -23 + e.max(-1) / 448, what + " scale")
        got = vals.reshape(-1, KV, d)[at[kept]] * sc[..., None]
        tol = 2.0 ** -4 * (np.abs(ref) + e) + 2.0 ** -10 * sc[..., None] + 2 * e + 2.0 ** -22 * np.abs(ref)
        within(got, ref, tol, what + " e4m3 cache")


def test_rope_rows_of_zeros_and_long_heads():
    # a zero row has scale 1 and codes 0 in an E4M3 cache; its norm divides by sqrt(eps)
    qkv = torch.zeros(3, 4 * 64, dtype=torch.bfloat16, device="cuda")
    qkv[1, 64:128] = 2.0 ** -130   # amax / 448 below fp32's normal range: scale 1, codes 0
    cache = attn.kv_cache(1, 1, 16, 64, torch.float8_e4m3fn)
    slots = torch.tensor([0, 5, 15], device="cuda")
    attn.qkv_rope(qkv, 2, 1, cache=cache, slots=slots)
    torch.cuda.synchronize()
    assert (cache.k.float() == 0).all() and (cache.v.float() == 0).all()
    assert cache.k_scale[0, 0].nonzero().flatten().tolist() == [0, 5, 15]
    assert (cache.k_scale[0, 0, [0, 5, 15]] == 1).all() and (cache.v_scale[0, 0, [0, 5, 15]] == 1).all()


def test_rope_slot_past_the_cache_is_reported_and_not_stored():
    qkv = normal(3, 4, 6 * 64)
    cache = attn.kv_cache(2, 2, 16, 64)
    slots = torch.tensor([31, 32, 1 << 40, -7], device="cuda")
    attn.qkv_rope(qkv, 2, 2, cache=cache, slots=slots)
    assert attn.decode_status(attn.last_device_error())["kind"] == 5
    assert torch.equal(cache.v[1, :, 15], qkv[0].view(6, 64)[4:]) and int((cache.v != 0).sum()) <= 128


BWD = ROPE + [(2, 611, 12, 3, 128, 128, False, True, 0, 1.0, 0)]


@pytest.mark.parametrize("B,N,H,KV,d,rot,inter,norm,far,rs,pad", BWD)
def test_qkv_rope_bwd(B, N, H, KV, d, rot, inter, norm, far, rs, pad):
    qkv, pos, f, wq, wk = rope_inputs(7 * N + H, B, N, H, KV, d, rot, norm, far, pad)
    dq, dk, dv = normal(1, B, H, N, d), normal(2, B, KV, N, d), normal(3, B, KV, N, d)
    call = lambda: attn.qkv_rope_bwd(dq, dk, dv, qkv, pos if rot else None, f, inter, wq, wk, EPS, rs)  # noqa: E731
    dx, dwq, dwk = call()
    again = call()
    torch.cuda.synchronize()
    assert all(a is None if b is None else torch.equal(a.view(torch.uint8), b.view(torch.uint8))
               for a, b in zip(again, (dx, dwq, dwk)))
    T = B * N
    x = f64(qkv).reshape(T, -1)
    ff = f64(f) if rot else np.zeros(0)
    ww = [None if w is None else f64(w) for w in (wq, wk)]
    pp = pos.cpu().numpy().reshape(-1)
    g = [f64(t).transpose(1, 0, 2, 3).reshape(t.shape[1], T, d) for t in (dq, dk, dv)]
    rdx, rdwq, rdwk = gen.qkv_rope_bwd(*g, x, H, KV, d, pp, ff, inter, *ww, EPS, rs)
    what = f"rope bwd B{B} N{N} H{H} KV{KV} d{d} rot{rot}"
    nf = len(ff)
    a, b = (np.arange(0, 2 * nf, 2), np.arange(1, 2 * nf, 2)) if inter else \
        (np.arange(nf), np.arange(nf, 2 * nf))
    tol = np.zeros((T, H + 2 * KV, d))
    x3 = x.reshape(T, H + 2 * KV, d)
    sums = [np.zeros(d), np.zeros(d)]
    for h in range(H + KV):
        gg = np.abs(g[0][h] if h < H else g[1][h - H])
        ga = gg.copy()
        ga[:, a] = ga[:, b] = (gg[:, a] + gg[:, b]) * abs(rs)
        w = ww[0] if h < H else ww[1]
        if w is None:
            tol[:, h] = 2.0 ** -18 * ga
            continue
        xh = np.abs(x3[:, h])
        r = 1 / np.sqrt(np.mean(xh * xh, axis=1, keepdims=True) + EPS)
        u = ga * np.abs(w)
        tol[:, h] = 2.0 ** -18 * (r * u + xh * r ** 3 * np.mean(u * xh, axis=1, keepdims=True))
        sums[0 if h < H else 1] += np.sum(ga * xh * r, axis=0)
    within(f64(dx).reshape(T, -1), rdx, bf16_tol(rdx, tol.reshape(T, -1)), what + " dx")
    for got, ref, s, name in ((dwq, rdwq, sums[0], "dwq"), (dwk, rdwk, sums[1], "dwk")):
        assert (got is None) == (ref is None)
        if got is not None:
            within(f64(got), ref, 2.0 ** -16 * s, f"{what} {name}")


def test_rope_one_norm_only_and_columns_past_the_heads():
    qkv, pos, f, wq, _ = rope_inputs(5, 1, 6, 4, 2, 64, 64, True, 0, 0)
    dq, dk, dv = normal(1, 1, 4, 6, 64), normal(2, 1, 2, 6, 64), normal(3, 1, 2, 6, 64)
    both = attn.qkv_rope_bwd(dq, dk, dv, qkv, pos, f, False, wq, None, EPS)
    assert both[2] is None
    full = attn.qkv_rope_bwd(dq, dk, dv, qkv, pos, f, False, wq, wq, EPS)
    assert torch.equal(both[1], full[1]) and torch.equal(both[0][..., :256], full[0][..., :256])
    # rows further apart than they are long: what lies between stays
    wide = torch.full((6, 600), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(attn.lib().attn_qkv_rope_bwd_workspace_bytes(1, 6, 4, 2, 64), dtype=torch.uint8,
                     device="cuda")
    dw = torch.empty(2, 64, device="cuda")
    p = [t.data_ptr() for t in (dq, dk, dv, qkv, wq, f, pos, wide, dw, ws)]
    rc = attn.lib().attn_qkv_rope_bwd(p[0], p[1], p[2], p[3], 512, p[4], None, EPS, p[5], 64, 0, 1.0, p[6],
                                      p[7], 600, p[8], None, 1, 6, 4, 2, 64, p[9], ws.numel(),
                                      torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert torch.equal(wide[:, :512], both[0][0]) and (wide[:, 512:] == 7).all()


# ------------------------------------------------------------------------------------------- slots
@pytest.mark.parametrize("B,old,lo,hi,page", [
    (1, 0, 1, 1, 16), (1, 0, 500, 500, 16), (3, 40, 0, 3, 16), (256, 3000, 1, 1, 16), (300, 100, 0, 9, 7),
    (16, 0, 128, 4096, 64), (5, 1000, 0, 300, 128), (1000, 20, 0, 2, 1), (16384, 50, 0, 1, 32),
])
def test_kv_slots(B, old, lo, hi, page):
    r = np.random.default_rng(B + page)
    lens, new = r.integers(0, old + 1, B), r.integers(lo, hi + 1, B)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    had = -(-lens // page)
    width = int((-(-(lens + new) // page)).max()) + 1
    order = r.permutation(int(had.sum()) + int(cu[-1]) // page + 2 * B + 5).astype(np.int32)
    table = np.full((B, width), -1, dtype=np.int32)
    at = 0
    for s in range(B):
        table[s, :had[s]] = order[at:at + had[s]]
        at += had[s]
    free = order[at:]
    dev = [torch.from_numpy(np.ascontiguousarray(a.astype(np.int32))).cuda()
           for a in (lens, cu, table, free, np.array([2]))]
    for _ in range(2):  # the same inputs again give the same answer
        got = attn.kv_slots(dev[0], dev[1], int(cu[-1]), dev[2], dev[3], dev[4], page)
    ref = gen.kv_slots(lens, cu, table, free, 2, page)
    for g, w in zip(got, ref):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))
    assert np.array_equal(dev[0].cpu().numpy(), lens) and int(dev[4]) == 2


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_kv_slots_without_room():
    table = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    table[0, 0] = 11
    slots, pos, t, lens, head = attn.kv_slots(i32(3, 0, 7), i32(0, 3, 8, 10), 10, table, i32(5, 6), i32(0), 4)
    assert attn.decode_status(attn.last_device_error())["kind"] == 4
    ref = gen.kv_slots([3, 0, 7], [0, 3, 8, 10], [[11, -1], [-1, -1], [-1, -1]], [5, 6], 0, 4)
    assert slots.tolist() == ref[0] and pos.tolist() == ref[1] and lens.tolist() == ref[3]
    assert t[:2].tolist() == ref[2][:2]


def test_kv_slots_bad_prefix_sums_and_no_tokens():
    table = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    slots, pos, *_ = attn.kv_slots(i32(0, 0), i32(0, 9, 4), 6, table, i32(1, 2, 3), i32(0), 16)
    assert attn.decode_status(attn.last_device_error())["kind"] == 2
    assert slots.shape == (6,) and int(slots.max()) < 64
    _, _, t, lens, head = attn.kv_slots(i32(5, 0), i32(0, 0, 0), 0, table, i32(1), i32(1), 16)
    assert lens.tolist() == [5, 0] and head.tolist() == [1]
    out = attn.kv_slots(i32()[:0], i32(0), 0, table[:0], i32(1), i32(3), 16)
    assert out[4].tolist() == [3] and out[0].numel() == 0


# -------------------------------------------------------------------------- attention over pages
def paged_inputs(seed, lens, H, KV, d, page, kind, sigma=1.0, spare=2, junk=True):
    """Requests' rows in shuffled pages; rows past a request's end and pages of nobody hold NaN."""
    r = np.random.default_rng(seed)
    used = [-(-n // page) for n in lens]
    pages = sum(used) + spare
    order = r.permutation(pages)
    width = max(max(used), 1) + 1
    table = np.full((len(lens), width), 10 ** 6, dtype=np.int32)  # entries not needed are not read
    live = np.zeros((pages, page), dtype=bool)
    at = 0
    for s, n in enumerate(used):
        table[s, :n] = order[at:at + n]
        at += n
        for j in range(n):
            live[table[s, j], :min(page, lens[s] - j * page)] = True
    mask = torch.from_numpy(live)[:, None, :, None].cuda()
    k, v = (normal(seed + i, pages, KV, page, d, sigma=sigma if i == 0 else 1.0) for i in (0, 1))
    q = normal(seed + 2, len(lens), H, 1, d, sigma=sigma)
    if kind == "bf16":
        vals = f64(k), f64(v)
        nan = torch.tensor(float("nan"), dtype=torch.bfloat16, device="cuda")
        cache = attn.KVCache(*(torch.where(mask, t, nan) if junk else t for t in (k, v)))
    else:
        both, vals = [], []
        for t in (k, v):
            s = t.float().abs().amax(-1) / 448 * torch.from_numpy(
                np.exp2(r.integers(-6, 7, t.shape[:3])).astype(np.float32)).cuda()
            codes = (t.float() / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            raw = codes.view(torch.uint8)
            vals.append(ofp8.e4m3_value(raw.cpu().numpy()) * f64(s)[..., None])
            if junk:
                raw = torch.where(mask, raw, torch.tensor(0x7F, dtype=torch.uint8, device="cuda"))
                s = torch.where(mask[..., 0], s, torch.tensor(float("nan"), device="cuda"))
            both += [raw.view(torch.float8_e4m3fn), s.contiguous()]
        cache = attn.KVCache(both[0], both[2], both[1], both[3])
    return q, cache, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), vals


def check_paged(o, lse, q, vals, table, lens, scale, kind, what):
    ro, rl, a, z = gen.paged_attention(f64(q)[:, :, 0], vals[0], vals[1], table.cpu().numpy(),
                                       [int(n) for n in lens], scale)
    es = 2.0 ** -16 * z + 2.0 ** -20
    low = 0.0
    if kind != "bf16":
        low = np.array([n * 2.0 ** -25 for n in lens])[:, None, None] * np.nanmax(np.abs(vals[1]))
    e = ((2.0 ** -8 if kind == "bf16" else 2.0 ** -11) + 2 * es)[..., None] * a + low
    within(f64(o)[:, :, 0], ro, bf16_tol(ro, e), what + " O")
    got = lse.cpu().numpy().astype(np.float64)[:, :, 0]
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(got), empty)
    within(got[~empty], rl[~empty], (es + 2.0 ** -20 * (1 + np.abs(rl)))[~empty], what + " lse")


PAGED = [
    ([1], 1, 1, 64, 16, 1.0),
    ([1, 0, 2], 4, 2, 128, 16, 1.0),
    ([63, 64, 65, 127, 128, 129], 8, 8, 64, 32, 1.0),
    ([15, 16, 17, 31, 33, 0, 0, 100], 8, 2, 128, 16, 1.0),
    ([0, 0], 2, 1, 64, 64, 1.0),
    ([1000, 3, 517], 12, 2, 128, 64, 1.0),
    ([333, 777], 20, 2, 64, 128, 1.0),            # 10 rows a K/V head
    ([2000, 1, 400], 16, 1, 128, 256, 1.0),       # 16 rows
    ([777, 64, 5], 24, 1, 64, 32, 1.0),           # 24 rows
    ([900, 31], 32, 1, 128, 16, 1.0),             # 32 rows
    ([500, 70], 71, 1, 64, 64, 1.0),              # 71 rows: three groups of 24
    ([130], 34, 1, 128, 16, 1.0),                 # two groups of 17
    ([4097, 129], 6, 2, 128, 64, 3.0),            # peaky rows: the reference maximum moves
    ([20000], 2, 1, 128, 64, 1.0),                # one unit over every CTA
    ([17] * 70, 8, 2, 64, 16, 1.0),               # more requests than a warp looks at together
    ([(37 * i) % 300 for i in range(150)], 4, 4, 64, 16, 1.0),
    ([(61 * i) % 200 for i in range(320)], 4, 4, 128, 16, 1.0),   # more units than CTAs
    ([3000, 2500] + [5] * 280 + [700], 20, 2, 64, 32, 1.0),       # long and short, two row slices
    ([1500] + [0] * 40 + [900], 64, 2, 128, 64, 1.0),             # empty requests between, 32 rows
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,H,KV,d,page,sigma", PAGED)
def test_fwd_paged(lens, H, KV, d, page, sigma, kind):
    q, cache, table, n, vals = paged_inputs(len(lens) + H, lens, H, KV, d, page, kind, sigma)
    scale = 1 / math.sqrt(d)
    o, lse = attn.attn_fwd_paged(q, cache, table, n)
    o2, lse2 = attn.attn_fwd_paged(q[:, :, 0], cache, table, n, scale)
    torch.cuda.synchronize()
    assert torch.equal(o[:, :, 0].view(torch.int16), o2.view(torch.int16)) and torch.equal(lse[:, :, 0], lse2)
    check_paged(o, lse, q, vals, table, lens, scale, kind,
                f"paged {kind} {lens[:4]}x{len(lens)} H{H} KV{KV} d{d} page{page}")


def test_paged_rising_scores():
    # every key beats the ones before it by more than the reference may trail
    d, n = 64, 700
    q, cache, table, lens, _ = paged_inputs(5, [n], 3, 1, d, 16, "bf16", junk=False)
    ids = table[0, : -(-n // 16)].long()
    ramp = torch.linspace(-300, 300, len(ids) * 16, device="cuda").reshape(len(ids), 1, 16, 1)
    cache.k[ids] = (ramp * torch.ones(d, device="cuda") / d).to(torch.bfloat16)
    q.fill_(1.0)
    o, lse = attn.attn_fwd_paged(q, cache, table, lens, 1.0)
    check_paged(o, lse, q, (f64(cache.k), f64(cache.v)), table, [n], 1.0, "bf16", "paged rising")


def test_paged_interleaved_pages_and_far_offsets():
    # K and V page by page in one tensor of over 2^33 bytes; the pages used lie at its end
    d, KV, page, H = 128, 8, 128, 16
    pages = (1 << 33) // (2 * KV * page * d * 2) + 50
    both = torch.empty(pages, 2, KV, page, d, dtype=torch.bfloat16, device="cuda")
    lens = [300, 128, 1]
    q, small, table, n, vals = paged_inputs(9, lens, H, KV, d, page, "bf16")
    m = small.k.shape[0]
    both[pages - m:, 0], both[pages - m:, 1] = small.k, small.v
    assert (pages - 1) * both.stride(0) > 1 << 32
    o, lse = attn.attn_fwd_paged(q, attn.KVCache(both[:, 0], both[:, 1]), table + (pages - m), n)
    check_paged(o, lse, q, vals, table, lens, 1 / math.sqrt(d), "bf16", "paged far")
    # rows written there by slot
    qkv = normal(4, 2, (H + 2 * KV) * d)
    slots = torch.tensor([pages * page - 1, (pages - 1) * page], device="cuda")
    attn.qkv_rope(qkv, H, KV, cache=attn.KVCache(both[:, 0], both[:, 1]), slots=slots)
    rows = qkv.view(2, H + 2 * KV, d)
    assert torch.equal(both[-1, 0, :, page - 1], rows[0, H:H + KV])
    assert torch.equal(both[-1, 1, :, 0], rows[1, H + KV:])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_paged_page_outside_the_cache_reads_as_zeros(kind):
    lens = [200, 50]
    q, cache, table, n, vals = paged_inputs(3, lens, 4, 2, 64, 16, kind)
    bad = table.clone()
    bad[0, 3], bad[0, 7], bad[1, 1] = -1, cache.k.shape[0], 2 ** 31 - 1
    o, lse = attn.attn_fwd_paged(q, cache, bad, n)
    assert attn.decode_status(attn.last_device_error())["kind"] == 5
    zk, zv = (np.concatenate([x, np.zeros_like(x[:1])]) for x in vals)
    ref = bad.clone()
    ref[0, 3] = ref[0, 7] = ref[1, 1] = cache.k.shape[0]
    check_paged(o, lse, q, (zk, zv), ref, lens, 1 / 8, kind, f"paged {kind} bad pages")


def test_paged_nan_and_infinity_of_live_rows_stay_in_their_request():
    lens = [90, 90, 90]
    q, cache, table, n, vals = paged_inputs(8, lens, 4, 2, 64, 16, "bf16", junk=False)
    cache.v[table[0, 2].long(), 0, 3, 5] = float("nan")
    cache.k[table[1, 0].long(), 1, 0, :] = float("nan")
    o, lse = attn.attn_fwd_paged(q, cache, table, n)
    nan = torch.isnan(o[:, :, 0])
    assert nan[0, :2, 5].all() and int(nan[0].sum()) == 2        # one column of one K/V head's rows
    assert nan[1, 2:].all() and not nan[1, :2].any() and torch.isnan(lse[1, 2:]).all()
    assert not nan[2].any() and not torch.isnan(lse[[0, 2]]).any()


def test_paged_lengths_past_the_table_are_clamped():
    lens = [48, 16]
    q, cache, table, n, vals = paged_inputs(2, lens, 2, 1, 64, 16, "bf16")
    o, lse = attn.attn_fwd_paged(q, cache, table[:, :3].contiguous(), i32(1000, 16))
    check_paged(o, lse, q, vals, table, lens, 1 / 8, "bf16", "paged clamped")
    o, lse = attn.attn_fwd_paged(q, cache, table[:, :3].contiguous(), i32(-5, 16))
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all()
    o, lse = attn.attn_fwd_paged(q, cache, table[:, :0].contiguous(), n)
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_paged_outputs_given_codes_as_bytes_and_one_page_of_any_stride():
    q, cache, table, n, vals = paged_inputs(31, [9, 16], 6, 3, 64, 16, "e4m3")
    out, lse = torch.full_like(q, 7.0), torch.full((2, 6, 1), 7.0, device="cuda")
    raw = attn.KVCache(cache.k.view(torch.uint8), cache.v.view(torch.uint8), *cache[2:])
    got = attn.attn_fwd_paged(q, raw, table, n, out=out, lse=lse)
    assert got[0].data_ptr() == out.data_ptr() and got[1].data_ptr() == lse.data_ptr()
    check_paged(out, lse, q, vals, table, [9, 16], 1 / 8, "e4m3", "paged outputs given")
    q, cache, table, n, vals = paged_inputs(32, [16], 2, 1, 64, 16, "bf16", spare=0)
    o, lse = attn.attn_fwd_paged(q, cache, table, n)
    check_paged(o, lse, q, vals, table, [16], 1 / 8, "bf16", "paged one page")


def test_refusals_of_the_library_name_the_entry_point():
    q, cache, table, n, _ = paged_inputs(33, [9], 2, 1, 64, 16, "bf16")
    small = attn.KVCache(cache.k[:, :, :8].contiguous(), cache.v[:, :, :8].contiguous())
    with pytest.raises(attn.AttnError, match="attn_fwd_paged failed: ATTN_ERR_UNSUPPORTED") as e:
        attn.attn_fwd_paged(q, small, table, n)
    assert e.value.code == -9
    with pytest.raises(attn.AttnError, match="ATTN_ERR_SCALE"):
        attn.attn_fwd_paged(q, cache, table, n, 0.0)
    with pytest.raises(attn.AttnError, match="ATTN_ERR_WORKSPACE"):
        attn.attn_fwd_paged(q, cache, table, n, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(attn.AttnError, match="attn_qkv_rope failed: ATTN_ERR_SHAPE"):
        attn.qkv_rope(normal(1, 3, 4 * 64), 2, 1, torch.zeros(3, dtype=torch.int32, device="cuda"),
                      torch.ones(5, dtype=torch.float64, device="cuda"))
    with pytest.raises(attn.AttnError, match="attn_kv_slots failed: ATTN_ERR_SHAPE"):
        attn.kv_slots(i32(1), i32(0, 1), 1, table, i32(1), i32(0), 0)
    attn.attn_fwd_paged(q, cache, table[:, ::2], n)  # one entry: its stride is free
    for bad in (dict(seq_lens=n.long()), dict(block_table=table.repeat(2, 1)[::2, ::2].expand(1, 3)),
                dict(q=q.float()),
                dict(out=torch.empty_like(q).float()), dict(seq_lens=n.cpu())):
        with pytest.raises(ValueError):
            attn.attn_fwd_paged(**{**dict(q=q, cache=cache, block_table=table, seq_lens=n), **bad})


def test_rope_without_tokens():
    f = attn.rope_inv_freq(64)
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for shape, lead in (((0, 4 * 64), ()), ((2, 0, 4 * 64), (2,)), ((0, 3, 4 * 64), (0,))):
        qkv = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        pos = torch.empty(shape[:-1], dtype=torch.int32, device="cuda")
        q, k, v = attn.qkv_rope(qkv, 2, 1, pos, f, wq=w, wk=w)
        T = shape[-2]
        assert q.shape == (*lead, 2, T, 64) and k.shape == v.shape == (*lead, 1, T, 64)
        dx, dwq, dwk = attn.qkv_rope_bwd(q, k, v, qkv, pos, f, wq=w, wk=w)
        assert dx.shape == qkv.shape and (dwq == 0).all() and (dwk == 0).all()


def test_paged_workspace_stays_inside():
    q, cache, table, n, vals = paged_inputs(6, [5000, 77], 16, 2, 128, 64, "bf16")
    need = attn.paged_workspace_bytes(2, 16, 2, 128)
    buf = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    o, lse = attn.attn_fwd_paged(q, cache, table, n, workspace=buf[:need])
    torch.cuda.synchronize()
    assert (buf[need:] == 0xA5).all()
    check_paged(o, lse, q, vals, table, [5000, 77], 1 / math.sqrt(128), "bf16", "paged workspace")


def test_paged_two_streams_at_once():
    work = [paged_inputs(20 + i, [3000 + 500 * i, 40], 8, 2, 128, 64, "bf16") for i in range(2)]
    alone = [attn.attn_fwd_paged(*w[:4]) for w in work]
    streams = [torch.cuda.Stream() for _ in work]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        got = [attn.attn_fwd_paged(*w[:4], stream=s) for w, s in zip(work, streams)]
    torch.cuda.synchronize()
    for (a, b), (c, e) in zip(alone, got):
        assert torch.equal(a.view(torch.int16), c.view(torch.int16)) and torch.equal(b, e)


# ------------------------------------------------------------------------------- all together
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,KV,d,page,inter", [(8, 2, 128, 16, False), (6, 6, 64, 64, True)])
def test_prompts_then_tokens(H, KV, d, page, inter, kind):
    """Prompts of unequal length through slots, the step before attention and packed attention, then new
    tokens one at a time, the last of them replayed from a captured graph."""
    prompts, steps, pages = [70, 1, 200], 4, 64
    B, width = len(prompts), (H + 2 * KV) * d
    f = attn.rope_inv_freq(d, factor=2.0, original_len=64)
    wq, wk = (1 + 0.2 * normal(50, 2, d)).unbind(0)
    cache = attn.kv_cache(pages, KV, page, d, torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn)
    table = torch.full((B, 20), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    lens, head = torch.zeros(B, dtype=torch.int32, device="cuda"), i32(0)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(prompts)]), dtype=torch.int32, device="cuda")
    T = sum(prompts)
    rows = normal(60, T, width)
    new = [normal(61 + i, B, 1, width) for i in range(steps)]
    kw = dict(inv_freq=f, interleaved=inter, wq=wq, wk=wk, eps=EPS)

    slots, pos, _, lens, head = attn.kv_slots(lens, cu, T, table, free, head, page)
    q, k, v = attn.qkv_rope(rows, H, KV, pos, cache=cache, slots=slots, **kw)
    o, _ = attn.attn_fwd(q, k, v, cu_seqlens=cu, causal=True)
    x = f64(rows)
    ff, w2 = f64(f), (f64(wq), f64(wk))
    for s in range(B):
        a, b = int(cu[s]), int(cu[s + 1])
        rq, rk, rv = gen.qkv_rope(x[a:b], H, KV, d, np.arange(b - a), ff, inter, *w2, EPS)
        for h in range(H):
            ref = orc.probabilities(rq[h], rk[h // (H // KV)], True, 1 / math.sqrt(d)) @ rv[h // (H // KV)]
            # q and k rounded to bf16 move a score by 2^-7 scale sum |q k| (about 7) at most, 0.055, a
            # weight by as much relative to it, and O by twice that of P|V| (about 0.8): under 0.1
            assert np.abs(f64(o)[h, a:b] - ref).max() < 0.1

    one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    buf = new[0].clone()
    ws = torch.empty(attn.paged_workspace_bytes(B, H, KV, d), dtype=torch.uint8, device="cuda")

    def step():
        slots, pos, _, nl, nh = attn.kv_slots(lens, one, B, table, free, head, page)
        q, _, _ = attn.qkv_rope(buf, H, KV, pos.view(B, 1), cache=cache, slots=slots, with_kv=False, **kw)
        o, lse = attn.attn_fwd_paged(q, cache, table, nl, workspace=ws)
        lens.copy_(nl)
        head.copy_(nh)
        return q, o, lse

    graph, out = None, None
    for i in range(steps):
        buf.copy_(new[i])
        if i < 2:
            out = step()
            continue
        if graph is None:
            graph = torch.cuda.CUDAGraph()
            keep = lens.clone(), head.clone()
            with torch.cuda.graph(graph):
                out = step()
            assert torch.equal(lens, keep[0]) and torch.equal(head, keep[1])
        graph.replay()
    torch.cuda.synchronize()
    assert lens.tolist() == [n + steps for n in prompts]
    if kind == "bf16":
        vals = f64(cache.k), f64(cache.v)
    else:
        vals = [ofp8.e4m3_value(c.view(torch.uint8).cpu().numpy()) * f64(s)[..., None]
                for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    q, o, lse = out
    check_paged(o, lse, q, vals, table, lens.tolist(), 1 / math.sqrt(d), kind, f"generation {kind}")
    # and the cache holds every row of every request, in order
    for s in range(B):
        xs = np.concatenate([x[int(cu[s]):int(cu[s + 1])]] + [f64(n)[s] for n in new])
        n = len(xs)
        _, rk, rv = gen.qkv_rope(xs, H, KV, d, np.arange(n), ff, inter, *w2, EPS)
        _, ek = rope_err(xs, H, KV, d, np.arange(n), ff, inter, *w2, 1.0)
        ids = table[s].cpu().numpy()[: -(-n // page)]
        for ref, val, e in ((rk, vals[0], ek), (rv, vals[1], 0 * rv)):
            got = np.concatenate([val[p] for p in ids], axis=1)[:, :n]
            if kind == "bf16":
                tol = bf16_tol(ref, e)
            else:
                sc = np.abs(ref).max(-1, keepdims=True) / 448
                tol = 2.0 ** -4 * (np.abs(ref) + e) + 2.0 ** -10 * sc * 1.001 + 2 * e + 2.0 ** -22 * np.abs(ref)
            within(got, ref, tol, f"generation {kind} cache")
