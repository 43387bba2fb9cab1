"""GPU parity of work over a paged cache beyond one new token a request, against the float64 oracle: attention of
several new tokens, attention behind a shared prefix, rows written into a cache and read back, and a run
of them together.

Tolerances, from the arithmetic (half a step of bf16 is 2^-8 of the value, of E4M3 2^-4, of fp32 2^-24):

* scores: e_s = 2^-16 Z + 2^-20, Z = scale max sum |q k|: a sum of 128 terms that may be truncated a term (2^-23
  each), and exp2's 2^-21.  Over E4M3 pages a query row enters as two E4M3 pieces of x / 2^f with a largest
  element of 2^7 to 2^8: a piece is off by half a step, 2^-4 of itself, or 2^-10 below E4M3's normal range
  (spacing 2^-9), so after two pieces x is exact (8 bits) or off by 2^-10, 2^-17 of the row's largest element: 2^-17 W
  more, W = scale max |q| max sum |k|; two more fp32 products (K scale, row factor) 2^-23 Z, within the first term.
* O: P rounded to bf16 (2^-8 of itself), relative errors e_s of P in the sum and its norm, A = sum P |v|:
  (2^-8 + 2 e_s) A, then one rounding to bf16.  Merged parts and prefixes add a few 2^-22, within e_s' 2^-20.
* lse: e_s + 2^-20 (1 + |lse|).
* read: code * scale, one rounding to bf16; the product of an E4M3 value (4 bits) and an fp32 scale is
  rounded to fp32 first: half a bf16 step + 2^-24.  write: bf16 exact; E4M3 scale amax / 448 within 2^-24, codes
  those of the fp32 quotient.
"""
import math

import numpy as np
import pytest
import torch

from io_aware_attention_attn_gb300 import accounting as acc
from io_aware_attention_attn_gb300 import attn
from oracle import fp8 as ofp8
from oracle import pages as orc
from test_parity_generation import _gpu, bf16_tol, f64, i32, normal, paged_inputs, within  # noqa: F401

pytestmark = pytest.mark.gpu


def sums(lens):
    return [0] + list(np.cumsum(lens))


def close(o, lse, ref, kind, what):
    ro, rl, a, z, w = ref
    es = 2.0 ** -16 * z + 2.0 ** -20 + (2.0 ** -17 * w if kind == "e4m3" else 0.0)
    within(o, ro, bf16_tol(ro, (2.0 ** -8 + 2 * es)[..., None] * a), what + " O")
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), empty)
    within(lse[~empty], rl[~empty], (es + 2.0 ** -20 * (1 + np.abs(rl)))[~empty], what + " lse")


def check_varlen(o, lse, q, vals, table, lens, cu, causal, scale, kind, what, tokens=None):
    ref = orc.varlen(f64(q), *vals, table.cpu().numpy(), lens, cu, causal, scale, tokens)
    at = [r[0] for r in ref]
    got = f64(o)[:, at].transpose(1, 0, 2), f64(lse)[:, at].T
    close(*got, [np.stack([r[i] for r in ref]) for i in range(1, 6)], kind, what)


# ---------------------------------------------------------------- several new tokens of a request
VARLEN = [
    # new tokens, rows before them, H, KV, d, page, sigma
    ([1], [0], 1, 1, 64, 16, 1.0),
    ([5], [295], 4, 1, 64, 16, 1.0),
    ([1, 0, 3, 2], [0, 7, 0, 500], 4, 2, 128, 16, 1.0),
    ([127, 128, 129], [0, 1, 127], 2, 2, 128, 64, 1.0),
    ([63, 64, 65], [65, 64, 63], 8, 2, 64, 32, 1.0),       # 128 rows a head exactly, one less, one more
    ([300, 1, 17], [0, 1000, 129], 6, 2, 128, 128, 1.0),   # three rows a token: 126 of 128 rows used
    ([40, 9], [200, 0], 20, 4, 64, 16, 1.0),               # five rows a token
    ([3, 30], [100, 256], 71, 1, 128, 256, 1.0),           # 71 rows: one token a CTA
    ([2, 11], [77, 0], 130, 1, 64, 64, 1.0),               # two groups of 65 rows
    ([700], [1400], 8, 8, 128, 16, 3.0),                   # peaky rows: the reference maximum moves
    ([8, 1, 4], [5000, 3, 0], 16, 2, 128, 16, 1.0),
    ([2], [20000], 1, 1, 128, 64, 1.0),                    # one unit over every pair of SMs
    ([(5 * i) % 4 for i in range(90)], [(37 * i) % 300 for i in range(90)], 4, 2, 64, 16, 1.0),
    ([(7 * i) % 3 for i in range(400)], [(61 * i) % 90 for i in range(400)], 2, 1, 128, 32, 1.0),
    ([0, 0, 60], [0, 9, 60], 3, 3, 128, 32, 1.0),          # requests without new tokens first
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,old,H,KV,d,page,sigma", VARLEN)
def test_varlen(new, old, H, KV, d, page, sigma, kind, causal):
    lens = [a + b for a, b in zip(new, old)]
    _, cache, table, n, vals = paged_inputs(len(lens) + H, lens, H, KV, d, page, kind, sigma)
    q, cu = normal(sum(lens), H, sum(new), d, sigma=sigma), sums(new)
    o, lse = attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu), causal=causal)
    again = attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu), causal, 1 / math.sqrt(d))
    torch.cuda.synchronize()
    assert torch.equal(o.view(torch.int16), again[0].view(torch.int16)) and torch.equal(lse, again[1])
    check_varlen(o, lse, q, vals, table, lens, cu, causal, 1 / math.sqrt(d), kind,
                 f"varlen {kind} {new[:3]}x{len(new)} H{H} KV{KV} d{d} page{page}")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_varlen_more_tokens_than_rows(kind):
    # tokens before the request's first row see nothing: O = 0, lse = -inf; so do all of a request without rows
    new, lens, H, KV, d = [10, 3, 200], [4, 0, 130], 4, 2, 128
    _, cache, table, n, vals = paged_inputs(3, lens, H, KV, d, 16, kind)
    q, cu = normal(4, H, sum(new), d), sums(new)
    for causal in (True, False):
        o, lse = attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu), causal=causal)
        check_varlen(o, lse, q, vals, table, lens, cu, causal, 1 / math.sqrt(d), kind, f"varlen {kind} few rows")
        if causal:
            assert (o[:, :6] == 0).all() and torch.isneginf(lse[:, :6]).all() and (o[:, 6] != 0).any()
        assert (o[:, 10:13] == 0).all() and torch.isneginf(lse[:, 10:13]).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_varlen_long_prompts_in_rounds(kind):
    # K and V of several row tiles beyond what a round keeps in L2, on sampled tokens
    new, old, H, KV, d, page = [5000, 3000], [3000, 9000], 16, 8, 128, 128
    lens = [a + b for a, b in zip(new, old)]
    _, cache, table, n, vals = paged_inputs(5, lens, H, KV, d, page, kind)
    q, cu = normal(6, H, sum(new), d), sums(new)
    o, lse = attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu))
    tokens = set(range(0, 8000, 397)) | {0, 4999, 5000, 7999, 127, 128, 5063, 5064}
    check_varlen(o, lse, q, vals, table, lens, cu, True, 1 / math.sqrt(d), kind, f"varlen {kind} long", tokens)
    assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_varlen_leaves_padding_alone(kind):
    new, lens, H, KV, d = [5, 33], [100, 33], 4, 2, 64
    _, cache, table, n, vals = paged_inputs(7, lens, H, KV, d, 16, kind)
    T, cu = 300, sums(new)
    q = normal(8, H, T, d)
    q[:, 38:] = float("nan")
    out = torch.full((H, T, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, T), 7.0, device="cuda")
    got = attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu), out=out, lse=lse)
    assert got[0].data_ptr() == out.data_ptr() and got[1].data_ptr() == lse.data_ptr()
    assert (out[:, 38:] == 7).all() and (lse[:, 38:] == 7).all()
    check_varlen(out[:, :38], lse[:, :38], q[:, :38], vals, table, lens, cu, True, 1 / 8, kind, f"varlen {kind} padding")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_varlen_page_outside_the_cache_reads_as_zeros(kind):
    lens, new, H, KV, d = [200, 50], [20, 50], 4, 2, 64
    _, cache, table, n, vals = paged_inputs(3, lens, H, KV, d, 16, kind)
    q, cu = normal(9, H, 70, d), sums(new)
    bad = table.clone()
    bad[0, 3], bad[0, 7], bad[1, 1] = -1, cache.k.shape[0], 2 ** 31 - 1
    o, lse = attn.attn_fwd_paged_varlen(q, cache, bad, n, i32(*cu))
    assert attn.decode_status(attn.last_device_error())["kind"] == 5
    zk, zv = (np.concatenate([x, np.zeros_like(x[:1])]) for x in vals)
    ref = bad.clone()
    ref[0, 3] = ref[0, 7] = ref[1, 1] = cache.k.shape[0]
    check_varlen(o, lse, q, (zk, zv), ref, lens, cu, True, 1 / 8, kind, f"varlen {kind} bad pages")


def test_varlen_bad_prefix_sums_are_reported():
    _, cache, table, n, _ = paged_inputs(3, [40, 40], 2, 1, 64, 16, "bf16")
    q = normal(2, 2, 30, 64)
    for cu in ((1, 10, 30), (0, 20, 10), (0, 10, 31)):
        attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu))
        assert attn.decode_status(attn.last_device_error())["kind"] == 2


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_varlen_nan_of_live_rows_stays_in_its_request(kind):
    lens, new = [90, 90, 90], [3, 40, 3]
    _, cache, table, n, _ = paged_inputs(8, lens, 4, 2, 64, 16, kind, junk=False)
    q = normal(1, 4, 46, 64)
    nan = 0x7F if kind == "e4m3" else 0x7FC0
    raw = torch.uint8 if kind == "e4m3" else torch.int16
    cache.v.view(raw)[table[0, 2].long(), 0, 3, 5] = nan
    cache.k.view(raw)[table[1, 0].long(), 1, 0, :] = nan
    q[3, 45, 7] = float("inf")
    o, lse = attn.attn_fwd_paged_varlen(q, cache, table, n, i32(0, 3, 43, 46))
    bad = torch.isnan(o)
    assert bad[:2, :3, 5].all() and int(bad[:, :3].sum()) == 6
    assert bad[2:, 3:43].all() and not bad[:2, 3:43].any() and torch.isnan(lse[2:, 3:43]).all()
    assert bad[3, 45].all() and int(bad[:, 43:].sum()) == 64


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_varlen_rising_scores(kind):
    # every tile of keys beats the ones before it by more than the reference may trail, over several shares
    d, n, new = 64, 3000, 9
    _, cache, table, lens, vals = paged_inputs(5, [n], 3, 1, d, 16, kind, junk=False)
    q = torch.ones(3, new, d, dtype=torch.bfloat16, device="cuda")
    ids = table[0, : -(-n // 16)].long()
    ramp = torch.linspace(-900, 900, len(ids) * 16, device="cuda").reshape(len(ids), 1, 16, 1)
    if kind == "bf16":
        cache.k[ids] = (ramp * torch.ones(d, device="cuda") / d).to(torch.bfloat16)
        kv = f64(cache.k)
    else:
        cache.k.view(torch.uint8)[ids] = 0x38  # 1
        cache.k_scale[ids] = ramp[..., 0] / d
        kv = ofp8.e4m3_value(cache.k.view(torch.uint8).cpu().numpy()) * f64(cache.k_scale)[..., None]
    o, lse = attn.attn_fwd_paged_varlen(q, cache, table, lens, i32(0, new), scale=1.0)
    check_varlen(o, lse, q, (kv, vals[1]), table, [n], [0, new], True, 1.0, kind, f"varlen {kind} rising")


def test_varlen_far_pages_and_interleaved():
    # K and V page by page in one tensor of over 2^33 bytes; the pages used lie at its end
    d, KV, page, H = 128, 8, 128, 16
    pages = (1 << 33) // (2 * KV * page * d * 2) + 50
    both = torch.empty(pages, 2, KV, page, d, dtype=torch.bfloat16, device="cuda")
    lens, new = [300, 128, 1], [40, 128, 1]
    _, small, table, n, vals = paged_inputs(9, lens, H, KV, d, page, "bf16")
    m = small.k.shape[0]
    both[pages - m:, 0], both[pages - m:, 1] = small.k, small.v
    cache = attn.KVCache(both[:, 0], both[:, 1])
    q, cu = normal(3, H, sum(new), d), sums(new)
    o, lse = attn.attn_fwd_paged_varlen(q, cache, table + (pages - m), n, i32(*cu))
    check_varlen(o, lse, q, vals, table, lens, cu, True, 1 / math.sqrt(d), "bf16", "varlen far")
    # written there by slot and read back
    k, v = normal(5, KV, 3, d), normal(6, KV, 3, d)
    last = (pages - 1) * page
    attn.kv_write(k, v, cache, torch.tensor([last + page - 1, last, last + 77], device="cuda"))
    assert torch.equal(both[-1, 0, :, page - 1], k[:, 0]) and torch.equal(both[-1, 1, :, 0], v[:, 1])
    rk, rv = attn.kv_read(cache, i32(pages - 1).view(1, 1), i32(0, page), page)
    assert torch.equal(rk, both[-1, 0]) and torch.equal(rv[:, 77], v[:, 2])


def test_varlen_workspace_stays_inside():
    lens, new, H, KV, d = [5000, 77], [300, 77], 16, 2, 128
    _, cache, table, n, vals = paged_inputs(6, lens, H, KV, d, 64, "bf16")
    q, cu = normal(2, H, sum(new), d), sums(new)
    for t in (sum(new), 5):
        need = attn.paged_varlen_workspace_bytes(t, H, KV, d)
        buf = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        c = cu if t != 5 else [0, 4, 5]
        o, lse = attn.attn_fwd_paged_varlen(q[:, :t].contiguous(), cache, table, n, i32(*c), workspace=buf[:need])
        torch.cuda.synchronize()
        assert (buf[need:] == 0xA5).all()
        check_varlen(o, lse, q[:, :t], vals, table, lens, c, True, 1 / math.sqrt(d), "bf16", "varlen workspace",
                     set(range(0, t, 29)))


def test_varlen_two_streams_at_once():
    work = []
    for i in range(2):
        lens, new = [3000 + 500 * i, 40], [33, 40 - i]
        _, cache, table, n, _ = paged_inputs(20 + i, lens, 8, 2, 128, 64, "bf16")
        work.append((normal(30 + i, 8, sum(new), 128), cache, table, n, i32(*sums(new))))
    alone = [attn.attn_fwd_paged_varlen(*w) for w in work]
    streams = [torch.cuda.Stream() for _ in work]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        got = [attn.attn_fwd_paged_varlen(*w, stream=s) for w, s in zip(work, streams)]
    torch.cuda.synchronize()
    for (a, b), (c, e) in zip(alone, got):
        assert torch.equal(a.view(torch.int16), c.view(torch.int16)) and torch.equal(b, e)


def test_varlen_replayed_with_other_lengths():
    H, KV, d, page, T = 8, 2, 128, 16, 64
    lens = [400, 700, 30]
    _, cache, table, n, vals = paged_inputs(11, lens, H, KV, d, page, "bf16")
    q, cu = normal(12, H, T, d), i32(0, 1, 2, 3)
    length = i32(1, 1, 1)
    attn.attn_fwd_paged_varlen(q, cache, table, length, cu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = attn.attn_fwd_paged_varlen(q, cache, table, length, cu)
    for new, rows in (([20, 40, 4], lens), ([0, 64, 0], [1, 699, 0]), ([1, 1, 1], [399, 16, 17])):
        cu.copy_(i32(*sums(new)))
        length.copy_(i32(*rows))
        graph.replay()
        t = sum(new)
        check_varlen(o[:, :t], lse[:, :t], q[:, :t], vals, table, rows, sums(new), True, 1 / math.sqrt(d), "bf16",
                     "varlen replayed")


# -------------------------------------------------------------------------- behind a shared prefix
SHARED = [
    # requests of each group, prefixes, H, KV, d, page, seed of the own lengths, most own rows
    ([1], [1], 1, 1, 64, 16, 1, 1),
    ([3], [1000], 4, 2, 128, 16, 2, 40),
    ([2, 0, 5], [130, 50, 0], 8, 2, 64, 32, 3, 100),         # a group without requests, a prefix without rows
    ([4] * 12, [97 * i for i in range(12)], 16, 4, 128, 16, 4, 64),
    ([70], [2000], 20, 4, 64, 64, 5, 300),                   # more than one run of requests
    ([9], [6000], 71, 1, 128, 128, 6, 5),                    # 71 rows a request
    ([300], [128], 2, 2, 128, 256, 7, 30),
    ([1] * 40, [31 * i for i in range(40)], 4, 1, 64, 16, 8, 20),
    ([2, 40], [9000, 10], 130, 1, 64, 16, 9, 700),
]


def shared_inputs(each, prefix, H, KV, d, page, seed, most, kind, sigma=1.0):
    B = sum(each)
    r = np.random.default_rng(seed)
    own = [int(x) for x in r.integers(0, most + 1, B)]
    _, cache, tables, _, vals = paged_inputs(seed + H, list(prefix) + own, H, KV, d, page, kind, sigma)
    G = len(each)
    return (normal(seed, B, H, 1, d, sigma=sigma), cache, tables[:G].contiguous(), i32(*prefix), i32(*sums(each)),
            tables[G:].contiguous(), i32(*own)), own, vals


def check_shared(o, lse, args, vals, scale, kind, what):
    q, _, pt, pl, cu, table, lens = args
    ref = orc.shared(f64(q)[:, :, 0], *vals, *(t.cpu().numpy() for t in (pt, pl, cu, table, lens)), scale)
    close(f64(o)[:, :, 0], f64(lse)[:, :, 0], ref, kind, what)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("each,prefix,H,KV,d,page,seed,most", SHARED)
def test_shared(each, prefix, H, KV, d, page, seed, most, kind):
    args, own, vals = shared_inputs(each, prefix, H, KV, d, page, seed, most, kind)
    o, lse = attn.attn_fwd_paged_shared(*args)
    q3, l3 = attn.attn_fwd_paged_shared(args[0][:, :, 0], *args[1:], 1 / math.sqrt(d))
    torch.cuda.synchronize()
    assert torch.equal(o[:, :, 0].view(torch.int16), q3.view(torch.int16)) and torch.equal(lse[:, :, 0], l3)
    check_shared(o, lse, args, vals, 1 / math.sqrt(d), kind, f"shared {kind} {each[:3]} {prefix[:3]} H{H} KV{KV} d{d}")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_shared_peaky_and_padding(kind):
    # what dominates lies in the prefix for some rows and in the own rows for others
    args, own, vals = shared_inputs([5, 6], [400, 333], 12, 4, 128, 32, 21, 200, kind, 3.0)
    o, lse = attn.attn_fwd_paged_shared(*args)
    check_shared(o, lse, args, vals, 1 / math.sqrt(128), kind, f"shared {kind} peaky")
    # the last three requests are padding (the work is cut differently then, so bits may differ)
    out, lse = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
    attn.attn_fwd_paged_shared(*args[:4], i32(0, 5, 8), *args[5:], out=out, lse=lse)
    assert (out[8:] == 7).all() and (lse[8:] == 7).all()
    q, cache, pt, pl, _, table, n = args
    check_shared(out[:8], lse[:8], (q[:8], cache, pt, pl, i32(0, 5, 8), table[:8], n[:8]), vals, 1 / math.sqrt(128), kind,
                 f"shared {kind} padded")


def test_shared_without_pages_of_one_kind():
    args, own, vals = shared_inputs([4], [90], 4, 2, 64, 16, 22, 50, "bf16")
    q, cache, pt, pl, cu, table, lens = args
    zero = torch.zeros_like(lens)
    a = attn.attn_fwd_paged_shared(q, cache, pt, pl, cu, table[:, :0].contiguous(), zero)
    check_shared(*a, (q, cache, pt, pl, cu, table, zero), vals, 1 / 8, "bf16", "shared prefix only")
    b = attn.attn_fwd_paged_shared(q, cache, pt[:, :0].contiguous(), pl, cu, table, lens)
    check_shared(*b, (q, cache, pt, torch.zeros_like(pl), cu, table, lens), vals, 1 / 8, "bf16", "shared own only")
    o, lse = attn.attn_fwd_paged_shared(q, cache, pt, torch.zeros_like(pl), cu, table, zero)
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_shared_workspace_and_replay():
    args, own, vals = shared_inputs([30, 3], [3000, 100], 16, 2, 128, 64, 23, 200, "bf16")
    need = attn.paged_shared_workspace_bytes(33, 16, 2, 128)
    buf = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    attn.attn_fwd_paged_shared(*args, workspace=buf[:need])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = attn.attn_fwd_paged_shared(*args, workspace=buf[:need])
    graph.replay()
    check_shared(o, lse, args, vals, 1 / math.sqrt(128), "bf16", "shared replayed")
    args[3].copy_(i32(17, 99))
    args[6].copy_((args[6] // 2).int())
    graph.replay()
    check_shared(o, lse, args, vals, 1 / math.sqrt(128), "bf16", "shared replayed with other lengths")
    assert (buf[need:] == 0xA5).all()


# ------------------------------------------------------------------------------ write and read
ROWS = [(1, 1, 1, 64, 16), (1, 77, 3, 128, 32), (5, 1, 8, 128, 16), (3, 50, 2, 64, 64), (2, 130, 5, 128, 256),
        (1, 3000, 16, 64, 128)]


@pytest.mark.parametrize("layout", ["heads", "tokens", "apart"])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,N,KV,d,page", ROWS)
def test_write_and_read(B, N, KV, d, page, kind, layout):
    if layout == "heads":
        k, v = normal(1, B, KV, N, d), normal(2, B, KV, N, d)
    elif layout == "tokens":
        k, v = (x.transpose(1, 2) for x in normal(3, B, N, 2 * KV, d).split(KV, 2))
    else:
        k, v = normal(4, B, KV, 2 * N, d + 8)[:, :, ::2, :d], normal(5, N, B, KV, d).permute(1, 2, 0, 3)
    k[:, :, N // 2] = 0
    T = B * N
    pages = -(-T // page) + 2
    cache = attn.kv_cache(pages, KV, page, d, torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn)
    for t in cache:
        if t is not None:
            t.view(torch.uint8).fill_(0x3A)
    order = torch.randperm(pages * page, generator=torch.Generator().manual_seed(N))[:T].cuda()
    slots = order.view(B, N).clone()
    slots.view(-1)[3::5] = -1
    assert attn.kv_write(k, v, cache, slots) is cache
    kept = (slots.view(-1) >= 0).cpu().numpy()
    at = order.cpu().numpy()
    other = np.ones(pages * page, dtype=bool)
    other[at[kept]] = False
    for x, codes, scale in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        raw = codes.view(torch.uint8)
        raw = raw.transpose(1, 2).reshape(pages * page, KV, -1).cpu().numpy()
        assert (raw[other] == 0x3A).all()
        ref = x.transpose(1, 2).reshape(T, KV, d)[torch.from_numpy(kept).cuda()]
        if kind == "bf16":
            assert (raw[at[kept]] == ref.contiguous().view(torch.uint8).cpu().numpy()).all()
            continue
        sc = scale.transpose(1, 2).reshape(pages * page, KV)
        assert (sc.view(torch.int32)[torch.from_numpy(other).cuda()] == 0x3A3A3A3A).all()
        amax = ref.float().abs().amax(-1).cpu()
        want = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))  # the fp32 quotient on the host
        assert torch.equal(sc.cpu()[torch.from_numpy(at[kept])], want)
        code = (ref.float().cpu() / want[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert (raw[at[kept]] == code).all()
    # back, request by request, from the middle too
    lens = [pages * page - 5, 0, 7, page]
    first = [5, 3, page - 3, 0]
    table = torch.stack([torch.randperm(pages, generator=torch.Generator().manual_seed(i)) for i in range(4)])
    table = table.to(torch.int32).cuda()
    total = sum(lens)
    out_k = torch.full((KV, total + 9, d), 7.0, dtype=torch.bfloat16, device="cuda")
    out_v = out_k.clone()
    got = attn.kv_read(cache, table, i32(*sums(lens)), total + 9, i32(*first), out_k, out_v)
    assert got[0].data_ptr() == out_k.data_ptr() and (out_k[:, total:] == 7).all() and (out_v[:, total:] == 7).all()
    for out, codes, scale in ((out_k, cache.k, cache.k_scale), (out_v, cache.v, cache.v_scale)):
        if kind == "bf16":
            vals = codes.float().cpu().numpy().astype(np.float64)
        else:
            vals = ofp8.e4m3_value(codes.view(torch.uint8).cpu().numpy()) * f64(scale)[..., None]
        ref = np.concatenate([orc.rows(vals, table[s].cpu().numpy(), first[s] + n)[:, first[s]:] for s, n in enumerate(lens)], 1)
        if kind == "bf16":
            assert np.array_equal(f64(out)[:, :total], ref)
        else:
            within(f64(out)[:, :total], ref, 2.0 ** -24 * np.abs(ref) + acc.bf16_half_ulp(np.abs(ref) * (1 + 2.0 ** -24)),
                   f"read e4m3 B{B} N{N}")
    if kind == "bf16":  # and without `first`, outputs made by the call
        rk, _ = attn.kv_read(cache, table[:1], i32(0, pages * page), pages * page)
        assert torch.equal(rk, cache.k[table[0].long()].transpose(0, 1).reshape(KV, -1, d))


def test_write_codes_are_those_of_the_step_before_attention():
    # rows of every size, among them the smallest and largest scales
    KV, d, T = 4, 128, 600
    x = normal(1, T, 3 * KV, d)
    x *= torch.exp2(torch.randint(-126, 120, (T, 3 * KV, 1), generator=torch.Generator().manual_seed(2)).float()).cuda().to(torch.bfloat16)
    caches = [attn.kv_cache(40, KV, 16, d, torch.float8_e4m3fn) for _ in range(2)]
    slots = torch.randperm(640, generator=torch.Generator().manual_seed(3))[:T].cuda()
    attn.qkv_rope(x.view(T, -1), KV, KV, cache=caches[0], slots=slots)
    attn.kv_write(x[:, KV:2 * KV].transpose(0, 1), x[:, 2 * KV:].transpose(0, 1), caches[1], slots)
    for a, b in zip(*caches):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and a.view(torch.uint8).any()


def test_write_slot_past_the_cache_is_reported_and_not_stored():
    cache = attn.kv_cache(2, 2, 16, 64)
    k, v = normal(3, 2, 4, 64), normal(4, 2, 4, 64)
    attn.kv_write(k, v, cache, torch.tensor([31, 32, 1 << 40, -7], device="cuda"))
    assert attn.decode_status(attn.last_device_error())["kind"] == 5
    assert torch.equal(cache.v[1, :, 15], v[:, 0]) and int((cache.v != 0).sum()) <= 128


def test_read_outside_the_table_is_zeros_and_reported():
    KV, d = 2, 64
    cache = attn.KVCache(normal(1, 3, KV, 16, d), normal(2, 3, KV, 16, d))
    table = torch.tensor([[0, 5, 2], [-1, 1, 0]], dtype=torch.int32, device="cuda")
    k, v = attn.kv_read(cache, table, i32(0, 60, 80), 80, i32(-4, 10))
    assert attn.decode_status(attn.last_device_error())["kind"] == 5
    for out, c in ((k, cache.k), (v, cache.v)):
        want = torch.zeros(KV, 80, d, dtype=torch.bfloat16, device="cuda")
        want[:, 4:20], want[:, 36:52] = c[0], c[2]
        want[:, 66:80] = c[1][:, :14]
        assert torch.equal(out, want)
    attn.kv_read(cache, table, i32(0, 9, 3), 9, None)
    assert attn.decode_status(attn.last_device_error())["kind"] == 2


# --------------------------------------------------------------------------------- refusals
def test_refusals_name_the_entry_point():
    q1, cache, table, n, _ = paged_inputs(33, [9], 2, 1, 64, 16, "bf16")
    q, cu = normal(1, 2, 5, 64), i32(0, 5)
    small = attn.KVCache(cache.k[:, :, :8].contiguous(), cache.v[:, :, :8].contiguous())
    tiny = torch.empty(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(attn.AttnError, match="attn_fwd_paged_varlen failed: ATTN_ERR_UNSUPPORTED"):
        attn.attn_fwd_paged_varlen(q, small, table, n, cu)
    with pytest.raises(attn.AttnError, match="attn_fwd_paged_varlen failed: ATTN_ERR_WORKSPACE"):
        attn.attn_fwd_paged_varlen(q, cache, table, n, cu, workspace=tiny)
    with pytest.raises(attn.AttnError, match="attn_fwd_paged_shared failed: ATTN_ERR_WORKSPACE"):
        attn.attn_fwd_paged_shared(q1, cache, table, n, i32(0, 1), table, n, workspace=tiny)
    with pytest.raises(attn.AttnError, match="attn_kv_write failed: ATTN_ERR_UNSUPPORTED"):
        attn.kv_write(normal(1, 1, 3, 64), normal(1, 1, 3, 64), small, torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(attn.AttnError, match="attn_kv_read failed: ATTN_ERR_UNSUPPORTED"):
        attn.kv_read(small, table, i32(0, 3), 3)
    for bad in (dict(q=q[:, ::2]), dict(q=q.float()), dict(q=q[:1].expand(3, 5, 64)), dict(seq_lens=n.long()),
                dict(cu_new=i32(0)), dict(block_table=table[0]), dict(out=q.float()), dict(seq_lens=n.cpu())):
        with pytest.raises(ValueError):
            attn.attn_fwd_paged_varlen(**{**dict(q=q, cache=cache, block_table=table, seq_lens=n, cu_new=cu), **bad})
    k = normal(1, 1, 3, 64)
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in (dict(k=k.float()), dict(v=k[:, :2]), dict(slots=slots.int()), dict(slots=slots[:2]),
                dict(k=normal(1, 1, 64, 3).transpose(1, 2)), dict(k=normal(1, 2, 3, 64), v=normal(1, 2, 3, 64))):
        with pytest.raises(ValueError):
            attn.kv_write(**{**dict(k=k, v=k, cache=cache, slots=slots), **bad})


def test_nothing_to_do():
    _, cache, table, n, _ = paged_inputs(33, [9], 2, 1, 64, 16, "bf16")
    o, lse = attn.attn_fwd_paged_varlen(normal(1, 2, 0, 64), cache, table, n, i32(0, 0))
    assert o.shape == (2, 0, 64) and lse.shape == (2, 0)
    o, lse = attn.attn_fwd_paged_shared(normal(1, 0, 2, 1, 64), cache, table, n, i32(0, 0), table[:0], n[:0])
    assert o.shape == (0, 2, 1, 64)
    k = torch.empty(1, 0, 64, dtype=torch.bfloat16, device="cuda")
    attn.kv_write(k, k, cache, torch.empty(0, dtype=torch.int64, device="cuda"))
    rk, rv = attn.kv_read(cache, table, i32(0, 0), 0)
    assert rk.shape == rv.shape == (1, 0, 64)


# ------------------------------------------------------------------------------- all together
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_prompt_in_chunks_then_samples_behind_it(kind):
    """Two prompts in chunks through slots, the step before attention and attention over their pages; then three
    samples of each, one new token at a time behind the shared prompt."""
    H, KV, d, page, pages, B = 8, 2, 128, 16, 80, 2
    f = attn.rope_inv_freq(d)
    kw = dict(inv_freq=f, wq=torch.ones(d, dtype=torch.bfloat16, device="cuda"))
    cache = attn.kv_cache(pages, KV, page, d, torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn)
    table = torch.full((B, 20), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    lens, head = i32(0, 0), i32(0)
    scale = 1 / math.sqrt(d)

    def values():
        if kind == "bf16":
            return f64(cache.k), f64(cache.v)
        return [ofp8.e4m3_value(c.view(torch.uint8).cpu().numpy()) * f64(s)[..., None]
                for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]

    for new in ([100, 37], [60, 0], [1, 120]):
        cu = i32(*sums(new))
        T = sum(new)
        slots, pos, _, lens, head = attn.kv_slots(lens, cu, T, table, free, head, page)
        q, _, _ = attn.qkv_rope(normal(T, T, (H + 2 * KV) * d), H, KV, pos, cache=cache, slots=slots, **kw)
        o, lse = attn.attn_fwd_paged_varlen(q, cache, table, lens, cu)
        check_varlen(o, lse, q, values(), table, lens.tolist(), sums(new), True, scale, kind, f"chunks {kind}")
    assert lens.tolist() == [161, 157]
    # the whole second prompt's rows read back give the last chunk's attention again
    k, v = attn.kv_read(cache, table, i32(0, 0, 157), 157)
    full = torch.zeros(H, 157, d, dtype=torch.bfloat16, device="cuda")
    full[:, 37:] = q[:, 1:]
    o2, lse2 = attn.attn_fwd(full, k, v, causal=True, cu_seqlens=i32(0, 157))
    # rows rounded to bf16 once more (2^-8 of k and v): a score moves by 2^-8 Z (Z about 7), a weight by
    # as much, O by twice that and 2^-8 of P|V| (about 0.8); under 0.06
    assert (o2[:, 37:].float() - o[:, 1:].float()).abs().max() < (0.06 if kind == "e4m3" else 0.02)
    n, own = 3, torch.full((2 * 3, 4), -1, dtype=torch.int32, device="cuda")
    mine = i32(*[0] * 6)
    one = i32(*range(7))
    for i in range(20):
        slots, pos, _, mine, head = attn.kv_slots(mine, one, 6, own, free, head, page)
        pos = pos + lens.repeat_interleave(n)
        q, _, _ = attn.qkv_rope(normal(900 + i, 6, 1, (H + 2 * KV) * d), H, KV, pos.view(6, 1).int(), cache=cache, slots=slots,
                                with_kv=False, **kw)
        o, lse = attn.attn_fwd_paged_shared(q, cache, table, lens, i32(0, 3, 6), own, mine)
    check_shared(o, lse, (q, cache, table, lens, i32(0, 3, 6), own, mine), values(), scale, kind, f"samples {kind}")
