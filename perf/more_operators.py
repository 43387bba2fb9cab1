"""Cases of work over a paged key-value cache that goes beyond one new token a request: attention of several new
tokens a request (a prompt in chunks, a second prompt of a conversation, proposed tokens to verify), attention
of one new token of requests that share a long prefix, rows written into a cache and read back from it.

``run`` computes an operator from elementary torch operations, or through the framework's entry
points when ``own`` is true."""
import math
import random

import torch

own = False

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # five proposed tokens of one short conversation of a small model: latency
        {"name": "varlen-B1-new5-L300-H16-KV4-d64", "op": "varlen", "B": 1, "H": 16, "KV": 4, "d": 64, "new_lo": 5, "new": 5,
         "old_lo": 295, "old": 295, "page": 16, "cache": "bf16", "causal": True, "lens": 1},
        # proposed tokens of a batch of requests of every age, verified over an 8-bit cache
        {"name": "varlen-B32-new1-8-old1-8191-e4m3", "op": "varlen", "B": 32, "H": 32, "KV": 8, "d": 128, "new_lo": 1,
         "new": 8, "old_lo": 1, "old": 8183, "page": 16, "cache": "e4m3", "causal": True, "lens": 2},
        # the prompts of the variable-length workload, attended to through their pages
        {"name": "varlen-B16-new128-4096-H16", "op": "varlen", "B": 16, "H": 16, "KV": 16, "d": 128, "new_lo": 128,
         "new": 4096, "old_lo": 0, "old": 0, "page": 64, "cache": "bf16", "causal": True, "lens": 3},
        # the last chunk of a long prompt: 2048 tokens that end at 16384
        {"name": "varlen-B1-new2048-L16384-H32-KV8", "op": "varlen", "B": 1, "H": 32, "KV": 8, "d": 128, "new_lo": 2048,
         "new": 2048, "old_lo": 14336, "old": 14336, "page": 128, "cache": "bf16", "causal": True, "lens": 4},
        # second prompts of conversations, five query heads a K/V head, 8-bit cache
        {"name": "varlen-B24-new1-700-old0-3000-d64-e4m3", "op": "varlen", "B": 24, "H": 20, "KV": 4, "d": 64, "new_lo": 1,
         "new": 700, "old_lo": 0, "old": 3000, "page": 32, "cache": "e4m3", "causal": True, "lens": 5},
        # a serving batch behind one system prompt
        {"name": "shared-G1x64-P8192-own1-512", "op": "shared", "groups": 1, "each": 64, "H": 32, "KV": 8, "d": 128,
         "prefix_lo": 8192, "prefix": 8192, "own": 512, "page": 64, "cache": "bf16", "lens": 6},
        # twelve requests of four samples each over their prompts, 8-bit cache
        {"name": "shared-G12x4-P128-4096-e4m3", "op": "shared", "groups": 12, "each": 4, "H": 16, "KV": 4, "d": 128,
         "prefix_lo": 128, "prefix": 4096, "own": 64, "page": 16, "cache": "e4m3", "lens": 7},
        # four samples of one prompt, as many K/V heads as query heads: latency
        {"name": "shared-G1x4-P1000-H16-KV16-d64", "op": "shared", "groups": 1, "each": 4, "H": 16, "KV": 16, "d": 64,
         "prefix_lo": 1000, "prefix": 1000, "own": 100, "page": 16, "cache": "bf16", "lens": 8},
        # rows of the variable-length workload's prompts into an 8-bit cache
        {"name": "write-T33333-KV16-e4m3", "op": "write", "B": 1, "N": 33333, "KV": 16, "d": 128, "page": 64, "cache": "e4m3",
         "rows": False},
        # one new row of 16 requests
        {"name": "write-B16-KV8-e4m3", "op": "write", "B": 16, "N": 1, "KV": 8, "d": 128, "page": 16, "cache": "e4m3", "rows": False},
        # the whole of an 8-bit cache's requests back as bf16 rows
        {"name": "read-B48-U1-16384-e4m3", "op": "read", "B": 48, "KV": 8, "d": 128, "lo": 1, "hi": 16384, "page": 16,
         "cache": "e4m3", "lens": 9},
        # three short requests of a small model
        {"name": "read-B3-U1-300-d64", "op": "read", "B": 3, "KV": 4, "d": 64, "lo": 1, "hi": 300, "page": 16, "cache": "bf16",
         "lens": 10},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["varlen", "varlen", "varlen", "shared", "shared", "write", "read"])
    d, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    cache, lens = rng.choice(["bf16", "bf16", "e4m3"]), rng.randrange(1 << 20)
    KV = rng.choice([1, 2, 4, 8, 16])
    c = {"op": op, "KV": KV, "d": d, "page": page, "cache": cache}
    row = 2 * KV * d * 2  # bytes of a token's K and V in bf16
    if op == "write":
        N = _spread(rng, 1, min(40000, 400_000_000 // row))
        if N < 200 and rng.random() < 0.5:  # one new row of each of so many requests
            return {**c, "B": N, "N": 1, "rows": rng.random() < 0.3}
        return {**c, "B": 1, "N": N, "rows": rng.random() < 0.3}
    if op == "read":
        hi = _spread(rng, 1, 20000)
        B = _spread(rng, 1, max(1, min(100, 1_500_000_000 // (row * hi))))
        return {**c, "B": B, "lo": rng.choice([1, hi]), "hi": hi, "lens": lens}
    H = KV * rng.choice([1, 2, 3, 4, 5, 8]) if KV > 1 else rng.choice([3, 8, 16, 32])
    H = min(H, 48) // KV * KV
    if op == "shared":
        n = rng.choice([1, 1, 2, rng.randint(3, 16)])
        b = _spread(rng, 2, 64 if n == 1 else 12)
        P = _spread(rng, 64, min(16000, 1_000_000_000 // (row * n)))
        return {**c, "H": H, "groups": n, "each": b, "prefix_lo": rng.choice([P, max(1, P // 8)]), "prefix": P,
                "own": _spread(rng, 1, 600), "lens": lens}
    most = 400_000_000_000  # operations
    new = _spread(rng, 1, 4096)
    old = rng.choice([0, 0, _spread(rng, 16, 12000)])
    B = _spread(rng, 1, max(1, min(40, most // (4 * H * d * new * (new + old)), 1_000_000_000 // (row * (new + old)),
                                   40000 // new)))
    return {**c, "H": H, "B": B, "new_lo": rng.choice([1, new]), "new": new, "old_lo": rng.choice([0, old]), "old": old,
            "causal": rng.random() < 0.85, "lens": lens}


def _lens(case):
    """New and earlier tokens of each request (varlen); prefixes and own rows (shared); rows (read)."""
    r = random.Random(case["lens"])
    if case["op"] == "varlen":
        return [[r.randint(case[x + "_lo"], case[x]) for _ in range(case["B"])] for x in ("new", "old")]
    if case["op"] == "shared":
        return [r.randint(case["prefix_lo"], case["prefix"]) for _ in range(case["groups"])], \
            [r.randint(1, case["own"]) for _ in range(case["groups"] * case["each"])]
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]


# ------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _codes(g, pages, KV, page, d):
    """Rows of an 8-bit cache as a writer leaves them: codes of x / scale, scale = amax / 448."""
    codes = torch.empty(pages, KV, page, d, dtype=E4M3, device="cuda")
    scale = torch.empty(pages, KV, page, device="cuda")
    step = max(1, (1 << 27) // (KV * page * d))
    for a in range(0, pages, step):
        x = _normal(g, min(step, pages - a), KV, page, d).float()
        s = x.abs().amax(-1) / 448.0
        scale[a:a + step] = s
        codes[a:a + step] = (x / s[..., None]).to(E4M3)
    return codes, scale


def _cache(st, g, case, lens_of_tables, seed):
    """A cache that holds the rows of every table's requests on scattered pages, and the tables."""
    page, KV, d = case["page"], case["KV"], case["d"]
    used = [[-(-n // page) for n in lens] for lens in lens_of_tables]
    pages = sum(map(sum, used)) + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    at, tables = 0, []
    for lens in used:
        table = torch.full((len(lens), max(lens + [1])), -1, dtype=torch.int32)
        for s, n in enumerate(lens):
            table[s, :n] = order[at:at + n]
            at += n
        tables.append(table.cuda())
    if case["cache"] == "bf16":
        st["k"], st["v"] = _normal(g, pages, KV, page, d), _normal(g, pages, KV, page, d)
        st["ks"] = st["vs"] = None
    else:
        st["k"], st["ks"] = _codes(g, pages, KV, page, d)
        st["v"], st["vs"] = _codes(g, pages, KV, page, d)
    return tables


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _sums(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def prepare(case, seed):
    g = _gen(seed)
    op, KV, d, page = case["op"], case["KV"], case["d"], case["page"]
    st = {"case": dict(case)}
    if op == "write":
        B, N = case["B"], case["N"]
        T = B * N
        if case["rows"]:  # as a projection leaves them, token by token
            kv = _normal(g, B, N, 2 * KV, d)
            st["kn"], st["vn"] = kv[:, :, :KV].transpose(1, 2), kv[:, :, KV:].transpose(1, 2)
        else:
            st["kn"], st["vn"] = _normal(g, B, KV, N, d), _normal(g, B, KV, N, d)
        pages = -(-T // page) + (T if N == 1 else 0) + 2
        kind = BF16 if case["cache"] == "bf16" else E4M3
        st["k"], st["v"] = (torch.zeros(pages, KV, page, d, device="cuda").to(kind) for _ in range(2))
        st["ks"] = st["vs"] = None
        if kind == E4M3:
            st["ks"], st["vs"] = (torch.zeros(pages, KV, page, device="cuda") for _ in range(2))
        order = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        if N == 1:  # each request's token somewhere in a page of its own
            slots = order[:T] * page + torch.randint(0, page, (T,), generator=g, device="cuda")
        else:
            slots = order[t // page] * page + t % page
        st["slots"] = slots.view(B, N)
        return st
    if op == "read":
        lens = _lens(case)
        st["table"], = _cache(st, g, case, [lens], seed)
        st["cu"], st["T"] = _i32(_sums(lens)), sum(lens)
        return st
    st["scale"] = 1.0 / math.sqrt(d)
    # a generating program keeps one workspace for all its steps
    st["ws"] = torch.empty(128 << 20, dtype=torch.uint8, device="cuda")
    if op == "varlen":
        new, old = _lens(case)
        total = [a + b for a, b in zip(new, old)]
        st["table"], = _cache(st, g, case, [total], seed)
        st["lens"], st["cu"] = _i32(total), _i32(_sums(new))
        st["q"] = _normal(g, case["H"], sum(new), d)
        return st
    prefix, mine = _lens(case)
    st["ptable"], st["table"] = _cache(st, g, case, [prefix, mine], seed)
    st["plens"], st["lens"], st["cug"] = _i32(prefix), _i32(mine), _i32(range(0, len(mine) + 1, case["each"]))
    st["q"] = _normal(g, len(mine), case["H"], 1, d)
    return st


# ------------------------------------------------------------------------------- plain forms
def _rows(codes, scale, table, n):
    """Rows [KV, n, d] in 32 bits of the pages in `table`."""
    at = table[:-(-n // codes.shape[2])].long()
    x = codes[at] if codes.dtype == BF16 else codes.view(torch.uint8)[at].view(E4M3)
    x = x.float()
    if scale is not None:
        x = x * scale[at][..., None]
    return x.transpose(0, 1).reshape(codes.shape[1], -1, codes.shape[3])[:, :n]


def _varlen_plain(st):
    c, q = st["case"], st["q"]
    H, KV, d = c["H"], c["KV"], c["d"]
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=q.device)
    new, old = _lens(c)
    for s, (n, before) in enumerate(zip(new, old)):
        L, t0 = n + before, sum(new[:s])
        k, v = _rows(st["k"], st["ks"], st["table"][s], L), _rows(st["v"], st["vs"], st["table"][s], L)
        step = max(1, (1 << 29) // (H * L))
        for a in range(0, n, step):
            b = min(n, a + step)
            x = q[:, t0 + a:t0 + b].float().reshape(KV, H // KV * (b - a), d)
            z = (torch.matmul(x, k.transpose(1, 2)) * st["scale"]).view(KV, H // KV, b - a, L)
            if c["causal"]:
                seen = torch.arange(L, device=q.device) <= torch.arange(before + a, before + b, device=q.device)[:, None]
                z = z.masked_fill(~seen, -math.inf)
            m = z.amax(-1, keepdim=True)
            p = torch.exp(z - m)
            total = p.sum(-1, keepdim=True)
            y = torch.matmul(p.view(KV, -1, L), v).view(KV, H // KV, b - a, d) / total
            o[:, t0 + a:t0 + b] = y.reshape(H, b - a, d).to(BF16)
            lse[:, t0 + a:t0 + b] = (m + torch.log(total)).reshape(H, b - a)
    return o, lse


def _shared_plain(st):
    c, q = st["case"], st["q"]
    H, KV, d, page = c["H"], c["KV"], c["d"], c["page"]
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=q.device)
    prefix, mine = _lens(c)
    b = c["each"]
    for s in range(c["groups"]):
        at = s * b
        P, W = prefix[s], max(mine[at:at + b])
        x = q[at:at + b].float().view(b, KV, H // KV, d)
        pk, pv = (_rows(t, u, st["ptable"][s], P) for t, u in ((st["k"], st["ks"]), (st["v"], st["vs"])))
        table = st["table"][at:at + b, :-(-W // page)].clamp(min=0).flatten()
        ok, ov = (_rows(t, u, table, table.numel() * page).view(KV, b, -1, d)[:, :, :W].transpose(0, 1)
                  for t, u in ((st["k"], st["ks"]), (st["v"], st["vs"])))
        dead = torch.arange(W, device=q.device) >= st["lens"][at:at + b, None]
        z = torch.cat((torch.matmul(x, pk.transpose(1, 2)), torch.matmul(x, ok.transpose(2, 3))), -1) * st["scale"]
        z[..., P:] = z[..., P:].masked_fill(dead[:, None, None], -math.inf)
        m = z.amax(-1, keepdim=True)
        p = torch.exp(z - m)
        total = p.sum(-1, keepdim=True)
        y = (torch.matmul(p[..., :P], pv) + torch.matmul(p[..., P:], ov)) / total
        o[at:at + b] = y.reshape(b, H, 1, d).to(BF16)
        lse[at:at + b] = (m + torch.log(total)).reshape(b, H, 1)
    return o, lse


def _write_plain(st):
    c = st["case"]
    B, N, KV, d = c["B"], c["N"], c["KV"], c["d"]
    slots = st["slots"].view(-1)
    page, off = slots // c["page"], slots % c["page"]
    for x, codes, scale in ((st["kn"], st["k"], st["ks"]), (st["vn"], st["v"], st["vs"])):
        x = x.transpose(1, 2).reshape(B * N, KV, d)
        if scale is None:
            codes[page, :, off] = x
            continue
        x = x.float()
        amax = x.abs().amax(-1)
        s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        scale[page, :, off] = s
        codes.view(torch.uint8)[page, :, off] = (x / s[..., None]).to(E4M3).view(torch.uint8)
    return [t for t in (st["k"], st["v"], st["ks"], st["vs"]) if t is not None]


def _read_plain(st):
    out = []
    for codes, scale in ((st["k"], st["ks"]), (st["v"], st["vs"])):
        out.append(torch.cat([_rows(codes, scale, st["table"][s], n).to(BF16) for s, n in enumerate(_lens(st["case"]))], 1))
    return out


# ---------------------------------------------------------------------------- the framework's
def _own(st):
    from io_aware_attention_attn_gb300 import attn
    c = st["case"]
    cache = attn.KVCache(st["k"], st["v"], st["ks"], st["vs"])
    if c["op"] == "varlen":
        return attn.attn_fwd_paged_varlen(st["q"], cache, st["table"], st["lens"], st["cu"], causal=c["causal"],
                                          scale=st["scale"], workspace=st["ws"])
    if c["op"] == "shared":
        return attn.attn_fwd_paged_shared(st["q"], cache, st["ptable"], st["plens"], st["cug"], st["table"], st["lens"],
                                          scale=st["scale"], workspace=st["ws"])
    if c["op"] == "write":
        attn.kv_write(st["kn"], st["vn"], cache, st["slots"])
        return [t for t in cache if t is not None]
    return attn.kv_read(cache, st["table"], st["cu"], st["T"])


def run(st):
    if own:
        return _own(st)
    return {"varlen": _varlen_plain, "shared": _shared_plain, "write": _write_plain, "read": _read_plain}[st["case"]["op"]](st)


# -------------------------------------------------------------------------------------- work
def work(case):
    KV, d, page = case["KV"], case["d"], case["page"]
    row = 2 * KV * (2 * d if case["cache"] == "bf16" else d + 4)  # a token's K and V in the cache
    if case["op"] == "write":
        T = case["B"] * case["N"]
        return {"bytes": T * (4 * KV * d + row + 8), "flops": 0 if case["cache"] == "bf16" else 4 * T * KV * d}
    if case["op"] == "read":
        T = sum(_lens(case))
        return {"bytes": T * (row + 4 * KV * d) + 4 * (T // page), "flops": 0 if case["cache"] == "bf16" else 2 * T * KV * d}
    H = case["H"]
    if case["op"] == "shared":
        prefix, mine = _lens(case)
        keys = case["each"] * sum(prefix) + sum(mine)
        return {"bytes": (sum(prefix) + sum(mine)) * row + len(mine) * H * (4 * d + 4), "flops": 4 * keys * H * d}
    new, old = _lens(case)
    keys = sum(n * b + (n * (n + 1) // 2 if case["causal"] else n * n) for n, b in zip(new, old))
    return {"bytes": (sum(new) + sum(old)) * row + sum(new) * H * (4 * d + 4), "flops": 4 * keys * H * d}


# --------------------------------------------------------------------- the definition, 64 bits
def _exact_rows(codes, scale, ids, n):
    """Rows [KV, n, d] page by page, in 64 bits."""
    pages = codes.view(torch.uint8).index_select(0, ids.long()).view(codes.dtype).double()
    if scale is not None:
        pages = pages * scale.index_select(0, ids.long()).double().unsqueeze(-1)
    return torch.cat(list(pages), 1)[:, :n]


def _exact_kv(st, table, n):
    ids = table[:-(-n // st["case"]["page"])]
    return [_exact_rows(st[a], st[b], ids, n) for a, b in (("k", "ks"), ("v", "vs"))]


def _exact_attend(q, k, v, scale, first=None):
    """q [H, n, d] against rows k, v [KV, L, d]; query i sees keys up to first + i (all without `first`)."""
    H, n, d = q.shape
    KV, L = k.shape[:2]
    o, lse = q.new_empty(H, n, d), q.new_empty(H, n)
    for h in range(H):
        for a in range(0, n, 1024):
            z = torch.einsum("id,jd->ij", q[h, a:a + 1024], k[h // (H // KV)]) * scale
            if first is not None:
                i = torch.arange(a, min(n, a + 1024), device=q.device)[:, None]
                z = torch.where(torch.arange(L, device=q.device)[None] > first + i, -math.inf, z)
            lse[h, a:a + 1024] = torch.logsumexp(z, 1)
            o[h, a:a + 1024] = torch.softmax(z, 1) @ v[h // (H // KV)]
    return o, lse


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "write":
        out, page = [], case["page"]
        for x, codes in ((st["kn"], st["k"]), (st["vn"], st["v"])):
            f = torch.zeros(codes.shape, dtype=torch.float64, device="cuda").transpose(1, 2).flatten(0, 1)
            s = f.new_zeros(f.shape[:2])
            rows = x.double().permute(0, 2, 1, 3).flatten(0, 1)
            f[st["slots"].flatten()] = rows
            s[st["slots"].flatten()] = rows.abs().amax(-1) / 448
            out.append((f.unflatten(0, (-1, page)).transpose(1, 2), s.unflatten(0, (-1, page)).transpose(1, 2)))
        if case["cache"] == "bf16":
            return [f for f, _ in out]
        return [None, None] + [s for _, s in out]  # the codes are decided by a rounding
    if case["op"] == "read":
        parts = [_exact_kv(st, st["table"][s], n) for s, n in enumerate(_lens(case))]
        return [torch.cat([p[i] for p in parts], 1) for i in range(2)]
    if case["op"] == "varlen":
        new, old = _lens(case)
        at, parts = 0, []
        for s, (n, before) in enumerate(zip(new, old)):
            k, v = _exact_kv(st, st["table"][s], n + before)
            parts.append(_exact_attend(st["q"][:, at:at + n].double(), k, v, st["scale"], before if case["causal"] else None))
            at += n
        return torch.cat([o for o, _ in parts], 1), torch.cat([z for _, z in parts], 1)
    prefix, mine = _lens(case)
    group = [s for s in range(case["groups"]) for _ in range(case["each"])]
    parts = []
    for s, n in enumerate(mine):
        kv = [torch.cat(x, 1) for x in zip(_exact_kv(st, st["ptable"][group[s]], prefix[group[s]]), _exact_kv(st, st["table"][s], n))]
        parts.append(_exact_attend(st["q"][s].double(), *kv, st["scale"]))
    return torch.stack([o for o, _ in parts]), torch.stack([z for _, z in parts])
