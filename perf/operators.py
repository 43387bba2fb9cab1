"""Cases of the generation path: the step before attention (norm, rotation, layout, cache write), its
backward, the slots of new tokens in a paged key-value cache, and the attention of one new token.

``run`` computes an operator from elementary torch operations, or through the framework's entry
points when ``own`` is true."""
import math
import random

import torch

own = False

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
EPS = 1e-6


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one stream far into a long context: latency of a step, 16384 tokens as in the long causal workload
        {"name": "paged-B1-H32-KV8-L16384", "op": "paged", "B": 1, "H": 32, "KV": 8, "d": 128, "lo": 16384, "hi": 16384,
         "page": 64, "cache": "bf16", "lens": 1},
        # a small model's batch with as many K/V heads as query heads, short contexts, small pages
        {"name": "paged-B4-H16-KV16-L1024-d64", "op": "paged", "B": 4, "H": 16, "KV": 16, "d": 64, "lo": 1024, "hi": 1024,
         "page": 16, "cache": "bf16", "lens": 2},
        # a full serving batch of long contexts: bandwidth
        {"name": "paged-B64-H32-KV8-L16384", "op": "paged", "B": 64, "H": 32, "KV": 8, "d": 128, "lo": 16384, "hi": 16384,
         "page": 128, "cache": "bf16", "lens": 3},
        # a batch of requests of every age over an 8-bit cache
        {"name": "paged-B48-H32-KV8-U1-16384-e4m3", "op": "paged", "B": 48, "H": 32, "KV": 8, "d": 128, "lo": 1, "hi": 16384,
         "page": 16, "cache": "e4m3", "lens": 4},
        # one K/V head for all query heads, ragged lengths
        {"name": "paged-B37-H32-KV1-U128-8191-d64", "op": "paged", "B": 37, "H": 32, "KV": 1, "d": 64, "lo": 128, "hi": 8191,
         "page": 32, "cache": "bf16", "lens": 5},
        # one step of 16 requests: q, k normed and rotated, K and V into an 8-bit cache
        {"name": "rope-step-B16-e4m3", "op": "rope", "B": 16, "N": 1, "H": 32, "KV": 8, "d": 128, "rot": 128, "inter": False,
         "norm": True, "base": 500000.0, "factor": 8.0, "far": 131072, "page": 16, "cache": "e4m3", "lens": 6},
        # the headline shape's training forward: projection rows to head-major q, k, v
        {"name": "rope-B2-N4096-H32-KV8", "op": "rope", "B": 2, "N": 4096, "H": 32, "KV": 8, "d": 128, "rot": 128,
         "inter": False, "norm": True, "base": 10000.0, "factor": 1.0, "far": 0, "page": 0, "cache": "none", "lens": 7},
        # packed prompts of the variable-length workload: q, k, v for attention and the rows into the cache;
        # half of each head rotated, neighbouring pairs, no norms
        {"name": "rope-packed-H16-U128-4096", "op": "rope", "B": 1, "N": 33333, "H": 16, "KV": 16, "d": 128, "rot": 64,
         "inter": True, "norm": False, "base": 10000.0, "factor": 1.0, "far": 0, "page": 64, "cache": "bf16", "lens": 8},
        # the headline shape's backward
        {"name": "rope-bwd-B2-N4096-H32-KV8", "op": "rope_bwd", "B": 2, "N": 4096, "H": 32, "KV": 8, "d": 128, "rot": 128,
         "inter": False, "norm": True, "base": 10000.0, "factor": 1.0, "far": 0, "lens": 9},
        # a short packed batch of odd length, a quarter of the head left alone
        {"name": "rope-bwd-T1001-H16-KV4-d64", "op": "rope_bwd", "B": 1, "N": 1001, "H": 16, "KV": 4, "d": 64, "rot": 48,
         "inter": True, "norm": True, "base": 10000.0, "factor": 1.0, "far": 0, "lens": 10},
        # one step of 256 requests: most have room in their last page
        {"name": "slots-step-B256", "op": "slots", "B": 256, "lo": 1, "hi": 1, "old": 16384, "page": 16, "lens": 11},
        # 16 prompts of the variable-length workload
        {"name": "slots-prompts-B16-U128-4096", "op": "slots", "B": 16, "lo": 128, "hi": 4096, "old": 0, "page": 64, "lens": 12},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["paged", "paged", "paged", "rope", "rope", "rope_bwd", "slots"])
    lens = rng.randrange(1 << 20)
    if op == "slots":
        if rng.random() < 0.5:
            return {"op": op, "B": _spread(rng, 1, 2000), "lo": 1, "hi": 1, "old": _spread(rng, 64, 20000),
                    "page": rng.choice([16, 32, 64, 128]), "lens": lens}
        return {"op": op, "B": _spread(rng, 1, 40), "lo": 1, "hi": _spread(rng, 100, 5000), "old": rng.choice([0, 0, 1000]),
                "page": rng.choice([16, 32, 64, 128]), "lens": lens}
    d = rng.choice([64, 128, 128])
    KV = rng.choice([1, 2, 4, 8, 16])
    H = KV * rng.choice([1, 2, 3, 4, 6, 8]) if KV > 1 else rng.choice([8, 16, 20, 32])
    H = min(H, 64) // KV * KV
    if op == "paged":
        most = 4_000_000_000  # bytes of live K and V rows
        cache = rng.choice(["bf16", "bf16", "e4m3"])
        hi = _spread(rng, 16, 50000)
        row = 2 * KV * d * (2 if cache == "bf16" else 1)
        B = _spread(rng, 1, max(1, min(256, most // (row * hi))))
        return {"op": op, "B": B, "H": H, "KV": KV, "d": d, "lo": rng.choice([1, hi]), "hi": hi,
                "page": rng.choice([16, 32, 64, 128]), "cache": cache, "lens": lens}
    rot = rng.choice([d, d, d // 2, d // 4, d - 16])
    c = {"op": op, "H": H, "KV": KV, "d": d, "rot": rot, "inter": rng.random() < 0.4, "norm": rng.random() < 0.7,
         "base": rng.choice([10000.0, 500000.0]), "factor": rng.choice([1.0, 4.0, 8.0]), "lens": lens}
    T = _spread(rng, 1, min(33000, 80_000_000 // ((H + 2 * KV) * d)))
    if op == "rope_bwd":
        B = rng.choice([1, 1, 2, 3])
        T = min(T, 8192)
        return {**c, "B": B, "N": max(1, T // B), "far": 0}
    if rng.random() < 0.4:  # one new token of each request
        return {**c, "B": min(T, 300), "N": 1, "far": _spread(rng, 1000, 1000000), "page": rng.choice([16, 64]),
                "cache": rng.choice(["bf16", "e4m3"])}
    B = rng.choice([1, 1, 2])
    return {**c, "B": B, "N": max(1, T // B), "far": 0, "page": rng.choice([16, 64]), "cache": rng.choice(["none", "bf16"])}


def _lens(case):
    r = random.Random(case["lens"])
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


def _inv_freq(case):
    i = torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64)
    return case["base"] ** (-i / case["rot"]) / case["factor"]


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": dict(case)}
    if case["op"] == "paged":
        B, KV, d, page = case["B"], case["KV"], case["d"], case["page"]
        lens = _lens(case)
        used = [-(-n // page) for n in lens]
        width = -(-case["hi"] // page)
        pages = sum(used) + 3
        table = torch.full((B, width), -1, dtype=torch.int32)
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        at = 0
        for s, n in enumerate(used):
            table[s, :n] = order[at:at + n]
            at += n
        st["table"] = table.cuda()
        st["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
        st["q"] = _normal(g, B, case["H"], 1, d)
        st["scale"] = 1.0 / math.sqrt(d)
        if case["cache"] == "bf16":
            st["k"], st["v"] = _normal(g, pages, KV, page, d), _normal(g, pages, KV, page, d)
            st["ks"] = st["vs"] = None
        else:
            st["k"], st["ks"] = _codes(g, pages, KV, page, d)
            st["v"], st["vs"] = _codes(g, pages, KV, page, d)
        # a generating program keeps one workspace for all its steps
        st["ws"] = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
        return st
    if case["op"] == "slots":
        B, page = case["B"], case["page"]
        r = random.Random(seed)
        new = _lens(case)
        old = [r.randint(0, case["old"]) for _ in range(B)]
        had = [-(-n // page) for n in old]
        width = -(-(case["old"] + case["hi"]) // page) + 1
        more = sum(-(-(o + n) // page) - h for o, n, h in zip(old, new, had))
        order = torch.randperm(sum(had) + more + 7, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(had):
            table[s, :n] = order[at:at + n]
            at += n
        cu = torch.zeros(B + 1, dtype=torch.int32)
        cu[1:] = torch.tensor(new, dtype=torch.int32).cumsum(0)
        st.update(table=table.cuda(), lens=torch.tensor(old, dtype=torch.int32).cuda(), cu=cu.cuda(), T=sum(new),
                  free=order[at:].contiguous().cuda(), head=torch.tensor([3], dtype=torch.int32).cuda())
        return st
    B, N, H, KV, d = case["B"], case["N"], case["H"], case["KV"], case["d"]
    T = B * N
    st["qkv"] = _normal(g, B, N, (H + 2 * KV) * d)
    st["inv_freq"] = _inv_freq(case)
    if case["far"]:
        st["pos"] = torch.randint(0, case["far"], (B, N), generator=g, device="cuda", dtype=torch.int32)
    else:
        st["pos"] = torch.arange(N, device="cuda", dtype=torch.int32).repeat(B, 1)
    st["wq"] = st["wk"] = None
    if case["norm"]:
        st["wq"], st["wk"] = (1 + 0.2 * _normal(g, 2, d)).unbind(0)
    if case["op"] == "rope_bwd":
        st["dq"], st["dk"], st["dv"] = _normal(g, B, H, N, d), _normal(g, B, KV, N, d), _normal(g, B, KV, N, d)
        return st
    st["k"] = st["v"] = st["ks"] = st["vs"] = st["slots"] = None
    if case["cache"] != "none":
        page = case["page"]
        pages = -(-T // page) + (T if N == 1 else 0) + 2
        kind = BF16 if case["cache"] == "bf16" else E4M3
        st["k"], st["v"] = (torch.zeros(pages, KV, page, d, device="cuda").to(kind) for _ in range(2))
        if kind == E4M3:
            st["ks"], st["vs"] = (torch.zeros(pages, KV, page, device="cuda") for _ in range(2))
        order = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        if N == 1:  # each request's token somewhere in a page of its own
            st["slots"] = order[:T] * page + torch.randint(0, page, (T,), generator=g, device="cuda")
        else:
            st["slots"] = order[t // page] * page + t % page
    return st


# ------------------------------------------------------------------------------- plain forms
def _paged_plain(st):
    c, q = st["case"], st["q"]
    B, H, KV, d, page = c["B"], c["H"], c["KV"], c["d"], c["page"]
    width = st["table"].shape[1]
    at = st["table"].clamp(min=0).long()

    def rows(codes, scale):
        x = codes[at] if codes.dtype == BF16 else codes.view(torch.uint8)[at].view(E4M3)
        x = x.float()
        if scale is not None:
            x = x * scale[at][..., None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, KV, width * page, d)

    dead = torch.arange(width * page, device=q.device)[None, :] >= st["lens"][:, None]
    s = torch.matmul(q.float().reshape(B, KV, H // KV, d), rows(st["k"], st["ks"]).transpose(2, 3)) * st["scale"]
    s = s.masked_fill(dead[:, None, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    v = rows(st["v"], st["vs"]).masked_fill(dead[:, None, :, None], 0.0)
    o = torch.matmul(p, v) / total
    return o.reshape(B, H, 1, d).to(BF16), (m + torch.log(total)).reshape(B, H, 1)


def _angles(st):
    a = st["pos"].double()[..., None] * st["inv_freq"]
    return a.cos().float(), a.sin().float()


def _turn(x, cos, sin, rot, inter):
    """Rotates the first `rot` columns of x [B, N, heads, d]; cos, sin [B, N, rot / 2]."""
    cos, sin = cos[:, :, None], sin[:, :, None]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((ya, yb), -1).flatten(-2) if inter else torch.cat((ya, yb), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _rope_plain(st):
    c = st["case"]
    B, N, H, KV, d = c["B"], c["N"], c["H"], c["KV"], c["d"]
    x = st["qkv"].float().view(B, N, H + 2 * KV, d)
    cos, sin = _angles(st)
    y = []
    for part, w in ((x[:, :, :H], st["wq"]), (x[:, :, H:H + KV], st["wk"])):
        if w is not None:
            part = part * torch.rsqrt((part * part).mean(-1, keepdim=True) + EPS) * w.float()
        y.append(_turn(part, cos, sin, c["rot"], c["inter"]))
    y.append(x[:, :, H + KV:])
    out = [t.to(BF16).transpose(1, 2).contiguous() for t in (y if N > 1 else y[:1])]
    if st["slots"] is None:
        return out
    page, off = st["slots"] // c["page"], st["slots"] % c["page"]
    for t, codes, scale in ((y[1], st["k"], st["ks"]), (y[2], st["v"], st["vs"])):
        t = t.reshape(B * N, KV, d)
        if scale is not None:
            amax = t.abs().amax(-1)
            s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
            scale[page, :, off] = s
            codes.view(torch.uint8)[page, :, off] = (t / s[..., None]).to(E4M3).view(torch.uint8)
        else:
            codes[page, :, off] = t.to(BF16)
    return out + [t for t in (st["k"], st["v"], st["ks"], st["vs"]) if t is not None]


def _rope_bwd_plain(st):
    c = st["case"]
    B, N, H, KV, d = c["B"], c["N"], c["H"], c["KV"], c["d"]
    x = st["qkv"].float().view(B, N, H + 2 * KV, d)
    cos, sin = _angles(st)
    dx, dw = [], []
    for part, dy, w in ((x[:, :, :H], st["dq"], st["wq"]), (x[:, :, H:H + KV], st["dk"], st["wk"])):
        g = _turn(dy.float().transpose(1, 2), cos, -sin, c["rot"], c["inter"])
        if w is not None:
            r = torch.rsqrt((part * part).mean(-1, keepdim=True) + EPS)
            n = part * r
            dw.append((g * n).sum((0, 1, 2)))
            g = g * w.float()
            g = r * (g - n * (g * n).mean(-1, keepdim=True))
        dx.append(g)
    dx.append(st["dv"].float().transpose(1, 2))
    return [torch.cat(dx, 2).to(BF16).view(B, N, -1)] + dw


def _slots_plain(st):
    page, T, table, lens = st["case"]["page"], st["T"], st["table"], st["lens"]
    cu = st["cu"].long()
    new = cu[1:] - cu[:-1]
    old = lens.long()
    had = (old + page - 1) // page
    need = (old + new + page - 1) // page - had
    first = need.cumsum(0) - need + st["head"].long()
    seq = torch.repeat_interleave(torch.arange(len(lens), device=cu.device), new, output_size=T)
    pos = old[seq] + torch.arange(T, device=cu.device) - cu[seq]
    j = pos // page
    fresh = j - had[seq]
    taken = st["free"][(first[seq] + fresh).clamp(0, len(st["free"]) - 1)].long()
    where = torch.where(fresh >= 0, taken, table[seq, j].long())
    table[seq, j] = where.to(torch.int32)
    return where * page + pos % page, pos.to(torch.int32), table, (old + new).to(torch.int32), \
        (st["head"].long() + need.sum()).to(torch.int32)


# ---------------------------------------------------------------------------- the framework's
def _own(st):
    from io_aware_attention_attn_gb300 import attn
    c = st["case"]
    if c["op"] == "paged":
        cache = attn.KVCache(st["k"], st["v"], st["ks"], st["vs"])
        return attn.attn_fwd_paged(st["q"], cache, st["table"], st["lens"], scale=st["scale"], workspace=st["ws"])
    if c["op"] == "slots":
        return attn.kv_slots(st["lens"], st["cu"], st["T"], st["table"], st["free"], st["head"], c["page"])
    rope = dict(inv_freq=st["inv_freq"], interleaved=c["inter"], wq=st["wq"], wk=st["wk"], eps=EPS)
    if c["op"] == "rope_bwd":
        out = attn.qkv_rope_bwd(st["dq"], st["dk"], st["dv"], st["qkv"], st["pos"], **rope)
        return [t for t in out if t is not None]
    cache = None if st["slots"] is None else attn.KVCache(st["k"], st["v"], st["ks"], st["vs"])
    out = attn.qkv_rope(st["qkv"], c["H"], c["KV"], st["pos"], cache=cache, slots=st["slots"], with_kv=c["N"] > 1, **rope)
    return [t for t in out if t is not None] + ([t for t in cache if t is not None] if cache else [])


def run(st):
    if own:
        return _own(st)
    return {"paged": _paged_plain, "rope": _rope_plain, "rope_bwd": _rope_bwd_plain, "slots": _slots_plain}[st["case"]["op"]](st)


# -------------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "paged":
        B, H, KV, d = case["B"], case["H"], case["KV"], case["d"]
        total = sum(_lens(case))
        row = 2 * KV * (2 * d if case["cache"] == "bf16" else d + 4)
        return {"bytes": total * row + B * H * (4 * d + 4) + 4 * (total // case["page"]), "flops": 4 * total * H * d}
    if case["op"] == "slots":
        T = sum(_lens(case))
        return {"bytes": 12 * T + 16 * case["B"], "flops": 0}
    T, H, KV, d = case["B"] * case["N"], case["H"], case["KV"], case["d"]
    rows = T * (H + 2 * KV) * d * 2
    if case["op"] == "rope_bwd":
        return {"bytes": 3 * rows + 4 * T, "flops": 20 * T * (H + KV) * d}
    byte = {"none": 0, "bf16": 2, "e4m3": 1}[case["cache"]]
    out = T * H * d * 2 + (2 * T * KV * d * 2 if case["N"] > 1 else 0) + 2 * T * KV * d * byte
    return {"bytes": rows + out + 12 * T, "flops": 10 * T * (H + KV) * d}


# --------------------------------------------------------------------- the definition, 64 bits
def _paged_exact(st):
    c = st["case"]
    B, H, KV, d, page = c["B"], c["H"], c["KV"], c["d"], c["page"]
    o = torch.empty(B, H, 1, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(B, H, 1, dtype=torch.float64, device="cuda")
    for s, n in enumerate(_lens(c)):
        ids = st["table"][s, :-(-n // page)].long()
        kv = []
        for codes, scale in ((st["k"], st["ks"]), (st["v"], st["vs"])):
            x = torch.stack([codes[i] for i in ids]).double() if codes.dtype == BF16 else \
                codes.view(torch.uint8).index_select(0, ids).view(E4M3).double() * scale.index_select(0, ids).double()[..., None]
            kv.append(x.transpose(0, 1).reshape(KV, -1, d)[:, :n])
        q = st["q"][s, :, 0].double().view(KV, H // KV, d)
        z = torch.einsum("hgd,hnd->hgn", q, kv[0]) * st["scale"]
        lse[s] = torch.logsumexp(z, -1).reshape(H, 1)
        o[s] = torch.einsum("hgn,hnd->hgd", torch.softmax(z, -1), kv[1]).reshape(H, 1, d)
    return o, lse


def _rope_exact_rows(x, st, w):
    """Rows x [B, N, heads, d] in 64 bits: normed, then each pair turned as a complex number."""
    c = st["case"]
    rot = c["rot"]
    if w is not None:
        x = x / (x.square().sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * w
    head = x[..., :rot].unflatten(-1, (rot // 2, 2) if c["inter"] else (2, rot // 2))
    if not c["inter"]:
        head = head.transpose(-1, -2)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       st["pos"].double()[:, :, None, None] * st["inv_freq"])
    z = torch.view_as_real(torch.view_as_complex(head.contiguous()) * turn)
    if not c["inter"]:
        z = z.transpose(-1, -2)
    return torch.cat((z.flatten(-2), x[..., rot:]), -1)


def _rope_exact(st):
    c = st["case"]
    B, N, H, KV, d = c["B"], c["N"], c["H"], c["KV"], c["d"]
    x = st["qkv"].double().unflatten(-1, (H + 2 * KV, d))
    w = [None if t is None else t.double() for t in (st["wq"], st["wk"])]
    q, k, v = x.split((H, KV, KV), 2)
    q, k = _rope_exact_rows(q, st, w[0]), _rope_exact_rows(k, st, w[1])
    out = [t.permute(0, 2, 1, 3) for t in ((q, k, v) if N > 1 else (q,))]
    if st["slots"] is None:
        return out
    page = c["page"]
    full = [torch.zeros(st["k"].shape, dtype=torch.float64, device="cuda").transpose(1, 2).flatten(0, 1) for _ in range(2)]
    if st["ks"] is not None:  # the codes are decided by a rounding: only their scales have a value in 64 bits
        scales = [f.new_zeros(f.shape[:2]) for f in full]
        for f, t in zip(scales, (k, v)):
            f[st["slots"]] = t.reshape(B * N, KV, d).abs().amax(-1) / 448
        return out + [None, None] + [f.unflatten(0, (-1, page)).transpose(1, 2) for f in scales]
    for f, t in zip(full, (k, v)):
        f[st["slots"]] = t.reshape(B * N, KV, d)
    return out + [f.unflatten(0, (-1, page)).transpose(1, 2) for f in full]


def _rope_bwd_exact(st):
    c = st["case"]
    H, KV, d = c["H"], c["KV"], c["d"]
    x = st["qkv"].double().requires_grad_()
    w = [None if t is None else t.double().requires_grad_() for t in (st["wq"], st["wk"])]
    q, k, v = x.unflatten(-1, (H + 2 * KV, d)).split((H, KV, KV), 2)
    q, k = _rope_exact_rows(q, st, w[0]), _rope_exact_rows(k, st, w[1])
    loss = sum((t.transpose(1, 2) * g.double()).sum() for t, g in ((q, st["dq"]), (k, st["dk"]), (v, st["dv"])))
    return list(torch.autograd.grad(loss, [x] + [t for t in w if t is not None]))


def _slots_exact(st):
    page, table, free = st["case"]["page"], st["table"].tolist(), st["free"].tolist()
    lens, cu, head = st["lens"].tolist(), st["cu"].tolist(), st["head"].item()
    slots, pos = [], []
    for s, n in enumerate(lens):
        for t in range(n, n + cu[s + 1] - cu[s]):
            if t % page == 0:
                table[s][t // page] = free[head]
                head += 1
            slots.append(table[s][t // page] * page + t % page)
            pos.append(t)
        lens[s] = n + cu[s + 1] - cu[s]
    i32 = dict(dtype=torch.int32)
    return torch.tensor(slots), torch.tensor(pos, **i32), torch.tensor(table, **i32), torch.tensor(lens, **i32), \
        torch.tensor([head], **i32)


def exact(case, seed):
    st = prepare(case, seed)
    return {"paged": _paged_exact, "rope": _rope_exact, "rope_bwd": _rope_bwd_exact, "slots": _slots_exact}[case["op"]](st)
