"""CPU oracle of the generation path: norm and rotation of query and key heads with their backward,
slots of new tokens in a paged cache, and attention of one new token over the cache.

TEST INFRASTRUCTURE ONLY, like the other oracles: the product never calls it and shares no code with
it.  Plain definitions in float64 (integers for the slots), written with loops over what the
kernels share out: heads, requests, tokens.
"""
from __future__ import annotations

import numpy as np


def rotate(x, pos, inv_freq, interleaved: bool, scale: float = 1.0, back: bool = False):
    """Rows x [T, d] turned by their positions' angles; the first 2 len(inv_freq) elements turn.
    ``back`` applies the transposed matrix (the gradient's direction)."""
    y = np.array(x, dtype=np.float64)
    nf = len(inv_freq)
    ang = np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)
    c, s = np.cos(ang) * scale, np.sin(ang) * scale
    if back:
        s = -s
    for i in range(nf):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + nf)
        xa, xb = y[:, a].copy(), y[:, b].copy()
        y[:, a] = xa * c[:, i] - xb * s[:, i]
        y[:, b] = xb * c[:, i] + xa * s[:, i]
    return y


def norm(x, w, eps: float):
    """RMS norm of rows x [T, d]; the rows themselves without a weight."""
    if w is None:
        return np.array(x, dtype=np.float64)
    return x * w / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps)


def qkv_rope(qkv, H, H_kv, d, pos, inv_freq, interleaved, wq, wk, eps, scale=1.0):
    """q [H, T, d], k, v [H_kv, T, d] of rows qkv [T, (H + 2 H_kv) d]."""
    x = qkv.reshape(len(qkv), H + 2 * H_kv, d)
    q = np.stack([rotate(norm(x[:, h], wq, eps), pos, inv_freq, interleaved, scale) for h in range(H)])
    k = np.stack([rotate(norm(x[:, H + h], wk, eps), pos, inv_freq, interleaved, scale)
                  for h in range(H_kv)])
    return q, k, np.stack([x[:, H + H_kv + h] for h in range(H_kv)])


def qkv_rope_bwd(dq, dk, dv, qkv, H, H_kv, d, pos, inv_freq, interleaved, wq, wk, eps, scale=1.0):
    """(d qkv [T, (H + 2 H_kv) d], dwq [d] or None, dwk) from the chain rule."""
    T = len(qkv)
    x = qkv.reshape(T, H + 2 * H_kv, d)
    dx = np.zeros_like(x)
    dw = []
    for dy, w, h0 in ((dq, wq, 0), (dk, wk, H)):
        dwi = np.zeros(d)
        for h in range(len(dy)):
            g = rotate(dy[h], pos, inv_freq, interleaved, scale, back=True)
            if w is not None:
                xh = x[:, h0 + h]
                r = 1.0 / np.sqrt(np.mean(xh * xh, axis=1, keepdims=True) + eps)
                dwi += np.sum(g * xh * r, axis=0)
                u = g * w
                g = r * (u - xh * r * r * np.mean(u * xh, axis=1, keepdims=True))
            dx[:, h0 + h] = g
        dw.append(dwi if w is not None else None)
    for h in range(H_kv):
        dx[:, H + H_kv + h] = dv[h]
    return dx.reshape(T, -1), dw[0], dw[1]


def kv_slots(seq_lens, cu_new, table, free_pages, free_head: int, page_size: int):
    """(slots, positions, table, new seq_lens, new free_head) token by token: a token that finds no
    page for its position takes the next free one.  A request's pages come in order; requests are
    served in order.  A page past the table or the free list: slot -1 (entry -1)."""
    table = [list(r) for r in table]
    max_pages = len(table[0]) if table else 0
    slots, pos, lens = [], [], []
    head = free_head
    for s, old in enumerate(seq_lens):
        old = max(int(old), 0)
        new = int(cu_new[s + 1]) - int(cu_new[s])
        for t in range(old, old + new):
            j = t // page_size
            if t % page_size == 0 and j < max_pages:
                table[s][j] = int(free_pages[head]) if 0 <= head < len(free_pages) else -1
                head += 1
            page = table[s][j] if j < max_pages else -1
            slots.append(page * page_size + t % page_size if page >= 0 else -1)
            pos.append(t)
        lens.append(old + new)
    return slots, pos, table, lens, head


def paged_attention(q, k, v, table, seq_lens, scale: float):
    """O [B, H, d], lse [B, H] and, for error bounds, A = sum_j P_j |v_j| [B, H, d] and
    Z = max_j scale sum |q k_j| [B, H].  q [B, H, d]; k, v [pages, H_kv, page_size, d] values."""
    B, H, d = q.shape
    H_kv, P = k.shape[1], k.shape[2]
    o, a = np.zeros((B, H, d)), np.zeros((B, H, d))
    lse, z = np.full((B, H), -np.inf), np.zeros((B, H))
    for s in range(B):
        n = int(seq_lens[s])
        if n <= 0:
            continue
        ids = [int(p) for p in table[s][: -(-n // P)]]
        for g in range(H_kv):
            kk = np.concatenate([k[p, g] for p in ids])[:n]
            vv = np.concatenate([v[p, g] for p in ids])[:n]
            for h in range(g * (H // H_kv), (g + 1) * (H // H_kv)):
                sc = scale * (kk @ q[s, h])
                m = sc.max()
                p = np.exp(sc - m)
                o[s, h] = p @ vv / p.sum()
                a[s, h] = p @ np.abs(vv) / p.sum()
                lse[s, h] = m + np.log(p.sum())
                z[s, h] = scale * (np.abs(kk) @ np.abs(q[s, h])).max()
    return o, lse, a, z
