"""CPU oracle of work over a paged cache beyond one new token a request: attention of several new tokens,
attention behind a shared prefix, rows written into a cache and read back.

TEST INFRASTRUCTURE ONLY, like the other oracles: the product never calls it and shares no code with
it.  Plain definitions in float64, request by request and head by head.
"""
from __future__ import annotations

import numpy as np


def rows(values, table, n):
    """Rows [H_kv, n, d] of a request: values [pages, H_kv, page_size, d]."""
    P = values.shape[2]
    out = [values[int(p)] for p in table[: -(-n // P)]]
    return np.concatenate(out, axis=1)[:, :n] if out else np.zeros((values.shape[1], 0, values.shape[3]))


def attend(q, k, v, seen, scale):
    """One head: q [n, d] against k, v [L, d], query i over its first seen[i] keys.  Returns O, lse and, for error
    bounds, A = sum_j P_j |v_j|, Z = max_j scale sum |q k_j|, W = scale max |q| max_j sum |k_j|."""
    n, d = q.shape
    o, a = np.zeros((n, d)), np.zeros((n, d))
    lse, z, w = np.full(n, -np.inf), np.zeros(n), np.zeros(n)
    for i in range(n):
        m = min(max(int(seen[i]), 0), len(k))
        if m == 0:
            continue
        s = scale * (k[:m] @ q[i])
        top = s.max()
        p = np.exp(s - top)
        o[i], a[i] = p @ v[:m] / p.sum(), p @ np.abs(v[:m]) / p.sum()
        lse[i] = top + np.log(p.sum())
        z[i] = scale * (np.abs(k[:m]) @ np.abs(q[i])).max()
        w[i] = scale * np.abs(q[i]).max() * np.abs(k[:m]).sum(1).max()
    return o, lse, a, z, w


def varlen(q, k, v, table, seq_lens, cu, causal, scale, tokens=None):
    """q [H, T, d]; per token of `tokens` (all of the requests'): (token, O [H, d], lse [H], A, Z [H], W [H])."""
    H = q.shape[0]
    out = []
    for s in range(len(seq_lens)):
        L, a, b = int(seq_lens[s]), int(cu[s]), int(cu[s + 1])
        mine = [t for t in range(a, b) if tokens is None or t in tokens]
        if not mine:
            continue
        kk, vv = rows(k, table[s], L), rows(v, table[s], L)
        seen = [L - (b - a) + (t - a) + 1 if causal else L for t in mine]
        parts = [attend(q[h, mine], kk[h * len(kk) // H], vv[h * len(vv) // H], seen, scale) for h in range(H)]
        for i, t in enumerate(mine):
            out.append((t, *(np.stack([p[x][i] for p in parts]) for x in range(5))))
    return out


def shared(q, k, v, prefix_table, prefix_lens, cu_groups, table, seq_lens, scale):
    """q [B, H, d]: (O, lse, A, Z, W) over the prefix's rows and the request's own."""
    B, H, d = q.shape
    o, a = np.zeros((B, H, d)), np.zeros((B, H, d))
    lse, z, w = np.full((B, H), -np.inf), np.zeros((B, H)), np.zeros((B, H))
    for g in range(len(prefix_lens)):
        for s in range(int(cu_groups[g]), int(cu_groups[g + 1])):
            kk, vv = (np.concatenate([rows(x, prefix_table[g], int(prefix_lens[g])), rows(x, table[s], int(seq_lens[s]))], 1)
                      for x in (k, v))
            for h in range(H):
                y = attend(q[s, h:h + 1], kk[h * len(kk) // H], vv[h * len(vv) // H], [kk.shape[1]], scale)
                o[s, h], lse[s, h], a[s, h], z[s, h], w[s, h] = (x[0] for x in y)
    return o, lse, a, z, w
