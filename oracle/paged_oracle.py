"""fp64 oracle of the paged key/value cache: block tables and slots from request lengths,
the cache's write, and each request's new tokens' attention over its pages.

TEST INFRASTRUCTURE ONLY (see the package docstring): the CUDA library never imports or
calls this module.
"""
from __future__ import annotations

import numpy as np

from .gqa_oracle import gqa_split


def kv_tables(ctx, new, free, head, table, T, P):
    """Plain loops over requests and tokens. Returns a dict of every output."""
    R, MP = table.shape
    table = table.copy()
    n_free = len(free)
    head = min(max(int(head), 0), n_free)
    cu, total, slots, pos = [0], [], [-1] * T, [-1] * T
    at = head
    for r in range(R):
        c, n = max(int(ctx[r]), 0), max(int(new[r]), 0)
        for p in range(min(-(-c // P), MP), min(-(-(c + n) // P), MP)):
            table[r, p] = free[at] if at < n_free else -1
            at += 1
        for i in range(n):
            t = cu[-1] + i
            if t >= T:
                break
            pos[t] = c + i
            pg = (c + i) // P
            if pg < MP and table[r, pg] >= 0:
                slots[t] = int(table[r, pg]) * P + (c + i) % P
        cu.append(cu[-1] + n)
        total.append(c + n)
    taken = min(at, n_free) - head
    return {"table": table, "total": total, "cu": cu, "slots": slots, "pos": pos,
            "head": head + taken,
            "counts": [cu[-1], taken, at - head - taken, max(cu[-1] - T, 0)]}


def qkv_heads(qkv, H, Hkv, N):
    """Queries (T, H, d), and keys and values (T, Hkv, d) of the first replicas, out of the
    sharded rows."""
    hq, hkv, rep = gqa_split(H, Hkv, N)
    T, W = qkv.shape
    blk = hq + 2 * hkv
    x = qkv.reshape(T, N, blk, W // (N * blk))
    q = x[:, :, :hq].reshape(T, H, -1)
    first = x[:, ::rep]
    return (q, first[:, :, hq:hq + hkv].reshape(T, Hkv, -1),
            first[:, :, hq + hkv:].reshape(T, Hkv, -1))


def kv_append(k, v, slots, kc, vc):
    """Rows k, v (T, Hkv, d) into copies of the caches (n_pages, Hkv, P, d)."""
    kc, vc = kc.copy(), vc.copy()
    n_pages, _, P, _ = kc.shape
    for t, s in enumerate(slots):
        if 0 <= s < n_pages * P:
            kc[s // P, :, s % P] = k[t]
            vc[s // P, :, s % P] = v[t]
    return kc, vc


def paged_attention(q, kc, vc, table, total, cu, causal):
    """q (T, H, d); caches (n_pages, Hkv, P, d). Returns o (T, H, d), lse (H, T), written (T)
    and, for error bounds, A = sum p |v| / sum p (T, H, d), B (H, T) = the largest
    sum |q k| / sqrt(d) over a row's keys, and n (H, T) the number of its keys."""
    T, H, d = q.shape
    n_pages, Hkv, P, _ = kc.shape
    MP = table.shape[1]
    o, A = np.zeros((T, H, d)), np.zeros((T, H, d))
    lse, B, cnt = np.full((H, T), -np.inf), np.zeros((H, T)), np.zeros((H, T))
    written = np.zeros(T, bool)
    for r in range(len(total)):
        n = max(cu[r + 1] - cu[r], 0)
        end = min(max(int(total[r]), 0), MP * P)
        keys = [k for k in range(end) if 0 <= table[r, k // P] < n_pages]
        pg = np.array([table[r, k // P] for k in keys], int)
        off = np.array([k % P for k in keys], int)
        pos = np.array(keys, int)
        K = kc[pg, :, off] if len(keys) else np.zeros((0, Hkv, d))
        V = vc[pg, :, off] if len(keys) else np.zeros((0, Hkv, d))
        for i in range(n):
            t = cu[r] + i
            if not 0 <= t < T:
                continue
            written[t] = True
            see = pos <= max(int(total[r]), 0) - n + i if causal else pos >= 0
            if not see.any():
                continue
            for h in range(H):
                j = h // (H // Hkv)
                s = K[see, j] @ q[t, h] / np.sqrt(d)
                m = s.max()
                p = np.exp(s - m)
                z = p.sum()
                o[t, h] = p @ V[see, j] / z
                A[t, h] = p @ np.abs(V[see, j]) / z
                lse[h, t] = m + np.log(z)
                B[h, t] = (np.abs(K[see, j]) @ np.abs(q[t, h])).max() / np.sqrt(d)
                cnt[h, t] = see.sum()
    return {"o": o, "lse": lse, "A": A, "B": B, "n": cnt, "written": written}
