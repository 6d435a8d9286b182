"""Attention over a paged cache in float64 torch, for sizes at which the oracle's loops take
too long, and the runner of the paged kernels that compares every element with it.

Tolerances, element by element, from A = sum p |v| / sum p and B = max_k sum |q k| / sqrt(d)
of the row, n its keys, u = 2^-24: a score's fp32 sum of d products is off by at most
(d + 4) u B, so p by twice that share (its own and the normaliser's); sums over n keys add
2 n u, exponentials and the joins of pieces 64 u. In bf16, P is rounded to 2^-8 of itself,
hence 2^-8 A, and the output to 2^-8 |o|; in fp32 the output's rounding is u |o|. lse: the
largest score's error, the sum's, and 4 u |lse| for the product with ln 2 and the additions.
"""
import math

import numpy as np
import torch

from attention_gemms_gb300 import tpmlp as T
from oracle import gqa_oracle as Q

U = 2.0 ** -24


def i32(a, device="cuda"):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(device)


def cols(H, Hkv, N, d):
    hq, hkv, _ = Q.gqa_split(H, Hkv, N)
    return N * (hq + 2 * hkv) * d


def queries(qkv, H, Hkv, N):
    """(T, H, d) view of the packed rows' query columns."""
    hq, hkv, _ = Q.gqa_split(H, Hkv, N)
    rows = qkv.shape[0]
    x = qkv.view(rows, N, hq + 2 * hkv, -1)
    return x[:, :, :hq].reshape(rows, H, -1)


def seen(table, tot, cu, rows, n_pages, P, causal):
    """(n_pages, P) truth values: the slots that some row below `rows` sees."""
    used = np.zeros((n_pages, P), bool)
    for r in range(len(tot)):
        n = max(int(cu[r + 1]) - int(cu[r]), 0)
        have = min(n, max(rows - int(cu[r]), 0))       # rows that exist
        if have == 0:
            continue
        end = int(tot[r]) - n + have if causal else int(tot[r])
        for k in range(max(min(end, table.shape[1] * P), 0)):
            pg = int(table[r, k // P])
            if 0 <= pg < n_pages:
                used[pg, k % P] = True
    return used


def reference(q, kc, vc, table, tot, cu, causal):
    """q (T, H, d), caches (n_pages, Hkv, P, d), tables and lengths on the host. NaN in keys
    and values is taken as zero (slots that no row sees); NaN in q reaches its row. Returns
    o, A (T, H, d), lse, B, n (H, T) and written (T)."""
    rows, H, d = q.shape
    n_pages, Hkv, P, _ = kc.shape
    G, dev, f64 = H // Hkv, q.device, torch.float64
    o = torch.zeros(rows, H, d, dtype=f64, device=dev)
    A = torch.zeros_like(o)
    lse = torch.full((H, rows), -math.inf, dtype=f64, device=dev)
    B, cnt = torch.zeros_like(lse), torch.zeros_like(lse)
    written = torch.zeros(rows, dtype=torch.bool, device=dev)
    for r in range(len(tot)):
        n = max(int(cu[r + 1]) - int(cu[r]), 0)
        t0, have = int(cu[r]), min(n, max(rows - int(cu[r]), 0))
        if have == 0:
            continue
        written[t0:t0 + have] = True
        end = min(max(int(tot[r]), 0), table.shape[1] * P)
        key = np.arange(end)
        key = key[(table[r, key // P] >= 0) & (table[r, key // P] < n_pages)]
        if len(key) == 0:
            continue
        page = torch.from_numpy(table[r, key // P].astype(np.int64)).to(dev)
        off, key = torch.from_numpy(key % P).to(dev), torch.from_numpy(key).to(dev)
        last = max(int(tot[r]), 0) - n + torch.arange(have, device=dev)
        hidden = key[None, :] > last[:, None] if causal else \
            torch.zeros(have, len(key), dtype=torch.bool, device=dev)
        none = hidden.all(1)
        for h in range(H):
            j = h // G
            k = kc[page, j, off].to(f64).nan_to_num(0.0)
            v = vc[page, j, off].to(f64).nan_to_num(0.0)
            qq = q[t0:t0 + have, h].to(f64)
            s = (qq @ k.T) / math.sqrt(d)
            s = s.masked_fill(hidden, -math.inf)
            m = s.amax(1, keepdim=True)
            m = torch.where(torch.isneginf(m), torch.zeros_like(m), m)
            p = torch.exp(s - m)
            z = p.sum(1, keepdim=True)
            zz = torch.where(none[:, None], torch.ones_like(z), z)
            o[t0:t0 + have, h] = p @ v / zz
            A[t0:t0 + have, h] = p @ v.abs() / zz
            lse[h, t0:t0 + have] = torch.where(none, -math.inf, (m + torch.log(zz))[:, 0])
            B[h, t0:t0 + have] = ((qq.abs() @ k.abs().T) / math.sqrt(d)) \
                .masked_fill(hidden, 0.0).amax(1)
            cnt[h, t0:t0 + have] = (~hidden).sum(1).to(f64)
    return {"o": o, "A": A, "lse": lse, "B": B, "n": cnt, "written": written}


def attend(lens, H, Hkv, N, d, P, dtype, causal=1, *, seed=1, rows=None, total=None, pad=0,
           max_new=None, spare=2, cu=None, width=None, fill=None):
    """The attention call on random data with scattered pages, NaN in every slot that no
    existing row sees and in the workspace; checks every element of o and lse. lens: (cached,
    new) per request, total and cu in their place where given; width: the table's, where the
    lengths want more; fill(qkv, keys, values, pos): edits the inputs, pos (n_pages, P) the
    position that a slot holds (-1: none)."""
    rng = np.random.default_rng(seed)
    tot = np.array([c + n for c, n in lens] if total is None else total)
    cu = np.concatenate([[0], np.cumsum([n for _, n in lens])]) if cu is None else np.array(cu)
    rows = int(cu[-1]) + pad if rows is None else rows
    pages = [min(max(-(-int(t) // P), 0), width or 1 << 30) for t in tot]
    n_pages = sum(pages) + spare
    perm = rng.permutation(n_pages)
    table = np.full((len(lens), max(pages + [1])), -1)
    pos = np.full((n_pages, P), -1)
    at = 0
    for r, k in enumerate(pages):
        table[r, :k] = perm[at:at + k]
        pos[perm[at:at + k]] = np.arange(k * P).reshape(k, P)
        at += k
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").to(tdt)
    qkv = rnd(rows, cols(H, Hkv, N, d))
    kc, vc = rnd(n_pages, Hkv, P, d), rnd(n_pages, Hkv, P, d)
    if fill:
        fill(qkv, kc, vc, torch.from_numpy(pos).cuda())
    used = seen(table, tot, cu, rows, n_pages, P, causal)
    dead = torch.from_numpy(~used).cuda()[:, None, :, None].expand_as(kc)
    kc[dead], vc[dead] = float("nan"), float("nan")
    ref = reference(queries(qkv, H, Hkv, N), kc, vc, table, tot, cu, bool(causal))
    h, dt = H * d, T.dtype_of(qkv)
    o = torch.full((rows, h), -768.0, dtype=tdt, device="cuda")
    lse = torch.full((H, rows), -768.0, device="cuda")
    wsb = T.tp_gqa_paged_attention_workspace_size(h, H, Hkv, N, dt)
    ws = torch.full((wsb,), 255, dtype=torch.uint8, device="cuda")  # NaN: must not be read
    new = max([n for _, n in lens]) if max_new is None else max_new
    T.tp_gqa_paged_attention_fwd(qkv, kc, vc, i32(table), i32(tot), i32(cu), o, lse, rows, len(lens),
                                 h, H, Hkv, N, n_pages, P, table.shape[1], new, causal, dt, ws, wsb)
    torch.cuda.synchronize()
    assert T.tp_check_status() == 0
    check(o.view(rows, H, d), lse, ref, d, dtype)
    return o, lse, ref


def check(o, lse, ref, d, dtype):
    w = ref["written"]
    assert (o[~w].float() == -768.0).all() and (lse[:, ~w] == -768.0).all()
    B, n = ref["B"].T[:, :, None], ref["n"].T[:, :, None]
    sums = U * (2 * (d + 4) * B + 2 * n + 64)
    half = 2.0 ** -8 if dtype == "bf16" else U
    tol = ref["A"] * (sums + (half if dtype == "bf16" else 0.0)) + ref["o"].abs() * half
    nan = ref["o"].isnan()
    assert (o.isnan() == nan)[w].all()
    err = (o.double() - ref["o"]).abs()
    bad = (err > tol) & ~nan & w[:, None, None]
    assert not bad.any(), (bad.nonzero()[:5].tolist(), err[bad].max().item())
    rl, gl = ref["lse"][:, w], lse[:, w].double()
    assert (gl.isnan() == rl.isnan()).all() and (gl.isneginf() == rl.isneginf()).all()
    fin = rl.isfinite()
    ltol = U * ((d + 4) * ref["B"] + ref["n"] + 64)[:, w] + 4 * U * rl.abs()
    over = ((gl - rl).abs() > ltol) & fin
    assert not over.any(), (over.nonzero()[:5].tolist(), (gl - rl).abs()[over].max().item())
