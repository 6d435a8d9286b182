"""Cases of the paged key/value cache's operators: block tables and slot maps built from
request lengths (tp_kv_tables), the cache's write (tp_kv_append), and grouped-query
attention of each request's new tokens over its cached pages, from one token per request
(decode) to long chunks (tp_gqa_paged_attention_fwd).

`own` False computes the operators with elementary torch operations, True with the
library's entry points. Pages are `page` tokens of one layout for both: caches are
(n_pages, kv_heads, page, d), the packed QKV rows are the sharded layout of tp_gqa_*.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one user's next token with the GQA benchmark's heads (2 replicas of each kv head)
        dict(name="decode-one", op="attention", dtype="bf16", H=32, Hkv=8, N=16, d=64, page=16,
             R=1, new_lo=1, new_hi=1, ctx_lo=700, ctx_hi=700, pad=0, causal=1),
        # a decode step of a served batch, hidden width 8192, ragged contexts, rows padded to a graph's size
        dict(name="decode-batch", op="attention", dtype="bf16", H=64, Hkv=8, N=8, d=128, page=64,
             R=61, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=8191, pad=3, causal=1),
        # few users with very long documents: the keys have to be split over the GPU
        dict(name="decode-long", op="attention", dtype="bf16", H=32, Hkv=4, N=1, d=128, page=128,
             R=3, new_lo=1, new_hi=1, ctx_lo=90001, ctx_hi=131071, pad=0, causal=1),
        # a draft's tokens verified at once: a few rows per request
        dict(name="verify-drafts", op="attention", dtype="bf16", H=32, Hkv=8, N=8, d=128, page=16,
             R=33, new_lo=2, new_hi=7, ctx_lo=100, ctx_hi=5000, pad=0, causal=1),
        # prompts split into chunks, the first one without a context
        dict(name="chunk-large", op="attention", dtype="bf16", H=64, Hkv=8, N=8, d=128, page=64,
             R=2, new_lo=2048, new_hi=2048, ctx_lo=0, ctx_hi=6000, pad=0, causal=1),
        # the GQA benchmark's heads, four ragged chunks of about its sequence length
        dict(name="chunk-d64", op="attention", dtype="bf16", H=32, Hkv=8, N=16, d=64, page=16,
             R=4, new_lo=401, new_hi=512, ctx_lo=0, ctx_hi=4001, pad=0, causal=1),
        # one scheduler step: decoding requests beside a chunk of a new prompt
        dict(name="mixed-step", op="attention", dtype="bf16", H=32, Hkv=8, N=1, d=128, page=32,
             R=48, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=6000, pad=0, causal=1, chunk=1025),
        # fp32 path: a small model's mixed step
        dict(name="f32-mixed", op="attention", dtype="f32", H=8, Hkv=2, N=2, d=64, page=16,
             R=9, new_lo=1, new_hi=1, ctx_lo=0, ctx_hi=1500, pad=0, causal=1, chunk=130),
        # the set-up of a decode step, and of a step with prompts
        dict(name="tables-decode", op="tables", R=64, page=16, new_lo=1, new_hi=1, ctx_lo=0,
             ctx_hi=8191, pad=0),
        dict(name="tables-prompts", op="tables", R=333, page=16, new_lo=1, new_hi=200, ctx_lo=0,
             ctx_hi=16000, pad=77),
        # the write of a decode step's keys and values, and of a long chunk's
        dict(name="append-decode", op="append", dtype="bf16", H=32, Hkv=8, N=16, d=64, page=16,
             R=64, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=1000, pad=0),
        dict(name="append-chunk", op="append", dtype="bf16", H=64, Hkv=8, N=8, d=128, page=64,
             R=8, new_lo=900, new_hi=1100, ctx_lo=0, ctx_hi=1000, pad=5),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["attention"] * 4 + ["tables", "append"])
    if op == "tables":
        return dict(op=op, R=_log(rng, 1, 400), page=rng.choice([8, 16, 32, 64, 128, 256]), new_lo=1,
                    new_hi=_log(rng, 1, 200), ctx_lo=0, ctx_hi=_log(rng, 1, 16000),
                    pad=rng.choice([0, 0, 1, 50]))
    Hkv, N, G = rng.choice([(8, 16, 4), (8, 8, 8), (4, 1, 8), (2, 2, 4), (8, 1, 1), (1, 1, 5),
                            (3, 3, 6), (2, 1, 16)])
    d = rng.choice([16, 32, 64, 64, 128, 128, 128])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), H=Hkv * G, Hkv=Hkv, N=N,
                d=d, page=rng.choice([8, 16, 32, 64, 128, 256]), pad=rng.choice([0, 0, 3]))
    if op == "append":
        return dict(case, R=_log(rng, 1, 64), new_lo=1, new_hi=_log(rng, 1, 120), ctx_lo=0,
                    ctx_hi=_log(rng, 1, 1000))
    case["causal"] = rng.choice([1, 1, 1, 0])
    kind = rng.choice(["decode", "decode", "drafts", "chunk", "mixed"])
    small = case["dtype"] == "f32"
    if kind == "decode":
        return dict(case, R=_log(rng, 1, 60), new_lo=1, new_hi=1, ctx_lo=0,
                    ctx_hi=_log(rng, 1, 2000 if small else 8000))
    if kind == "drafts":
        return dict(case, R=_log(rng, 1, 33), new_lo=1, new_hi=rng.randint(2, 9), ctx_lo=0,
                    ctx_hi=_log(rng, 1, 1500 if small else 5000))
    if kind == "chunk":
        new = _log(rng, 10, 200 if small else 1500)
        return dict(case, R=rng.randint(1, 3), new_lo=max(1, new // 2), new_hi=new, ctx_lo=0,
                    ctx_hi=_log(rng, 1, 600 if small else 5000))
    return dict(case, R=_log(rng, 2, 48), new_lo=1, new_hi=1, ctx_lo=0,
                ctx_hi=_log(rng, 1, 1500 if small else 6000),
                chunk=_log(rng, 17, 150 if small else 1100))


def _lengths(case):
    """(cached, new) lengths: the same for every seed, so that `work` knows them. The ends
    of the ranges occur; the rest is spread evenly in a shuffled order."""
    R = case["R"]
    rs = np.random.RandomState(1000 * R + case["ctx_hi"] + case["new_hi"])
    ctx = np.linspace(case["ctx_lo"], case["ctx_hi"], R).astype(np.int64) if R > 1 else \
        np.array([case["ctx_hi"]])
    new = np.linspace(case["new_lo"], case["new_hi"], R).astype(np.int64) if R > 1 else \
        np.array([case["new_hi"]])
    rs.shuffle(ctx)
    rs.shuffle(new)
    if case.get("chunk"):
        new[R // 2] = case["chunk"]
    return ctx, new


def _tables(case, seed, spare=3):
    """Host block tables of the requests' pages in a shuffled order: (table, n_pages)."""
    ctx, new = _lengths(case)
    P = case["page"]
    pages = [-(-int(t) // P) for t in ctx + new]
    n = sum(pages) + spare
    perm = np.random.RandomState(seed).permutation(n).astype(np.int32)
    table = np.full((len(pages), max(max(pages), 1)), -1, np.int32)
    at = 0
    for r, k in enumerate(pages):
        table[r, :k] = perm[at:at + k]
        at += k
    return table, n, perm[at:]


def _qkv_cols(case):
    hq = case["H"] // case["N"]
    hkv = max(case["Hkv"] // case["N"], 1)
    return hq, hkv, (hq + 2 * hkv) * case["d"]


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def prepare(case, seed):
    ctx, new = _lengths(case)
    R, P, T = case["R"], case["page"], int(new.sum()) + case["pad"]
    st = dict(case, T=T)
    if case["op"] == "tables":
        table, n_pages, spare = _tables(case, seed)
        have = -(-ctx // P)
        free = np.concatenate([table[r, have[r]:][table[r, have[r]:] >= 0] for r in range(R)] +
                              [spare])
        rs = np.random.RandomState(seed + 1)
        rs.shuffle(free)
        taken = rs.randint(0, 50)  # pages that earlier steps took off the list
        free = np.concatenate([np.arange(taken), free])
        cached = table.copy()
        for r in range(R):
            cached[r, have[r]:] = -1
        st.update(ctx=_i32(ctx), new=_i32(new), free=_i32(free), head=_i32([taken]),
                  table=_i32(cached), max_pages=table.shape[1])
        if own:
            e = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
            st.update(total=e(R), cu=e(R + 1), slots=e(T), pos=e(T), counts=e(4), head_out=e(1))
        return st
    dt = DTYPES[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.float32).to(dt)
    _, _, S = _qkv_cols(case)
    table, n_pages, _ = _tables(case, seed)
    cu = np.concatenate([[0], np.cumsum(new)])
    st.update(qkv=rnd(T, case["N"] * S), n_pages=n_pages, max_pages=table.shape[1],
              kc=rnd(n_pages, case["Hkv"], P, case["d"]), vc=rnd(n_pages, case["Hkv"], P, case["d"]))
    if case["op"] == "append":
        slots = np.full(T, -1, np.int64)
        for r in range(R):
            p = ctx[r] + np.arange(new[r])
            slots[cu[r]:cu[r + 1]] = table[r, p // P].astype(np.int64) * P + p % P
        st.update(slots=_i32(slots))
        return st
    h = case["H"] * case["d"]
    st.update(table=_i32(table), total=_i32(ctx + new), cu=_i32(cu), h=h, max_new=int(new.max()),
              lens=[(int(a), int(b)) for a, b in zip(ctx, new)],
              o=torch.zeros(T, h, dtype=dt, device="cuda"),
              lse=torch.zeros(case["H"], T, dtype=torch.float32, device="cuda"))
    if own:
        from attention_gemms_gb300 import tpmlp as L
        st["dt"] = L.dtype_of(st["qkv"])
        wsb = L.tp_gqa_paged_attention_workspace_size(h, case["H"], case["Hkv"], case["N"], st["dt"])
        st["ws"] = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ the operators

def run(st):
    if st["op"] == "tables":
        return _tables_own(st) if own else _tables_plain(st)
    if st["op"] == "append":
        return _append_own(st) if own else _append_plain(st)
    return _attention_own(st) if own else _attention_plain(st)


def _tables_own(st):
    from attention_gemms_gb300 import tpmlp as L
    L.tp_kv_tables(st["ctx"], st["new"], st["free"], st["free"].numel(), st["head"], st["head_out"],
                   st["table"], st["total"], st["cu"], st["slots"], st["pos"], st["counts"], st["R"],
                   st["T"], st["page"], st["max_pages"])
    return (st["table"], st["total"], st["cu"], st["slots"], st["pos"], st["counts"],
            st["head_out"])


def _tables_plain(st):
    P, MP, T, R = st["page"], st["max_pages"], st["T"], st["R"]
    ctx, new, free, head = st["ctx"].long(), st["new"].long(), st["free"], st["head"].long()
    n_free = free.numel()
    zero = torch.zeros(1, dtype=torch.long, device="cuda")
    total = ctx + new
    cu = torch.cat([zero, torch.cumsum(new, 0)])
    have = ((ctx + P - 1) // P).clamp(max=MP)
    want = ((total + P - 1) // P).clamp(max=MP)
    need = want - have
    base = head + torch.cat([zero, torch.cumsum(need, 0)])
    col = torch.arange(MP, device="cuda")[None, :]
    idx = base[:-1, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < want[:, None])
    page = torch.where(idx < n_free, free[idx.clamp(0, n_free - 1)], -1)
    table = torch.where(fresh, page, st["table"])
    t = torch.arange(T, device="cuda")
    r = torch.searchsorted(cu[1:], t, right=True).clamp(max=R - 1)
    live = t < cu[-1]
    pos = ctx[r] + t - cu[r]
    page = torch.where(pos // P < MP, table[r, (pos // P).clamp(max=MP - 1)], -1).long()
    slots = torch.where(live & (page >= 0), page * P + pos % P, -1)
    taken = torch.minimum(base[-1:], torch.full_like(zero, n_free)) - head
    counts = torch.cat([cu[-1:], taken, base[-1:] - head - taken, (cu[-1:] - T).clamp(min=0)])
    i32 = torch.int32
    return (table, total.to(i32), cu.to(i32), slots.to(i32), torch.where(live, pos, -1).to(i32),
            counts.to(i32), (head + taken).to(i32))


def _append_own(st):
    from attention_gemms_gb300 import tpmlp as L
    L.tp_kv_append(st["qkv"], st["slots"], st["kc"], st["vc"], st["T"], st["H"] * st["d"], st["H"],
                   st["Hkv"], st["N"], st["n_pages"], st["page"], L.dtype_of(st["qkv"]))
    return st["kc"], st["vc"]


def _kv_of(st):
    """The new rows' keys and values (T, Hkv, d) out of the sharded blocks (one replica)."""
    hq, hkv, S = _qkv_cols(st)
    N, Hkv, d = st["N"], st["Hkv"], st["d"]
    blocks = st["qkv"].view(st["T"], N, S // d, d)[:, ::max(N // Hkv, 1)]
    k = blocks[:, :, hq:hq + hkv].reshape(st["T"], Hkv, d)
    v = blocks[:, :, hq + hkv:].reshape(st["T"], Hkv, d)
    return k, v


def _append_plain(st):
    k, v = _kv_of(st)
    slots = st["slots"].long()
    t = torch.nonzero(slots >= 0).squeeze(1)
    page, off = slots[t] // st["page"], slots[t] % st["page"]
    st["kc"][page, :, off] = k[t]
    st["vc"][page, :, off] = v[t]
    return st["kc"], st["vc"]


def _attention_own(st):
    from attention_gemms_gb300 import tpmlp as L
    L.tp_gqa_paged_attention_fwd(st["qkv"], st["kc"], st["vc"], st["table"], st["total"], st["cu"],
                                 st["o"], st["lse"], st["T"], st["R"], st["h"], st["H"], st["Hkv"],
                                 st["N"], st["n_pages"], st["page"], st["max_pages"], st["max_new"],
                                 st["causal"], st["dt"], st["ws"], st["ws"].numel())
    return st["o"], st["lse"]


def _queries(st):
    hq, _, S = _qkv_cols(st)
    q = st["qkv"].view(st["T"], st["N"], S // st["d"], st["d"])[:, :, :hq]
    return q.reshape(st["T"], st["H"], st["d"])


def _attention_plain(st):
    H, Hkv, d, P = st["H"], st["Hkv"], st["d"], st["page"]
    G = H // Hkv
    q_all = _queries(st).float()
    o, lse = torch.zeros_like(st["o"]), torch.zeros_like(st["lse"])
    at = 0
    for r, (c, n) in enumerate(st["lens"]):
        if n == 0:
            continue
        L = c + n
        pages = st["table"][r, :-(-L // P)].long()
        k = st["kc"][pages].transpose(0, 1).reshape(Hkv, 1, -1, d)[:, :, :L].float()
        v = st["vc"][pages].transpose(0, 1).reshape(Hkv, 1, -1, d)[:, :, :L].float()
        q = q_all[at:at + n].view(n, Hkv, G, d).permute(1, 2, 0, 3)
        s = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(d))
        if st["causal"] and n > 1:
            seen = torch.arange(L, device="cuda")[None] <= torch.arange(c, L, device="cuda")[:, None]
            s = s.masked_fill(~seen, -math.inf)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        z = p.sum(-1, keepdim=True)
        out = (p @ v) / z
        o[at:at + n] = out.permute(2, 0, 1, 3).reshape(n, H * d).to(o.dtype)
        lse[:, at:at + n] = (m + torch.log(z)).squeeze(-1).view(H, n)
        at += n
    return o, lse


# ------------------------------------------------------------------ least work and exact values

def work(case):
    ctx, new = _lengths(case)
    R, P, T = case["R"], case["page"], int(new.sum())
    if case["op"] == "tables":
        fresh = int((-(-(ctx + new) // P) + (ctx // -P)).sum())
        return {"bytes": 4 * (2 * R + 2 * fresh + int((ctx % P > 0).sum()) + 2 * R + 2 * T + 8),
                "flops": 0}
    e = 2 if case["dtype"] == "bf16" else 4
    kv = 2 * case["Hkv"] * case["d"] * e
    if case["op"] == "append":
        return {"bytes": 2 * T * kv + 4 * T, "flops": 0}
    # with a causal mask row i sees c + i + 1 keys; K and V of every request are read once
    seen = sum(int(n) * int(c) + (int(n) * (int(n) + 1) // 2 if case["causal"] else int(n) ** 2)
               for c, n in zip(ctx, new))
    toks = int(sum((c + n) for c, n in zip(ctx, new) if n > 0))
    return {"bytes": toks * kv + 2 * T * case["H"] * case["d"] * e + 4 * T * case["H"] +
            4 * (toks // P + 2 * R), "flops": 4 * case["d"] * case["H"] * seen}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "tables":
        return None  # whole numbers
    if case["op"] == "append":
        hq, hkv, S = _qkv_cols(case)
        rep, d, P = max(case["N"] // case["Hkv"], 1), case["d"], case["page"]
        slots = st["slots"].cpu().numpy()
        kc, vc = st["kc"].double(), st["vc"].double()
        t = np.nonzero(slots >= 0)[0]
        page, off = torch.from_numpy(slots[t] // P).long().cuda(), \
            torch.from_numpy(slots[t] % P).long().cuda()
        rows = st["qkv"][torch.from_numpy(t).cuda()].double()
        for j in range(case["Hkv"]):
            col = (j // hkv * rep) * S + (hq + j % hkv) * d
            kc[page, j, off] = rows[:, col:col + d]
            vc[page, j, off] = rows[:, col + hkv * d:col + (hkv + 1) * d]
        return kc, vc
    ctx, new = _lengths(case)
    H, Hkv, d, P, T = case["H"], case["Hkv"], case["d"], case["page"], st["T"]
    hq, _, S = _qkv_cols(case)
    if work(case)["flops"] > 4e12:
        return None
    o = torch.zeros(T, H * d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(H, T, dtype=torch.float64, device="cuda")
    at = 0
    for r in range(case["R"]):
        n, L = int(new[r]), int(ctx[r] + new[r])
        key = torch.arange(L, device="cuda")
        page, off = st["table"][r][key // P].long(), key % P
        limit = torch.arange(L - n, L, device="cuda") if case["causal"] else \
            torch.full((n,), L - 1, device="cuda")
        hidden = key[None, :] > limit[:, None]
        for j in range(Hkv):
            k, v = st["kc"][page, j, off].double(), st["vc"][page, j, off].double()
            for t in range(j * (H // Hkv), (j + 1) * (H // Hkv)):
                col = (t // hq) * S + (t % hq) * d
                q = st["qkv"][at:at + n, col:col + d].double()
                s = torch.matmul(q, k.T).div(d ** 0.5)
                s[hidden] = -math.inf
                z = torch.logsumexp(s, dim=1)
                o[at:at + n, t * d:(t + 1) * d] = torch.exp(s - z[:, None]) @ v
                lse[t, at:at + n] = z
        at += n
    return o, lse
