"""GPU parity of the paged key/value cache (tp_kv_tables, tp_kv_append,
tp_gqa_paged_attention_fwd, tp_gqa_paged_attn_proj_fwd) against the fp64 oracle.

Attention tolerances, element by element, from the oracle's A = sum p |v| / sum p and B =
max_k sum |q k| / sqrt(d) of the row, n its keys: u = 2^-24. A score's fp32 sum of d
products is off by at most (d + 4) u B, so p by twice that share (its own and the
normaliser's); sums over n keys add 2 n u, exponentials and the joins of pieces 64 u. In
bf16, P is rounded to 2^-8 of itself, hence 2^-8 A, and the output to 2^-8 |o|; in fp32 the
output's rounding is u |o|.
"""
import numpy as np
import pytest
import torch

from attention_gemms_gb300 import tpmlp as T
from oracle import gqa_oracle as Q
from oracle import paged_oracle as P
from tests.helpers import BF16_TOL, F32_TOL, host, rel, tensor

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    T.lib()
    torch.cuda.set_device(0)
    T.tp_set_wait_timeout_ns(1_000_000_000)
    yield
    T.tp_set_wait_timeout_ns(0)
    assert T.tp_check_status() == 0


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def cols(H, Hkv, N, d):
    hq, hkv, _ = Q.gqa_split(H, Hkv, N)
    return N * (hq + 2 * hkv) * d


# ------------------------------------------------------------------ block tables

@pytest.mark.parametrize("R,hi_ctx,hi_new,P_,pad,short", [
    (1, 0, 1, 16, 0, 0), (1, 5, 300, 8, 0, 0), (7, 100, 1, 16, 2, 0), (64, 900, 40, 32, 0, 0),
    (333, 50, 9, 8, 5, 0), (1025, 300, 3, 64, 0, 0), (8192, 40, 2, 256, 0, 0), (40, 64, 64, 16, 0, 11),
    (33, 200, 200, 8, -500, 0), (5, 0, 0, 16, 4, 0)])
@pytest.mark.parametrize("inplace", [0, 1])
def test_tables(R, hi_ctx, hi_new, P_, pad, short, inplace):
    """Against the loops of the oracle: every output, in place and not; the list running
    out (short), rows beyond T (negative pad), lengths of zero, untouched table entries."""
    rng = np.random.default_rng(R + hi_ctx)
    ctx, new = rng.integers(0, hi_ctx + 1, R), rng.integers(0, hi_new + 1, R)
    need = int((-(-(ctx + new) // P_) - -(-ctx // P_)).sum())
    MP = max(int((-(-(ctx + new) // P_)).max()), 1)
    n_free = max(need + 6 - short, 1)
    free = rng.permutation(n_free + 1000)[:n_free]
    table = np.full((R, MP), -7)
    for r in range(R):
        table[r, :-(-int(ctx[r]) // P_)] = rng.integers(0, 5000, -(-int(ctx[r]) // P_))
    rows = max(int(new.sum()) + pad, 0)
    want = P.kv_tables(ctx, new, free, 3, table, rows, P_)
    c, n, f, h, tb = i32(ctx), i32(new), i32(free), i32([3]), i32(table)
    e = lambda k: torch.full((max(k, 1),), -99, dtype=torch.int32, device="cuda")
    total, ho = (c, h) if inplace else (e(R), e(1))
    cu, slots, pos, counts = e(R + 1), e(rows), e(rows), e(4)
    T.tp_kv_tables(c, n, f, n_free, h, ho, tb, total, cu, slots, pos, counts, R, rows, P_, MP)
    torch.cuda.synchronize()
    g = lambda t: t.cpu().numpy().tolist()
    assert g(total)[:R] == want["total"] and g(cu) == want["cu"]
    assert g(tb) == want["table"].tolist()
    assert g(slots)[:rows] == want["slots"] and g(pos)[:rows] == want["pos"]
    assert g(counts) == want["counts"] and g(ho) == [want["head"]]


def test_tables_narrow_table_and_odd_lengths():
    """More tokens than the table's width, negative lengths, a missing old page, a list
    position outside the list; without positions and counts; no requests at all."""
    ctx, new = [30, -4, 9, 0], [20, 5, -1, 7]
    table = np.array([[3, 9], [-1, -1], [-1, 4], [-1, -1]])
    want = P.kv_tables(ctx, new, [11, 12], 0, table, 32, 16)
    tb, total, cu, slots, ho = i32(table), i32([0] * 4), i32([0] * 5), i32([0] * 32), i32([0])
    T.tp_kv_tables(i32(ctx), i32(new), i32([11, 12]), 2, i32([-3]), ho, tb, total, cu, slots, None,
                   None, 4, 32, 16, 2)
    torch.cuda.synchronize()
    assert tb.cpu().tolist() == want["table"].tolist() and slots.cpu().tolist() == want["slots"]
    assert total.cpu().tolist() == want["total"] and ho.item() == want["head"]
    cu, slots = i32([5]), i32([5, 5, 5])
    T.tp_kv_tables(i32([0]), i32([0]), None, 0, i32([9]), ho, tb, total, cu, slots, None, None, 0, 3,
                   16, 2)
    torch.cuda.synchronize()
    assert cu.item() == 0 and slots.cpu().tolist() == [-1] * 3 and ho.item() == 0


# ------------------------------------------------------------------ the cache's write

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv,N,d,P_", [(8, 2, 2, 64, 16), (8, 2, 4, 32, 8), (6, 3, 1, 16, 32),
                                          (4, 4, 1, 128, 64), (5, 1, 5, 128, 256)])
@pytest.mark.parametrize("rows", [1, 7, 130])
def test_append(dtype, H, Hkv, N, d, P_, rows):
    """Bit for bit; skipped slots (negative, past the cache) and the other slots as before."""
    rng = np.random.default_rng(rows)
    n_pages = -(-rows // P_) + 2
    slots = rng.permutation(n_pages * P_)[:rows]
    if rows > 3:
        slots[1], slots[2] = -1, n_pages * P_
    qo, qkv = tensor((rows, cols(H, Hkv, N, d)), 700 + rows, dtype=dtype)
    ko, kc = tensor((n_pages, Hkv, P_, d), 701, dtype=dtype)
    vo, vc = tensor((n_pages, Hkv, P_, d), 702, dtype=dtype)
    _, k, v = P.qkv_heads(qo, H, Hkv, N)
    wk, wv = P.kv_append(k, v, slots, ko, vo)
    dt = T.DType.BF16 if dtype == "bf16" else T.DType.F32
    T.tp_kv_append(qkv, i32(slots), kc, vc, rows, H * d, H, Hkv, N, n_pages, P_, dt)
    torch.cuda.synchronize()
    assert np.array_equal(host(kc), wk) and np.array_equal(host(vc), wv)


# ------------------------------------------------------------------ attention

def run_attention(lens, H, Hkv, N, d, P_, dtype, causal, seed=1, pad=0, total=None, rows=None,
                  max_new=None, edit=None, spare=2):
    """Random cache with scattered pages, unused slots NaN; checks every element."""
    rng = np.random.default_rng(seed)
    R = len(lens)
    tot = np.array([c + n for c, n in lens]) if total is None else np.array(total)
    new = np.array([n for _, n in lens])
    cu = np.concatenate([[0], np.cumsum(new)])
    rows = int(cu[-1]) + pad if rows is None else rows
    pages = [-(-int(t) // P_) for t in tot]
    n_pages = sum(pages) + spare
    perm = rng.permutation(n_pages)
    table = np.full((R, max(pages + [1])), -1)
    at = 0
    for r, k in enumerate(pages):
        table[r, :k] = perm[at:at + k]
        at += k
    qo, qkv = tensor((rows, cols(H, Hkv, N, d)), 800 + seed, dtype=dtype)
    ko, kc = tensor((n_pages, Hkv, P_, d), 801 + seed, dtype=dtype)
    vo, vc = tensor((n_pages, Hkv, P_, d), 802 + seed, dtype=dtype)
    if edit:
        edit(table)
    used = np.zeros((n_pages, P_), bool)
    for r in range(R):
        for k in range(min(int(tot[r]), table.shape[1] * P_)):
            if 0 <= table[r, k // P_] < n_pages:
                used[table[r, k // P_], k % P_] = True
    dead = torch.from_numpy(~used).cuda()[:, None, :, None].expand_as(kc)
    kc[dead], vc[dead] = float("nan"), float("nan")
    ko, vo = np.nan_to_num(host(kc)), np.nan_to_num(host(vc))
    q, _, _ = P.qkv_heads(qo, H, Hkv, N)
    ref = P.paged_attention(q, ko, vo, table, tot, cu, bool(causal))
    dt = T.DType.BF16 if dtype == "bf16" else T.DType.F32
    o = torch.full((rows, H * d), -768.0, dtype=qkv.dtype, device="cuda")
    lse = torch.full((H, rows), -768.0, device="cuda")
    h = H * d
    wsb = T.tp_gqa_paged_attention_workspace_size(h, H, Hkv, N, dt)
    ws = torch.full((wsb,), 255, dtype=torch.uint8, device="cuda")  # NaN: must not be read
    T.tp_gqa_paged_attention_fwd(qkv, kc, vc, i32(table), i32(tot), i32(cu), o, lse, rows, R, h, H,
                                 Hkv, N, n_pages, P_, table.shape[1],
                                 int(new.max()) if max_new is None else max_new, causal, dt, ws, wsb)
    torch.cuda.synchronize()
    assert T.tp_check_status() == 0
    got, gl = host(o).reshape(rows, H, d), host(lse)
    w = ref["written"]
    assert (got[~w] == -768.0).all() and (gl[:, ~w] == -768.0).all()
    Bt, nt = ref["B"].T[:, :, None], ref["n"].T[:, :, None]
    sums = U * (2 * (d + 4) * Bt + 2 * nt + 64)
    tol = ref["A"] * sums + np.abs(ref["o"]) * U
    if dtype == "bf16":
        tol = ref["A"] * (sums + 2.0 ** -8) + np.abs(ref["o"]) * 2.0 ** -8
    bad = np.abs(got - ref["o"])[w] > tol[w]
    assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - ref["o"])[w].max())
    assert np.isfinite(got[w]).all()
    rl = ref["lse"][:, w]
    assert (np.isneginf(gl[:, w]) == np.isneginf(rl)).all()
    fin = np.isfinite(rl)
    ltol = U * ((d + 4) * ref["B"] + ref["n"] + 64)[:, w] + 4 * U * np.abs(np.where(fin, rl, 0))
    assert (np.abs(np.where(fin, gl[:, w] - np.where(fin, rl, 0), 0)) <= ltol).all()
    return o, lse


HEADS = [(8, 2, 2), (8, 2, 4), (4, 4, 1), (5, 1, 1), (40, 2, 1), (12, 4, 2)]
DECODE = [(0, 1), (700, 1), (63, 1), (64, 1), (15, 1), (16, 1), (1, 1), (129, 1)]


@pytest.mark.parametrize("H,Hkv,N", HEADS)
@pytest.mark.parametrize("d,P_", [(64, 16), (128, 64), (32, 8), (16, 256), (128, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode(H, Hkv, N, d, P_, dtype):
    run_attention(DECODE, H, Hkv, N, d, P_, dtype, 1, seed=d + P_, pad=2)


CHUNKS = [(0, 70), (33, 1), (130, 129), (5, 0), (0, 3), (257, 40)]


@pytest.mark.parametrize("H,Hkv,N", [(8, 2, 2), (5, 1, 1), (40, 2, 1), (3, 3, 1)])
@pytest.mark.parametrize("d,P_", [(64, 16), (128, 32), (32, 16), (16, 8), (128, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [0, 1])
def test_chunks(H, Hkv, N, d, P_, dtype, causal):
    """Chunks beside decoding requests, a request without new tokens, padding rows."""
    run_attention(CHUNKS, H, Hkv, N, d, P_, dtype, causal, seed=d + P_ + causal, pad=3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("max_new", [0, 1, 9, 5000, 1 << 62])
def test_max_new_is_a_hint(dtype, d, max_new):
    run_attention([(20, 9), (300, 1), (0, 40)], 8, 2, 1, d, 16, dtype, 1, seed=5, max_new=max_new)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("new", [1, 60])
def test_rows_without_keys_and_bad_pages(dtype, d, causal, new):
    """total_lens below the number of new tokens (rows before the cache's start), a length
    of zero, page ids outside the cache at the front, in the middle and everywhere, a table
    narrower than the length, rows beyond T."""
    def edit(tab):
        tab[2, 0] = -1
        tab[3, 2] = 1 << 30
        tab[4, :] = -5
    lens = [(0, new)] * 6
    total = [max(new - 1, 0), 0, 100, 200, 90, 150]
    kw = dict(total=total, edit=edit, rows=6 * new - new // 2)
    run_attention(lens, 8, 2, 1, d, 16, dtype, causal, seed=6, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R", [1, 257, 700])
def test_many_requests(dtype, R):
    lens = [((7 * r) % 90, 1 + (r % 3 == 0)) for r in range(R)]
    run_attention(lens, 4, 2, 1, 64, 16, dtype, 1, seed=R)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 32)])
@pytest.mark.parametrize("lens", [[(40000, 1)], [(9000, 33), (3, 1)]])
def test_long_context(dtype, d, lens):
    run_attention(lens, 4, 1, 1, d, 128, dtype, 1, seed=9)


@pytest.mark.parametrize("d,new", [(128, 1), (128, 40), (64, 1)])
def test_cache_past_32_bits(d, new):
    """A cache of more than 2^32 elements: pages at its far end."""
    H, Hkv, P_ = 8, 4, 64
    n_pages = (2 ** 32 + 2 ** 26) // (Hkv * P_ * d)
    kc = torch.empty(n_pages, Hkv, P_, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    assert kc.numel() > 2 ** 32
    table = np.array([[n_pages - 1, 0, n_pages - 3]])
    L, BF = 150, T.DType.BF16
    ko, ks = tensor((3, Hkv, P_, d), 41)
    vo, vs = tensor((3, Hkv, P_, d), 42)
    for i, pg in enumerate(table[0]):
        kc[pg], vc[pg] = ks[i], vs[i]
    qo, qkv = tensor((new, cols(H, Hkv, 1, d)), 43)
    o = torch.empty(new, H * d, dtype=torch.bfloat16, device="cuda")
    wsb = T.tp_gqa_paged_attention_workspace_size(H * d, H, Hkv, 1, BF)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    # the new rows' own keys and values are written at the far end first
    pos = np.arange(L - new, L)
    slots = table[0][pos // P_] * P_ + pos % P_
    T.tp_kv_append(qkv, i32(slots), kc, vc, new, H * d, H, Hkv, 1, n_pages, P_, BF)
    T.tp_gqa_paged_attention_fwd(qkv, kc, vc, i32(table), i32([L]), i32([0, new]), o, None, new, 1,
                                 H * d, H, Hkv, 1, n_pages, P_, 3, new, 1, BF, ws, wsb)
    torch.cuda.synchronize()
    q, k, v = P.qkv_heads(qo, H, Hkv, 1)
    small = np.array([[0, 1, 2]])
    ko, vo = P.kv_append(k, v, pos, ko, vo)
    ref = P.paged_attention(q, ko, vo, small, [L], [0, new], True)
    tol = ref["A"] * (2.0 ** -8 + U * (2 * (d + 4) * ref["B"].T[:, :, None] + 2 * L + 64)) + \
        np.abs(ref["o"]) * 2.0 ** -8
    assert (np.abs(host(o).reshape(new, H, d) - ref["o"]) <= tol).all()
    del kc, vc
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores(dtype):
    """Scores of +-1000 and a running maximum that grows from tile to tile."""
    H, Hkv, d, P_, L = 2, 1, 64, 16, 300
    _, qkv = tensor((1, cols(H, Hkv, 1, d)), 50, dtype=dtype)
    _, kc = tensor((19, Hkv, P_, d), 51, dtype=dtype)
    _, vc = tensor((19, Hkv, P_, d), 52, dtype=dtype)
    qkv[:] = 4.0
    kc[:] = (torch.arange(19, device="cuda") * 2.0 - 20)[:, None, None, None].to(kc.dtype)
    dt = T.dtype_of(qkv)
    o = torch.empty(1, H * d, dtype=qkv.dtype, device="cuda")
    lse = torch.empty(H, 1, device="cuda")
    wsb = T.tp_gqa_paged_attention_workspace_size(H * d, H, Hkv, 1, dt)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    table = np.arange(19)[None]
    T.tp_gqa_paged_attention_fwd(qkv, kc, vc, i32(table), i32([L]), i32([0, 1]), o, lse, 1, 1, H * d,
                                 H, Hkv, 1, 19, P_, 19, 1, 1, dt, ws, wsb)
    torch.cuda.synchronize()
    q, _, _ = P.qkv_heads(host(qkv), H, Hkv, 1)
    ref = P.paged_attention(q, host(kc), host(vc), table, [L], [0, 1], True)
    # every product and sum of the scores is a whole number below 2^24: exact; the last
    # page's 12 keys tie and the others' weights vanish (2^-90)
    r = 2.0 ** -8 if dtype == "bf16" else U * 64
    assert (np.abs(host(o).reshape(1, H, d) - ref["o"]) <= r * (ref["A"] + np.abs(ref["o"]))).all()
    assert np.abs(host(lse) - ref["lse"]).max() <= 4 * U * np.abs(ref["lse"]).max()


# ------------------------------------------------------------------ together

def _block_setup(H, Hkv, N, d, dtype, seed=900):
    h = H * d
    sig = 1.0 / np.sqrt(h)
    go, g = tensor((h,), seed + 1, 0.2, dtype="f32")
    g += 1.0
    bo, be = tensor((h,), seed + 2, 0.2, dtype="f32")
    Wq, Wk, Wv = (tensor((h, w * d), seed + 3 + i, sig, dtype=dtype)[0]
                  for i, w in enumerate((H, Hkv, Hkv)))
    Wsh = Q.gqa_pack(Wq, Wk, Wv, H, Hkv, N)
    Woo, Wo = tensor((h, h), seed + 6, sig, dtype=dtype)
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    return go + 1.0, g, bo, be, Wsh, torch.from_numpy(Wsh).cuda().to(tdt), Woo, Wo, tdt


@pytest.mark.parametrize("H,Hkv,N,d,dtype,mode", [
    (8, 2, 4, 64, "bf16", 0), (8, 4, 2, 128, "bf16", 1), (8, 2, 2, 32, "bf16", 0),
    (6, 3, 3, 16, "f32", 0), (4, 2, 2, 64, "f32", 1)])
@pytest.mark.parametrize("graph", [0, 1])
def test_serving_run(H, Hkv, N, d, dtype, mode, graph):
    """Three requests served step by step (prompt chunks of several lengths, then decoding,
    one of them starting late) through tables, cache write and block, eagerly or each
    step replayed from one captured graph of a fixed number of rows: every row equals the
    dense causal block over its whole sequence."""
    h, P_, R, rows, MP = H * d, 16, 3, 100, 16
    go, g, bo, be, Wsho, Wsh, Woo, Wo, tdt = _block_setup(H, Hkv, N, d, dtype)
    dt = T.DType.BF16 if dtype == "bf16" else T.DType.F32
    steps = [(60, 0, 33), (61, 0, 1), (1, 40, 1), (1, 1, 1), (1, 1, 1), (7, 1, 0), (1, 5, 1)]
    length = [sum(s[r] for s in steps) for r in range(R)]
    xs = [tensor((length[r], h), 950 + r, dtype=dtype) for r in range(R)]
    W = cols(H, Hkv, N, d)
    n_pages = 40
    z = lambda *s, t=tdt: torch.zeros(s, dtype=t, device="cuda")
    zi = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    kc, vc = z(n_pages, Hkv, P_, d), z(n_pages, Hkv, P_, d)
    x, xn, qkv, o, out = z(rows, h), z(rows, h), z(rows, W), z(rows, h), z(rows, h)
    mean, rstd = z(rows, t=torch.float32), z(rows, t=torch.float32)
    ctx, new, head, table, cu = zi(R), zi(R), zi(1), zi(R, MP) - 1, zi(R + 1)
    slots, pos, counts = zi(rows), zi(rows), zi(4)
    free = i32(np.random.default_rng(2).permutation(n_pages))
    md = T.Reduce.SPLITK if mode else T.Reduce.BUFFERS
    wsb = T.tp_gqa_paged_workspace_size(rows, h, H, Hkv, N, dt, md)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")

    def step():
        T.tp_kv_tables(ctx, new, free, n_pages, head, head, table, ctx, cu, slots, pos, counts, R,
                       rows, P_, MP)
        T.tp_gqa_paged_attn_proj_fwd(x, g, be, Wsh, Wo, xn, mean, rstd, qkv, kc, vc, table, ctx, cu,
                                     slots, o, None, out, rows, R, h, H, Hkv, N, n_pages, P_, MP,
                                     61, 1, dt, md, ws, wsb)

    cg = None
    if graph:
        step()                               # a step without new tokens, outside the capture
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            step()
    done = [0] * R
    got = [[] for _ in range(R)]
    for st in steps:
        new.copy_(i32(st))
        at = 0
        for r, n in enumerate(st):
            x[at:at + n] = xs[r][1][done[r]:done[r] + n]
            at += n
        cg.replay() if cg else step()
        torch.cuda.synchronize()
        assert counts.cpu().tolist()[::2] == [sum(st), 0]
        at = 0
        for r, n in enumerate(st):
            got[r].append(out[at:at + n].clone())
            assert pos[at:at + n].cpu().tolist() == list(range(done[r], done[r] + n))
            at += n
            done[r] += n
    assert T.tp_check_status() == 0
    assert ctx.cpu().tolist() == length
    for r in range(R):
        ref = Q.gqa_block_fwd(xs[r][0], 1, length[r], go, bo, Wsho, Woo, H, Hkv, N, True)["out"]
        assert rel(host(torch.cat(got[r])), ref) <= (BF16_TOL if dtype == "bf16" else F32_TOL)


@pytest.mark.parametrize("dtype,new", [("bf16", 1), ("bf16", 90), ("f32", 1), ("f32", 50)])
def test_streams_graphs_and_repeats(dtype, new):
    """Two calls at once on two streams with a workspace each, repeats, and a graph replay
    after another graph has used the same workspace: all bit for bit alike."""
    H, Hkv, N, d, P_ = 8, 2, 2, 64, 16
    h, dt = H * d, (T.DType.BF16 if dtype == "bf16" else T.DType.F32)
    lens = [(500, new), (30, 1), (1200, new)]
    tot, cu = [c + n for c, n in lens], np.concatenate([[0], np.cumsum([n for _, n in lens])])
    MP = -(-max(tot) // P_)
    table = np.arange(3 * MP).reshape(3, MP)[:, ::-1]
    rows = int(cu[-1])
    _, qkv = tensor((rows, cols(H, Hkv, N, d)), 60, dtype=dtype)
    _, kc = tensor((3 * MP, Hkv, P_, d), 61, dtype=dtype)
    _, vc = tensor((3 * MP, Hkv, P_, d), 62, dtype=dtype)
    tb, tt, cc = i32(table), i32(tot), i32(cu)
    wsb = T.tp_gqa_paged_attention_workspace_size(h, H, Hkv, N, dt)
    mk = lambda: (torch.zeros(rows, h, dtype=qkv.dtype, device="cuda"),
                  torch.empty(wsb, dtype=torch.uint8, device="cuda"))

    def call(o, ws, causal=1, stream=None):
        T.tp_gqa_paged_attention_fwd(qkv, kc, vc, tb, tt, cc, o, None, rows, 3, h, H, Hkv, N, 3 * MP,
                                     P_, MP, new, causal, dt, ws, wsb, stream)
    ref, ws0 = mk()
    call(ref, ws0)
    full, _ = mk()
    call(full, ws0, causal=0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [mk() for _ in streams]
    for _ in range(5):
        for s, (o, ws) in zip(streams, outs):
            call(o, ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o, _ in outs)
    o1, o2 = mk()[0], mk()[0]
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        call(o1, ws0)
    with torch.cuda.graph(g2):
        call(o2, ws0, causal=0)
    for g in (g2, g1, g2, g1):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o1, ref) and torch.equal(o2, full)


@pytest.mark.parametrize("d,new,mx", [(64, 1, 1), (128, 1, 1), (64, 40, 40), (128, 40, 40)])
def test_expired_waits_are_reported_and_recovered_from(d, new, mx):
    """The injected wait runs out (a barrier that nothing arrives on): the call stops, the
    status says so, and the next call on the same buffers is right."""
    lens = [(300, new), (5, 1)]
    T.tp_set_wait_timeout_ns(20_000_000)
    T.tp_debug_inject_wait_fault(True)
    try:
        H, Hkv, P_ = 8, 2, 16
        rows, MP = new + 1, -(-(300 + new) // P_)
        _, qkv = tensor((rows, cols(H, Hkv, 1, d)), 70)
        _, kc = tensor((2 * MP, Hkv, P_, d), 71)
        o = torch.zeros(rows, H * d, dtype=torch.bfloat16, device="cuda")
        wsb = T.tp_gqa_paged_attention_workspace_size(H * d, H, Hkv, 1, T.DType.BF16)
        ws = torch.zeros(wsb, dtype=torch.uint8, device="cuda")
        T.tp_gqa_paged_attention_fwd(qkv, kc, kc, i32(np.arange(2 * MP).reshape(2, MP)),
                                     i32([300 + new, 6]), i32([0, new, rows]), o, None, rows, 2,
                                     H * d, H, Hkv, 1, 2 * MP, P_, MP, mx, 1, T.DType.BF16, ws, wsb)
        assert T.tp_check_status() == T.Status.TIMEOUT
    finally:
        T.tp_debug_inject_wait_fault(False)
        T.tp_set_wait_timeout_ns(1_000_000_000)
    assert T.tp_check_status() == 0
    run_attention(lens, 8, 2, 1, d, 16, "bf16", 1, seed=12)


@pytest.mark.parametrize("H,Hkv,N", [(128, 1, 1), (130, 1, 1), (256, 2, 4), (100, 1, 100), (7, 7, 7)])
@pytest.mark.parametrize("new", [1, 3])
def test_wide_and_narrow_groups(H, Hkv, N, new):
    """Query heads per key/value head from 1 to 130: a row tile's whole tokens, more than one
    tile's heads, replicas across all shards."""
    run_attention([(37, new), (0, 2)], H, Hkv, N, 64, 16, "bf16", 1, seed=H)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 64)])
def test_chunked_equals_whole(dtype, d):
    """A prompt in one call and in pieces (the kernel for few rows among them) agree to the
    rounding of P and the output."""
    H, Hkv, P_, L = 8, 2, 16, 333
    h, dt = H * d, (T.DType.BF16 if dtype == "bf16" else T.DType.F32)
    MP = -(-L // P_)
    _, qkv = tensor((L, cols(H, Hkv, 1, d)), 80, dtype=dtype)
    z = lambda *s: torch.zeros(s, dtype=qkv.dtype, device="cuda")
    kc, vc = z(MP, Hkv, P_, d), z(MP, Hkv, P_, d)
    tb = i32(np.random.default_rng(1).permutation(MP)[None])
    wsb = T.tp_gqa_paged_attention_workspace_size(h, H, Hkv, 1, dt)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    pos = np.arange(L)
    slots = tb.cpu().numpy()[0][pos // P_] * P_ + pos % P_
    T.tp_kv_append(qkv, i32(slots), kc, vc, L, h, H, Hkv, 1, MP, P_, dt)
    outs = []
    for cuts in ([0, L], [0, 1, 2, 5, 130, 131, 300, L]):
        o = z(L, h)
        for a, b in zip(cuts[:-1], cuts[1:]):
            T.tp_gqa_paged_attention_fwd(qkv[a:], kc, vc, tb, i32([b]), i32([0, b - a]), o[a:], None,
                                         b - a, 1, h, H, Hkv, 1, MP, P_, MP, b - a, 1, dt, ws, wsb)
        outs.append(host(o))
    torch.cuda.synchronize()
    q, k, v = P.qkv_heads(host(qkv), H, Hkv, 1)
    ref = P.paged_attention(q, host(kc), host(vc), tb.cpu().numpy(), [L], [0, L], True)
    tol = 2.0 ** -8 if dtype == "bf16" else U * 2 * L
    lim = 2 * tol * (ref["A"] + np.abs(ref["o"])) + \
        2 * ref["A"] * U * (2 * (d + 4) * ref["B"].T[:, :, None] + 2 * L + 64)
    assert (np.abs(outs[0] - outs[1]).reshape(L, H, d) <= lim).all()
