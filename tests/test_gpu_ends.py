"""The output layer's cross-entropy without logits, and the scaled embedding with its gradient by
sorted tokens, against float64 (tests/ends_ref.py), element by element within counted roundings."""
import pytest
import torch

from attention_gemms_gb300 import tpmlp as T
from tests import ends_ref as R
from tests.helpers import gemm_tiles

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DT = {BF: T.DType.BF16, F32: T.DType.F32}
SENT = -768.0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *s, sigma=1.0, dt=BF):
    return (torch.randn(s, generator=g, device="cuda") * sigma).to(dt)


def tokens(g, M, v, kind="mixed"):
    u = torch.rand(M, generator=g, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * torch.log(torch.tensor(v + 1.0, device="cuda"))) - 1).long().clamp(0, v - 1)
    if kind == "uniform":
        ids = (u * v).long().clamp(0, v - 1)
    if kind == "same":
        ids = torch.full_like(ids, v // 2)
    if kind == "sorted":
        ids = torch.sort(ids).values
    if kind == "none":
        ids = torch.where(u < 0.5, -1, v)
    if kind == "mixed" and M >= 4:  # the ends of the vocabulary, and what lies outside it
        ids[0], ids[1] = v - 1, 0
        ids[2], ids[3] = -1, v
        if M >= 8:
            ids[4], ids[5] = -2 ** 31, 2 ** 31 - 1
    return ids.to(torch.int32)


def guarded(n, dt=F32, extra=64):
    return torch.full((n + extra,), SENT, dtype=dt, device="cuda")


def poison(n):
    return torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")


def run_fwd(x, E, t, N, stream=None, ws=None):
    M, h = x.shape
    v = E.shape[0]
    d = DT[x.dtype]
    n = T.tp_vocab_linear_ce_workspace_size(1, M, v, h, N, d)
    ws = poison(n) if ws is None else ws
    out = [guarded(k) for k in (M, M, N, 1)]
    T.tp_vocab_linear_ce_fwd(x, E, t, *out, M, v, h, N, d, ws, n, stream)
    torch.cuda.synchronize()
    assert T.tp_check_status() == 0
    assert torch.all(ws[n:] == 255)
    for o, k in zip(out, (M, M, N, 1)):
        assert torch.all(o[k:] == SENT)
    lse, rows, shards, loss = (o[:k] for o, k in zip(out, (M, M, N, 1)))
    return loss, lse, rows, shards


def run_bwd(x, E, t, lse, scale, N=1, want=(True, True), ws=None):
    M, h = x.shape
    v = E.shape[0]
    d = DT[x.dtype]
    n = T.tp_vocab_linear_ce_workspace_size(0, M, v, h, N, d)
    ws = poison(n) if ws is None else ws
    dx = guarded(M * h, x.dtype) if want[0] else None
    dE = guarded(v * h, x.dtype) if want[1] else None
    T.tp_vocab_linear_ce_bwd(x, E, t, lse, dx, dE, M, v, h, N, scale, d, ws, n)
    torch.cuda.synchronize()
    assert T.tp_check_status() == 0
    assert torch.all(ws[n:] == 255)
    for o, k in ((dx, M * h), (dE, v * h)):
        assert o is None or torch.all(o[k:] == SENT)
    return (dx[:M * h].view(M, h) if want[0] else None, dE[:v * h].view(v, h) if want[1] else None)


def within(got, ref, bound, what=""):
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)  # NaN counts
    if bad.any():
        i = int(torch.nonzero(bad.view(-1))[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: got "
                             f"{got.reshape(-1)[i].item()} want {ref.reshape(-1)[i].item()} within "
                             f"{bound.expand_as(ref).reshape(-1)[i].item():.3g}")


def ce_case(M, v, h, dt, seed=1, kind="mixed", sigma=0.1):
    g = gen(seed)
    x, E = rnd(g, M, h, dt=dt), rnd(g, v, h, sigma=sigma, dt=dt)
    return x, E, tokens(g, M, v, kind)


def check_ce(x, E, t, N, scale=None, want=(True, True)):
    scale = 1.0 / x.shape[0] if scale is None else scale
    got = run_fwd(x, E, t, N)
    ref, b = R.ce_fwd(x, E, t, N), R.ce_fwd_bounds(x, E, t, N)
    for g_, r_, b_, n_ in zip(got, ref, (b[3], b[0], b[1], b[2]), ("loss", "lse", "rows", "shards")):
        within(g_, r_, b_, n_)
    lse = got[1].clone()
    dx, dE = run_bwd(x, E, t, lse, scale, N, want)
    rx, rE = R.ce_bwd(x, E, t, lse, scale)
    bx, bE = R.ce_bwd_bounds(x, E, t, lse, scale)
    if want[0]:
        within(dx, rx, bx, "dx")
    if want[1]:
        within(dE, rE, bE, "dE")
    return got, dx, dE


CE = [(1, 1, 8, 1), (1, 7, 8, 7), (1, 2000, 64, 8), (2, 256, 16, 1), (3, 65, 24, 5), (4, 300, 72, 3),
      (5, 4097, 128, 1), (37, 1000, 136, 8), (63, 129, 64, 3), (64, 5000, 200, 4), (65, 2048, 128, 2),
      (127, 31, 1032, 1), (128, 256, 128, 2), (129, 257, 264, 1), (255, 640, 64, 16),
      (256, 511, 72, 7), (257, 3001, 512, 1), (300, 12345, 64, 3), (1000, 4099, 1032, 1),
      (2049, 8192, 256, 16), (1300, 20000, 128, 5), (400, 500, 6144, 1), (2500, 2000, 304, 1),
      (1000, 4000, 1024, 1), (10000, 50, 64, 1), (300, 1500, 256, 1), (130, 990, 64, 33),
      (5000, 1280, 64, 40)]


@pytest.mark.parametrize("M,v,h,N", CE)
def test_linear_ce_bf16(M, v, h, N):
    check_ce(*ce_case(M, v, h, BF, seed=M + v), N)


@pytest.mark.parametrize("M,v,h,N", [(1, 1, 1, 1), (1, 3, 2, 3), (3, 64, 5, 2), (64, 65, 33, 5),
                                     (65, 257, 128, 1), (128, 256, 128, 2), (130, 1000, 77, 8),
                                     (300, 4097, 64, 17), (700, 3000, 129, 3), (1025, 128, 300, 16),
                                     (90, 770, 40, 35)])
def test_linear_ce_fp32(M, v, h, N):
    check_ce(*ce_case(M, v, h, F32, seed=M + v), N)


@pytest.mark.parametrize("pair,wide", [(0, 0), (2, 0), (2, 2), (1, 0)])
@pytest.mark.parametrize("M,v,h", [(300, 777, 136), (513, 2304, 320), (1500, 9000, 72)])
def test_linear_ce_every_tile_form(M, v, h, pair, wide):
    with gemm_tiles(pair, wide):
        check_ce(*ce_case(M, v, h, BF, seed=7), 1)


@pytest.mark.parametrize("kind", ["none", "same", "uniform"])
@pytest.mark.parametrize("dt", [BF, F32])
def test_linear_ce_targets(kind, dt):
    x, E, t = ce_case(200, 300, 64, dt, kind=kind)
    got, dx, dE = check_ce(x, E, t, 3)
    if kind == "none":
        assert got[0].item() == 0 and torch.all(got[2] == 0) and torch.all(dx == 0) and torch.all(dE == 0)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("sigma", [0.0, 1e-4, 3.0])
def test_linear_ce_flat_and_peaked(dt, sigma):
    """Equal logits (lse = log v), and logits of some hundreds."""
    check_ce(*ce_case(150, 1000, 256, dt, sigma=sigma), 2)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("scale", [0.0, -2.5, 1024.0])
def test_linear_ce_scale(dt, scale):
    check_ce(*ce_case(90, 500, 64, dt), 1, scale=scale)


@pytest.mark.parametrize("dt", [BF, F32])
def test_linear_ce_one_gradient_only(dt):
    x, E, t = ce_case(300, 700, 128, dt)
    _, dx, dE = check_ce(x, E, t, 1)
    a, _ = check_ce(x, E, t, 1, want=(True, False))[1:]
    _, b = check_ce(x, E, t, 1, want=(False, True))[1:]
    assert torch.equal(a, dx) and torch.equal(b, dE)


def test_linear_ce_several_pieces():
    """More of q than a piece holds: the pieces' shares of dx are added up, by one-CTA and by pair
    tiles, in one part and in two."""
    for M, v, h, N in ((8192, 50304, 64, 8), (70000, 4111, 72, 1), (33000, 8300, 512, 1),
                       (8192, 33000, 4096, 1)):
        assert M * v * 2 > 512 << 20
        x, E, t = ce_case(M, v, h, BF)
        lse = run_fwd(x, E, t, N)[1].clone()
        dx, dE = run_bwd(x, E, t, lse, 1.0 / M, N)
        # the bounds of some rows and columns (the whole would take 3 GB matrices)
        r = torch.arange(0, M, 61, device="cuda")
        rx, bx = R.ce_bwd(x[r], E, t[r], lse[r], 1.0 / M)[0], R.ce_bwd_bounds(x[r], E, t[r], lse[r], 1.0 / M)[0]
        within(dx[r], rx, bx, "dx")
        p = torch.exp(x.double() @ E.double().T - lse.double()[:, None])
        own = R.has_target(t, v)
        i = torch.nonzero(own).squeeze(1)
        p[i, t[i].long()] -= 1
        p *= own[:, None] / M
        rE = p.T @ x.double()
        aE = p.abs().T @ x.double().abs()
        # relative to the absolute products: q's rounding and its error of p (logits within 1, lse
        # below 16: some 1e-5), the sums, the result's rounding
        within(dE, rE, aE * (2.0 ** -8 + 2e-5 + (M + 64) * 2.0 ** -23) + rE.abs() * 2.0 ** -8 * 1.01, "dE")
        del p, rE, aE


def test_linear_ce_pieces_fp32():
    x, E, t = ce_case(40000, 4000, 8, F32)
    assert 40000 * 4000 * 4 > 512 << 20
    check_ce(x, E, t, 2)


@pytest.mark.parametrize("dt", [BF, F32])
def test_linear_ce_repeats_bit_for_bit(dt):
    x, E, t = ce_case(777, 3000, 136, dt)
    a, ax, aE = check_ce(x, E, t, 6)
    for _ in range(3):
        b = run_fwd(x, E, t, 6)
        bx, bE = run_bwd(x, E, t, b[1].clone(), 1.0 / 777)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        assert torch.equal(ax, bx) and torch.equal(aE, bE)


def test_linear_ce_values_that_are_not_finite():
    """A row's NaN or infinity stays in its own loss."""
    x, E, t = ce_case(200, 600, 64, BF, kind="uniform")
    clean = run_fwd(x, E, t, 1)
    x[7, 3] = float("nan")
    x[150, 0] = float("inf")
    got = run_fwd(x, E, t, 1)
    bad = torch.tensor([7, 150], device="cuda")
    assert torch.isnan(got[1][7]) and torch.isnan(got[2][7])
    assert not torch.isfinite(got[1][150])
    keep = torch.ones(200, dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert torch.equal(got[1][keep], clean[1][keep]) and torch.equal(got[2][keep], clean[2][keep])


def test_linear_ce_agrees_with_the_kernels_on_logits():
    """tp_gemm + tp_vocab_ce_fwd on the same fp32 inputs."""
    x, E, t = ce_case(256, 1000, 128, F32, kind="uniform")
    M, v, h = 256, 1000, 128
    logits, lse, rows = (torch.empty(s, device="cuda") for s in ((M, v), (M,), (M,)))
    shards, loss = torch.empty(2, device="cuda"), torch.empty(1, device="cuda")
    T.tp_gemm(x, E, logits, M, v, h, 0, 1, T.DType.F32)
    T.tp_vocab_ce_fwd(logits, t, lse, rows, shards, loss, M, v, 2, T.DType.F32)
    got = run_fwd(x, E, t, 2)
    b = R.ce_fwd_bounds(x, E, t, 2)
    for g_, r_, b_ in zip(got, (loss, lse, rows, shards), (b[3], b[0], b[1], b[2])):
        within(g_, r_.double(), 2 * b_)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M", [1, 100, 1300, 5000])
def test_linear_ce_vocabulary_of_one_entry(M, dt):
    """The softmax is 1 and every loss 0, not a rounding of it."""
    x, E, t = ce_case(M, 1, 72, dt, kind="uniform", sigma=2.0)
    (loss, lse, rows, shards), _, _ = check_ce(x, E, t, 1)
    assert torch.all(rows == 0) and loss == 0 and shards == 0


def test_linear_ce_empty_batch():
    E = rnd(gen(0), 50, 64)
    dE = guarded(50 * 64, BF)
    z = torch.empty(0, 64, dtype=BF, device="cuda")
    one = torch.empty(16, device="cuda")
    T.tp_vocab_linear_ce_bwd(one, E, one, one, None, dE, 0, 50, 64, 1, 1.0, T.DType.BF16, None, 0)
    torch.cuda.synchronize()
    assert torch.all(dE[:3200] == 0) and torch.all(dE[3200:] == SENT) and z.numel() == 0


# ------------------------------------------------------------------ embedding

EMB = [(1, 1, 1), (1, 5, 8), (2, 3, 7), (5, 1000, 64), (33, 40, 72), (128, 256, 128), (1000, 50, 24),
       (3000, 50304, 136), (5000, 4000, 33), (20000, 7, 520), (500, 300001, 8), (70000, 30000, 16),
       (700, 900, 5000), (300, 200, 4101), (9000, 12000, 1024)]


def run_embed_bwd(ids, dx, v, scale, dE0=None):
    M, h = dx.shape
    d = DT[dx.dtype]
    n = T.tp_vocab_embed_scaled_workspace_size(M, v, h, d)
    ws = poison(n)
    dE = guarded(v * h, dx.dtype)
    if dE0 is not None:
        dE[:v * h] = dE0.reshape(-1)
    T.tp_vocab_embed_scaled_bwd(ids, dx, dE, M, v, h, 1, scale, dE0 is not None, d, ws, n)
    torch.cuda.synchronize()
    assert torch.all(ws[n:] == 255) and torch.all(dE[v * h:] == SENT)
    return dE[:v * h].view(v, h)


def check_embed_bwd(ids, dx, v, scale, dE0=None):
    got = run_embed_bwd(ids, dx, v, scale, dE0)
    g, a, n = R.embed_bwd(ids, dx, v, scale, dE0)
    within(got, g, R.embed_bwd_bound(g, a, n, scale, dx.dtype), "dE")
    empty = n == 0
    if dE0 is None:
        assert torch.all(got[empty] == 0)
    else:
        assert torch.equal(got[empty].view(torch.uint8), dE0[empty].view(torch.uint8))
    assert torch.equal(got, run_embed_bwd(ids, dx, v, scale, dE0))  # the same bits again
    return got


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,v,h", EMB)
def test_embed_scaled_fwd(M, v, h, dt):
    g = gen(M)
    ids, E = tokens(g, M, v), rnd(g, v, h, dt=dt)
    for scale in (1.0, 11.3125, -0.37):
        x = guarded(M * h, dt)
        T.tp_vocab_embed_scaled_fwd(ids, E, x, M, v, h, 1, scale, DT[dt])
        torch.cuda.synchronize()
        assert torch.all(x[M * h:] == SENT)
        ref = R.embed_fwd(ids, E, torch.tensor(scale, dtype=F32).double().item())
        within(x[:M * h].view(M, h), ref, ref.abs() * (R.HALF[dt] * 1.01 + 2.0 ** -24))
    same = guarded(M * h, dt)
    T.tp_vocab_embed_fwd(ids, E, same, M, v, h, 1, DT[dt])
    T.tp_vocab_embed_scaled_fwd(ids, E, x, M, v, h, 1, 1.0, DT[dt])
    assert torch.equal(x, same)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,v,h", EMB)
def test_embed_scaled_bwd(M, v, h, dt):
    g = gen(M + 1)
    ids, dx = tokens(g, M, v), rnd(g, M, h, dt=dt)
    check_embed_bwd(ids, dx, v, 2.5)
    check_embed_bwd(ids, dx, v, 0.75, rnd(g, v, h, dt=dt))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("kind", ["same", "none", "sorted", "uniform"])
@pytest.mark.parametrize("M,v,h", [(16, 9, 8), (17, 9, 64), (4096, 33, 256), (40001, 5000, 40)])
def test_embed_scaled_bwd_orders(M, v, h, kind, dt):
    g = gen(5)
    ids, dx = tokens(g, M, v, kind), rnd(g, M, h, dt=dt)
    check_embed_bwd(ids, dx, v, 1.5)
    dE0 = rnd(g, v, h, dt=dt)
    dE0[0] = -0.0  # a row without a token keeps its bits, which -0.0 + 0.0 would not
    check_embed_bwd(torch.where(ids == 0, 1, ids).to(torch.int32), dx, v, 1.5, dE0)


def test_embed_scaled_bwd_rows_of_every_count():
    """1, 2, ..., 60 tokens of a row, in a shuffled order: rows that units share and rows they do not."""
    g = gen(9)
    ids = torch.repeat_interleave(torch.arange(60, device="cuda"), torch.arange(1, 61, device="cuda"))
    ids = ids[torch.randperm(ids.numel(), generator=g, device="cuda")].to(torch.int32)
    for h in (8, 130, 2048):
        for dt in (BF, F32):
            check_embed_bwd(ids, rnd(g, ids.numel(), h, dt=dt), 60, 1.0)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("h", [64, 1032, 5])
@pytest.mark.parametrize("counts", [(260, 3836), (257, 3839), (263, 30, 3803), (516, 9, 3571), (256, 3840),
                                    (100, 420, 300, 3276), (260, 512, 512, 2812)])
def test_embed_scaled_bwd_row_ends_where_the_next_begins(counts, h, dt):
    """4096 tokens are cut into 512 units of 8. A row of more than 32 units ends in a unit that is a
    multiple of 32, and the next row begins in it and is split as well: each counts its own."""
    assert sum(counts) == 4096
    ids = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), torch.tensor(counts, device="cuda"))
    g = gen(sum(counts[:1]) + h)
    ids = ids[torch.randperm(4096, generator=g, device="cuda")].to(torch.int32)
    check_embed_bwd(ids, rnd(g, 4096, h, dt=dt), len(counts), 1.5)
    check_embed_bwd(ids, rnd(g, 4096, h, dt=dt), len(counts), 1.5, rnd(g, len(counts), h, dt=dt))


@pytest.mark.parametrize("seed", range(12))
def test_embed_scaled_bwd_lists_of_every_shape(seed):
    g = gen(seed)
    M = 3000 + 5000 * seed
    v = (3, 7, 40, 700)[seed % 4]
    u = torch.rand(M, generator=g, device="cuda")
    ids = (u ** (2 + seed % 3) * v).long().clamp(max=v - 1).to(torch.int32)
    check_embed_bwd(ids, rnd(g, M, 24), v, 0.75)


def test_embed_scaled_bwd_without_tokens():
    for M in (0, 5):
        ids = torch.full((max(M, 1),), -1, dtype=torch.int32, device="cuda")
        dx = torch.ones(max(M, 1), 72, dtype=BF, device="cuda")
        n = T.tp_vocab_embed_scaled_workspace_size(M, 100, 72, T.DType.BF16)
        ws, dE = poison(n), guarded(7200, BF)
        T.tp_vocab_embed_scaled_bwd(ids, dx, dE, M, 100, 72, 4, 2.0, 1, T.DType.BF16, ws, n)
        torch.cuda.synchronize()
        assert torch.all(dE == SENT)
        T.tp_vocab_embed_scaled_bwd(ids, dx, dE, M, 100, 72, 4, 2.0, 0, T.DType.BF16, ws, n)
        torch.cuda.synchronize()
        assert torch.all(dE[:7200] == 0) and torch.all(dE[7200:] == SENT)


def test_embed_scaled_bwd_agrees_with_the_scan():
    g = gen(11)
    ids, dx = tokens(g, 900, 500), rnd(g, 900, 96, dt=F32)
    want = torch.empty(500, 96, device="cuda")
    T.tp_vocab_embed_bwd(ids, dx, want, 900, 500, 96, 4, 0, T.DType.F32)
    g_, a, n = R.embed_bwd(ids, dx, 500, 1.0)
    within(run_embed_bwd(ids, dx, 500, 1.0), want.double(), 2 * R.embed_bwd_bound(g_, a, n, 1.0, F32))


@pytest.mark.parametrize("M,v,h", [(1, 70_000, 264), (15, 65_601, 256), (16, 2049, 8200), (17, 131_080, 136),
                                   (33, 50_257, 520), (63, 16_385, 1032), (64, 2_100_001, 8), (64, 16_384, 1024),
                                   (65, 16_385, 1032), (64, 16_383, 1024)])
def test_linear_ce_few_rows_of_a_large_gradient(M, v, h):
    """dE of up to 64 rows and from 2^24 elements has a kernel of its own; the sizes on both sides."""
    x, E, t = ce_case(M, v, h, BF, seed=M)
    _, dx, dE = check_ce(x, E, t, 1)
    _, only_x, _ = check_ce(x, E, t, 1, want=(True, False))
    _, _, only_E = check_ce(x, E, t, 1, want=(False, True))
    assert torch.equal(only_x, dx) and torch.equal(only_E, dE)


@pytest.mark.parametrize("M,v,h,dt", [(200_000, 1000, 64, BF), (5, 1_000_003, 64, BF), (70, 600_001, 24, BF),
                                      (100_000, 130, 8, F32), (3, 400_000, 5, F32)])
def test_linear_ce_long(M, v, h, dt):
    check_ce(*ce_case(M, v, h, dt, seed=21), 1)


@pytest.mark.parametrize("M,v,h,kind", [(2_200_000, 300, 8, "mixed"), (2_200_000, 40_000, 2, "same"),
                                        (300, 2_000_000, 16, "mixed"), (900_000, 151_000, 3, "uniform"),
                                        (131_072, 128 * 1152, 64, "mixed")])
def test_embed_scaled_bwd_long(M, v, h, kind):
    """More tokens of a warp than 16 bits number, more rows than 128 CTAs count."""
    g = gen(31)
    ids, dx = tokens(g, M, v, kind), rnd(g, M, h)
    check_embed_bwd(ids, dx, v, 1.25)
    check_embed_bwd(ids, dx, v, 1.25, rnd(g, v, h))
