"""The paged kernels where a block has many key tiles and several segments: rings that refill,
row tiles that share their rows, maxima that move from half to half, and writes of more
vectors than one pass of the grid. Against the float64 form (tests/paged_ref.py, which derives
the tolerances); NaN in every slot that no row sees."""
import math

import pytest
import torch

from attention_gemms_gb300 import tpmlp as T
from oracle import gqa_oracle as Q
from tests.paged_ref import attend, cols, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    T.lib()
    torch.cuda.set_device(0)
    T.tp_set_wait_timeout_ns(1_000_000_000)
    yield
    T.tp_set_wait_timeout_ns(0)
    assert T.tp_check_status() == 0
    torch.cuda.empty_cache()


def spread(R, ctx_lo, ctx_hi, new_lo, new_hi):
    """R (cached, new) pairs over both ranges, their ends among them, in a mixed order."""
    f = lambda i, k, lo, hi: lo + (hi - lo) * ((i * k) % R) // max(R - 1, 1)
    return [(f(i, 7, ctx_lo, ctx_hi), f(i, 5, new_lo, new_hi)) for i in range(R)]


# One row tile per unit (bf16, d = 128, 17 to 128 rows per request and key/value head): 6 to 36
# key tiles per block and up to a dozen segments; one request's pieces joined four groups at a
# time, the others' by one
@pytest.mark.parametrize("lens,H,Hkv,N,P", [
    (spread(33, 100, 5000, 2, 7), 32, 8, 8, 16), (spread(16, 1000, 6000, 20, 64), 8, 4, 1, 8),
    ([(80000, 8)], 8, 2, 2, 256), ([(100001, 30)], 4, 2, 1, 64), (spread(8, 1, 9000, 5, 25), 20, 4, 4, 32)])
@pytest.mark.parametrize("causal", [0, 1])
def test_one_row_tile(lens, H, Hkv, N, P, causal):
    attend(lens, H, Hkv, N, 128, P, "bf16", causal, seed=P, pad=3)


# Two row tiles, beside requests and chunk ends whose rows both tiles share
MIXED = [(6000, 700), (2500, 1), (0, 900), (4001, 3), (77, 130), (0, 0), (5000, 31), (3333, 2)]


@pytest.mark.parametrize("lens,H,Hkv,N,P", [
    (MIXED, 16, 4, 2, 32), (MIXED, 10, 2, 1, 8), ([(9000, 2500)], 8, 1, 1, 256),
    ([(0, 3000), (1, 2049)], 4, 4, 4, 16)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [0, 1])
def test_chunks(lens, H, Hkv, N, P, d, causal):
    attend(lens, H, Hkv, N, d, P, "bf16", causal, seed=P + d, pad=1)


@pytest.mark.parametrize("lens,H,Hkv,N,P", [
    (spread(64, 0, 8000, 1, 1), 32, 8, 8, 64), ([(131071, 1), (90001, 1)], 8, 4, 1, 128),
    (spread(40, 10, 4000, 1, 4), 6, 2, 1, 8), ([(50000, 3)], 40, 2, 2, 16)])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
def test_few_rows(lens, H, Hkv, N, P, d):
    attend(lens, H, Hkv, N, d, P, "bf16", 1, seed=P + d, max_new=1)


@pytest.mark.parametrize("lens,H,Hkv,N,P", [
    (spread(40, 0, 3000, 1, 3), 8, 4, 4, 16), ([(20000, 1)], 8, 2, 1, 256),
    ([(3000, 300), (0, 900), (1000, 1)], 8, 2, 2, 32), ([(500, 1000), (7, 700)], 5, 1, 1, 8)])
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("causal", [0, 1])
def test_f32(lens, H, Hkv, N, P, d, causal):
    attend(lens, H, Hkv, N, d, P, "f32", causal, seed=P + d, pad=2)


@pytest.mark.parametrize("dtype,d,new", [
    ("bf16", 16, 1), ("bf16", 64, 1), ("bf16", 128, 1), ("bf16", 128, 20), ("bf16", 64, 20),
    ("bf16", 64, 70), ("bf16", 128, 70), ("f32", 64, 1), ("f32", 64, 20), ("f32", 128, 70)])
@pytest.mark.parametrize("R,Hkv", [(24, 8), (2, 1)])
def test_growing_maxima(dtype, d, new, R, Hkv):
    """Scores that grow by 12 (base 2, more than the 8 that move a row's maximum) every 64 keys,
    in odd halves of the key tiles for some rows, in even ones for others, in all or in none
    (falling) for the rest; values shrink alike, so that earlier keys still count: a lost or
    repeated factor on the sum or the output, or one applied to another half, is far off."""
    H, N = 4 * Hkv, 1
    hq, hkv, _ = Q.gqa_split(H, Hkv, N)
    c = 12.0 * math.sqrt(d) / (16.0 * math.log2(math.e))

    def fill(qkv, kc, vc, pos):
        half = (pos.clamp(min=0) // 64)[:, None, :]
        kc[..., 0] = (16 * ((half + 1) // 2)).to(kc.dtype)   # grows in odd halves
        kc[..., 1] = (16 * (half // 2)).to(kc.dtype)         # in even ones
        vc.mul_(torch.exp2(60.0 - 6.0 * half)[..., None].to(vc.dtype))
        x = qkv.view(-1, N, hq + 2 * hkv, d)
        t = torch.arange(x.shape[0], device="cuda")[:, None]
        kind = (t + torch.arange(hq, device="cuda")[None]) % 4
        x[:, 0, :hq, 0] = torch.where(kind == 3, -c, torch.where(kind == 1, 0.0, c)).to(x.dtype)
        x[:, 0, :hq, 1] = torch.where(kind == 3, -c, torch.where(kind == 0, 0.0, c)).to(x.dtype)
    lens = [(1150 - 37 * (r % 5), new) for r in range(R)]
    attend(lens, H, Hkv, N, d, 16, dtype, 1, seed=d + new, fill=fill)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_of_many_rows(dtype):
    """More vectors than two per thread of the grid, an odd number of rows, skipped slots; bit
    for bit."""
    rows, H, Hkv, N, d, P, n_pages = 3001, 16, 8, 4, 128, 32, 101
    qkv = torch.randn(rows, cols(H, Hkv, N, d), device="cuda").to(dtype)
    kc, vc = (torch.randn(n_pages, Hkv, P, d, device="cuda").to(dtype) for _ in range(2))
    slots = torch.randperm(n_pages * P, device="cuda")[:rows]
    slots[5::97] = -1
    slots[7::101] = n_pages * P
    wk, wv = kc.clone(), vc.clone()
    hq, hkv, _ = Q.gqa_split(H, Hkv, N)
    x = qkv.view(rows, N, hq + 2 * hkv, d)
    ok = (slots >= 0) & (slots < n_pages * P)
    page, off = slots[ok] // P, slots[ok] % P
    wk[page, :, off] = x[:, :, hq:hq + hkv].reshape(rows, Hkv, d)[ok]
    wv[page, :, off] = x[:, :, hq + hkv:].reshape(rows, Hkv, d)[ok]
    T.tp_kv_append(qkv, slots.int(), kc, vc, rows, H * d, H, Hkv, N, n_pages, P, T.dtype_of(qkv))
    torch.cuda.synchronize()
    assert torch.equal(kc, wk) and torch.equal(vc, wv)


def test_append_past_31_bits():
    """2^31 vectors of 16 bytes and more, of which a few rows have slots: the last ones, and
    those on both sides of 2^31 elements and of 2^31 vectors."""
    H = Hkv = 8
    d, P, n_pages = 128, 16, 2
    per_row = 2 * Hkv * d * 4 // 16
    rows = 2 ** 31 // per_row + 3
    W = cols(H, Hkv, 1, d)
    qkv = torch.empty(rows, W, device="cuda")
    kc = torch.zeros(n_pages, Hkv, P, d, device="cuda")
    vc = torch.zeros_like(kc)
    slots = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    at = [0, 2 ** 31 // W - 1, 2 ** 31 // W, 2 ** 31 // W + 1, 2 ** 31 // per_row - 1,
          2 ** 31 // per_row, rows - 1]
    x = torch.randn(len(at), W, device="cuda")
    for i, t in enumerate(at):
        qkv[t] = x[i]
        slots[t] = 3 * i
    T.tp_kv_append(qkv, slots, kc, vc, rows, H * d, H, Hkv, 1, n_pages, P, T.DType.F32)
    torch.cuda.synchronize()
    k, v = x.view(len(at), 3, Hkv, d)[:, 1], x.view(len(at), 3, Hkv, d)[:, 2]
    for i in range(len(at)):
        s = 3 * i
        assert torch.equal(kc[s // P, :, s % P], k[i]) and torch.equal(vc[s // P, :, s % P], v[i])
    assert kc.count_nonzero() == k.count_nonzero() and vc.count_nonzero() == v.count_nonzero()


@pytest.mark.parametrize("d,new", [(64, 1), (128, 1), (128, 20), (64, 70), (128, 70)])
def test_expired_waits_with_full_rings(d, new):
    """The injected wait (a barrier that nothing arrives on) runs out while every block has a
    ring of loads and several segments ahead: the call ends, the status says so, and the next
    call is right."""
    lens, H, Hkv, P = spread(24, 800, 3000, new, new), 32, 8, 16
    tot = [c + n for c, n in lens]
    MP, rows = -(-max(tot) // P), 24 * new
    qkv = torch.randn(rows, cols(H, Hkv, 1, d), device="cuda").bfloat16()
    kc = torch.randn(24 * MP, Hkv, P, d, device="cuda").bfloat16()
    table = torch.arange(24 * MP, device="cuda", dtype=torch.int32)
    cu = torch.arange(25, device="cuda", dtype=torch.int32) * new
    o = torch.zeros(rows, H * d, dtype=torch.bfloat16, device="cuda")
    wsb = T.tp_gqa_paged_attention_workspace_size(H * d, H, Hkv, 1, T.DType.BF16)
    ws = torch.zeros(wsb, dtype=torch.uint8, device="cuda")
    total = i32(tot)
    T.tp_set_wait_timeout_ns(20_000_000)
    T.tp_debug_inject_wait_fault(True)
    try:
        T.tp_gqa_paged_attention_fwd(qkv, kc, kc, table, total, cu, o, None, rows, 24, H * d, H, Hkv,
                                     1, 24 * MP, P, MP, new, 1, T.DType.BF16, ws, wsb)
        assert T.tp_check_status() == T.Status.TIMEOUT
    finally:
        T.tp_debug_inject_wait_fault(False)
        T.tp_set_wait_timeout_ns(1_000_000_000)
    assert T.tp_check_status() == 0
    attend(lens[:9], H, Hkv, 1, d, P, "bf16", 1, seed=d)
