"""Paged attention where rows, keys or values end or are not finite, against the float64
form (tests/paged_ref.py, which derives the tolerances)."""
import pytest
import torch

from attention_gemms_gb300 import tpmlp as T
from oracle import gqa_oracle as Q
from tests.helpers import BF16_TOL, F32_TOL, host, rel, tensor
from tests.paged_ref import attend, cols, i32
from tests.test_gpu_paged import _block_setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    T.lib()
    torch.cuda.set_device(0)
    T.tp_set_wait_timeout_ns(1_000_000_000)
    yield
    T.tp_set_wait_timeout_ns(0)
    assert T.tp_check_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("P", [8, 16, 256])
@pytest.mark.parametrize("lens,rows,max_new", [
    ([(0, 60)], 30, None), ([(90, 60)], 30, None), ([(90, 60)], 30, 1), ([(90, 100)], 70, None),
    ([(0, 40), (300, 200), (5, 9)], 171, None), ([(700, 3), (0, 2)], 2, None)])
def test_rows_cut_off_at_T(dtype, d, P, lens, rows, max_new):
    """New rows at or past T do not exist: nothing wrote their keys and values, and the rows
    below T do not see them. NaN in those slots must not reach any row."""
    attend(lens, 8, 2, 1, d, P, dtype, 1, seed=d + P, rows=rows, max_new=max_new)


@pytest.mark.parametrize("H,Hkv,N,d,dtype", [(8, 2, 2, 64, "bf16"), (8, 4, 2, 128, "bf16"),
                                             (4, 2, 2, 64, "f32")])
def test_step_with_more_tokens_than_rows(H, Hkv, N, d, dtype):
    """A step that T has no room for, through tables, cache write and block over a cache of
    NaN: tp_kv_tables says how many rows are missing, and the rows that exist equal the dense
    causal block over their tokens."""
    h, P, rows, MP = H * d, 16, 45, 5
    go, g, bo, be, Wsho, Wsh, Woo, Wo, tdt = _block_setup(H, Hkv, N, d, dtype)
    xo, x = tensor((rows, h), 960, dtype=dtype)
    z = lambda *s: torch.full(s, float("nan"), dtype=tdt, device="cuda")
    zi = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    kc, vc = z(MP + 1, Hkv, P, d), z(MP + 1, Hkv, P, d)
    total, cu, slots, counts, head, table = zi(1), zi(2), zi(rows), zi(4), zi(1), zi(1, MP) - 1
    T.tp_kv_tables(i32([0]), i32([70]), i32([3, 1, 5, 0, 2]), 5, head, head, table, total, cu, slots,
                   None, counts, 1, rows, P, MP)
    dt, md = T.dtype_of(x), T.Reduce.SPLITK
    wsb = T.tp_gqa_paged_workspace_size(rows, h, H, Hkv, N, dt, md)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    out = z(rows, h)
    T.tp_gqa_paged_attn_proj_fwd(x, g, be, Wsh, Wo, z(rows, h), None, None, z(rows, cols(H, Hkv, N, d)),
                                 kc, vc, table, total, cu, slots, z(rows, h), None, out, rows, 1, h, H,
                                 Hkv, N, MP + 1, P, MP, 70, 1, dt, md, ws, wsb)
    torch.cuda.synchronize()
    assert counts.cpu().tolist() == [70, 5, 0, 25]
    ref = Q.gqa_block_fwd(xo, 1, rows, go, bo, Wsho, Woo, H, Hkv, N, True)["out"]
    assert rel(host(out), ref) <= (BF16_TOL if dtype == "bf16" else F32_TOL)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("lens", [
    [(700, 1), (3, 1), (130, 1)], [(20000, 1)], [(3000, 5), (40, 3)], [(300, 40), (0, 70), (9, 1)],
    [(100, 700), (0, 400)]])
def test_query_that_is_not_finite(dtype, d, causal, lens):
    """A NaN, or an infinity whose scores are +-inf, in the query of some rows makes o and lse
    of these rows NaN, and no others: lse = -inf says that a row sees no key."""
    H, Hkv, N = 8, 2, 2
    hq, hkv, _ = Q.gqa_split(H, Hkv, N)
    rows = sum(n for _, n in lens)
    n0 = lens[0][1]
    spots = [(0, 0, float("nan")), (n0 - 1, 3, float("inf")), (n0 // 2, 5, float("-inf")),
             (rows - 1, 7, float("nan"))]

    def fill(qkv, kc, vc, pos):
        x = qkv.view(-1, N, hq + 2 * hkv, d)
        for t, h, v in spots:
            x[t, h // hq, h % hq, 5 + h] = v
    _, _, ref = attend(lens, H, Hkv, N, d, 16, dtype, causal, seed=3 + d, pad=1, fill=fill)
    assert ref["lse"].isnan().sum() == len(spots)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("P", [8, 16, 256])
@pytest.mark.parametrize("max_new", [1, 9, 100])
@pytest.mark.parametrize("total", [[7, 3, 100, 2 ** 31 - 1], [0, 0, 30, 0], [9, -5, -(2 ** 31), 60]])
def test_lengths_that_do_not_fit(dtype, d, P, max_new, total):
    """A negative number of new tokens, one that ends at 2^31 - 1, totals that are negative,
    below the new tokens or far past the table: rows and keys are those that exist, and rows
    that no request has stay as they were."""
    cu, T_rows = [40, 2, 2, 40, 2 ** 31 - 1], 60
    attend([(0, 0)] * 4, 8, 2, 1, d, P, dtype, 1, seed=d, rows=T_rows, total=total, cu=cu,
           width=80 // P or 1, max_new=max_new)
