"""The cross-entropy of stored logits at its edges: targets outside the vocabulary, small losses."""
import pytest
import torch

from attention_gemms_gb300 import tpmlp as T
from tests.test_gpu_ends import BF, DT, F32, gen, guarded, rnd, within

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M,v,N", [(1, 8, 1), (100, 1000, 5), (300, 256, 4), (33, 77, 7)])
@pytest.mark.parametrize("in_place", [False, True])
def test_ce_bwd_of_a_target_outside_the_vocabulary_is_a_row_of_zeros(M, v, N, dt, in_place):
    g = gen(v)
    L = rnd(g, M, v, sigma=2.0, dt=dt)
    t = torch.randint(0, v, (M,), generator=g, device="cuda").to(torch.int32)
    for i, bad in zip(range(0, M, 3), (-1, v, 2 ** 31 - 1, -2 ** 31) * M):
        t[i] = bad
    out = t < 0
    out |= t >= v
    L[out, 0] = float("inf")  # whatever such a row holds
    lse = torch.logsumexp(L.double(), 1).float()
    d = L.clone() if in_place else guarded(M * v, dt)
    keep = L.clone()
    T.tp_vocab_ce_bwd(d if in_place else L, t, lse, d, M, v, N, 1.0 / M, DT[dt])
    torch.cuda.synchronize()
    got = d.reshape(-1)[:M * v].view(M, v)
    assert torch.all(got[out] == 0)
    p = torch.exp(keep.double() - lse.double()[:, None])
    i = torch.nonzero(~out).squeeze(1)
    p[i, t[i].long()] -= 1.0
    half = 2.0 ** -8 if dt == BF else U
    # p's exponent: lse in base 2 and the multiply-add round 2^-23 of up to 16 log2(e), the power 2^-22
    tol = (p.abs() * 1.01 * half + (1.0 + p.abs()) * 2.0 ** -18) / M
    within(got[~out], (p / M)[~out], tol[~out], "dlogits")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("v,N", [(64, 4), (1000, 5), (77, 7)])
def test_ce_fwd_has_no_loss_below_zero(v, N, dt):
    """A target that is above the other logits by 20 to 30: vectorised rows and the others."""
    g = gen(v)
    M = 4000
    a = (torch.rand(M, generator=g, device="cuda") * 200.0 - 100.0).to(BF)
    L = (a.float()[:, None] - 20.0 - 10.0 * torch.rand(M, v, generator=g, device="cuda")).to(dt)
    t = torch.randint(0, v, (M,), generator=g, device="cuda").to(torch.int32)
    L[torch.arange(M, device="cuda"), t.long()] = a.to(dt)
    e = lambda n: torch.empty(n, device="cuda")
    lse, rows, shards, loss = e(M), e(M), e(N), e(1)
    T.tp_vocab_ce_fwd(L, t, lse, rows, shards, loss, M, v, N, DT[dt])
    torch.cuda.synchronize()
    assert torch.all(rows >= 0), f"{int((rows < 0).sum())} of {M}, {rows.min().item():.3g}"
    assert torch.all(shards >= 0) and loss.item() >= 0
    L[5, 0] = float("nan")
    T.tp_vocab_ce_fwd(L, t, lse, rows, shards, loss, M, v, N, DT[dt])
    torch.cuda.synchronize()
    assert torch.isnan(rows[5]) and torch.isnan(loss)
