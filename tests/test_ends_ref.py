"""The float64 torch forms of the training step's ends against the oracle's definitions, plain
loops and finite differences (CPU)."""
import numpy as np
import torch

from oracle import gpt_oracle as G
from tests import ends_ref as R


def _case(M=6, v=12, h=5, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, h, generator=g, dtype=torch.float64)
    E = torch.randn(v, h, generator=g, dtype=torch.float64)
    t = torch.randint(0, v, (M,), generator=g, dtype=torch.int32)
    return x, E, t


def test_ce_is_the_oracles_on_logits():
    x, E, t = _case()
    t[2] = -1
    t[4] = 12
    loss, lse, rows, shards = R.ce_fwd(x, E, t, 3)
    o = G.vocab_ce_fwd((x @ E.T).numpy(), t.numpy(), 3)
    for a, b in zip((loss.item(), lse.numpy(), rows.numpy(), shards.numpy()), o):
        np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-12)
    assert rows[2] == 0 and rows[4] == 0
    live = torch.tensor([0, 1, 3, 5])
    _, q = R.ce_grad_logits(x, E, t, lse, 0.5)
    want = G.vocab_ce_bwd((x @ E.T).numpy(), t.numpy(), lse.numpy(), 3, 0.5)
    np.testing.assert_allclose(q[live].numpy(), want[live], atol=1e-13)
    assert torch.all(q[2] == 0) and torch.all(q[4] == 0)


def test_ce_gradients_by_differences():
    x, E, t = _case()
    t[3] = -7
    lse = R.ce_fwd(x, E, t, 1)[1]
    dx, dE = R.ce_bwd(x, E, t, lse, 1.0 / 6)
    for z, dz in ((x, dx), (E, dE)):
        for i in range(z.numel()):
            old = z.view(-1)[i].item()
            f = []
            for s in (1e-6, -1e-6):
                z.view(-1)[i] = old + s
                f.append(R.ce_fwd(x, E, t, 1)[0].item())
            z.view(-1)[i] = old
            assert abs((f[0] - f[1]) / 2e-6 - dz.view(-1)[i].item()) < 1e-8


def test_embedding_is_the_oracles_times_the_factor():
    _, E, t = _case(M=9)
    t[1] = t[0]
    dx = torch.randn(9, 5, dtype=torch.float64)
    np.testing.assert_allclose(R.embed_fwd(t, E, 3.0).numpy(), 3 * G.vocab_embed_fwd(t.numpy(), E.numpy(), 2))
    want = G.vocab_embed_bwd(t.numpy(), dx.numpy(), 12, 2)
    g, a, n = R.embed_bwd(t, dx, 12, 3.0)
    np.testing.assert_allclose(g.numpy(), 3 * want, atol=1e-12)
    assert int(n.sum()) == 9 and torch.all(a >= 0)
    old = torch.randn(12, 5, dtype=torch.float64)
    g2 = R.embed_bwd(t, dx, 12, 3.0, old)[0]
    np.testing.assert_allclose(g2.numpy(), old.numpy() + 3 * want, atol=1e-12)
    # the lookup's transpose: <y, S(E)> = <S^T(y), E>
    assert abs((dx * R.embed_fwd(t, E, 3.0)).sum() - (g * E).sum()) < 1e-10


def test_bounds_cover_fp32_and_bf16_arithmetic():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(40, 64, generator=g).to(torch.bfloat16)
    E = (torch.randn(300, 64, generator=g) * 0.1).to(torch.bfloat16)
    t = torch.randint(0, 300, (40,), generator=g, dtype=torch.int32)
    logits = x.float() @ E.float().T
    lse = torch.logsumexp(logits, 1)
    ref = R.ce_fwd(x, E, t, 4)
    b = R.ce_fwd_bounds(x, E, t, 4)
    assert torch.all((lse - ref[1]).abs() <= b[0]) and float(b[0].max()) < 1e-3
    q = torch.exp(logits - lse[:, None])
    q[torch.arange(40), t.long()] -= 1.0
    q = (q * (1 / 40)).to(torch.bfloat16).float()
    dx, dE = R.ce_bwd(x, E, t, lse, 1 / 40)
    bx, bE = R.ce_bwd_bounds(x, E, t, lse, 1 / 40)
    assert torch.all(((q @ E.float()).to(torch.bfloat16).double() - dx).abs() <= bx)
    assert torch.all(((q.T @ x.float()).to(torch.bfloat16).double() - dE).abs() <= bE)
    # and notice a wrong value: a target's share left out
    assert not torch.all((dE + 0.02 * x.double()[0] - dE).abs() <= bE)
