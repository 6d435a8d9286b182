"""Values at the edges of the cross-entropy without logits: rows whose target has all of the
probability, logits of any finite size."""
import pytest
import torch

from tests import ends_ref as R
from tests.helpers import gemm_tiles
from tests.test_gpu_ends import BF, F32, gen, rnd, run_bwd, run_fwd, within

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # an fp32 rounding, of a number up to 1


def two_levels(M, v, h, dt, seed, top=100.0, gap=(8.0, 25.0)):
    """Logits without a rounding: a_r for the row's entry `at`, a_r - b_r for every other one. Two
    features: x_r = (a_r, b_r, 0 ...), E_c = (1, -[c != at], 0 ...); the other features are zero."""
    g = gen(seed)
    u = lambda: torch.rand(M, generator=g, device="cuda")
    a = ((2.0 * u() - 1.0) * top).to(BF).to(dt)
    b = (gap[0] + u() * (gap[1] - gap[0])).to(BF).to(dt)
    x, E = torch.zeros(M, h, dtype=dt, device="cuda"), torch.zeros(v, h, dtype=dt, device="cuda")
    x[:, 0], x[:, 1] = a, b
    at = v // 2
    E[:, 0], E[:, 1] = 1.0, -1.0
    E[at, 1] = 0.0
    return x, E, torch.full((M,), at, dtype=torch.int32, device="cuda"), a.double(), b.double()


def check_two_levels(M, v, h, N, dt, **kw):
    x, E, t, a, b = two_levels(M, v, h, dt, seed=M + v, **kw)
    t[3::7] = -1
    loss, lse, rows, shards = run_fwd(x, E, t, N)
    small = torch.log1p((v - 1) * torch.exp(-b))
    own = t >= 0
    # s = 1 + (v - 1) exp(-b), the largest logit's power 1 exactly. The others': a - b, its difference
    # to a and that times log2(e) round 2^-20, 2^-20 and 2^-19 log(2) at the most (b <= 25), the power
    # 2^-22: 2^-18 relative. s rounds in a column's 16 terms, 16 chunks, a thread's slots and ten joins,
    # 2^-24 of it each; the logarithm twice. a - at is 0.
    adds = 16 + 16 + 16 + -(-(-(-v // 64)) // 8) + 10
    err = adds * U + (2.0 ** -18 + 2 * U) * small
    assert torch.all(rows >= 0), f"{int((rows < 0).sum())} of {M} losses below 0, {rows.min().item():.3g}"
    within(rows, torch.where(own, small, torch.zeros_like(small)), err, "row_loss")
    # lse = a + that logarithm, rounded once
    within(lse, a + small, err + (a + small).abs() * U, "lse")
    assert loss.item() >= 0 and torch.all(shards >= 0)
    return x, E, t, lse


FORMS = [(1, 2, 8, 1), (37, 2, 8, 1), (64, 1000, 64, 1), (37, 50257, 136, 1), (100, 300, 64, 3), (600, 9000, 320, 1),
         (1000, 65, 8, 5), (2000, 40000, 64, 8), (512, 25600, 2048, 1), (5000, 130, 128, 1), (400, 70, 16, 35),
         (20000, 3, 8, 3)]


@pytest.mark.parametrize("M,v,h,N", FORMS)
def test_loss_of_a_target_with_all_of_the_probability_bf16(M, v, h, N):
    check_two_levels(M, v, h, N, BF)


@pytest.mark.parametrize("M,v,h,N", [(1, 2, 2, 1), (37, 65, 8, 1), (128, 256, 128, 2), (300, 5000, 40, 1),
                                     (2048, 1280, 16, 5), (3000, 3000, 33, 40), (64, 7, 700, 1)])
def test_loss_of_a_target_with_all_of_the_probability_fp32(M, v, h, N):
    check_two_levels(M, v, h, N, F32)


@pytest.mark.parametrize("pair,wide", [(0, 0), (2, 0), (2, 2)])
@pytest.mark.parametrize("h", [64, 1088])
def test_loss_of_a_target_with_all_of_the_probability_in_every_tile_form(pair, wide, h):
    with gemm_tiles(pair, wide):
        check_two_levels(700, 1100, h, 1, BF)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("v", [1, 2, 700])
def test_lse_does_not_depend_on_the_target(v, dt):
    g = gen(v)
    x, E = rnd(g, 300, 64, dt=dt), rnd(g, v, 64, sigma=0.5, dt=dt)
    t = torch.randint(0, v, (300,), generator=g, device="cuda").to(torch.int32)
    some = run_fwd(x, E, t, 1)[1]
    none = run_fwd(x, E, torch.full_like(t, -1), 1)[1]
    assert torch.equal(some, none)


@pytest.mark.parametrize("M,v", [(40, 300), (200, 700), (700, 2200), (2048, 1280)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_logits_of_any_finite_size(M, v, dt):
    """Logits of 1e5 to 1e37, one of a row above the others by two thousandths of that at the least: p
    is 1 there, and 0 elsewhere."""
    for top in (1.0e5, 1.0e10, 1.0e37):
        x, E, t, a, b = two_levels(M, v, 64, dt, seed=3, top=top, gap=(top * 0.002, top * 0.01))
        loss, lse, rows, _ = run_fwd(x, E, t, 1)
        assert torch.all(rows == 0) and loss.item() == 0
        assert torch.equal(lse.double(), a)
        # another target: its loss is the distance
        rows = run_fwd(x, E, torch.zeros_like(t), 1)[2]
        assert torch.equal(rows.double(), b)


@pytest.mark.parametrize("M,v", [(40, 300), (200, 700), (700, 2200), (2048, 1280)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_gradients_of_logits_of_any_finite_size(M, v, dt):
    for top in (1.0e5, 1.0e10, 1.0e37):
        x, E, t, a, _ = two_levels(M, v, 64, dt, seed=3, top=top, gap=(top * 0.002, top * 0.01))
        dx, dE = run_bwd(x, E, t, a.float(), 0.5)
        assert torch.all(dx == 0) and torch.all(dE == 0)
        # another target: q is the scale at the largest logit, its negative at the target
        dx, _ = run_bwd(x, E, torch.zeros_like(t), a.float(), 0.5)
        want = torch.zeros_like(dx)
        want[:, 1] = 0.5
        assert torch.equal(dx, want)


@pytest.mark.parametrize("dt", [BF, F32])
def test_gradient_of_a_certain_target_is_zero(dt):
    """exp(l - lse) = 1 where the target's logit is lse itself: no residue of a change of base."""
    x, E, t, a, _ = two_levels(500, 900, 64, dt, seed=5, gap=(120.0, 130.0))
    dx, dE = run_bwd(x, E, t, a.float(), 1.0)
    assert torch.all(dx == 0) and torch.all(dE == 0)  # e^-120 is below every fp32 number


@pytest.mark.parametrize("scale", [1.0 / 1003, -1.0 / 777, 1.0 / 300])
@pytest.mark.parametrize("M,v,h", [(5, 5003, 1024), (40, 20000, 1024), (100, 5003, 256), (300, 4100, 256),
                                   (1003, 5003, 256), (700, 9000, 1088), (2100, 6000, 64)])
def test_gradients_are_not_shifted_by_the_scale(M, v, h, scale):
    """bf16 holds these more than 1.5e-3 off. What is rounded is p - 1, here about -1: no term may bring
    such a factor in."""
    assert abs(torch.tensor(scale).bfloat16().item() / scale - 1) > 1.5e-3
    g = gen(M)
    x, E = rnd(g, M, h), rnd(g, v, h, sigma=1e-4)
    t = torch.randint(0, v, (M,), generator=g, device="cuda").to(torch.int32)
    lse = torch.logsumexp(x.double() @ E.double().T, 1).float()
    dx, dE = run_bwd(x, E, t, lse, scale)
    for got, ref, name in zip((dx, dE), R.ce_bwd(x, E, t, lse, scale), ("dx", "dE")):
        got = got.double()
        # p = 1/v within 2 % or so, which p - 1 may lose to its rounding; the results' roundings, up to
        # 2^-8 each and independent: six of their standard deviations
        tol = 1.1 / v + 6 * 2.0 ** -8 / 3 ** 0.5 * ((ref ** 4).sum().sqrt() / (ref ** 2).sum()).item()
        shift = ((got - ref) * ref).sum() / (ref ** 2).sum()
        assert abs(shift.item()) <= tol < 1e-3, (name, shift.item(), tol)
