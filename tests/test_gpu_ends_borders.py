"""The training step's ends on both sides of the sizes where their kernels change form."""
import pytest
import torch

from tests import ends_ref as R
from tests.test_gpu_ends import BF, F32, ce_case, check_ce, check_embed_bwd, gen, rnd, run_fwd, tokens, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [1, 32])
@pytest.mark.parametrize("v", [1280, 16384])
@pytest.mark.parametrize("M", [1, 127, 128, 129, 303, 304, 305, 4863, 4864, 4865, 9001])
def test_join_of_the_partials(M, v, N):
    """One CTA up to 128 rows of few slots; 2, 8 or 32 rows of a CTA."""
    x, E, t = ce_case(M, v, 16, BF, seed=M + v)
    got = run_fwd(x, E, t, N)
    ref, b = R.ce_fwd(x, E, t, N), R.ce_fwd_bounds(x, E, t, N)
    for g, r, d, n in zip(got, ref, (b[3], b[0], b[1], b[2]), ("loss", "lse", "rows", "shards")):
        within(g, r, d, n)
    assert all(torch.equal(p, q) for p, q in zip(got, run_fwd(x, E, t, N)))


@pytest.mark.parametrize("M,v", [(300, 700), (4864, 130)])
def test_join_in_fp32(M, v):
    check_ce(*ce_case(M, v, 12, F32, seed=M), 2)


@pytest.mark.parametrize("kind", ["mixed", "same", "uniform", "sorted"])
@pytest.mark.parametrize("M", [4095, 4096, 4097, 8191])
@pytest.mark.parametrize("v,h", [(5, 24), (3000, 40), (128 * 1152, 8), (128 * 1152 + 1, 8)])
def test_sort_of_few_and_of_many_tokens(M, v, h, kind):
    """8 warps of a sorting CTA up to 4096 tokens, each of which may be one row's; more CTAs than SMs."""
    g = gen(M + v)
    ids, dx = tokens(g, M, v, kind), rnd(g, M, h)
    check_embed_bwd(ids, dx, v, 1.25)
    check_embed_bwd(ids, dx, v, 1.25, rnd(g, v, h))
