"""The oracle's cross-entropy where a target lies outside the vocabulary: its gradient is that of its
loss, by differences (CPU)."""
import numpy as np
import pytest

from oracle import gpt_oracle as G


@pytest.mark.parametrize("N", [1, 3])
def test_gradient_is_the_losss_with_targets_outside(N):
    rng = np.random.default_rng(4)
    M, v = 5, 12
    L = rng.normal(size=(M, v))
    t = np.array([3, -1, 11, 12, 0])
    lse = G.vocab_ce_fwd(L, t, N)[1]
    d = G.vocab_ce_bwd(L, t, lse, N, 1.0 / M)
    assert np.all(d[[1, 3]] == 0)
    for i in range(M):
        for j in range(v):
            f = []
            for e in (1e-6, -1e-6):
                K = L.copy()
                K[i, j] += e
                f.append(G.vocab_ce_fwd(K, t, N)[0])
            assert abs((f[0] - f[1]) / 2e-6 - d[i, j]) < 1e-9
