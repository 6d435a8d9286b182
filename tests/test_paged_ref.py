"""The float64 torch form of paged attention equals the oracle's loops (CPU)."""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from tests import paged_ref as R


@pytest.mark.parametrize("H,Hkv,N", [(4, 2, 1), (8, 2, 4), (3, 3, 3)])
@pytest.mark.parametrize("causal", [0, 1])
def test_equals_the_oracle(H, Hkv, N, causal):
    """Rows without keys, page ids outside the cache, a table narrower than the length, rows
    beyond T, padding; NaN in every slot that no row sees."""
    rng = np.random.default_rng(4)
    d, PS, n_pages = 8, 8, 9
    table = np.array([[3, -1, 5], [0, 1 << 20, 2], [7, 4, -1], [6, 1, 8]])
    tot, cu, rows = [20, 2, 13, 40], [0, 3, 8, 9, 15], 13
    qkv = rng.normal(size=(rows, R.cols(H, Hkv, N, d)))
    kc, vc = rng.normal(size=(2, n_pages, Hkv, PS, d))
    dead = ~R.seen(table, tot, cu, rows, n_pages, PS, causal)
    assert dead.any()
    want = P.paged_attention(P.qkv_heads(qkv, H, Hkv, N)[0], kc, vc, table, tot, cu, bool(causal))
    kc, vc = kc.copy(), vc.copy()
    kc[np.repeat(dead[:, None], Hkv, 1)] = np.nan
    vc[np.repeat(dead[:, None], Hkv, 1)] = np.nan
    t = torch.from_numpy
    got = R.reference(R.queries(t(qkv), H, Hkv, N), t(kc), t(vc), table, tot, cu, bool(causal))
    assert (got["written"].numpy() == want["written"]).all()
    for k in ("o", "A", "lse", "B", "n"):
        g, w = got[k].numpy(), want[k]
        assert (np.isneginf(g) == np.isneginf(w)).all()
        assert np.abs(np.where(np.isneginf(w), 0, g) - np.where(np.isneginf(w), 0, w)).max() < 1e-12


def test_nan_query_reaches_its_row_alone():
    q, kc = torch.ones(3, 2, 4, dtype=torch.float64), torch.ones(1, 1, 8, 4, dtype=torch.float64)
    q[1, 0, 2] = float("nan")
    f = R.reference(q, kc, kc, np.array([[0]]), [3], [0, 3], True)
    assert f["o"][1, 0].isnan().all() and f["lse"][0, 1].isnan()
    assert f["o"].isnan().sum() == 4 and f["lse"].isnan().sum() == 1
