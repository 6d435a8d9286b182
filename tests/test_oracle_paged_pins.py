"""Pins of the paged-cache oracle (CPU): pages and slots by hand, the cache's write, and
attention over pages against the dense grouped-query oracle, whole and in chunks."""
import numpy as np
import pytest

from oracle import gqa_oracle as Q
from oracle import paged_oracle as P


def test_tables_by_hand():
    table = np.full((3, 4), -1)
    table[0, :2] = [7, 3]                     # 10 cached tokens, pages of 8
    table[2, 0] = 5
    f = P.kv_tables([10, 0, 8], [7, 3, 1], [50, 51, 52, 53], 1, table, 12, 8)
    assert f["cu"] == [0, 7, 10, 11] and f["total"] == [17, 3, 9]
    assert f["table"].tolist() == [[7, 3, 51, -1], [52, -1, -1, -1], [5, 53, -1, -1]]
    assert f["slots"] == [26, 27, 28, 29, 30, 31, 51 * 8, 52 * 8, 52 * 8 + 1, 52 * 8 + 2, 53 * 8, -1]
    assert f["pos"] == [10, 11, 12, 13, 14, 15, 16, 0, 1, 2, 8, -1]
    assert f["head"] == 4 and f["counts"] == [11, 3, 0, 0]


def test_tables_list_runs_out_and_rows_overflow():
    f = P.kv_tables([0, 0], [9, 8], [4], 0, np.full((2, 2), -1), 10, 8)
    assert f["table"].tolist() == [[4, -1], [-1, -1]]
    assert f["slots"] == [32, 33, 34, 35, 36, 37, 38, 39, -1, -1]
    assert f["counts"] == [17, 1, 2, 7] and f["head"] == 1


@pytest.mark.parametrize("H,Hkv,N", [(4, 2, 1), (4, 2, 2), (8, 2, 4)])
@pytest.mark.parametrize("causal", [0, 1])
def test_attention_equals_the_dense_oracle(H, Hkv, N, causal):
    """A prompt written page by page and attended at once, or (causal) in two chunks,
    equals the dense attention on the same rows."""
    rng = np.random.default_rng(3)
    s, d, PS = 21, 8, 8
    hq, hkv, _ = Q.gqa_split(H, Hkv, N)
    qkv = rng.normal(size=(s, N * (hq + 2 * hkv) * d))
    q, k, v = P.qkv_heads(qkv, H, Hkv, N)
    if N > Hkv:                                # replicas hold equal keys and values
        x = qkv.reshape(s, N, hq + 2 * hkv, d)
        for i in range(N):
            x[:, i, hq:] = x[:, i // (N // Hkv) * (N // Hkv), hq:]
        q, k, v = P.qkv_heads(qkv, H, Hkv, N)
    ref = Q.gqa_attention_fwd(qkv, 1, s, H, Hkv, N, bool(causal))
    table = np.array([[4, 0, 2]])
    f = P.kv_tables([0], [s], [4, 0, 2], 0, np.full((1, 3), -1), s, PS)
    assert (f["table"] == table).all()
    kc = np.full((5, Hkv, PS, d), np.nan)      # unused slots are never read
    kc, vc = P.kv_append(k, v, f["slots"], kc, kc.copy())
    o = P.paged_attention(q, kc, vc, table, [s], [0, s], causal)["o"]
    assert np.abs(o.reshape(s, -1) - ref).max() < 1e-12
    if causal:
        a = P.paged_attention(q[:13], kc, vc, table, [13], [0, 13], 1)["o"]
        b = P.paged_attention(q[13:], kc, vc, table, [s], [0, s - 13], 1)["o"]
        assert np.abs(np.concatenate([a, b]).reshape(s, -1) - ref).max() < 1e-12


def test_rows_without_keys():
    q, kc = np.ones((3, 1, 4)), np.ones((1, 1, 8, 4))
    f = P.paged_attention(q, kc, kc, np.array([[0]]), [1], [0, 3], 1)
    assert f["lse"][0, 0] == -np.inf and f["lse"][0, 1] == -np.inf and f["o"][:2].max() == 0
    assert np.allclose(f["o"][2], 1.0)
