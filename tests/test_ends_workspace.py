"""The forward cross-entropy's workspace is what its declaration says (CPU)."""
import pytest

from attention_gemms_gb300 import build as B
from attention_gemms_gb300 import tpmlp as T

ROWS = [1, 2, 7, 8, 9, 127, 128, 129, 303, 304, 305, 1216, 1217, 4863, 4864, 4865, 8192, 19456, 19457, 65537, 1 << 20]


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


@pytest.mark.parametrize("dtype", [T.DType.BF16, T.DType.F32])
@pytest.mark.parametrize("v", [1, 2, 63, 64, 65, 256, 50257, 50304, 262144])
def test_forward_bytes(v, dtype):
    last = 0
    for M in ROWS:
        n = T.tp_vocab_linear_ce_workspace_size(1, M, v, 8, 1, dtype)
        assert M * 8 * -(-v // 64) < n <= M * (8 * -(-v // 64) + 20) + (24 << 10), (M, v)
        assert n >= last, (M, v)  # what is enough for more rows is enough for fewer
        last = n
