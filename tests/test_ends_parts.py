"""Into how many parts the gradients of the cross-entropy split their sums, by the workspace that they
ask for (CPU)."""
import pytest

from attention_gemms_gb300 import build as B
from attention_gemms_gb300 import tpmlp as T


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def up(n, to):
    return -(-n // to) * to


def parts(M, v, h):
    """Of dx and of dE, one piece of the vocabulary (bf16; M * h and h whole 64-element blocks, so that
    the two are told apart by the rows)."""
    q = up(M * up(v, 256) * 2, 256)
    rest = T.tp_vocab_linear_ce_workspace_size(0, M, v, h, 1, T.DType.BF16) - q
    x, e = M * h * 4, up(v, 256) * h * 4
    found = [(a, b) for a in range(33) for b in range(33) if a * x + b * e == rest and 1 not in (a, b)]
    assert len(found) == 1, found
    return found[0]


@pytest.mark.parametrize("M,v,h", [(65, 8200, 128), (1, 4336, 1664), (65, 4336, 1664), (37, 50257, 4096),
                                   (256, 2064, 256), (300, 1500, 256), (130, 32000, 512), (1003, 50257, 1024)])
def test_every_part_of_dx_holds_something(M, v, h):
    a, _ = parts(M, v, h)
    if a:
        each = up(-(-v // a), 64)
        assert (a - 1) * each < v, f"{a} parts of {each} for {v}"


@pytest.mark.parametrize("M,v,h", [(2064, 256, 256), (8200, 65, 128), (4336, 70, 128), (5000, 513, 256),
                                   (20000, 130, 192)])
def test_every_part_of_dE_holds_something(M, v, h):
    _, b = parts(M, v, h)
    assert b > 1
    each = up(-(-M // b), 64)
    assert (b - 1) * each < M, f"{b} parts of {each} for {M}"
