"""Refusals of the output layer's cross-entropy and of the scaled embedding, before any launch."""
import pytest

from attention_gemms_gb300 import build as B
from attention_gemms_gb300 import tpmlp as T

A = 1 << 20  # a fake, 16-byte-aligned address: never dereferenced (validation fails first)
BF, F32 = T.DType.BF16, T.DType.F32
S = T.Status


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def status(fn, base, **kw):
    try:
        fn(**{**base, **kw})
    except T.TpError as e:
        return e.status
    return S.OK


FWD = dict(x=A, E=A, targets=A, lse=A, row_loss=A, shard_loss=A, loss=A, M=10, vocab=100, h=64, N=2,
           dtype=BF, ws=A, ws_bytes=1 << 30)
BWD = dict(x=A, E=A, targets=A, lse=A, dx=A, dE=A, M=10, vocab=100, h=64, N=2, scale=0.1, dtype=BF,
           ws=A, ws_bytes=1 << 30)
EF = dict(ids=A, E=A, x=A, M=10, vocab=100, h=64, N=2, scale=2.0, dtype=BF)
EB = dict(ids=A, dx=A, dE=A, M=10, vocab=100, h=64, N=2, scale=2.0, accumulate=0, dtype=BF, ws=A,
          ws_bytes=1 << 30)

COMMON = [(dict(M=-1), S.INVALID_ARG), (dict(N=0), S.INVALID_ARG), (dict(vocab=0), S.INVALID_ARG),
          (dict(h=0), S.INVALID_ARG), (dict(N=3), S.SHAPE), (dict(dtype=7), S.DTYPE),
          (dict(M=(1 << 30) + 1), S.SHAPE), (dict(vocab=1 << 31), S.SHAPE),
          (dict(h=(1 << 20) + 8), S.SHAPE), (dict(vocab=1 << 30, h=1 << 20), S.SHAPE)]


@pytest.mark.parametrize("fn,base", [(T.tp_vocab_linear_ce_fwd, FWD), (T.tp_vocab_linear_ce_bwd, BWD),
                                     (T.tp_vocab_embed_scaled_fwd, EF),
                                     (T.tp_vocab_embed_scaled_bwd, EB)])
def test_sizes_types_and_pointers(fn, base):
    for kw, want in COMMON:
        assert status(fn, base, **kw) == want, kw
    for name, v in base.items():
        if v != A:
            continue
        if name not in ("shard_loss", "dx", "dE") or (base is EB and name != "ws"):
            want = S.WORKSPACE if name == "ws" else S.INVALID_ARG
            assert status(fn, base, **{name: None}) == want, name
        words = name in ("targets", "ids", "lse", "row_loss", "shard_loss", "loss")
        assert status(fn, base, **{name: A + 2}) == S.ALIGNMENT, name
        if not words:
            assert status(fn, base, **{name: A + 8}) == S.ALIGNMENT, name


def test_linear_ce_rules():
    assert status(T.tp_vocab_linear_ce_fwd, FWD, h=60) == S.SHAPE
    assert status(T.tp_vocab_linear_ce_bwd, BWD, h=60) == S.SHAPE
    assert status(T.tp_vocab_linear_ce_bwd, BWD, dx=None, dE=None) == S.INVALID_ARG
    for fn, base, fwd in ((T.tp_vocab_linear_ce_fwd, FWD, 1), (T.tp_vocab_linear_ce_bwd, BWD, 0)):
        assert status(fn, base, dtype=F32, M=64 * 65535 + 1) == S.SHAPE
        assert T.tp_vocab_linear_ce_workspace_size(fwd, 64 * 65535 + 1, 100, 64, 2, F32) == 0
    assert status(T.tp_vocab_linear_ce_fwd, FWD, M=0, ws=None) == S.OK  # nothing launched
    assert status(T.tp_vocab_linear_ce_bwd, BWD, M=0, dE=None, ws=None) == S.OK
    assert status(T.tp_vocab_embed_scaled_fwd, EF, M=0) == S.OK


@pytest.mark.parametrize("dtype", [BF, F32])
def test_workspaces(dtype):
    for fwd, fn, base in ((1, T.tp_vocab_linear_ce_fwd, FWD), (0, T.tp_vocab_linear_ce_bwd, BWD)):
        n = T.tp_vocab_linear_ce_workspace_size(fwd, 10, 100, 64, 2, dtype)
        assert n > 0
        assert status(fn, base, dtype=dtype, ws_bytes=n - 1) == S.WORKSPACE
    n = T.tp_vocab_embed_scaled_workspace_size(10, 100, 64, dtype)
    assert n > 0 and status(T.tp_vocab_embed_scaled_bwd, EB, dtype=dtype, ws_bytes=n - 1) == S.WORKSPACE
    for bad in (dict(M=-1), dict(vocab=0), dict(h=0), dict(N=0), dict(N=3), dict(dtype=5),
                dict(vocab=1 << 40), dict(M=1 << 40)):
        a = dict(M=10, vocab=100, h=64, N=2, dtype=dtype)
        assert T.tp_vocab_linear_ce_workspace_size(1, **{**a, **bad}) == 0
        assert T.tp_vocab_linear_ce_workspace_size(0, **{**a, **bad}) == 0
        a.pop("N")
        if "N" not in bad:
            assert T.tp_vocab_embed_scaled_workspace_size(**{**a, **bad}) == 0


def test_workspaces_stay_small():
    """What the backward keeps does not grow with the vocabulary, nor with rows beyond dx's own: q
    and the parts of the sums, 512 MiB each, and one fp32 dx."""
    size = T.tp_vocab_linear_ce_workspace_size
    M, h = 8192, 2048
    dx = M * h * 4
    for v in (50304, 262144, 1 << 20):
        assert size(0, M, v, h, 1, BF) <= (2 * 512 << 20) + dx + 4096
        assert size(1, M, v, h, 1, BF) <= M * v // 8 + M * 64 * 8 + 4096 + 64 * M
    assert size(0, 1 << 20, 50304, h, 1, BF) <= (2 * 512 << 20) + (1 << 20) * h * 4 + 4096
