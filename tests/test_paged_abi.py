"""Argument checks of the paged-cache entry points (no GPU: they return before any launch)."""
import pytest

from attention_gemms_gb300 import build as B
from attention_gemms_gb300 import tpmlp as T

S = T.Status
BF, F32 = T.DType.BF16, T.DType.F32
A = 1 << 20  # a fake, 16-byte-aligned address: never dereferenced


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    T.lib()


def _status(call, base, **kw):
    try:
        call(**{**base, **kw})
    except T.TpError as e:
        return e.status
    return S.OK


TABLES = dict(ctx_lens=A, new_lens=A, free_pages=A, n_free=4, free_head=A, free_head_out=A,
              block_table=A, total_lens=A, cu_new=A, slots=A, positions=None, counts=None, R=2,
              T=8, page_size=16, max_pages=4)
APPEND = dict(qkv=A, slots=A, kcache=A, vcache=A, T=0, h=512, n_heads=8, n_kv_heads=2, N=2,
              n_pages=4, page_size=16, dtype=BF)
ATTN = dict(qkv=A, kcache=A, vcache=A, block_table=A, total_lens=A, cu_new=A, o=A, lse=None, T=0,
            R=1, h=512, n_heads=8, n_kv_heads=2, N=2, n_pages=4, page_size=16, max_pages=4,
            max_new=1, causal=1, dtype=BF, ws=None, ws_bytes=0)
PROJ = dict(x=A, gamma=A, beta=A, Wqkv=A, Wo=A, xn=A, mean=None, rstd=None, qkv=A, kcache=A,
            vcache=A, block_table=A, total_lens=A, cu_new=A, slots=A, o=A, lse=None, out=A, T=0,
            R=1, h=512, n_heads=8, n_kv_heads=2, N=2, n_pages=4, page_size=16, max_pages=4,
            max_new=1, causal=1, dtype=BF, mode=T.Reduce.BUFFERS, ws=None, ws_bytes=0)


@pytest.mark.parametrize("kw,want", [
    (dict(ctx_lens=None), S.INVALID_ARG), (dict(slots=None), S.INVALID_ARG),
    (dict(free_pages=None), S.INVALID_ARG), (dict(n_free=-1), S.INVALID_ARG),
    (dict(R=-1), S.INVALID_ARG), (dict(T=-1), S.INVALID_ARG), (dict(R=8193), S.SHAPE),
    (dict(page_size=4), S.SHAPE), (dict(page_size=24), S.SHAPE), (dict(page_size=512), S.SHAPE),
    (dict(max_pages=0), S.INVALID_ARG), (dict(max_pages=1 << 28), S.SHAPE),
    (dict(n_free=1 << 31), S.SHAPE), (dict(ctx_lens=A + 2), S.ALIGNMENT),
    (dict(slots=A + 1), S.ALIGNMENT), (dict(counts=A + 2), S.ALIGNMENT)])
def test_tables(kw, want):
    assert _status(T.tp_kv_tables, TABLES, **kw) == want


SHAPES = [
    (dict(h=0), S.INVALID_ARG), (dict(n_kv_heads=0), S.INVALID_ARG), (dict(N=0), S.INVALID_ARG),
    (dict(T=-1), S.INVALID_ARG), (dict(n_pages=0), S.INVALID_ARG), (dict(h=510), S.SHAPE),
    (dict(h=8 * 48), S.SHAPE), (dict(h=8 * 256), S.SHAPE), (dict(n_kv_heads=3), S.SHAPE),
    (dict(N=3), S.SHAPE), (dict(page_size=12), S.SHAPE), (dict(page_size=1), S.SHAPE),
    (dict(n_pages=1 << 26), S.SHAPE), (dict(n_pages=1 << 40), S.SHAPE), (dict(T=1 << 31), S.SHAPE),
    (dict(dtype=5), S.DTYPE), (dict(kcache=A + 8), S.ALIGNMENT), (dict(qkv=A + 4), S.ALIGNMENT),
    (dict(vcache=None), S.INVALID_ARG)]


@pytest.mark.parametrize("kw,want", SHAPES + [(dict(slots=None), S.INVALID_ARG), (dict(), S.OK)])
def test_append(kw, want):
    assert _status(T.tp_kv_append, APPEND, **kw) == want


@pytest.mark.parametrize("kw,want", SHAPES + [
    (dict(block_table=None), S.INVALID_ARG), (dict(total_lens=None), S.INVALID_ARG),
    (dict(cu_new=None), S.INVALID_ARG), (dict(o=None), S.INVALID_ARG), (dict(o=A + 2), S.ALIGNMENT),
    (dict(max_pages=0), S.INVALID_ARG), (dict(max_pages=1 << 28), S.SHAPE),
    (dict(max_new=-1), S.INVALID_ARG), (dict(R=-1), S.INVALID_ARG), (dict(T=3), S.WORKSPACE),
    (dict(R=(1 << 20) + 1), S.SHAPE), (dict(lse=A + 2), S.ALIGNMENT),
    (dict(block_table=A + 2), S.ALIGNMENT), (dict(max_pages=(1 << 26) + 1), S.SHAPE),
    (dict(T=3, ws=A, ws_bytes=64), S.WORKSPACE), (dict(ws=A + 8), S.ALIGNMENT), (dict(), S.OK),
    (dict(R=0, T=3), S.OK)])
def test_attention(kw, want):
    assert _status(T.tp_gqa_paged_attention_fwd, ATTN, **kw) == want


@pytest.mark.parametrize("kw,want", SHAPES + [
    (dict(slots=None), S.INVALID_ARG), (dict(xn=None), S.INVALID_ARG), (dict(mode=7), S.INVALID_ARG),
    (dict(h=8 * 16, n_kv_heads=8, N=8), S.SHAPE),   # bf16 tile rule: shard block of 48 columns
    (dict(T=3), S.WORKSPACE), (dict(), S.OK)])
def test_block(kw, want):
    assert _status(T.tp_gqa_paged_attn_proj_fwd, PROJ, **kw) == want


def test_workspace_sizes():
    ws = T.tp_gqa_paged_attention_workspace_size
    assert ws(512, 8, 2, 2, BF) > 0 and ws(512, 8, 2, 2, F32) > 0
    assert ws(512, 8, 3, 2, BF) == 0 and ws(500, 8, 2, 2, BF) == 0 and ws(512, 8, 2, 2, 9) == 0
    blk = T.tp_gqa_paged_workspace_size
    assert blk(64, 512, 8, 2, 2, BF, T.Reduce.BUFFERS) >= max(ws(512, 8, 2, 2, BF), 2 * 64 * 512 * 4)
    assert blk(-1, 512, 8, 2, 2, BF, T.Reduce.BUFFERS) == 0
