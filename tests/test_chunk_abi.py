"""Contract checks of moe_attn_chunk that need no GPU: refusals on the host before any launch,
calls without work, and the workspace's size."""
import ctypes
import math

import pytest

import quantized_expert_ffn_router_amd as q
from attn_ref import BF16, NVFP4, Q8_0

OK, BAD, UNSUP, WS = q.MOE_OK, q.MOE_ERR_INVALID_ARG, q.MOE_ERR_UNSUPPORTED, q.MOE_ERR_WORKSPACE
A, B = 0x1000, 0x40000000  # addresses that must never be read


def cache(fmt=NVFP4, n_kv=2, D=128, P=64, n_pages=4, ks=1.0, vs=1.0, pool=A):
    return q.KvCacheDesc(fmt, n_kv, D, P, n_pages, ks, vs, pool)


def chunk(c=None, n=2, width=128, start=A, lens=A, table=A, n_q=8, x=A, xs=1024, T=40, max_len=8192, scale=0.1, out=B, os=1024,
          ws=A, wb=1 << 30):
    c, s = c or cache(), q.SeqBatch(n, width, start, lens, table)
    return q.lib().moe_attn_chunk(ctypes.byref(c), ctypes.byref(s), n_q, x, xs, T, max_len, scale, out, os, ws, wb, None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(c=cache(fmt=7)), UNSUP, "cache format 7"), (dict(c=cache(D=96)), UNSUP, "D=96"), (dict(c=cache(P=48)), UNSUP, "page_tokens=48"),
    (dict(c=cache(n_pages=0)), BAD, "n_pages=0"), (dict(c=cache(ks=0.0)), BAD, "k_scale"), (dict(c=cache(pool=None)), BAD, "pool is NULL"),
    (dict(c=cache(pool=A + 16)), BAD, "256-byte"), (dict(n=-1), BAD, "n_seq=-1"), (dict(n=65536), UNSUP, "n_seq=65536"),
    (dict(width=0), BAD, "max_pages=0"), (dict(start=None), BAD, "row_start is NULL"), (dict(lens=None), BAD, "kv_len is NULL"),
    (dict(table=None), BAD, "page_table is NULL"), (dict(n_q=7), BAD, "n_q=7"), (dict(n_q=1026), UNSUP, "n_q=1026"),
    (dict(T=-1), BAD, "T=-1"), (dict(T=1 << 24), UNSUP, "too large"), (dict(scale=0.0), BAD, "scale"), (dict(scale=math.nan), BAD, "scale"),
    (dict(max_len=-1), BAD, "max_len=-1"), (dict(x=None), BAD, "q is NULL"), (dict(xs=1016), BAD, "q stride"), (dict(xs=1028), BAD, "q stride"),
    (dict(out=None), BAD, "out is NULL"), (dict(os=512), BAD, "out stride"), (dict(out=B + 8), BAD, "16-byte"),
    (dict(ws=None), BAD, "ws is NULL"), (dict(wb=100), WS, "workspace"), (dict(ws=A + 8), BAD, "16-byte"),
    (dict(out=A + 1024), BAD, "out overlaps q"), (dict(out=A, os=2048), BAD, "out overlaps q"),
])
def test_refusals(kw, status, msg):
    assert chunk(**kw) == status, q.last_error()
    assert msg in q.last_error()


def test_calls_without_rows_do_nothing():
    assert chunk(T=0, x=None, out=None, ws=None) == OK and chunk(n=0, x=None, out=None, start=None) == OK


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16])
@pytest.mark.parametrize("n_q,n_kv,D", [(32, 4, 128), (8, 8, 64), (5, 1, 256)])
def test_a_workspace_serves_every_smaller_step(fmt, n_q, n_kv, D):
    """The size for T rows is enough for any fewer, and for any shorter longest cache."""
    c = cache(fmt, n_kv, D)
    for n_seq in (1, 3, 40):
        for T in (1, 17, 300, 2048, 5000):
            most = q.moe_attn_chunk_workspace_bytes(c, n_q, n_seq, T, 100_000)
            assert most % 256 == 0
            for t in range(1, T + 1, max(1, T // 37)):
                for m in (1, 900, 33_000, 100_000):
                    assert q.moe_attn_chunk_workspace_bytes(c, n_q, n_seq, t, m) <= most
            assert q.moe_attn_chunk_workspace_bytes(c, n_q, n_seq, T, 0) >= most
    assert q.moe_attn_chunk_workspace_bytes(c, n_q, 1, 0, 1000) == 0


def test_workspace_refusals():
    c = cache()
    assert q.moe_attn_chunk_workspace_bytes(c, 7, 1, 5, 100) == 0 and "n_q=7" in q.last_error()
    assert q.moe_attn_chunk_workspace_bytes(c, 8, -1, 5, 100) == 0 and "n_seq=-1" in q.last_error()
    assert q.moe_attn_chunk_workspace_bytes(c, 8, 1, 5, -100) == 0 and "max_len=-100" in q.last_error()
    assert q.lib().moe_attn_chunk_workspace_bytes(None, 8, 1, 5, 100) == 0 and "c is NULL" in q.last_error()
