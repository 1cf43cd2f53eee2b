"""Contract checks of the norm, the microscaled formats and the product that need no GPU:
sizes, refusals on the host before any launch, and calls without work.  The reference of
the GPU tests is checked here too, against facts outside itself."""
import ctypes
import math

import numpy as np
import pytest
import torch

import attn_ref as ref
import mx_ref
import quantized_expert_ffn_router_amd as q
from mx_ref import MXFP4, MXFP8

OK, BAD, UNSUP, WS = q.MOE_OK, q.MOE_ERR_INVALID_ARG, q.MOE_ERR_UNSUPPORTED, q.MOE_ERR_WORKSPACE


def at(mib):  # addresses that must never be read, 1 MiB apart
    return 0x10000000 + (mib << 20)


def norm(H=256, T=4, x=at(0), xs=256, res=at(1), rs=256, w=at(2), eps=1e-6, sum=at(3), ss=256, out=at(4), os=256,
         fmt=MXFP8, codes=at(5), scales=at(6)):
    return q.lib().moe_add_norm(H, T, x, xs, res, rs, w, eps, sum, ss, out, os, fmt, codes, scales, None)


def quant(fmt=MXFP8, K=256, T=4, x=at(0), xs=256, codes=at(5), scales=at(6)):
    return q.lib().moe_mx_quant(fmt, K, T, x, xs, codes, scales, None)


def pack(N=64, K=256, codes=at(5), scales=at(6), packed=at(7)):
    return q.lib().moe_mx_pack(N, K, codes, scales, packed, None)


def matrix(N=64, K=256, packed=at(7), bias=None):
    return q.MxMatrix(N, K, packed, bias)


def linear(w=None, fmt=MXFP8, codes=at(5), scales=at(6), T=4, y=at(8), ys=64, dt=q.MOE_DTYPE_BF16):
    w = matrix() if w is None else w
    return q.lib().moe_mx_linear(ctypes.byref(w), fmt, codes, scales, T, y, ys, dt, None)


def rows(w=None, fmt=MXFP8, x=at(0), xs=256, T=4, y=at(8), ys=64, dt=q.MOE_DTYPE_BF16, ws=at(9), wb=1 << 20):
    w = matrix() if w is None else w
    return q.lib().moe_mx_linear_rows(ctypes.byref(w), fmt, x, xs, T, y, ys, dt, ws, wb, None)


def refused(status, want, msg):
    assert status == want, (status, q.last_error())
    assert msg in q.last_error()


@pytest.mark.parametrize("kw,status,msg", [
    (dict(H=0), BAD, "H=0"), (dict(H=100), UNSUP, "H=100"), (dict(H=16512), UNSUP, "H=16512"),
    (dict(T=-1), BAD, "T=-1"), (dict(T=(1 << 20) + 1), UNSUP, "2^20"), (dict(eps=-1.0), BAD, "eps"),
    (dict(eps=math.nan), BAD, "eps"), (dict(fmt=1), UNSUP, "row format 1"), (dict(fmt=0), BAD, "without a format"),
    (dict(fmt=0, codes=None, scales=None, sum=None, out=None), BAD, "no output"), (dict(x=None), BAD, "x is NULL"),
    (dict(xs=248), BAD, "x stride"), (dict(xs=257), BAD, "x stride"), (dict(x=at(0) + 2), BAD, "16-byte"),
    (dict(res=at(1) + 8), BAD, "16-byte"), (dict(rs=128), BAD, "residual stride"), (dict(ss=8), BAD, "sum stride"),
    (dict(os=8), BAD, "out stride"), (dict(w=None), BAD, "weight is NULL"), (dict(w=at(2) + 4), BAD, "16-byte"),
    (dict(codes=None), BAD, "codes is NULL"), (dict(scales=None), BAD, "scales is NULL"),
    (dict(codes=at(5) + 4), BAD, "16-byte"), (dict(scales=at(6) + 4), BAD, "16-byte"),
    (dict(sum=at(0), ss=512, xs=256), BAD, "sum overlaps x"), (dict(sum=at(0) + 512), BAD, "sum overlaps x"),
    (dict(out=at(1) + 32), BAD, "out overlaps residual"), (dict(out=at(3)), BAD, "out overlaps sum"),
    (dict(out=at(0), sum=at(0)), BAD, "out overlaps sum"), (dict(out=at(2)), BAD, "out overlaps weight"),
    (dict(codes=at(0)), BAD, "codes overlaps x"), (dict(codes=at(4) + 1024), BAD, "codes overlaps out"),
    (dict(scales=at(5) + 1008), BAD, "scales overlaps codes"), (dict(scales=at(3)), BAD, "scales overlaps sum"),
])
def test_norm_refusals(kw, status, msg):
    refused(norm(**kw), status, msg)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(fmt=0), UNSUP, "row format 0"), (dict(fmt=q.MOE_FMT_NVFP4), UNSUP, "row format 1"), (dict(K=0), BAD, "K=0"),
    (dict(K=64), UNSUP, "K=64"), (dict(K=32896), UNSUP, "K=32896"), (dict(T=-3), BAD, "T=-3"), (dict(x=None), BAD, "x is NULL"),
    (dict(xs=250), BAD, "stride"), (dict(codes=None), BAD, "codes is NULL"), (dict(scales=at(6) + 8), BAD, "16-byte"),
    (dict(codes=at(0) + 1024), BAD, "codes overlaps x"), (dict(scales=at(0)), BAD, "scales overlaps x"),
    (dict(scales=at(5)), BAD, "scales overlaps codes"),
])
def test_quant_refusals(kw, status, msg):
    refused(quant(**kw), status, msg)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(N=0), BAD, "N=0"), (dict(N=(1 << 20) + 1), UNSUP, "2^20"), (dict(K=129), UNSUP, "K=129"),
    (dict(codes=None), BAD, "codes is NULL"), (dict(scales=None), BAD, "scales is NULL"), (dict(packed=None), BAD, "packed is NULL"),
    (dict(packed=at(7) + 128), BAD, "256-byte"), (dict(packed=at(5)), BAD, "packed overlaps codes"),
    (dict(packed=at(6) - 256), BAD, "packed overlaps scales"),
])
def test_pack_refusals(kw, status, msg):
    refused(pack(**kw), status, msg)


PRODUCT = [
    (dict(w=matrix(N=0)), BAD, "N=0"), (dict(w=matrix(K=100)), UNSUP, "K=100"), (dict(w=matrix(packed=None)), BAD, "packed is NULL"),
    (dict(w=matrix(packed=at(7) + 16)), BAD, "256-byte"), (dict(w=matrix(bias=at(10) + 4)), BAD, "16-byte"),
    (dict(fmt=5), UNSUP, "row format 5"), (dict(T=-1), BAD, "T=-1"), (dict(T=1 << 21), UNSUP, "2^20"), (dict(dt=2), BAD, "y_dtype"),
    (dict(y=None), BAD, "y is NULL"), (dict(ys=56), BAD, "y stride"), (dict(ys=65), BAD, "y stride"), (dict(y=at(8) + 2), BAD, "16-byte"),
    (dict(y=at(7)), BAD, "y overlaps the weights"), (dict(w=matrix(bias=at(8) + 16)), BAD, "y overlaps bias"),
]


@pytest.mark.parametrize("kw,status,msg", PRODUCT + [
    (dict(codes=None), BAD, "codes is NULL"), (dict(scales=at(6) + 2), BAD, "16-byte"), (dict(codes=at(8)), BAD, "y overlaps codes"),
    (dict(scales=at(8) + 496, dt=q.MOE_DTYPE_F32), BAD, "y overlaps scales"),
])
def test_product_refusals(kw, status, msg):
    refused(linear(**kw), status, msg)


@pytest.mark.parametrize("kw,status,msg", PRODUCT + [
    (dict(x=None), BAD, "x is NULL"), (dict(xs=128), BAD, "x stride"), (dict(x=at(8)), BAD, "y overlaps x"), (dict(ws=None), BAD, "ws is NULL"),
    (dict(wb=4 * 256 + 255), WS, "workspace"), (dict(ws=at(9) + 8), BAD, "16-byte"), (dict(ws=at(8)), BAD, "y overlaps ws"),
    (dict(ws=at(0), T=100, wb=1 << 20), BAD, "ws overlaps x"),
])
def test_product_of_rows_refusals(kw, status, msg):
    refused(rows(**kw), status, msg)


def test_calls_without_rows_do_nothing():
    assert norm(T=0, x=None) == OK and quant(T=0, x=None) == OK and linear(T=0, y=None) == OK and rows(T=0, ws=None) == OK


def test_sizes():
    assert q.moe_mx_matrix_bytes(16, 128) == 1024 + 256  # 64 bytes of scales, to the next 256
    assert q.moe_mx_matrix_bytes(17, 256) == 2 * 2 * 1024 + 256
    assert q.moe_mx_matrix_bytes(1 << 20, 32768) == (1 << 20) * (16384 + 1024)
    assert q.moe_mx_matrix_bytes(0, 128) == 0 and q.moe_mx_matrix_bytes(16, 130) == 0
    assert q.moe_mx_workspace_bytes(MXFP4, 256, 0) == 0
    assert q.moe_mx_workspace_bytes(MXFP8, 256, 5) == 1280 + 256
    last = 0
    for T in range(1, 300):
        n = q.moe_mx_workspace_bytes(MXFP4, 384, T)
        assert n >= max(last, T * (192 + 12)) and n % 256 == 0
        last = n
    assert q.moe_mx_workspace_bytes(3, 256, 5) == 0 and q.moe_mx_workspace_bytes(MXFP4, 100, 5) == 0


def test_reference_grids():
    assert np.array_equal(mx_ref.e4m3_value(np.arange(256))[~np.isnan(ref.e4m3_val(np.arange(256)))],
                          ref.e4m3_val(np.arange(256))[~np.isnan(ref.e4m3_val(np.arange(256)))])
    v = np.random.default_rng(0).uniform(0, 460, 20000)
    assert np.array_equal(mx_ref.nearest(MXFP8, np.minimum(v, 448.0)), ref.e4m3_byte(np.minimum(v, 448.0).astype(np.float32).astype(np.float64)))
    v = (np.arange(0, 1200) / 160).astype(np.float32)
    assert np.array_equal(mx_ref.nearest(MXFP4, v.astype(np.float64)), ref.e2m1_code(v) & 7)


def test_reference_scales():
    """Hand-made blocks: the largest magnitude lands in the highest binade, whole blocks scale
    by powers of two, and what is beyond the largest code is held to it."""
    for fmt, hi in ((MXFP4, 4.0), (MXFP8, 256.0)):
        for k in (-30, 0, 7, 100):
            x = np.zeros((1, 32))
            x[0, 3], x[0, 5] = hi * 2.0 ** k, -hi * 1.984375 * 2.0 ** k  # the largest bf16 of the binade is 1.9921875
            c, s = mx_ref.quantise(fmt, ref.bf16_bits(x))
            assert s[0, 0] == 127 + k
            v = mx_ref.values(fmt, c, s)[0]
            assert v[3] == x[0, 3] and v[5] == -(6.0 if fmt == MXFP4 else 448.0) * 2.0 ** k and not v[[0, 31]].any()
    c, s = mx_ref.quantise(MXFP8, np.array([[0x0001] + [0] * 31], np.uint16))  # 2^-133
    assert s[0, 0] == 0 and mx_ref.values(MXFP8, c, s)[0, 0] == 2.0 ** -133
    for bad in (0x7f80, 0xff80, 0x7fc0):
        c, s = mx_ref.quantise(MXFP4, np.array([[bad] + [0x3f80] * 31], np.uint16))
        assert s[0, 0] == 255 and not c.any()


def test_reference_norm():
    x = torch.randn(5, 256).bfloat16()
    w = torch.randn(256)
    _, z = mx_ref.norm(x.view(torch.int16).numpy().view(np.uint16), None, w.numpy(), 1e-5)
    want = torch.nn.functional.rms_norm(x.double(), (256,), w.double(), float(np.float32(1e-5)))
    assert np.abs(ref.bf16_val(z) - want.numpy()).max() <= 2.0 ** -8 * want.abs().max()
