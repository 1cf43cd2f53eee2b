"""moe_add_norm, moe_mx_quant, moe_mx_pack, moe_mx_linear and moe_mx_linear_rows against the
64-bit reference in mx_ref.py: sizes around every tile, both formats, both output types,
extreme values, infinities and NaN, strides, in-place outputs, untouched surroundings,
offsets beyond 32 bits, other streams and captured graphs.

Bounds: sums, normed rows, codes and scales are equal bit for bit (both sides compute what
is rounded in 64 bits); products are within mx_ref.product_bound."""
import numpy as np
import pytest
import torch

import attn_ref as ref
import mx_ref
import quantized_expert_ffn_router_amd as q
from mx_ref import MXFP4, MXFP8

pytestmark = pytest.mark.gpu

dev = "cuda"
EPS = 1e-6


def to_dev(u16):
    return torch.from_numpy(np.ascontiguousarray(u16).view(np.int16)).to(dev).view(torch.bfloat16)


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def u8(*shape, fill=0xA5):
    return torch.full(shape, fill, dtype=torch.uint8, device=dev)


def wide(rng, T, K):
    """Rows whose blocks lie binades apart, as bf16 bits."""
    return ref.bf16_bits(rng.standard_normal((T, K)) * 2.0 ** np.repeat(rng.integers(-8, 8, (T, K // 32)), 32, 1))


def width(fmt, K):
    return K // 2 if fmt == MXFP4 else K


# ------------------------------------------------------------------ norm and quantiser

def run_norm(x, res, w, fmt, want_sum=True, want_out=True, xs=None):
    T, H = x.shape
    stride = xs or H
    pad = lambda a: torch.cat((to_dev(a), torch.zeros(T, stride - H, dtype=torch.bfloat16, device=dev)), 1)  # noqa: E731
    xd, rd = pad(x), None if res is None else pad(res)
    s = torch.full((T + 1, stride), 9.0, dtype=torch.bfloat16, device=dev) if want_sum else None
    o = torch.full((T + 1, stride), 9.0, dtype=torch.bfloat16, device=dev) if want_out else None
    c, f = (u8(T + 1, width(fmt, H)), u8(T + 1, H // 32)) if fmt else (None, None)
    q.moe_add_norm(H, T, xd, stride, rd, stride, torch.from_numpy(w).to(dev), EPS, s, stride, o, stride, fmt, c, f)
    torch.cuda.synchronize()
    for t in (s, o):  # nothing beside the rows' own elements
        assert t is None or ((t[T] == 9.0).all() and (t[:T, H:] == 9.0).all())
    for t in (c, f):
        assert t is None or (t[T] == 0xA5).all()
    return (None if s is None else bits(s[:T, :H]), None if o is None else bits(o[:T, :H]),
            None if c is None else c[:T].cpu().numpy(), None if f is None else f[:T].cpu().numpy())


def check_codes(fmt, want_bits, codes, scales):
    c, s = mx_ref.quantise(fmt, want_bits)
    assert np.array_equal(scales, s)
    assert np.array_equal(codes, mx_ref.pack_codes(fmt, c))


@pytest.mark.parametrize("fmt", [0, MXFP4, MXFP8])
@pytest.mark.parametrize("H", [128, 256, 384, 512, 640, 1024, 2048, 2176, 5120, 8192, 8320, 16384])
def test_norm_widths(H, fmt):
    rng = np.random.default_rng(H)
    for T in (1, 3, 5):
        x, res = wide(rng, T, H), wide(rng, T, H)
        w = (1 + 0.3 * rng.standard_normal(H)).astype(np.float32)
        s, o, c, f = run_norm(x, res, w, fmt)
        h, z = mx_ref.norm(x, res, w, EPS)
        assert np.array_equal(s, h) and np.array_equal(o, z)
        if fmt:
            check_codes(fmt, z, c, f)


@pytest.mark.parametrize("fmt,res,want_sum,want_out", [(MXFP8, True, True, False), (MXFP4, True, False, False), (0, True, False, True),
                                                       (0, True, True, False), (MXFP8, False, False, True), (MXFP8, False, True, False)])
def test_norm_outputs_left_out(fmt, res, want_sum, want_out):
    rng = np.random.default_rng(3)
    x, r = wide(rng, 37, 384), wide(rng, 37, 384) if res else None
    w = rng.standard_normal(384).astype(np.float32)
    s, o, c, f = run_norm(x, r, w, fmt, want_sum, want_out, xs=400)
    h, z = mx_ref.norm(x, r, w, EPS)
    assert s is None or np.array_equal(s, h)
    assert o is None or np.array_equal(o, z)
    if fmt:
        check_codes(fmt, z, c, f)


def test_norm_extremes():
    """Rows whose squares leave fp32 at both ends, zero rows, one value alone, infinities, NaN, a
    sum that overflows: each row is answered by itself."""
    H, rng = 256, np.random.default_rng(5)
    x = np.zeros((9, H), np.uint16)
    x[0] = ref.bf16_bits(rng.standard_normal(H) * 2.0 ** 120)
    x[1] = ref.bf16_bits(rng.standard_normal(H) * 2.0 ** -130)
    x[3, 77] = 0x3f80
    x[4], x[5], x[6], x[8] = x[0], wide(rng, 1, H)[0], wide(rng, 1, H)[0], wide(rng, 1, H)[0]
    x[4, 9], x[5, 10], x[6, 11] = 0x7f7f, 0xff80, 0x7fc1
    res = np.zeros_like(x)
    res[4, 9] = 0x7f7f  # 2 * the largest: infinite
    w = rng.standard_normal(H).astype(np.float32)
    s, o, c, f = run_norm(x, res, w, MXFP8)
    h, z = mx_ref.norm(x, res, w, EPS)
    val = ref.bf16_val
    assert np.array_equal(np.isnan(val(s)), np.isnan(val(h))) and np.array_equal(s[~np.isnan(val(h))], h[~np.isnan(val(h))])
    assert np.array_equal(np.isnan(val(o)), np.isnan(val(z))) and np.array_equal(o[~np.isnan(val(z))], z[~np.isnan(val(z))])
    for t in range(9):
        cc, ff = mx_ref.quantise(MXFP8, o[t:t + 1])
        assert np.array_equal(f[t:t + 1], ff) and np.array_equal(c[t:t + 1], cc), t
    assert (f[5] == 255).any() and (f[6] == 255).all() and (f[8] != 255).all()


def test_norm_in_place():
    rng = np.random.default_rng(6)
    x, res = wide(rng, 700, 1152), wide(rng, 700, 1152)
    w = rng.standard_normal(1152).astype(np.float32)
    h, z = mx_ref.norm(x, res, w, EPS)
    xd, rd, wd = to_dev(x), to_dev(res), torch.from_numpy(w).to(dev)
    c, f = u8(700, 576), u8(700, 36)
    q.moe_add_norm(1152, 700, xd, 1152, rd, 1152, wd, EPS, rd, 1152, xd, 1152, MXFP4, c, f)  # sum over the residual, out over x
    assert np.array_equal(bits(rd), h) and np.array_equal(bits(xd), z)
    check_codes(MXFP4, z, c.cpu().numpy(), f.cpu().numpy())


@pytest.mark.parametrize("fmt", [MXFP4, MXFP8])
@pytest.mark.parametrize("T,K", [(1, 128), (3, 512), (5, 640), (2, 4096), (700, 1152), (9, 16384), (2, 32768), (3000, 2176)])
def test_quant(T, K, fmt):
    rng = np.random.default_rng(T + K)
    x = wide(rng, T, K)
    xd = torch.zeros(T, K + 8, dtype=torch.bfloat16, device=dev)
    xd[:, :K] = to_dev(x)
    c, f = u8(T + 1, width(fmt, K)), u8(T + 1, K // 32)
    q.moe_mx_quant(fmt, K, T, xd, K + 8, c, f)
    assert (c[T] == 0xA5).all() and (f[T] == 0xA5).all()
    check_codes(fmt, x, c[:T].cpu().numpy(), f[:T].cpu().numpy())


@pytest.mark.parametrize("fmt", [MXFP4, MXFP8])
def test_quant_of_every_value(fmt):
    """Every bf16 value as a block's largest and beside a larger one: ties, subnormal numbers,
    what the largest code holds, zeros of both signs, infinities and NaN."""
    v = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    x = np.zeros((1 << 16, 128), np.uint16)
    x[:, 0] = v  # alone
    x[:, 32], x[:, 33] = v, np.roll(v, 1)
    x[:, 64], x[:, 65] = v, np.where((v & 0x7f80) < 0x7f00, (v & 0x7f80) + 0x80 | 0x7f, v)  # a binade below the largest
    x[:, 96], x[:, 97] = v, np.minimum((v & 0x7fff).astype(np.uint32) + 0x200, 0x7f7f).astype(np.uint16)
    c, f = u8(1 << 16, width(fmt, 128)), u8(1 << 16, 4)
    q.moe_mx_quant(fmt, 128, 1 << 16, to_dev(x), 128, c, f)
    check_codes(fmt, x, c.cpu().numpy(), f.cpu().numpy())


# ------------------------------------------------------------------ product

def matrix(rng, N, K, bias=False):
    """A packed matrix, its values and its bias."""
    w = wide(rng, N, K)
    wd = to_dev(w)
    c, f = u8(N, K // 2), u8(N, K // 32)
    q.moe_mx_quant(MXFP4, K, N, wd, K, c, f)
    nb = q.moe_mx_matrix_bytes(N, K)
    packed = u8(nb, fill=0xFF)
    q.moe_mx_pack(N, K, c, f, packed)
    b = torch.from_numpy(rng.standard_normal((N + 3) // 4 * 4).astype(np.float32)).to(dev) if bias else None
    cc, ss = mx_ref.quantise(MXFP4, w)
    m = q.MxMatrix(N, K, packed.data_ptr(), None if b is None else b.data_ptr())
    m.keep = (packed, b)
    return m, mx_ref.values(MXFP4, cc, ss), 0.0 if b is None else b[:N].double().cpu().numpy()


def run_product(m, fmt, x, f32, as_rows, codes=None, stream=None):
    """x: bf16 bits [T, K], or codes (one byte each) and scales -> values [T, N] float64."""
    N, K = m.N, m.K
    T = len(x if codes is None else codes[0])
    stride = (N + 7) // 8 * 8 + 8
    y = torch.full((T + 1, stride), 9.0, dtype=torch.float32 if f32 else torch.bfloat16, device=dev)
    dt = q.MOE_DTYPE_F32 if f32 else q.MOE_DTYPE_BF16
    if as_rows:
        xd = torch.zeros(T, K + 8, dtype=torch.bfloat16, device=dev)
        xd[:, :K] = to_dev(x)
        nb = q.moe_mx_workspace_bytes(fmt, K, T)
        q.moe_mx_linear_rows(m, fmt, xd, K + 8, T, y, stride, dt, u8(nb, fill=0xFF), nb, stream)
    else:
        c, s = mx_ref.quantise(fmt, x) if codes is None else codes
        q.moe_mx_linear(m, fmt, torch.from_numpy(mx_ref.pack_codes(fmt, c)).to(dev), torch.from_numpy(s).to(dev), T, y, stride, dt, stream)
    torch.cuda.synchronize()
    assert (y[T] == 9.0).all() and (y[:T, N:] == 9.0).all()
    return y[:T, :N].double().cpu().numpy()


def exact(fmt, x, w, b, codes=None):
    c, s = mx_ref.quantise(fmt, x) if codes is None else codes
    a = mx_ref.values(fmt, c, s)
    return a @ w.T + b, np.abs(a) @ np.abs(w).T + np.abs(b), tops(a, w)


def tops(a, w):
    """Sum over the groups of 8 neighbouring products of the group's largest magnitude [T, N]."""
    (T, K), N = a.shape, len(w)
    ad, wd = (torch.from_numpy(np.abs(v)).to(dev).view(len(v), K // 8, 8) for v in (a, w))
    out = torch.zeros(T, N, dtype=torch.float64, device=dev)
    step = max(1, (1 << 26) // (T * N * 8))
    for j in range(0, K // 8, step):
        out += (ad[:, None, j:j + step] * wd[None, :, j:j + step]).amax(-1).sum(-1)
    return out.cpu().numpy()


def check_product(fmt, x, w, b, got, f32, K, codes=None):
    y, ab, top = exact(fmt, x, w, b, codes)
    err = np.abs(got - y)
    bound = mx_ref.product_bound(fmt, y, ab, top, K, f32)
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("fmt", [MXFP4, MXFP8])
@pytest.mark.parametrize("N,K", [(1, 128), (16, 256), (17, 384), (100, 1152), (333, 2048), (40, 4224), (9, 8320), (5000, 128)])
def test_product_of_few_rows(N, K, fmt):
    rng = np.random.default_rng(N + K)
    m, w, b = matrix(rng, N, K, bias=N % 2 == 0)
    for T in (1, 2, 15, 16, 17, 32, 33, 64):
        x = wide(rng, T, K)
        for f32 in (False, True):
            got = run_product(m, fmt, x, f32, False)
            check_product(fmt, x, w, b, got, f32, K)
            assert np.array_equal(run_product(m, fmt, x, f32, True), got)  # quantised on the way: the same bit for bit


@pytest.mark.parametrize("fmt", [MXFP4, MXFP8])
@pytest.mark.parametrize("T,N,K", [(65, 1, 128), (65, 127, 384), (100, 129, 640), (128, 256, 256), (129, 400, 128), (300, 1000, 1152),
                                   (2049, 2051, 256), (2048, 2100, 128), (4100, 4099, 384), (8192, 2048, 128)])
def test_product_of_many_rows(T, N, K, fmt):
    rng = np.random.default_rng(T + N + K)
    m, w, b = matrix(rng, N, K, bias=N % 2 == 1)
    x = wide(rng, T, K)
    got = run_product(m, fmt, x, False, False)
    check_product(fmt, x, w, b, got, False, K)
    if T * N < 1 << 19:
        check_product(fmt, x, w, b, run_product(m, fmt, x, True, False), True, K)
    assert np.array_equal(run_product(m, fmt, x, False, True), got)


@pytest.mark.parametrize("fmt", [MXFP4, MXFP8])
@pytest.mark.parametrize("T", [1, 20, 64, 70, 300])
def test_product_of_extreme_scales(T, fmt):
    """Any scale bytes with any codes: products far below and above 1; a NaN scale of a row makes
    that row NaN and no other, one of the matrix its column."""
    rng = np.random.default_rng(T)
    K, N = 384, 75
    m, w, b = matrix(rng, N, K)
    c = rng.integers(0, 16 if fmt == MXFP4 else 127, (T, K)).astype(np.uint8)
    s = rng.integers(60, 190, (T, K // 32)).astype(np.uint8)
    if fmt == MXFP8:
        c ^= (rng.integers(0, 2, (T, K)) << 7).astype(np.uint8)
    s[T // 2, 5] = 255
    got = run_product(m, fmt, None, True, False, codes=(c, s))
    y, ab, top = exact(fmt, None, w, b, codes=(c, s))
    assert np.isnan(got[T // 2]).all()
    keep = np.arange(T) != T // 2
    assert (np.abs(got - y)[keep] <= mx_ref.product_bound(fmt, y, ab, top, K, True)[keep]).all()


@pytest.mark.parametrize("fmt", [MXFP4, MXFP8])
@pytest.mark.parametrize("T", [3, 64, 200])
def test_product_of_rows_with_infinities(T, fmt):
    rng = np.random.default_rng(T)
    m, w, b = matrix(rng, 50, 512)
    x = wide(rng, T, 512)
    x[1, 300], x[2, 7] = 0x7f80, 0x7fc0
    for as_rows in (False, True):
        got = run_product(m, fmt, x, False, as_rows)
        assert np.isnan(got[1:3]).all() and np.isfinite(got[np.arange(T) > 2]).all() and np.isfinite(got[0]).all()


def test_weights_of_a_nan_scale():
    rng = np.random.default_rng(1)
    w = wide(rng, 40, 256)
    w[7, 33] = 0x7f80
    c, f = u8(40, 128), u8(40, 8)
    q.moe_mx_quant(MXFP4, 256, 40, to_dev(w), 256, c, f)
    packed = u8(q.moe_mx_matrix_bytes(40, 256))
    q.moe_mx_pack(40, 256, c, f, packed)
    m = q.MxMatrix(40, 256, packed.data_ptr(), None)
    for T in (2, 90):
        got = run_product(m, MXFP8, wide(rng, T, 256), False, False)
        assert np.isnan(got[:, 7]).all() and np.isfinite(np.delete(got, 7, 1)).all()


def test_long_sums():
    """K = 32768, which takes several passes of a workgroup's waves."""
    rng = np.random.default_rng(8)
    m, w, b = matrix(rng, 70, 32768)
    for T in (1, 16, 40, 100):
        x = wide(rng, T, 32768)
        for fmt in (MXFP4, MXFP8):
            got = run_product(m, fmt, x, True, False)
            check_product(fmt, x, w, b, got, True, 32768)
            assert np.array_equal(run_product(m, fmt, x, True, True), got)


def test_offsets_beyond_32_bits():
    """Rows and a matrix of more than 4 GiB each; ends and places around 2^32 bytes are looked at."""
    K, T = 8192, 600_000
    g = torch.Generator(dev).manual_seed(1)
    x = torch.empty(T, K, dtype=torch.bfloat16, device=dev)
    pick = torch.tensor([0, 1, 262143, 262144, 262145, 524287, 524288, 524289, T - 1], device=dev)
    x.zero_()
    x[pick] = torch.randn(len(pick), K, generator=g, device=dev).bfloat16()
    c, f = torch.empty(T, K, dtype=torch.uint8, device=dev), torch.empty(T, K // 32, dtype=torch.uint8, device=dev)
    q.moe_mx_quant(MXFP8, K, T, x, K, c, f)
    check_codes(MXFP8, bits(x[pick]), c[pick].cpu().numpy(), f[pick].cpu().numpy())
    s, o = torch.empty_like(x), torch.empty_like(x)
    w = torch.rand(K, generator=g, device=dev)
    q.moe_add_norm(K, T, x, K, x, K, w, EPS, s, K, o, K)
    h, z = mx_ref.norm(bits(x[pick]), bits(x[pick]), w.cpu().numpy(), EPS)
    assert np.array_equal(bits(s[pick]), h) and np.array_equal(bits(o[pick]), z)
    del s, o
    rng = np.random.default_rng(2)
    m, wv, b = matrix(rng, 24, K)
    y = torch.zeros(T, 24, dtype=torch.bfloat16, device=dev)
    q.moe_mx_linear(m, MXFP8, c, f, T, y, 24, q.MOE_DTYPE_BF16)
    check_product(MXFP8, bits(x[pick]), wv, b, y[pick].double().cpu().numpy(), False, K)
    del x, c, f, y
    torch.cuda.empty_cache()
    N, K = 600_000, 16384
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device=dev)
    scales = torch.full((N, K // 32), 127, dtype=torch.uint8, device=dev)
    pick = torch.tensor([0, 524287, 524288, 524289, N - 17, N - 1], device=dev)
    codes[pick] = torch.randint(0, 256, (len(pick), K // 2), generator=g, device=dev, dtype=torch.int32).to(torch.uint8)
    packed = torch.empty(q.moe_mx_matrix_bytes(N, K), dtype=torch.uint8, device=dev)
    q.moe_mx_pack(N, K, codes, scales, packed)
    cc = codes[pick].cpu().numpy()
    wv = mx_ref.E2M1[np.stack((cc & 15, cc >> 4), -1).reshape(len(pick), K)]
    del codes, scales
    m = q.MxMatrix(N, K, packed.data_ptr(), None)
    for T in (2, 65):
        x = wide(rng, T, K)
        y = torch.empty(T, N, dtype=torch.float32, device=dev)
        cx, sx = mx_ref.quantise(MXFP4, x)
        q.moe_mx_linear(m, MXFP4, torch.from_numpy(mx_ref.pack_codes(MXFP4, cx)).to(dev), torch.from_numpy(sx).to(dev), T, y, N, q.MOE_DTYPE_F32)
        got = y[:, pick].double().cpu().numpy()
        check_product(MXFP4, x, wv, 0.0, got, True, K)
        assert not y[:, 1000:2000].any()


def test_another_stream_and_a_captured_graph():
    """A step's norm, product of its codes, and product of 16-bit rows on a stream of its own and
    in a graph replayed on other inputs between eager calls: the same bits."""
    rng = np.random.default_rng(9)
    H, N = 1024, 700
    m, _, _ = matrix(rng, N, H, bias=True)
    back, _, _ = matrix(rng, H, 768)
    for T in (5, 150):
        x, res = torch.empty(T, H, dtype=torch.bfloat16, device=dev), torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        w = torch.rand(H, device=dev)
        c, f = u8(T, H), u8(T, H // 32)
        y, z, v = (torch.empty(T, n, dtype=torch.bfloat16, device=dev) for n in (704, 768, H))
        nb = q.moe_mx_workspace_bytes(MXFP4, 768, T)
        ws = u8(nb)

        def step(stream=None):
            q.moe_add_norm(H, T, x, H, res, H, w, EPS, res, H, None, H, MXFP8, c, f, stream)
            q.moe_mx_linear(m, MXFP8, c, f, T, y, 704, q.MOE_DTYPE_BF16, stream)
            q.moe_mx_linear_rows(back, MXFP4, z, 768, T, v, H, q.MOE_DTYPE_BF16, ws, nb, stream)

        def fill(seed):
            g = torch.Generator(dev).manual_seed(seed)
            for t in (x, res, z):
                t.copy_(torch.randn(t.shape, generator=g, device=dev))

        def run(call, seed):
            fill(seed)
            torch.cuda.synchronize()
            call()
            torch.cuda.synchronize()
            return [t.clone() for t in (res, y, v, c, f)]

        y.zero_()
        want = [run(step, s) for s in range(4)]
        side = torch.cuda.Stream()
        got = run(lambda: step(side), 1)
        assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
        graph = torch.cuda.CUDAGraph()
        fill(0)
        with torch.cuda.graph(graph):
            step()
        for s in (2, 0, 3, 1):
            got = run(graph.replay, s)
            assert all(torch.equal(a, b) for a, b in zip(got, want[s])), s
            again = run(step, s)
            assert all(torch.equal(a, b) for a, b in zip(again, want[s]))
