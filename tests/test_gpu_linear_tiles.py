"""moe_mx_linear and moe_mx_linear_rows at every tile and cut of their rule (linear_rule.py, checked
against the source on the CPU), against 64 bits and closer than mx_ref.product_bound.

Bound of an fp32 result, from what include/moe.h states.  8-bit rows: among 8 neighbouring products
(elements 8i..8i+7, one block each) let 2^E be the largest sum of the exponents of a product's two
factors; each product is cut to a multiple of 2^(E - 13).  One that is such a multiple loses nothing,
another less than 2^(E - 13): the bound counts the latter.  What is left of 8 products are
multiples of 2^(E - 13) below 2^(E + 2) each, whose sum below 2^(E + 5) has 18 bits: exact in fp32.  4-bit
rows: products between 1/4 and 36 are multiples of 2^-2 and nothing is cut.  The groups' sums are then
added in fp32, K / 8 additions and up to 17 more (the parts of 16 waves, the bias), each off by 2^-24 of
a partial sum if it is rounded and by 2^-23 if it is cut; a partial sum is at most the sum of |a||w|.
bf16: half a step more, 2^-8 of the value.

The same norm over norm: cuts as above, and additions whose errors are as good as independent,
2^-23 of partial sums that are as large as the products' own sum is expected to be, the root of the
sum of their squares: 2^-23 (K / 8 + 17)^1/2 of that."""
import pytest
import torch

import mx_ref
import quantized_expert_ffn_router_amd as q
from linear_rule import FEW, MANY
from mx_ref import MXFP4, MXFP8

pytestmark = pytest.mark.gpu

dev = "cuda"


def pow2(k):
    """2^k in float64, exactly."""
    return ((k.long() + 1023) << 52).view(torch.float64)


class Rows:
    """Normal rows in a microscaled format: codes and scales as the library makes them, and the codes'
    values and exponents from mx_ref's tables, without the library."""

    def __init__(self, fmt, T, K, gen, size=1.0):
        self.x = (size * torch.randn(T, K, generator=gen, device=dev)).bfloat16()
        self.fmt, self.T, self.K = fmt, T, K
        self.codes = torch.empty(T, K // 2 if fmt == MXFP4 else K, dtype=torch.uint8, device=dev)
        self.scales = torch.empty(T, K // 32, dtype=torch.uint8, device=dev)
        q.moe_mx_quant(fmt, K, T, self.x, K, self.codes, self.scales)

    def unpack(self):
        c = self.codes
        if self.fmt == MXFP4:
            c = torch.stack((c & 15, c >> 4), -1).flatten(-2)
        table = mx_ref.E2M1 if self.fmt == MXFP4 else mx_ref.e4m3_value(range(256))
        c, power = c.int(), (self.scales.int() - 127).repeat_interleave(32, -1)
        # (a subnormal code, or 0, has the smallest exponent)
        e = ((c >> 1) & 3).clamp(min=1) - 1 if self.fmt == MXFP4 else ((c >> 3) & 15).clamp(min=1) - 7
        return torch.from_numpy(table).to(dev)[c] * pow2(power), e + power


def matrix(N, K, gen, bias):
    w = Rows(MXFP4, N, K, gen, 0.05)
    m = q.MxLinear(w.codes, w.scales, torch.randn(N, generator=gen, device=dev) if bias else None)
    return m, *w.unpack(), 0.0 if m.bias is None else m.bias.double()


def exact(a, w, bias):
    """The product, the sums of |a||w| and of (a w)^2, float64."""
    y = a @ w.t().contiguous() + bias
    ab = a.abs() @ w.abs().t().contiguous() + (bias.abs() if torch.is_tensor(bias) else 0.0)
    return y, ab, a.square() @ w.square().t().contiguous()


def cuts(a, ea, w, ew):
    """What 8-bit rows may lose in each product, float64 [T, N]."""
    out = torch.zeros(len(a), len(w), dtype=torch.float64, device=dev)
    step = max(1, (1 << 25) // len(w))
    for t in range(0, len(a), step):
        r = slice(t, t + step)
        for j in range(0, a.shape[1], 8):
            e = (ea[r, None, j:j + 8] + ew[None, :, j:j + 8]).amax(-1) - 13
            p = a[r, None, j:j + 8] * w[None, :, j:j + 8] * pow2(-e)[..., None]
            out[r] += (p != p.round()).sum(-1) * pow2(e)
    return out


def run(m, rows, f32, as_rows=False):
    """-> [T, N] float64; nothing beside the results is written."""
    T, N, K = rows.T, m.N, rows.K
    stride = (N + 7) // 8 * 8 + 8
    y = torch.full((T + 1, stride), 9.0, dtype=torch.float32 if f32 else torch.bfloat16, device=dev)
    dt = q.MOE_DTYPE_F32 if f32 else q.MOE_DTYPE_BF16
    if as_rows:
        nb = q.moe_mx_workspace_bytes(rows.fmt, K, T)
        ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device=dev)
        q.moe_mx_linear_rows(m.mat, rows.fmt, rows.x, K, T, y, stride, dt, ws, nb)
    else:
        q.moe_mx_linear(m.mat, rows.fmt, rows.codes, rows.scales, T, y, stride, dt)
    torch.cuda.synchronize()
    assert (y[T] == 9.0).all() and (y[:T, N:] == 9.0).all()
    return y[:T, :N].double()


def check(m, w, ew, bias, rows, as_rows):
    a, ea = rows.unpack()
    y, ab, squares = exact(a, w, bias)
    lost = cuts(a, ea, w, ew) if rows.fmt == MXFP8 else torch.zeros_like(y)
    adds = rows.K / 8 + 17
    bound = lost + adds * 2.0 ** -23 * ab
    got = run(m, rows, True)
    over = float(((got - y).abs() / bound).max())
    assert over <= 1, over
    whole = float((got - y).norm() / y.norm())
    allowed = float((lost.norm() + 2.0 ** -23 * adds ** 0.5 * squares.sum().sqrt()) / y.norm())
    print(f"    worst {over:.3f} of the bound; norm over norm {whole:.2e} of {allowed:.2e}", flush=True)
    assert whole <= allowed
    half = run(m, rows, False)
    assert bool(((half - y).abs() <= bound + (y.abs() + bound) * 2.0 ** -8).all())
    if as_rows:  # quantised on the way: the same bit for bit
        assert torch.equal(run(m, rows, True, True), got) and torch.equal(run(m, rows, False, True), half)


@pytest.mark.parametrize("fmt", [MXFP4, MXFP8], ids=["4 bits", "8 bits"])
@pytest.mark.parametrize("tile", MANY, ids=lambda t: f"{t[0]}x{t[1]}")
def test_every_tile(tile, fmt):
    T, N, K = MANY[tile]
    print("tile", tile, T, N, K, fmt, flush=True)
    gen = torch.Generator(dev).manual_seed(T)
    m, w, ew, bias = matrix(N, K, gen, bias=True)
    check(m, w, ew, bias, Rows(fmt, T, K, gen), T < 1000)


@pytest.mark.parametrize("fmt", [MXFP4, MXFP8], ids=["4 bits", "8 bits"])
@pytest.mark.parametrize("cut", FEW, ids=lambda c: "{} steps, {} passes, {}".format(*c))
def test_every_cut_of_few_rows(cut, fmt):
    N, K = FEW[cut]
    print("few", cut, N, K, fmt, flush=True)
    gen = torch.Generator(dev).manual_seed(N)
    m, w, ew, bias = matrix(N, K, gen, bias=N % 2 == 1)
    for T in (1, 5, 16):
        check(m, w, ew, bias, Rows(fmt, T, K, gen), True)


def test_norm_over_norm_of_8_bit_rows():
    """The cut of 8-bit products costs a few 1e-6 of the result; 4-bit rows, nothing."""
    gen = torch.Generator(dev).manual_seed(4)
    m, w, ew, bias = matrix(2000, 2048, gen, False)
    err = {}
    for fmt in (MXFP4, MXFP8):
        for T in (16, 300):
            rows = Rows(fmt, T, 2048, gen)
            y = exact(rows.unpack()[0], w, bias)[0]
            err[fmt, T] = float((run(m, rows, True) - y).norm() / y.norm())
    print(err, flush=True)
    assert max(err[MXFP8, 16], err[MXFP8, 300]) <= 2e-5 and max(err[MXFP4, 16], err[MXFP4, 300]) <= 2e-6


@pytest.mark.parametrize("T", [3, 40, 300])
def test_a_nan_code(T):
    """E4M3 has codes for NaN, too: a row that holds one is NaN, no other."""
    gen = torch.Generator(dev).manual_seed(T)
    m, w, _, bias = matrix(77, 1152, gen, True)
    rows = Rows(MXFP8, T, 1152, gen)
    want = run(m, rows, True)
    rows.codes[1, 700], rows.codes[2, 3] = 0x7F, 0xFF
    got = run(m, rows, True)
    assert bool(got[1:3].isnan().all())
    keep = torch.arange(T, device=dev).sub(1.5).abs() > 1
    assert torch.equal(got[keep], want[keep])
