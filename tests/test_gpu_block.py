"""The norm, the projections, the cache, the attention and the experts together, as a step of a
layer uses them: block_forward and attention_forward's chunk steps, each stage against the
64-bit reference of what the stage before it left, over prompts in chunks, mixed steps and
decode steps, eager and captured.

Bounds: codes, sums and normed rows bit for bit; products within mx_ref.product_bound;
attention within attn_ref.attend_bound (decode) or test_gpu_chunk.chunk_bound (chunks); the
experts bit for bit what layer_forward gives for the same rows."""
import math

import numpy as np
import pytest
import torch

import attn_ref as ref
import moegen
import mx_ref
import quantized_expert_ffn_router_amd as q
from attn_ref import BF16, NVFP4, Q8_0
from mx_ref import MXFP4, MXFP8
from test_gpu_attention import FMT, bits, i32, to_dev
from test_gpu_chunk import chunk_bound
from test_gpu_norm_linear import tops

pytestmark = pytest.mark.gpu

dev = "cuda"
H, N_Q, N_KV, P = 512, 8, 2, 32


class Model:
    """L layers, their caches and buffers for two sequences."""

    def __init__(self, fmt, row_fmt, D=64, L=1, T_max=64, pages=6, n_q=N_Q):
        rng = np.random.default_rng(D + fmt + row_fmt)
        self.D, self.n_q, self.fmt, self.row_fmt, self.T_max = D, n_q, fmt, row_fmt, T_max
        qw, kw = n_q * D, N_KV * D
        self.experts = q.DeviceLayer(moegen.make_layer(moegen.Workload("block", E=8, k=2, H=H, I=128, T=T_max)))
        self.blocks, self.host = [], []
        rope = q.moe_rope_freqs(q.MOE_ROPE_PLAIN, D, 10000.0)
        for _ in range(L):
            mats, host = [], []
            for N, K in ((qw + 2 * kw, H), (H, qw)):
                w = ref.bf16_bits(rng.standard_normal((N, K)) / math.sqrt(K))
                b = (0.1 * rng.standard_normal(N)).astype(np.float32)
                c, s = mx_ref.quantise(MXFP4, w)
                # one matrix from its values, one from its codes
                lin = q.MxLinear(to_dev(w), bias=torch.from_numpy(b).to(dev)) if not mats else q.MxLinear(
                    torch.from_numpy(mx_ref.pack_codes(MXFP4, c)).to(dev), torch.from_numpy(s).to(dev),
                    torch.from_numpy(b).to(dev))
                mats.append(lin)
                host.append((mx_ref.values(MXFP4, c, s), b.astype(np.float64)))
            norms = [rng.uniform(0.5, 1.5, H).astype(np.float32) for _ in range(2)]
            a, f = (torch.from_numpy(n).to(dev) for n in norms)
            self.blocks.append(q.BlockWeights(a, mats[0], mats[1], f, 1e-5, row_fmt))
            self.host.append((host, norms))
        self.caches = [q.KvCache(fmt, n_q, N_KV, D, P, 2 * pages, np.ones(D), np.ones(D), rope) for _ in range(L)]
        self.table = i32(np.random.default_rng(5).permutation(2 * pages).reshape(2, pages))
        self.buf = q.BlockBuffers(self.blocks[0], T_max)
        self.step = q.StepBuffers(self.experts, T_max)
        self.attn = q.AttnBuffers(self.caches[0], 2, T_max, pages, chunk=True)
        self.attn.page_table.copy_(self.table)
        self.lens = [0, 0]

    def begin(self, rows):
        self.lens = [n + r for n, r in zip(self.lens, rows)]
        self.attn.row_start.copy_(i32(np.concatenate([[0], np.cumsum(rows)])))
        self.attn.kv_len.copy_(i32(self.lens))

    def run(self, l, x, T, chunk, stream=None, **kw):
        return q.block_forward(self.blocks[l], self.experts, self.caches[l], self.buf, self.attn, self.step, x, T,
                               1 / math.sqrt(self.D), stream=stream, chunk=chunk, **kw)[:T]


def product(fmt, c, s, w, b, got):
    a = mx_ref.values(fmt, c, s)
    y, ab = a @ w.T + b, np.abs(a) @ np.abs(w).T + np.abs(b)
    assert (np.abs(got - y) <= mx_ref.product_bound(fmt, y, ab, tops(a, w), a.shape[1], False)).all()


def check_stages(m, l, x, rows, T, chunk, out):
    """Every stage of the step that just ran, from what the buffers hold."""
    host = lambda t: bits(t[:T])  # noqa: E731
    (wq, wo), (n1, n2) = m.host[l]
    fmt, b, D = m.row_fmt, m.buf, m.D
    _, z = mx_ref.norm(x, None, n1, 1e-5)
    c, s = mx_ref.quantise(fmt, z)
    assert np.array_equal(b.codes[:T].cpu().numpy(), mx_ref.pack_codes(fmt, c))
    assert np.array_equal(b.scales[:T].cpu().numpy(), s)
    product(fmt, c, s, *wq, ref.bf16_val(host(b.qkv)))
    # attention over what the cache holds, from the rows that the cache's write left in attn.q
    Tk = sum(m.lens)
    start = np.concatenate([[0], np.cumsum(m.lens)])
    kv = [torch.empty(Tk, N_KV * D, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    q.moe_kv_read(m.caches[l].desc, m.attn.seqs, None, i32(start), Tk, kv[0], N_KV * D, kv[1], N_KV * D)
    k, v = (ref.bf16_val(bits(t)).reshape(Tk, N_KV, D) for t in kv)
    qs, o = ref.bf16_val(host(m.attn.q)), ref.bf16_val(host(m.attn.out))
    scale, t = float(np.float32(1 / math.sqrt(D))), 0
    for i, n in enumerate(rows):
        for r in range(n):
            for h in range(m.n_q):
                col, kvh = slice(h * D, h * D + D), h // (m.n_q // N_KV)
                lim = m.lens[i] - n + r
                span = slice(start[i], start[i + 1])
                want, pv, qk = ref.attend(qs[t, col], k[span, kvh], v[span, kvh], lim, scale)
                vmax = float(np.abs(v[span, kvh]).max())
                bound = (chunk_bound(m.fmt, want, pv, qk, D, lim + 1, vmax) if chunk
                         else ref.attend_bound(want, pv, qk, lim + 1, vmax, D, m.fmt))
                if m.fmt == Q8_0:  # (what is read back is rounded to bf16, 2^-8: the values and, in the scores, the keys)
                    bound = bound + pv * (2.0 ** -8 + 2 * math.expm1(min(qk * 2.0 ** -8, 1.0))) * (1 + 2.0 ** -6)
                assert (np.abs(o[t, col] - want) <= bound).all(), (i, r, h)
            t += 1
    c, s = mx_ref.quantise(fmt, host(m.attn.out))
    product(fmt, c, s, *wo, ref.bf16_val(host(b.proj)))
    hsum, z = mx_ref.norm(host(b.proj), x, n2, 1e-5)
    assert np.array_equal(host(b.sum), hsum) and np.array_equal(host(b.z), z)
    other = q.StepBuffers(m.experts, m.T_max)
    want = q.layer_forward(m.experts, other, b.z, T, b.sum)[:T]
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))


STEPS = [((37, 0), True), ((20, 9), True), ((1, 30), True), ((1, 1), False), ((2, 1), True), ((3, 1), False),
         ((0, 1), False), ((1, 0), True)]


@pytest.mark.parametrize("fmt,row_fmt,D,n_q", [(NVFP4, MXFP8, 64, 8), (Q8_0, MXFP8, 128, 8), (BF16, MXFP8, 64, 2),
                                               (NVFP4, MXFP4, 128, 16), (Q8_0, MXFP4, 256, 4)],
                         ids=lambda v: FMT.get(v, str(v)))
def test_stages_of_a_step(fmt, row_fmt, D, n_q):
    m = Model(fmt, row_fmt, D, L=2, n_q=n_q)
    gen = torch.Generator(device=dev).manual_seed(D)
    for rows, chunk in STEPS:
        print("step", rows, chunk, flush=True)
        T = sum(rows)
        m.begin(rows)
        x = torch.randn(T, H, generator=gen, device=dev).bfloat16()
        for l in range(2):
            xin = bits(x)
            out = m.run(l, x, T, chunk)
            torch.cuda.synchronize()
            out = out.clone()
            check_stages(m, l, xin, rows, T, chunk, out)
            x = m.step.out[:T]  # as it is used: the next layer reads what this one wrote
            assert torch.equal(x, out)


@pytest.mark.parametrize("chunk", [False, True])
@pytest.mark.parametrize("keep_y", [False, True])
def test_step_captured_and_replayed(chunk, keep_y):
    """A step of two layers in a graph: each replay, with other rows and longer sequences, gives what
    the eager calls give, bit for bit; eager work in between; another graph of the same weights."""
    rows, start = (1, 1) if not chunk else (9, 1), (40, 25)
    T = sum(rows)
    m = Model(NVFP4, MXFP8, L=2)
    gen = torch.Generator(device=dev).manual_seed(3)
    m.begin(start)
    prompt = torch.randn(sum(start), H, generator=gen, device=dev).bfloat16()
    m2 = q.StepBuffers(m.experts, 80)
    x = prompt
    b80 = q.BlockBuffers(m.blocks[0], 80)
    a80 = q.AttnBuffers(m.caches[0], 2, 80, 6, chunk=True)
    for name in ("row_start", "kv_len", "page_table"):
        getattr(a80, name).copy_(getattr(m.attn, name))
    for l in range(2):
        x = q.block_forward(m.blocks[l], m.experts, m.caches[l], b80, a80, m2, x, 65, 0.125, chunk=True)[:65].clone()
    held = torch.zeros(T, H, dtype=torch.bfloat16, device=dev)

    def both(stream=None):
        out = m.run(0, held, T, chunk, stream, keep_y=keep_y)
        return m.run(1, out, T, chunk, stream, keep_y=keep_y)

    m.begin(rows)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        both(side)
    for turn in range(4):
        if turn:
            m.begin(rows)
        held.copy_(torch.randn(T, H, generator=gen, device=dev).bfloat16())
        torch.cuda.synchronize()
        m.step.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = m.step.out[:T].clone()
        want = both().clone()  # (writes the same tokens into the caches again)
        torch.cuda.synchronize()
        assert torch.isfinite(got.view(torch.bfloat16).float()).all()
        assert torch.equal(got, want), turn


def test_two_streams_of_steps_at_once():
    """Two sets of buffers and caches on two streams, the weights shared: as one after the other."""
    m = [Model(NVFP4, MXFP8), Model(NVFP4, MXFP8)]
    gen = torch.Generator(device=dev).manual_seed(9)
    xs = [torch.randn(40, H, generator=gen, device=dev).bfloat16() for _ in m]
    want = []
    for s, x in zip(m, xs):
        s.begin((30, 10))
        want.append(s.run(0, x, 40, True).clone())
    torch.cuda.synchronize()
    m[1].blocks = m[0].blocks  # (the same seed: the same weights)
    streams = [torch.cuda.Stream() for _ in m]
    for _ in range(5):
        got = []
        for s, x, st in zip(m, xs, streams):
            s.step.out.zero_()
        torch.cuda.synchronize()
        for s, x, st in zip(m, xs, streams):
            got.append(s.run(0, x, 40, True, st))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
def test_chunk_steps_of_attention_forward(fmt):
    """A prompt's chunks straight over the cache against the same chunks with the keys and values
    read back, and the rows behind the step's are left as they were."""
    D, n_q, kw = 128, 8, N_KV * 128
    gen = torch.Generator(device=dev).manual_seed(4)
    qkv = torch.randn(150, (n_q + 2 * N_KV) * D, generator=gen, device=dev).bfloat16()
    outs, lens = [], []
    for chunk in (True, False):
        cache = q.KvCache(fmt, n_q, N_KV, D, P, 5, np.ones(D), np.ones(D))
        buf = q.AttnBuffers(cache, 1, 100, 5, chunk=True)
        buf.page_table.copy_(i32([[4, 0, 3, 1, 2]]))
        at = 0
        for n in (100, 1, 49):
            buf.row_start.copy_(i32([0, n]))
            buf.kv_len.copy_(i32([at + n]))
            buf.out.fill_(7.0)
            at += n
            kv = [torch.empty(at, kw, dtype=torch.bfloat16, device=dev) for _ in range(2)]
            prompt = None if chunk else (i32([0, at]), at, *kv)
            o = q.attention_forward(cache, buf, qkv[at - n:at], n, D ** -0.5, prompt, chunk=chunk)
            torch.cuda.synchronize()
            assert (o[n:] == 7.0).all()
            outs.append(o[:n].double())
            lens.append(kv)
    one, two = torch.cat(outs[:3]), torch.cat(outs[3:])
    v = lens[-1][1].double().view(150, N_KV, 1, D).abs().amax(0).expand(-1, n_q // N_KV, -1).reshape(-1)
    # each rounds its weights to 2^-8 or finer, in numerator and denominator, and the result
    # (2^-8); scores of normed keys and queries: |s| <= D^1/2, fp32 sums of D products, D 2^-24
    # of it; Q8_0 keys and values: rounded to 2^-8 or finer; sum p|v| is at most the largest |v|
    e_kv = 2.0 ** -8 if fmt == Q8_0 else 0.0
    w = 2.0 ** -7 + e_kv + 2 * math.expm1(D ** 0.5 * 1.02 * (D * 2.0 ** -24 + e_kv)) + 2.0 ** -20 + 150 * 2.0 ** -24
    assert ((one - two).abs() <= 2 * (w + 2.0 ** -8 * (1 + w)) * v).all()


def test_a_step_without_rows_changes_nothing():
    m = Model(NVFP4, MXFP8)
    x = torch.zeros(4, H, dtype=torch.bfloat16, device=dev)
    for chunk in (False, True):
        q.attention_forward(m.caches[0], m.attn, m.buf.qkv, 0, 0.125, chunk=chunk)
    pool, m.buf.qkv[:] = m.caches[0].pool.clone(), 7.0
    q.moe_add_norm(H, 0, x, H, None, 0, m.blocks[0].attn_norm, 1e-5, None, 0, x, H)
    q.moe_mx_linear_rows(m.blocks[0].out.mat, MXFP8, m.attn.out, m.n_q * m.D, 0, m.buf.qkv, m.buf.qkv.shape[1],
                         q.MOE_DTYPE_BF16, m.buf.ws, m.buf.ws_bytes)
    torch.cuda.synchronize()
    assert torch.equal(m.caches[0].pool, pool) and (m.buf.qkv == 7.0).all() and (x == 0).all()
