"""block_forward over prompts whose keys and values are read back, and with rows and streams as callers
give them: the same bits as its stages called one by one."""
import pytest
import torch

import quantized_expert_ffn_router_amd as q
from attn_ref import BF16, NVFP4, Q8_0
from mx_ref import MXFP4, MXFP8
from test_gpu_attention import FMT, i32
from test_gpu_block import H, N_KV, Model

pytestmark = pytest.mark.gpu

dev = "cuda"


def stages(m, x, T, prompt, chunk):
    """The step's stages on buffers of their own; the cache gets the same tokens once more."""
    w, D, qw = m.blocks[0], m.D, m.n_q * m.D
    attn = q.AttnBuffers(m.caches[0], 2, m.T_max, m.table.shape[1], chunk=True)
    for name in ("row_start", "kv_len", "page_table"):
        getattr(attn, name).copy_(getattr(m.attn, name))
    bf16 = lambda n: torch.empty(T, n, dtype=torch.bfloat16, device=dev)  # noqa: E731
    z, s, qkv, proj, ffn = bf16(H), bf16(H), bf16(w.qkv.N), bf16(H), bf16(H)
    nb = max(q.moe_mx_workspace_bytes(w.fmt, k, T) for k in (H, qw))
    ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    q.moe_add_norm(H, T, x, H, None, 0, w.attn_norm, w.eps, None, 0, z, H)
    q.moe_mx_linear_rows(w.qkv.mat, w.fmt, z, H, T, qkv, w.qkv.N, q.MOE_DTYPE_BF16, ws, nb)
    a = q.attention_forward(m.caches[0], attn, qkv, T, 0.125, prompt, chunk=chunk)
    q.moe_mx_linear_rows(w.out.mat, w.fmt, a, qw, T, proj, H, q.MOE_DTYPE_BF16, ws, nb)
    q.moe_add_norm(H, T, proj, H, x, H, w.ffn_norm, w.eps, s, H, ffn, H)
    out = q.layer_forward(m.experts, q.StepBuffers(m.experts, m.T_max), ffn, T, s)[:T].clone()
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("fmt,row_fmt", [(NVFP4, MXFP8), (Q8_0, MXFP4), (BF16, MXFP8)], ids=lambda v: FMT.get(v, str(v)))
def test_prompts_in_chunks(fmt, row_fmt):
    m = Model(fmt, row_fmt)
    gen = torch.Generator(device=dev).manual_seed(2)
    for rows, read in (((40, 9), True), ((20, 1), True), ((1, 1), False), ((3, 30), True)):
        T = sum(rows)
        m.begin(rows)
        Tk, prompt = sum(m.lens), None
        if read:
            k, v = torch.empty(2, Tk, N_KV * m.D, dtype=torch.bfloat16, device=dev)
            prompt = (i32([0, m.lens[0], Tk]), Tk, k, v)
        x = torch.randn(T, H, generator=gen, device=dev).bfloat16()
        want = stages(m, x, T, prompt, False)
        got = m.run(0, x, T, False, prompt=prompt).clone()
        torch.cuda.synchronize()
        assert torch.equal(got, want), rows


@pytest.mark.parametrize("chunk", [False, True])
def test_rows_given_as_bits_and_as_an_address_on_another_stream(chunk):
    m = Model(NVFP4, MXFP8)
    m.begin((20, 7))
    x = torch.randn(27, H, generator=torch.Generator(device=dev).manual_seed(6), device=dev).bfloat16()
    want = stages(m, x, 27, None, chunk)
    side = torch.cuda.Stream()
    for rows in (x, x.view(torch.int16), x.data_ptr()):
        for stream in (None, side, side.cuda_stream):
            m.step.out.zero_()
            torch.cuda.synchronize()
            got = m.run(0, rows, 27, chunk, stream)
            torch.cuda.synchronize()
            assert torch.equal(got, want)


def test_rows_in_the_layers_own_output():
    """In place: the step reads them before it writes its output there; and where the sum or the
    normed rows of the step before lie."""
    m = Model(Q8_0, MXFP8)
    m.begin((30, 2))
    x = torch.randn(32, H, generator=torch.Generator(device=dev).manual_seed(7), device=dev).bfloat16()
    want = stages(m, x, 32, None, True)
    for t in (m.step.out.view(torch.bfloat16), m.buf.sum, m.buf.z):
        t[:32] = x
        got = m.run(0, t[:32], 32, True).clone()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
