"""What MxLinear, BlockWeights, block_forward and the chunk steps of attention_forward refuse
before anything reaches the GPU."""
import types

import pytest
import torch

import quantized_expert_ffn_router_amd as q

H, N_Q, N_KV, D, T = 256, 4, 2, 64, 6
WIDTH = (N_Q + 2 * N_KV) * D


def linear(N, K, device="cpu"):
    """An MxLinear's fields without its packing, which runs on the GPU."""
    m = q.MxLinear.__new__(q.MxLinear)
    m.N, m.K, m.device, m.bias = N, K, torch.device(device), None
    m.packed = torch.zeros(q.moe_mx_matrix_bytes(N, K), dtype=torch.uint8)
    m.mat = q.MxMatrix(N, K, m.packed.data_ptr(), None)
    return m


def weights(**kw):
    a = dict(attn_norm=torch.ones(H), qkv=linear(WIDTH, H), out=linear(H, N_Q * D), ffn_norm=torch.ones(H))
    a.update(kw)
    return q.BlockWeights(**a)


def setup(chunk=True):
    w = weights()
    cache = q.KvCache(q.MOE_FMT_NVFP4, N_Q, N_KV, D, 32, 4, device="cpu")
    rows = lambda n: torch.zeros(T, n)  # noqa: E731
    return dict(w=w, layer=types.SimpleNamespace(H=H, E=8, k=2, blobs=torch.zeros(1)), cache=cache,
                buf=q.BlockBuffers(w, T), attn=q.AttnBuffers(cache, 2, T, 2, device="cpu", chunk=chunk),
                step=types.SimpleNamespace(T_max=T, out=rows(H), logits=rows(8), idx=rows(2)),
                x=torch.zeros(T, H, dtype=torch.bfloat16), T=T, scale=0.125)


@pytest.mark.parametrize("weight,scales,bias,msg", [
    (torch.zeros(16, 128), None, None, "bf16"), (torch.zeros(16, 128, dtype=torch.bfloat16)[0], None, None, "contiguous"),
    (torch.zeros(128, 16, dtype=torch.bfloat16).t(), None, None, "contiguous"),
    (torch.zeros(16, 120, dtype=torch.bfloat16), None, None, "K"), (torch.zeros(0, 128, dtype=torch.bfloat16), None, None, "N"),
    (torch.zeros(16, 64, dtype=torch.bfloat16), torch.zeros(16, 4, dtype=torch.uint8), None, "uint8 codes"),
    (torch.zeros(16, 64, dtype=torch.uint8), None, None, "bf16"),
    (torch.zeros(16, 64, dtype=torch.uint8), torch.zeros(16, 2, dtype=torch.uint8), None, "scales must"),
    (torch.zeros(16, 64, dtype=torch.uint8), torch.zeros(16, 4), None, "scales must"),
    (torch.zeros(16, 128, dtype=torch.bfloat16), None, torch.zeros(15), "bias must"),
    (torch.zeros(16, 128, dtype=torch.bfloat16), None, torch.zeros(16, dtype=torch.bfloat16), "bias must"),
    (torch.zeros(16, 128, dtype=torch.bfloat16), None, torch.zeros(16, device="meta"), "bias must"),
    (torch.zeros(16, 128, dtype=torch.bfloat16), None, torch.zeros(16), "not the current GPU"),
])
def test_a_projection_is_checked(weight, scales, bias, msg):
    with pytest.raises(q.MoeError, match=msg):
        q.MxLinear(weight, scales, bias)


@pytest.mark.parametrize("change,msg", [
    (dict(fmt=q.MOE_FMT_Q8_0), "no form of rows"), (dict(out=linear(H + 128, N_Q * D)), "out gives"),
    (dict(attn_norm=torch.ones(H - 1)), "attn_norm"), (dict(ffn_norm=torch.ones(H, dtype=torch.float64)), "ffn_norm"),
    (dict(ffn_norm=torch.ones(2 * H)[::2]), "ffn_norm"), (dict(attn_norm=torch.ones(H, device="meta")), "attn_norm"),
])
def test_block_weights_are_checked(change, msg):
    with pytest.raises(q.MoeError, match=msg):
        weights(**change)


def changed(**kw):
    a = setup()
    for name, v in kw.items():
        a[name] = v(a) if callable(v) else v
    return a


@pytest.mark.parametrize("change,msg", [
    (dict(T=T + 1), "T=7"), (dict(T=-1), "T=-1"), (dict(x=torch.zeros(T, H)), "x must be bf16"),
    (dict(x=torch.zeros(T - 1, H, dtype=torch.bfloat16)), "x has"),
    (dict(x=torch.zeros(T, 2 * H, dtype=torch.bfloat16)[:, :H]), "contiguous"),
    (dict(x=torch.zeros(T, H, dtype=torch.bfloat16, device="meta")), "x is on meta"),
    (dict(layer=types.SimpleNamespace(H=2 * H, E=8, k=2, blobs=torch.zeros(1))), "experts' rows"),
    (dict(layer=types.SimpleNamespace(H=H, E=16, k=2, blobs=torch.zeros(1))), "another layer"),
    (dict(layer=types.SimpleNamespace(H=H, E=8, k=2, blobs=torch.zeros(1, device="meta"))), "experts are on meta"),
    (dict(cache=q.KvCache(q.MOE_FMT_NVFP4, N_Q, N_KV, 128, 32, 4, device="cpu")), "heads"),
    (dict(buf=lambda a: q.BlockBuffers(weights(fmt=q.MOE_FMT_MXFP4), T)), "other weights"),
    (dict(buf=lambda a: q.BlockBuffers(a["w"], T - 1)), "buffers of 5"),
    (dict(), "not the current GPU"), (dict(chunk=True), "not the current GPU"),
])
def test_a_step_is_checked(change, msg):
    with pytest.raises(q.MoeError, match=msg):
        q.block_forward(**changed(**change))


def test_chunk_steps_need_their_buffers():
    c = q.KvCache(q.MOE_FMT_NVFP4, N_Q, N_KV, D, 32, 4, device="cpu")
    qkv = torch.zeros(T, WIDTH, dtype=torch.bfloat16)
    with pytest.raises(q.MoeError, match="without chunk=True"):
        q.attention_forward(c, q.AttnBuffers(c, 2, T, 2, device="cpu"), qkv, T, 0.125, chunk=True)
    kv = (torch.zeros(3, dtype=torch.int32), 8, *torch.zeros(2, 8, N_KV * D, dtype=torch.bfloat16))
    buf = q.AttnBuffers(c, 2, T, 2, device="cpu", chunk=True)
    with pytest.raises(q.MoeError, match="no prompt"):
        q.attention_forward(c, buf, qkv, T, 0.125, kv, chunk=True)
    assert buf.ws.numel() >= max(buf.ws_bytes, buf.chunk_bytes)


@pytest.mark.parametrize("n_seq,T_max,pages", [(1, 1, 1), (3, 4096, 40), (64, 600, 300)])
def test_chunk_buffers_hold_every_smaller_step(n_seq, T_max, pages):
    for fmt, n_q, n_kv, d in ((q.MOE_FMT_NVFP4, 32, 4, 128), (q.MOE_FMT_Q8_0, 5, 5, 64), (q.MOE_FMT_BF16, 8, 1, 256)):
        c = q.KvCache(fmt, n_q, n_kv, d, 32, 1, device="cpu")
        whole = q.moe_attn_chunk_workspace_bytes(c.desc, n_q, n_seq, T_max, 32 * pages)
        for t in {1, T_max // 3, T_max - 1, T_max}:
            for m in (1, 32 * pages // 2, 32 * pages):
                if t > 0:
                    assert q.moe_attn_chunk_workspace_bytes(c.desc, n_q, n_seq, t, m) <= whole
