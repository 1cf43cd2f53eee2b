"""block_forward reads its rows twice, before the first norm and as the second one's residual: rows in
a buffer that the step has written by then are refused, others are not."""
import pytest
import torch

import quantized_expert_ffn_router_amd as q
from test_block_checks import H, N_KV, D, T, setup


def view(t):
    """The first rows of a buffer as the step's (buffers narrower than the rows: the first of them)."""
    return t.view(torch.bfloat16).flatten()[:T * H].view(-1, H) if t.numel() * t.element_size() >= 2 * T * H else t.data_ptr()


def buffers(a):
    b, n = a["buf"], a["attn"]
    return dict(qkv=b.qkv, proj=b.proj, ws=b.ws, q=n.q, k=n.k, out=n.out, attn_ws=n.ws)


@pytest.mark.parametrize("name", ["qkv", "proj", "ws", "q", "k", "out", "attn_ws"])
@pytest.mark.parametrize("address", [False, True])
def test_rows_in_a_buffer_of_the_step(name, address):
    a = setup()
    t = buffers(a)[name]
    a["x"] = t.data_ptr() if address else view(t)
    with pytest.raises(q.MoeError, match="x lies in a buffer"):
        q.block_forward(**a)


def test_rows_that_end_in_a_buffer():
    a = setup()
    a["x"] = a["buf"].proj.data_ptr() - 2 * T * H + 16
    with pytest.raises(q.MoeError, match="x lies in a buffer"):
        q.block_forward(**a)


@pytest.mark.parametrize("which", [0, 1])
def test_rows_in_a_prompts_buffers(which):
    a = setup()
    kv = torch.zeros(2, 32, N_KV * D, dtype=torch.bfloat16)
    a.update(prompt=(torch.zeros(3, dtype=torch.int32), 32, kv[0], kv[1]), x=kv[which].view(-1, H)[4:4 + T])
    with pytest.raises(q.MoeError, match="x lies in a buffer"):
        q.block_forward(**a)


def test_rows_elsewhere():
    """The layer's own output, the sum and the normed rows: not refused for where they lie."""
    a = setup()
    for x in (torch.zeros(T, H, dtype=torch.int16), a["buf"].sum, a["buf"].z):
        a["x"] = x
        with pytest.raises(q.MoeError, match="not the current GPU"):
            q.block_forward(**a)
