"""What the binding's attention classes and calls refuse before anything reaches
the GPU: sizes, types, layouts and devices that do not fit."""
import numpy as np
import pytest
import torch

import quantized_expert_ffn_router_amd as q

N_Q, N_KV, D, ROWS = 8, 2, 64, 6


def setup(n_seq=2, **kw):
    c = q.KvCache(q.MOE_FMT_NVFP4, N_Q, N_KV, D, 32, 4, device="cpu", **kw)
    return c, q.AttnBuffers(c, n_seq, ROWS, 2, device="cpu")


def rows(n, heads, dtype=torch.bfloat16):
    return torch.zeros(n, heads * D, dtype=dtype)


@pytest.mark.parametrize("name", ["q_norm", "k_norm"])
@pytest.mark.parametrize("n", [0, 1, D - 1, D + 1, 2 * D])
def test_norm_weights_are_as_many_as_a_head_has_elements(name, n):
    with pytest.raises(q.MoeError, match=f"{name} has {n} weights"):
        setup(**{name: np.ones(n)})
    c, _ = setup(**{name: torch.ones(D, dtype=torch.float64)})
    assert getattr(c, name).dtype == torch.float32


@pytest.mark.parametrize("qkv,msg", [
    (rows(ROWS - 1, 12), "qkv has"), (rows(ROWS, 11), "qkv has"), (rows(ROWS, 12, torch.float32), "bf16"),
    (rows(ROWS, 12, torch.float16), "bf16"), (rows(ROWS, 13)[:, :12 * D], "contiguous"),
    (rows(12 * D, 1)[:, :ROWS].t(), "contiguous"), (rows(ROWS, 12).to("meta"), "is on meta"),
])
@pytest.mark.parametrize("prompt", [False, True])
def test_projections_must_fit(qkv, msg, prompt):
    c, buf = setup()
    kv = (torch.zeros(3, dtype=torch.int32), 20, rows(20, N_KV), rows(20, N_KV)) if prompt else None
    with pytest.raises(q.MoeError, match=msg):
        q.attention_forward(c, buf, qkv, ROWS, 0.125, kv)


@pytest.mark.parametrize("change,msg", [
    (dict(start=torch.zeros(2, dtype=torch.int32)), "kv_start"), (dict(start=torch.zeros(3, dtype=torch.int64)), "kv_start"),
    (dict(start=torch.zeros(3, 2, dtype=torch.int32)[:, 0]), "kv_start"), (dict(k=rows(20, N_KV, torch.float32)), "k must"),
    (dict(v=rows(20, N_KV, torch.float16)), "v must"), (dict(k=rows(20, 2 * N_KV)[:, :N_KV * D]), "k must"),
    (dict(v=rows(19, N_KV)), "Tk=20"), (dict(v=rows(20, N_KV).to("meta")), "v is on meta"),
])
def test_prompt_arguments_must_fit(change, msg):
    c, buf = setup()
    a = dict(start=torch.zeros(3, dtype=torch.int32), k=rows(20, N_KV), v=rows(20, N_KV))
    a.update(change)
    with pytest.raises(q.MoeError, match=msg):
        q.attention_forward(c, buf, rows(ROWS, 12), ROWS, 0.125, (a["start"], 20, a["k"], a["v"]))


def test_buffers_of_another_cache_are_refused():
    c, _ = setup()
    for n_q, n_kv, d in ((16, 2, 64), (8, 4, 64), (8, 2, 128), (4, 1, 64)):
        other = q.KvCache(q.MOE_FMT_NVFP4, n_q, n_kv, d, 32, 4, device="cpu")
        with pytest.raises(q.MoeError, match="buffers for heads"):
            q.attention_forward(c, q.AttnBuffers(other, 2, ROWS, 2, device="cpu"), rows(ROWS, 12), ROWS, 0.125)


def test_a_step_without_rows_passes_the_checks():
    """(The library launches nothing for it, so the pool is never read.)"""
    c, buf = setup()
    c.desc.pool = (c.desc.pool + 255) & ~255
    for qkv in (rows(0, 12), rows(ROWS, 12), rows(ROWS, 12).view(torch.int16)):
        assert q.attention_forward(c, buf, qkv, 0, 0.125, stream=0) is buf.out


def test_a_cache_that_is_not_on_the_current_gpu_is_refused(monkeypatch):
    """Host memory, buffers elsewhere, and another GPU than the current one."""
    c, buf = setup()
    with pytest.raises(q.MoeError, match="the cache is on cpu"):
        q.attention_forward(c, buf, rows(ROWS, 12), ROWS, 0.125)
    with pytest.raises(q.MoeError, match="buffers on meta"):
        q.attention_forward(c, q.AttnBuffers(c, 2, ROWS, 2, device="meta"), rows(ROWS, 12), ROWS, 0.125)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert q._launches_on(torch.device("cuda", 0), None) and not q._launches_on(torch.device("cuda", 1), None)
    assert q._launches_on(torch.device("cuda", 1), 0x1000) and not q._launches_on(torch.device("cpu"), 0x1000)
