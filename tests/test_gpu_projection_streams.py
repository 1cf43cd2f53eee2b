"""MxLinear on a stream of its own, beside work that the current stream has not done yet."""
import pytest
import torch

import quantized_expert_ffn_router_amd as q

pytestmark = pytest.mark.gpu

dev = "cuda"
N, K = 1000, 2048


def keep_busy():
    """Some milliseconds of work on the current stream."""
    a = torch.full((4096, 4096), 0.01, dtype=torch.bfloat16, device=dev)
    for _ in range(60):
        a = (a @ a).tanh_()


def rows(seed):
    return torch.randn(N, K, generator=torch.Generator(dev).manual_seed(seed), device=dev).bfloat16()


def plain(w):
    m = q.MxLinear(w)
    torch.cuda.synchronize()
    return m.packed.clone()


def test_weights_that_are_still_being_written():
    src = rows(1)
    want, side = plain(src), torch.cuda.Stream()
    weight = torch.zeros_like(src)
    torch.cuda.synchronize()
    keep_busy()
    weight.copy_(src)
    assert torch.equal(q.MxLinear(weight, stream=side).packed, want)


def test_memory_that_is_still_being_used():
    """Blocks that the allocator hands out again are written by the current stream until then."""
    src = rows(2)
    want, side = plain(src), torch.cuda.Stream()
    late = [torch.empty(n, dtype=torch.uint8, device=dev) for n in (len(want), N * K // 2, N * K // 32)]
    torch.cuda.synchronize()
    keep_busy()
    for t in late:
        t.fill_(0xAA)
    del late, t
    m = q.MxLinear(src, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(m.packed, want)


def test_raw_handles():
    src = rows(3)
    want, side = plain(src), torch.cuda.Stream()
    for handle in (side.cuda_stream, torch.cuda.current_stream().cuda_stream, 0):
        weight = torch.zeros_like(src)
        torch.cuda.synchronize()
        keep_busy()
        weight.copy_(src)
        assert torch.equal(q.MxLinear(weight, stream=handle).packed, want)
