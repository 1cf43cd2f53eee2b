"""Decode steps over caches long enough for every way in which chunks of a sequence
are joined: 32 to 256 of them, more than were likely for the step, rows of unequal
sequences, and a longest cache understated; against a 64-bit reference on the GPU."""
import math

import pytest
import torch

import attn_pages
import quantized_expert_ffn_router_amd as q
from attn_pages import BF16, NVFP4, Q8_0

pytestmark = pytest.mark.gpu

dev = "cuda"
FMT = {NVFP4: "nvfp4", Q8_0: "q8_0", BF16: "bf16"}
i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731


def check(fmt, n_kv, G, D, P, lens, rows, max_lens=(None,), seed=1):
    gen = torch.Generator(device=dev).manual_seed(seed)
    k_ts, v_ts = (0.75, 1.25) if fmt == NVFP4 else (1.0, 1.0)
    pool, table, kv = attn_pages.make(fmt, n_kv, D, P, lens, gen, dev, k_ts, v_ts)
    assert pool.data_ptr() % 256 == 0
    n_q, T = n_kv * G, sum(rows)
    start = [sum(rows[:b]) for b in range(len(rows) + 1)]
    start_d, len_d, table = i32(start), i32(lens), table.contiguous()
    cache = q.KvCacheDesc(fmt, n_kv, D, P, pool.numel() // q.moe_kv_page_bytes(fmt, n_kv, D, P), k_ts, v_ts, pool.data_ptr())
    seqs = q.SeqBatch(len(lens), table.shape[1], start_d.data_ptr(), len_d.data_ptr(), table.data_ptr())
    x = (1.5 * torch.randn(T, n_q * D, generator=gen, device=dev)).bfloat16()
    scale = D ** -0.5
    for m in max_lens:
        print("long", FMT[fmt], n_kv, G, D, P, lens[:4], rows[:4], "max_len", m, flush=True)
        nb = q.moe_attn_workspace_bytes(cache, n_q, len(lens), T, max(lens) if m is None else m)
        ws = torch.full((max(nb, 1),), 0xff, dtype=torch.uint8, device=dev)
        out = torch.full((T, n_q * D), 7.0, dtype=torch.bfloat16, device=dev)
        q.moe_attn_decode(cache, seqs, n_q, x, n_q * D, T, max(lens) if m is None else m, scale, out, n_q * D, ws, nb)
        for b, (L, n) in enumerate(zip(lens, rows)):
            if n == 0:
                continue
            at = slice(start[b], start[b + 1])
            limit = (L - n + torch.arange(n, device=dev)).repeat_interleave(G)
            for h in range(n_kv):
                cut = lambda t: t[at, h * G * D:(h + 1) * G * D].double().reshape(n * G, D)  # noqa: E731
                # (a wave's share of a chunk is at most 64 units of 32 tokens here)
                want, bound = attn_pages.attend(cut(x), kv[b][0][:, h], kv[b][1][:, h], limit, float(torch.tensor(scale)), fmt, 4096)
                over = (cut(out) - want).abs() / bound
                assert float(over.max()) <= 1, (b, h, m, float(over.max()))


@pytest.mark.parametrize("fmt,D,P", [(NVFP4, 128, 64), (NVFP4, 64, 256), (Q8_0, 128, 32), (BF16, 256, 64)])
@pytest.mark.parametrize("L", [40001, 262144])
def test_decode_one_long_sequence(fmt, D, P, L):
    """Up to 256 chunks of one sequence."""
    if fmt == BF16:
        L = min(L, 131072)
    check(fmt, 1, 2, D, P, [L], [1])


@pytest.mark.parametrize("fmt,n_kv,G,D,P", [
    (NVFP4, 8, 1, 128, 64), (NVFP4, 4, 2, 128, 32), (NVFP4, 4, 8, 64, 64), (Q8_0, 4, 2, 128, 64), (Q8_0, 2, 4, 64, 128),
    (BF16, 4, 1, 64, 64), (BF16, 2, 2, 128, 32), (Q8_0, 1, 4, 256, 64)])
def test_decode_one_long_sequence_among_short_ones(fmt, n_kv, G, D, P):
    """More chunks of it than the step's shape lets expect (33 to 256, also in a
    second round of the join), whatever the longest cache is said to be."""
    for lens, rows in (([33000, 300], [1, 1]), ([100, 60000, 7, 33, 1, 500, 64, 20], [1] * 8), ([90, 41000, 600], [3, 2, 1])):
        check(fmt, n_kv, G, D, P, lens, rows, (None, 2000, 1 << 20))


@pytest.mark.parametrize("fmt,n_kv,G,D,n,short,L,rows", [
    (BF16, 4, 2, 64, 66, 50, 40000, 1), (Q8_0, 4, 2, 128, 66, 50, 40000, 1), (NVFP4, 8, 1, 64, 140, 40, 30000, 1),
    (Q8_0, 8, 2, 256, 16, 60, 20000, 5), (BF16, 8, 1, 64, 70, 33, 9000, 1)])
def test_decode_one_long_sequence_among_many(fmt, n_kv, G, D, n, short, L, rows):
    """Steps whose short sequences alone take more than half, or all, of the GPU."""
    lens = [1 + (short * b) % (2 * short) for b in range(n)]
    lens[n // 2], lens[-1] = L, rows
    check(fmt, n_kv, G, D, 64, lens, [min(rows, x) for x in lens], (None, 1 << 20))


def test_decode_many_rows_of_long_sequences():
    """The work of a step over its workgroups exceeds any one sequence: as many rows
    as are still split, heads enough that few chunks fit beside them."""
    check(BF16, 64, 1, 64, 32, [1500, 8300, 90, 8300], [60, 60, 60, 60], (None, 1 << 20))
    check(NVFP4, 2, 8, 128, 64, [9000, 300, 12000], [300, 200, 350], (None,))
