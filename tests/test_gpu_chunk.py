"""moe_attn_chunk against the 64-bit references in attn_ref.py and attn_pages.py: every cache
format and head size, groups of heads that do and do not divide a tile, one row to many,
lengths around tiles, halves and pages, sequences split and not, rows that see nothing,
tokens that rows do not see holding NaN or infinity, bad pages, claims that do not fit,
strides, in-place outputs, long caches, other streams and captured graphs.

Bound: half a step of the bf16 result, 2^-8 of it; the weights' rounding, 2^-11 each (16-bit
caches: to bf16, 2^-8), in numerator and denominator; Q8_0 keys and values rounded once to
fp16, 2^-11 of a value and of sum |q||k| in a score; fp32 sums over D in a score (D 2^-24 of
sum |q||k|) and over the tokens; 2^-20 for exponentials and the division.  fp16 weights are
held to 2^7 or more for the largest: one below 2^-14 is off by 2^-25, 2^-32 of the sum, in
numerator and denominator."""
import math

import numpy as np
import pytest
import torch

import attn_pages
import attn_ref as ref
import quantized_expert_ffn_router_amd as q
from attn_ref import BF16, NVFP4, Q8_0
from test_gpu_attention import FMT, Setup, bits, i32, to_dev
from test_gpu_attention_edges import starts_before_row_0

pytestmark = pytest.mark.gpu

dev = "cuda"


def chunk_bound(fmt, want, pv, qk, D, n_tok, v_max):
    """Works on arrays and on tensors."""
    e_p = 2.0 ** -8 if fmt == BF16 else 2.0 ** -11
    e_kv = 2.0 ** -11 if fmt == Q8_0 else 0.0
    tiny = 0.0 if fmt == BF16 else n_tok * 2.0 ** -31 * v_max
    w = 2 * e_p + e_kv + 2 * math.expm1(min(qk * (D * 2.0 ** -24 + e_kv), 1.0)) + 2.0 ** -20 + n_tok * 2.0 ** -24
    return abs(want) * 2.0 ** -8 * (1 + w) + (pv * w + tiny) * (1 + 2.0 ** -8) + 1e-30


def run_chunk(s, n_q, qv, max_len=None, out=None, stride=None, stream=None):
    """qv: bf16 bits [T, n_q * D]; returns bf16 bits."""
    w = n_q * s.D
    stride = stride or w
    qd = torch.zeros(s.T, stride, dtype=torch.bfloat16, device=dev)
    qd[:, :w] = to_dev(qv)
    out = torch.full((s.T, stride), 7.0, dtype=torch.bfloat16, device=dev) if out is None else qd
    m = max(s.lens + [1]) if max_len is None else max_len
    nb = q.moe_attn_chunk_workspace_bytes(s.cache, n_q, len(s.lens), s.T, m)
    ws = torch.full((max(nb, 1),), 0xff, dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    q.moe_attn_chunk(s.cache, s.seqs, n_q, qd, stride, s.T, m, 1 / math.sqrt(s.D), out, stride, ws, nb, stream)
    torch.cuda.synchronize()
    return bits(out[:, :w])


def check_chunk(s, n_q, qv, got, skip=()):
    G = n_q // s.n_kv
    scale = float(np.float32(1 / math.sqrt(s.D)))
    for b, (n, L) in enumerate(zip(s.rows, s.lens)):
        if b in skip or n == 0:
            continue
        for h in range(s.n_kv):
            k, v = s.ref.tokens(s.table[b], L, h)
            for i in range(n):
                t = int(s.start[b]) + i
                lim = L - n + i
                for g in range(G):
                    c = slice((h * G + g) * s.D, (h * G + g + 1) * s.D)
                    want, pv, qk = ref.attend(ref.bf16_val(qv[t, c]), k, v, lim, scale)
                    have = ref.bf16_val(got[t, c])
                    fin = np.isfinite(want)
                    assert np.array_equal(np.isnan(want), np.isnan(have)), (b, i, h, g)
                    assert np.array_equal(want[~fin & ~np.isnan(want)], have[~fin & ~np.isnan(want)])
                    seen = v[:lim + 1][np.isfinite(v[:lim + 1])]
                    bound = chunk_bound(s.fmt, want[fin], pv[fin], qk, s.D, max(lim + 1, 0), np.abs(seen).max(initial=0.0))
                    assert (np.abs(have[fin] - want[fin]) <= bound).all(), (b, i, h, g)


CASES = [  # fmt, n_kv, G, D, P, lens, rows
    (NVFP4, 2, 8, 128, 64, [1, 31, 64, 65, 300], [1, 30, 1, 20, 33]),
    (NVFP4, 1, 1, 64, 32, [700, 0, 150, 129], [140, 1, 129, 128]),
    (NVFP4, 2, 5, 256, 128, [129, 1, 260], [27, 1, 52]),
    (NVFP4, 1, 4, 128, 256, [63, 257], [63, 33]),
    (Q8_0, 2, 8, 128, 32, [32, 97, 5], [17, 40, 1]),
    (Q8_0, 2, 1, 64, 256, [257, 20], [130, 5]),
    (Q8_0, 1, 4, 256, 32, [100, 31], [33, 31]),
    (BF16, 2, 8, 128, 64, [63, 130], [16, 17]),
    (BF16, 1, 5, 64, 32, [1, 600], [1, 60]),
    (BF16, 2, 2, 256, 64, [65, 140], [65, 64]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{FMT[c[0]]}-{c[1]}x{c[2]}-D{c[3]}-P{c[4]}")
def test_chunk_matches_reference(case):
    fmt, n_kv, G, D, P, lens, rows = case
    print("chunk", case, flush=True)
    s = Setup(fmt, n_kv, D, P, lens, rows, seed=len(lens) + D, k_ts=0.75, v_ts=1.3)
    qv = ref.bf16_bits(1.5 * s.rng.standard_normal((s.T, n_kv * G * D)))
    for m in (None, 1, 1 << 20):  # the split of the work: as it falls, none, and the finest
        got = run_chunk(s, n_kv * G, qv, max_len=m)
        check_chunk(s, n_kv * G, qv, got)
        assert (got[int(s.start[-1]):] == ref.bf16_bits([7.0])[0]).all(), "rows behind the last sequence"


@pytest.mark.parametrize("fmt,n_kv,G,D,P,lens,rows", [
    (NVFP4, 1, 8, 128, 32, [2500, 3, 0, 700, 33, 1500], [40, 1, 1, 0, 1, 3]),
    (Q8_0, 2, 4, 64, 64, [1, 2049, 500, 64, 0, 1100], [2, 9, 0, 1, 1, 70]),
    (BF16, 1, 2, 256, 32, [1200, 31, 1000], [65, 12, 1]),
    (Q8_0, 1, 2, 64, 32, [1 + (37 * b) % 90 for b in range(75)] + [1500, 2, 900], [b % 3 for b in range(76)] + [0, 80]),
], ids=["nvfp4", "q8_0", "bf16", "78 sequences"])
def test_chunk_beside_decode_steps(fmt, n_kv, G, D, P, lens, rows):
    """One sequence's chunk among single rows and none, whatever the longest cache is said to
    be (too short, right, far too long): same answers."""
    print("mixed", FMT[fmt], len(lens), flush=True)
    s = Setup(fmt, n_kv, D, P, lens, rows, seed=len(lens), k_ts=0.75, v_ts=1.3)
    qv = ref.bf16_bits(1.5 * s.rng.standard_normal((s.T, n_kv * G * D)))
    for m in (None, 32, 500, 1 << 20):
        print("  max_len", m, flush=True)
        got = run_chunk(s, n_kv * G, qv, max_len=m)
        check_chunk(s, n_kv * G, qv, got)
        assert (got[int(s.start[-1]):] == ref.bf16_bits([7.0])[0]).all(), "rows behind the last sequence"


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunk_empty_rows_strides_and_in_place(fmt, D):
    """Rows before a sequence's first token give zero, row strides beyond the width, output in
    place of the queries (the same bits, with and without a split)."""
    s = Setup(fmt, 2, D, 32, [3, 50, 9, 140, 0], [5, 0, 1, 75, 2], seed=3)
    n_q = 6
    qv = ref.bf16_bits(s.rng.standard_normal((s.T, n_q * D)))
    print("rows", FMT[fmt], D, flush=True)
    for m in (1, 1 << 20):
        want = run_chunk(s, n_q, qv, max_len=m)
        check_chunk(s, n_q, qv, want)
        assert (want[:2] == 0).all() and (want[int(s.start[4]):int(s.start[5])] == 0).all()
        end = int(s.start[-1])
        for _ in range(3):
            got = run_chunk(s, n_q, qv, max_len=m, out="q", stride=n_q * D + 24)
            assert np.array_equal(got[:end], want[:end]) and (got[end:] == qv[end:]).all()


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
@pytest.mark.parametrize("val", [math.nan, math.inf])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunk_unseen_tokens_have_no_influence(fmt, val, D):
    """One token in the midst of a chunk is NaN or infinite, in keys or values: rows before it
    are as if it were not there; those from it on show it."""
    for which in (0, 1):
        s = Setup(fmt, 1, D, 32, [150, 45], [40, 1], seed=5)
        x = s.rng.standard_normal(D)
        x[17] = val
        s.ref.put(which, s.table[0, 130 // 32], 130 % 32, 0, ref.bf16_bits(x))
        s.to_device()
        qv = ref.bf16_bits(s.rng.standard_normal((s.T, 4 * D)))
        print("unseen", FMT[fmt], val, which, flush=True)
        got = run_chunk(s, 4, qv)
        if which == 1:
            check_chunk(s, 4, qv, got)
        else:
            check_chunk(s, 4, qv, got, skip=(0,))
            assert np.isnan(ref.bf16_val(got[25])).any()
            s.ref.put(0, s.table[0, 130 // 32], 130 % 32, 0, ref.bf16_bits(np.zeros(D)))
            s.to_device()
            assert np.array_equal(run_chunk(s, 4, qv)[:20], got[:20])
        assert np.isfinite(ref.bf16_val(got[:20])).all()


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
@pytest.mark.parametrize("P", [32, 128])
def test_chunk_bad_pages_give_nan(fmt, P):
    """Pages outside the pool, and lengths past the page table, are not read: the rows that
    would need them are NaN, those before them and the others are right."""
    for page in (-1, 10 ** 6):
        s = Setup(fmt, 2, 128, P, [2 * P + 70, 200, 64], [75, 3, 1], seed=7)
        qv = ref.bf16_bits(s.rng.standard_normal((s.T, 8 * 128)))
        whole = run_chunk(s, 8, qv, max_len=1)
        check_chunk(s, 8, qv, whole)
        s.table[0, 2 * P // s.P] = page  # tokens 2 P on: rows 5 on
        s.lens[2] = P * s.width + 1
        s.to_device()
        print("bad page", FMT[fmt], P, page, flush=True)
        for m in (1, 300, 1 << 20):
            got = run_chunk(s, 8, qv, max_len=m)
            val = ref.bf16_val(got)
            assert np.isnan(val[5:75]).all() and np.isnan(val[int(s.start[2])]).all()
            assert np.isfinite(val[:5]).all()
            check_chunk(s, 8, qv, got, skip=(0, 2))
        assert np.array_equal(run_chunk(s, 8, qv, max_len=1)[:5], whole[:5])


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
@pytest.mark.parametrize("L", [3, 60, 700, 2100])
def test_chunk_rows_outside_the_step(fmt, L):
    """Rows claimed before row 0 or from T on are left out, the others answered at their own
    positions; no row outside the sequences is touched."""
    for skipped, rows in ((4, [6, 2]), (39, [140, 1]), (5, [5, 3])):
        print("rows before row 0", FMT[fmt], L, skipped, rows, flush=True)
        s = Setup(fmt, 2, 64, 32, [L, 40], rows, seed=4, pad_rows=1)
        starts_before_row_0(s, skipped)
        qv = ref.bf16_bits(s.rng.standard_normal((s.T, 4 * 64)))
        got = run_chunk(s, 4, qv)
        check_chunk(s, 4, qv, got)
        assert (got[int(s.start[-1]):] == ref.bf16_bits([7.0])[0]).all()
    s = Setup(fmt, 1, 64, 32, [L, 90], [7, 60], seed=4, pad_rows=0)
    s.start_d.copy_(i32([0, 7, 1 << 30]))  # claims rows far beyond T: it has 2^30 - 7 rows and 90 tokens
    qv = ref.bf16_bits(s.rng.standard_normal((s.T, 4 * 64)))
    got = run_chunk(s, 4, qv)
    check_chunk(s, 4, qv, got, skip=(1,))
    assert (got[7:] == 0).all()  # rows before their sequence's first token


def test_chunk_starts_that_do_not_ascend():
    """(Nothing but the rows' own answers may be touched; which rows are answered is not said.)"""
    s = Setup(NVFP4, 2, 128, 32, [90, 40, 70], [30, 10, 20], seed=4)
    s.start_d.copy_(i32([0, 50, 20, 55]))
    qv = ref.bf16_bits(s.rng.standard_normal((s.T, 8 * 128)))
    for m in (1, 1 << 20):
        got = run_chunk(s, 8, qv, max_len=m)
        assert (got[55:] == ref.bf16_bits([7.0])[0]).all()


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
def test_chunk_scores_far_apart(fmt):
    """Scores that grow along the sequence by far more than fp32's exponent range, and queries far
    from one in magnitude."""
    for mag in (1e-20, 40.0, 3e3):
        s = Setup(fmt, 1, 128, 64, [300], [50], seed=9)
        grow = np.linspace(0, 3, 300)
        for j in range(300):
            s.ref.put(0, s.table[0, j // 64], j % 64, 0, ref.bf16_bits(np.full(128, grow[j])))
        s.to_device()
        qv = ref.bf16_bits(mag * (1 + 0.2 * s.rng.standard_normal((s.T, 2 * 128))))
        got = run_chunk(s, 2, qv)
        val = ref.bf16_val(got)
        assert np.isfinite(val[:50]).all()
        if mag < 1:
            check_chunk(s, 2, qv, got)
        else:  # the last token of a row that sees it has all the weight, where the steps are large
            k, v = s.ref.tokens(s.table[0], 300, 0)
            for i in (0, 25, 49):
                sc = (k[:251 + i] @ ref.bf16_val(qv[i, :128])) / math.sqrt(128)
                p = np.exp(sc - sc.max())
                top = np.abs(v[:251 + i][p > 1e-3 * p.sum()]).max(0)
                assert (np.abs(val[i, :128]) <= top * 1.02 + 1e-2).all()


# ------------------------------------------------------------------ long caches

def long_chunk(fmt, n_kv, G, D, P, lens, rows, max_lens=(None,), seed=1):
    gen = torch.Generator(device=dev).manual_seed(seed)
    k_ts, v_ts = (0.75, 1.25) if fmt == NVFP4 else (1.0, 1.0)
    pool, table, kv = attn_pages.make(fmt, n_kv, D, P, lens, gen, dev, k_ts, v_ts)
    n_q, T = n_kv * G, sum(rows)
    start = [sum(rows[:b]) for b in range(len(rows) + 1)]
    start_d, len_d, table = i32(start), i32(lens), table.contiguous()
    cache = q.KvCacheDesc(fmt, n_kv, D, P, pool.numel() // q.moe_kv_page_bytes(fmt, n_kv, D, P), k_ts, v_ts, pool.data_ptr())
    seqs = q.SeqBatch(len(lens), table.shape[1], start_d.data_ptr(), len_d.data_ptr(), table.data_ptr())
    x = (1.5 * torch.randn(T, n_q * D, generator=gen, device=dev)).bfloat16()
    scale = D ** -0.5
    for m in max_lens:
        print("long", FMT[fmt], n_kv, G, D, P, lens[:4], rows[:4], "max_len", m, flush=True)
        m = max(lens) if m is None else m
        nb = q.moe_attn_chunk_workspace_bytes(cache, n_q, len(lens), T, m)
        ws = torch.full((max(nb, 1),), 0xff, dtype=torch.uint8, device=dev)
        out = torch.full((T, n_q * D), 7.0, dtype=torch.bfloat16, device=dev)
        q.moe_attn_chunk(cache, seqs, n_q, x, n_q * D, T, m, scale, out, n_q * D, ws, nb)
        for b, (L, n) in enumerate(zip(lens, rows)):
            if n == 0:
                continue
            at = slice(start[b], start[b + 1])
            limit = (L - n + torch.arange(n, device=dev)).repeat_interleave(G)
            for h in range(n_kv):
                cut = lambda t: t[at, h * G * D:(h + 1) * G * D].double().reshape(n * G, D)  # noqa: E731
                k, v = kv[b][0][:, h], kv[b][1][:, h]
                s = (cut(x) @ k.T) * float(torch.tensor(scale))
                s.masked_fill_(torch.arange(L, device=dev) > limit[:, None], -math.inf)
                e = (s - s.max(1, keepdim=True).values).exp_()
                e /= e.sum(1, keepdim=True)
                want, pv = e @ v, e @ v.abs()
                qk = float((cut(x).abs() @ k.abs().T).max()) * scale
                over = (cut(out) - want).abs() / chunk_bound(fmt, want, pv, qk, D, L, float(v.abs().max()))
                assert float(over.max()) <= 1, (b, h, m, float(over.max()))


@pytest.mark.parametrize("fmt,D,P", [(NVFP4, 128, 64), (NVFP4, 64, 256), (Q8_0, 128, 32), (BF16, 256, 64)])
def test_chunk_behind_a_long_cache(fmt, D, P):
    long_chunk(fmt, 1, 4, D, P, [40001], [33], (None, 100, 1 << 20))
    long_chunk(fmt, 2, 8, D, P, [20000], [64])


@pytest.mark.parametrize("fmt,n_kv,G,D,P", [(NVFP4, 4, 8, 128, 64), (Q8_0, 8, 3, 64, 32), (BF16, 2, 2, 128, 128)])
def test_chunk_of_many_rows_among_decode_steps(fmt, n_kv, G, D, P):
    """A chunk of several tiles, a long and a short sequence's single rows: split and joined."""
    long_chunk(fmt, n_kv, G, D, P, [9000, 15000, 300, 7], [500, 1, 1, 1], (None, 2000, 1 << 20))


def test_prompts_and_rows_too_many_to_split():
    long_chunk(NVFP4, 4, 8, 128, 64, [1500, 700, 333], [1500, 500, 333])
    long_chunk(BF16, 8, 2, 64, 32, [4200], [4200])
    long_chunk(Q8_0, 2, 8, 128, 32, [3000, 20000], [2500, 1600])


def test_chunk_in_a_captured_graph_and_on_another_stream():
    """Lengths, tables and queries change between replays; eager calls between them use the same
    workspace."""
    gen = torch.Generator(device=dev).manual_seed(3)
    fmt, n_kv, G, D, P = NVFP4, 2, 8, 128, 64
    n_q, T, B = n_kv * G, 70, 3
    page = q.moe_kv_page_bytes(fmt, n_kv, D, P)
    pools, tables = [], []
    for i in range(2):
        pool, table, _ = attn_pages.make(fmt, n_kv, D, P, [6000, 500, 800], gen, dev)
        pools.append(pool)
        tables.append(table)
    pool, table = pools[0].clone(), tables[0].clone()
    start, lens = i32([0, 60, 65, 70]), i32([6000, 500, 800])
    cache = q.KvCacheDesc(fmt, n_kv, D, P, pool.numel() // page, 1.0, 1.0, pool.data_ptr())
    seqs = q.SeqBatch(B, table.shape[1], start.data_ptr(), lens.data_ptr(), table.data_ptr())
    x, out = (torch.empty(T, n_q * D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    nb = q.moe_attn_chunk_workspace_bytes(cache, n_q, B, T, 6000)
    assert nb > 0
    ws = torch.full((nb,), 0xff, dtype=torch.uint8, device=dev)

    def call(stream=None):
        q.moe_attn_chunk(cache, seqs, n_q, x, n_q * D, T, 6000, 0.1, out, n_q * D, ws, nb, stream)

    def set_inputs(i):
        pool.copy_(pools[i % 2])
        table.copy_(tables[i % 2])
        lens.copy_(i32([[6000, 500, 800], [130, 499, 5], [5000, 64, 65], [61, 5, 700]][i]))
        start.copy_(i32([[0, 60, 65, 70], [0, 1, 30, 69], [0, 0, 10, 70], [0, 61, 62, 62]][i]))
        x.copy_(torch.randn(T, n_q * D, generator=torch.Generator(device=dev).manual_seed(i), device=dev))
        out.fill_(7.0)

    def run(f, i):
        set_inputs(i)
        torch.cuda.synchronize()
        f()
        torch.cuda.synchronize()
        return out.clone()

    want = [run(call, i) for i in range(4)]
    side = torch.cuda.Stream()
    assert torch.equal(run(lambda: call(side), 2), want[2])
    graph = torch.cuda.CUDAGraph()
    set_inputs(0)
    with torch.cuda.graph(graph):
        call()
    for i in (1, 3, 0, 2, 1):
        assert torch.equal(run(graph.replay, i), want[i]), i
        assert torch.equal(run(call, (i + 1) % 4), want[(i + 1) % 4])


# ------------------------------------------------------------------ the ends of the ranges

@pytest.mark.parametrize("fmt,G,D,lens,rows", [(NVFP4, 96, 128, [70, 33], [5, 1]), (Q8_0, 300, 64, [100, 3], [3, 2]),
                                               (BF16, 1024, 64, [66, 1], [2, 1]), (NVFP4, 130, 256, [40], [3])])
def test_chunk_groups_wider_than_a_tile(fmt, G, D, lens, rows):
    """A tile ends within a row's heads; in place, too."""
    s = Setup(fmt, 1, D, 32, lens, rows, seed=G)
    qv = ref.bf16_bits(1.5 * s.rng.standard_normal((s.T, G * D)))
    for m in (None, 1, 1 << 20):
        got = run_chunk(s, G, qv, max_len=m)
        check_chunk(s, G, qv, got)
    end = int(s.start[-1])
    assert np.array_equal(run_chunk(s, G, qv, max_len=1 << 20, out="q")[:end], got[:end])


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
@pytest.mark.parametrize("B", [64, 65, 150])
def test_chunk_of_many_sequences(fmt, B):
    """More sequences than lanes, some without rows, some without tokens."""
    rng = np.random.default_rng(B)
    lens = [int(n) for n in rng.integers(0, 90, B)]
    rows = [int(n) for n in rng.integers(0, 4, B)]
    lens[B - 1], rows[B - 1], lens[3] = 400, 40, 0
    s = Setup(fmt, 1, 64, 32, lens, rows, seed=B)
    qv = ref.bf16_bits(s.rng.standard_normal((s.T, 3 * 64)))
    for m in (None, 1, 1 << 20):
        print("sequences", FMT[fmt], B, m, flush=True)
        got = run_chunk(s, 3, qv, max_len=m)
        check_chunk(s, 3, qv, got)
        assert (got[int(s.start[-1]):] == ref.bf16_bits([7.0])[0]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunk_values_at_the_end_of_fp16(D):
    """Q8_0 values up to 65024, whose scale is 512, in tokens that some rows do not see: those are
    as if the token were not there, and the others right."""
    s = Setup(Q8_0, 1, D, 32, [150, 45], [40, 1], seed=5)
    qv = ref.bf16_bits(s.rng.standard_normal((s.T, 4 * D)))
    before = run_chunk(s, 4, qv)
    x = np.zeros(D)
    x[17], x[40] = 65024.0, -6e4
    s.ref.put(1, s.table[0, 130 // 32], 130 % 32, 0, ref.bf16_bits(x))
    s.ref.put(1, s.table[0, 2], 7, 0, ref.bf16_bits(s.rng.standard_normal(D) * 2e4))
    s.to_device()
    got = run_chunk(s, 4, qv)
    check_chunk(s, 4, qv, got)
    assert np.isfinite(ref.bf16_val(got[:41])).all() and np.array_equal(got[40], before[40])


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
def test_chunk_queries_near_nothing(fmt):
    """Queries far below one, of zero, and a cache's small scale: rows still see only their own."""
    s = Setup(fmt, 2, 128, 32, [100, 70], [40, 3], seed=6, k_ts=1e-30 if fmt == NVFP4 else 1.0)
    qv = ref.bf16_bits(1e-36 * s.rng.standard_normal((s.T, 4 * 128)))
    qv[5] = 0
    got = run_chunk(s, 4, qv)
    check_chunk(s, 4, qv, got)


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
def test_chunk_pages_beyond_32_bit_offsets(fmt):
    """A pool of more than 4 GiB: the same answers from its last pages as from a small one's."""
    n_kv, D, P, n_q = 8, 256, 256, 8
    far = (1 << 32) // q.moe_kv_page_bytes(fmt, n_kv, D, P) + 3
    qkv = torch.randn(600, (n_q + 2 * n_kv) * D, generator=torch.Generator(device=dev).manual_seed(6), device=dev).bfloat16()
    got = []
    for n_pages, pages in ((3, [2, 0, 1]), (far, [far - 1, far - 3, far - 2])):
        print("pool", FMT[fmt], n_pages, flush=True)
        cache = q.KvCache(fmt, n_q, n_kv, D, P, n_pages)
        buf = q.AttnBuffers(cache, 1, 600, 3, chunk=True)
        buf.page_table.copy_(i32([pages]))
        buf.row_start.copy_(i32([0, 600]))
        buf.kv_len.copy_(i32([600]))
        got.append(q.attention_forward(cache, buf, qkv, 600, 1 / 16, chunk=True).clone())
        torch.cuda.synchronize()
        del cache, buf
    assert torch.isfinite(got[0].float()).all() and torch.equal(*got)
