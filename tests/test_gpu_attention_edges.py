"""Corners of the key/value cache and attention operators that the cases of
test_gpu_attention.py do not reach, against the same 64-bit reference and bounds."""
import math

import numpy as np
import pytest
import torch

import attn_ref as ref
import quantized_expert_ffn_router_amd as q
from attn_ref import BF16, NVFP4, Q8_0
from test_gpu_attention import (FMT, Setup, append_inputs, bits, check_append, check_decode, check_prompt, i32,
                                run_append, run_decode, run_prompt)

pytestmark = pytest.mark.gpu

dev = "cuda"


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode_tiles_do_not_depend_on_other_tiles_rows(fmt, D):
    """5 rows of 8 heads a group: the last tile holds the last row alone, and its
    bits are the same whatever the first row's queries are."""
    print("other tiles", FMT[fmt], D, flush=True)
    s = Setup(fmt, 1, D, 32, [384], [5], seed=3, pad_rows=0)
    qv = ref.bf16_bits(3 * s.rng.standard_normal((s.T, 8 * D)))
    got = []
    for mag in (1.0, 0.0, 3.0, 10.0):
        x = qv.copy()
        x[0] = ref.bf16_bits(mag * ref.bf16_val(qv[0]))
        got.append(run_decode(s, 8, x))
    check_decode(s, 8, qv, got[0])
    for g in got[1:]:
        assert np.array_equal(g[4], got[0][4])


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
@pytest.mark.parametrize("D,rows", [(128, [5, 3, 9]), (64, [7, 1, 13]), (256, [3, 5, 1])])
def test_decode_in_place_is_bit_for_bit_the_same(fmt, D, rows):
    """Several tiles a sequence, the last ones partly filled, without a split (so
    each tile stores its own output): the output in the queries' place."""
    print("in place", FMT[fmt], D, rows, flush=True)
    s = Setup(fmt, 2, D, 32, [300, 64, 340], rows, seed=6, pad_rows=1)
    qv = ref.bf16_bits(3 * s.rng.standard_normal((s.T, 16 * D)))
    want = run_decode(s, 16, qv)
    n = int(s.start[-1])
    for _ in range(5):
        assert np.array_equal(run_decode(s, 16, qv, out="q")[:n], want[:n])


def starts_before_row_0(s, skipped):
    """The first sequence's first `skipped` rows lie before row 0."""
    s.start = s.start - skipped
    s.T -= skipped
    s.to_device()
    s.start, s.rows = np.maximum(s.start, 0), [s.rows[0] - skipped, *s.rows[1:]]


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
@pytest.mark.parametrize("L", [3, 60, 700, 2100])
def test_decode_rows_before_row_0_are_left_out(fmt, L):
    """A sequence's rows inside 0..T are answered at their own positions, with and
    without a split, wherever its first row lies (3 tokens: rows that see nothing)."""
    for skipped, rows in ((4, [6, 2]), (39, [40, 1]), (5, [5, 3])):
        print("rows before row 0", FMT[fmt], L, skipped, rows, flush=True)
        s = Setup(fmt, 2, 64, 32, [L, 40], rows, seed=4, pad_rows=1)
        starts_before_row_0(s, skipped)
        qv = ref.bf16_bits(s.rng.standard_normal((s.T, 4 * 64)))
        got = run_decode(s, 4, qv)
        check_decode(s, 4, qv, got)
        assert (got[int(s.start[-1]):] == ref.bf16_bits([7.0])[0]).all()


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
def test_append_rows_before_row_0_are_left_out(fmt):
    print("append, rows before row 0", FMT[fmt], flush=True)
    s = Setup(fmt, 2, 64, 32, [50, 9], [21, 5], seed=7, pad_rows=1)
    starts_before_row_0(s, 9)
    qkv = append_inputs(s, 4, 9)
    freq, _ = q.moe_rope_freqs(q.MOE_ROPE_PLAIN, 32, 10000.0)
    norm = [np.ones(64, np.float32)] * 2
    got_q, got_k, _ = run_append(s, 4, qkv, norm, 32, 0, freq, 1.0)
    check_append(s, 4, qkv, norm, 32, 0, freq, 1.0, got_q, got_k)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prompt_rows_before_row_0_are_left_out(D):
    """Sequences whose first row lies before row 0, behind longer keys or not: the
    rows inside are answered at their own positions, a row alone in the first
    tile's place among them."""
    rng = np.random.default_rng(D)
    for first, ends, keys in ((-127, [2], [129]), (-1000, [130, 180], [1130, 60]), (-3, [40, 41, 300], [20, 1, 259])):
        print("prompt, rows before row 0", D, first, ends, flush=True)
        T, ks = ends[-1] + 1, np.concatenate([[0], np.cumsum(keys)]).tolist()
        qv = ref.bf16_bits(rng.standard_normal((T, 2 * D)))
        kv, vv = (ref.bf16_bits(rng.standard_normal((ks[-1], D))) for _ in range(2))
        got = run_prompt(2, 1, D, [first, *ends], ks, T, ks[-1], qv, kv, vv)
        check_prompt(2, 1, D, [0, *ends], ks, qv, kv, vv, got)
        assert (got[ends[-1]:] == ref.bf16_bits([7.0])[0]).all()


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
@pytest.mark.parametrize("first,start", [
    ([0, 60], [-370, 30, 40]),   # the first rows before row 0
    ([17, 0], [-30, -3, 40]),    # a whole sequence, and a few rows of the next
    ([-5, 65], [0, 20, 40]),     # tokens before the sequence's first: their rows stay as they are
    ([-40, -3], [-20, 10, 60]),  # both; rows from R on
    ([-(2 ** 31), 2 ** 31 - 1], [-(2 ** 31), 0, 40]),
])
def test_read_outside_the_rows_and_tokens(fmt, first, start):
    print("read outside", FMT[fmt], first, start, flush=True)
    D, R = 64, 40
    s = Setup(fmt, 2, D, 32, [400, 70], [0, 0], seed=8)
    ko, vo = (torch.full((R, 2 * D), 7.0, dtype=torch.bfloat16, device=dev) for _ in range(2))
    q.moe_kv_read(s.cache, s.seqs, i32(first), i32(start), R, ko, 2 * D, vo, 2 * D)
    torch.cuda.synchronize()
    for w, got in ((0, bits(ko)), (1, bits(vo))):
        want = np.full((R, 2 * D), ref.bf16_bits([7.0])[0], np.uint16)
        for b in range(2):
            for r in range(max(start[b], 0), min(start[b + 1], R)):
                j = first[b] + r - start[b]
                if 0 <= j < s.lens[b]:
                    want[r] = np.concatenate([ref.bf16_bits(s.ref.get(w, s.table[b, j // 32], j % 32, h)) for h in range(2)])
        assert np.array_equal(ref.bf16_val(got), ref.bf16_val(want)), w


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prompt_tiles_do_not_depend_on_other_tiles_rows(D):
    """Partly filled tiles of three prompts, the first row of all being NaN, or far
    larger than the others: the rows of the other tiles keep their bits, also with
    the output in the queries' place.  (The keys of a prompt's first tile are
    small, so a pass with a running maximum would round the weights differently.)"""
    rng = np.random.default_rng(D)
    qs = [0, 130, 330, 375]
    T = qs[-1]
    small = np.concatenate([np.arange(n) < 64 for n in np.diff(qs)])[:, None]
    qv = ref.bf16_bits(2 * rng.standard_normal((T, 2 * D)))
    kv = ref.bf16_bits(rng.standard_normal((T, D)) * np.where(small, 0.05, 1.0))
    vv = ref.bf16_bits(rng.standard_normal((T, D)))
    want = run_prompt(2, 1, D, qs, None, T, T, qv, kv, vv)
    check_prompt(2, 1, D, qs, None, qv, kv, vv, want, [0, 64, 127, 128, 129, 199, 44])
    for row0 in (np.full(2 * D, math.nan), 1e5 * ref.bf16_val(qv[0])):
        x = qv.copy()
        x[0] = ref.bf16_bits(row0)
        for in_place in (False, True, True, True):
            print("prompt, other tiles", D, row0[0], in_place, flush=True)
            got = run_prompt(2, 1, D, qs, None, T, T, x, kv, vv, in_place=in_place)
            assert np.array_equal(got[128:], want[128:])


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
@pytest.mark.parametrize("L", [380, 2001])
@pytest.mark.parametrize("gap", [12, 20, 24, 26])
def test_decode_small_weights_beside_a_large_one(fmt, L, gap):
    """The first token outweighs every other 2^gap to 2^(5 gap / 6) times and has the
    value 0, so that the output is what the others add up to.  A weight is off by
    2^-11 of it (2^-8 for the 16-bit cache) or, below fp16's normal numbers, by
    2^-25 where the largest is 2^7 or more: 2^-32 of the largest."""
    print("small weights", FMT[fmt], L, gap, flush=True)
    D = 64
    s = Setup(fmt, 1, D, 32, [L], [1], seed=5, pad_rows=0)
    rng = np.random.default_rng(6)
    for j in range(L):
        k, v = np.zeros(D), 0.5 + rng.random(D)
        k[0], k[1] = 0.5 * rng.integers(0, 3), 6.0  # (the same scale for every token)
        if j == 0:
            k[0], v[:] = 6.0, 0.0
        for w, x in ((0, k), (1, v)):
            s.ref.put(w, s.table[0, j // 32], j % 32, 0, ref.bf16_bits(x))
    s.to_device()
    x = np.zeros((1, D))
    x[0, 0] = gap * math.log(2) / 6 * math.sqrt(D)
    qv = ref.bf16_bits(x)
    have = ref.bf16_val(run_decode(s, 1, qv)[0])
    k, v = s.ref.tokens(s.table[0], L, 0)
    want, pv, qk = ref.attend(ref.bf16_val(qv[0]), k, v, L - 1, float(np.float32(D ** -0.5)))
    bound = ref.attend_bound(want, pv, qk, L, 0.0, D, fmt)  # (without its own term for small weights)
    if fmt != BF16:
        bound += (np.abs(v).sum(0) + L * np.abs(want)) * 2.0 ** -32
    assert (np.abs(have - want) <= bound).all(), float((np.abs(have - want) / bound).max())


@pytest.mark.parametrize("ts", [2.0 ** -118, 2.0 ** 100])
def test_decode_value_scales_of_any_size(ts):
    """The values' scale of the whole cache is applied to the weighted mean: with
    values and scale times a power of two, so are the outputs, up to a step of
    bf16's subnormal numbers."""
    got = []
    for t in (1.0, ts):
        print("value scale", t, flush=True)
        s = Setup(NVFP4, 1, 64, 32, [40, 700], [1, 1], seed=5, pad_rows=0, v_ts=t, vary=(1.0, t))
        qv = ref.bf16_bits(s.rng.standard_normal((s.T, 2 * 64)))
        got.append(ref.bf16_val(run_decode(s, 2, qv)))
        if t == 1.0:
            check_decode(s, 2, qv, ref.bf16_bits(got[0]))
    assert (np.abs(got[1] - ts * got[0]) <= 2.0 ** -133).all()


def test_outputs_beside_their_inputs_in_one_buffer():
    """Rows of one wide buffer may hold inputs and outputs side by side: the same
    bits as with buffers of their own."""
    D, n_q, n_kv, P, L = 64, 4, 2, 32, 50
    qw, kw = n_q * D, n_kv * D
    gen = torch.Generator(device=dev).manual_seed(3)
    qkv = torch.randn(L, qw + 2 * kw, generator=gen, device=dev).bfloat16()
    f = torch.from_numpy(q.moe_rope_freqs(q.MOE_ROPE_PLAIN, D, 10000.0)[0]).to(dev)
    d = q.QkvDesc(n_q, 1e-6, None, None, D, 0, f.data_ptr(), 1.0)
    got = []
    for wide in (False, True):
        print("one buffer", wide, flush=True)
        cache = q.KvCache(Q8_0, n_q, n_kv, D, P, 2)
        buf = q.AttnBuffers(cache, 1, L, 2)
        buf.page_table.copy_(i32([[1, 0]]))
        buf.row_start.copy_(i32([0, L]))
        buf.kv_len.copy_(i32([L]))
        widths = [qw + 2 * kw, qw, kw, kw, kw, qw, qw]
        if wide:  # projections, queries, keys, keys and values read back, two outputs
            st, whole = sum(widths), torch.full((L, sum(widths)), 7.0, dtype=torch.bfloat16, device=dev)
            parts = list(torch.split(whole, widths, 1))
        else:
            parts = [torch.full((L, n), 7.0, dtype=torch.bfloat16, device=dev) for n in widths]
        strides = [st if wide else n for n in widths]
        parts[0].copy_(qkv)
        x, qo, ko, kr, vr, o1, o2 = parts
        xs, qs, ks, krs, vrs, s1, s2 = strides
        q.moe_kv_append(cache.desc, d, buf.seqs, x, xs, L, None, qo, qs, ko, ks)
        q.moe_kv_read(cache.desc, buf.seqs, None, buf.row_start, L, kr, krs, vr, vrs)
        q.moe_attn_prompt(n_q, n_kv, D, 1, buf.row_start, None, L, L, qo, qs, kr, krs, vr, vrs, 0.125, o1, s1)
        q.moe_attn_decode(cache.desc, buf.seqs, n_q, qo, qs, L, 0, 0.125, o2, s2, buf.ws, buf.ws_bytes)
        torch.cuda.synchronize()
        got.append([p.clone() for p in parts])
    for a, b in zip(*got):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
@pytest.mark.parametrize("D,n_q,n_kv", [(64, 9, 3), (128, 10, 5), (256, 3, 3)])
def test_append_in_place_with_whole_quads(fmt, D, n_q, n_kv):
    """Queries and keys in their own place of the projections, prompts of whole and
    part quads: cache bytes and rows as stated, the values' part untouched."""
    print("append in place", FMT[fmt], D, flush=True)
    s = Setup(fmt, n_kv, D, 32, [13, 43, 3, 8, 70], [13, 38, 5, 8, 2], seed=D, v_ts=1.5, pad_rows=2)
    qkv = append_inputs(s, n_q, 6)
    norm = [np.full(D, 1.25, np.float32), np.ones(D, np.float32)]
    freq, _ = q.moe_rope_freqs(q.MOE_ROPE_PLAIN, 32, 10000.0)
    got_q, got_k, whole = run_append(s, n_q, qkv, norm, 32, 0, freq, 1.0, in_place=True)
    check_append(s, n_q, qkv, norm, 32, 0, freq, 1.0, got_q, got_k)
    n = int(s.start[-1])
    assert np.array_equal(whole[:n, (n_q + n_kv) * D:], qkv[:n, (n_q + n_kv) * D:])
    assert np.array_equal(whole[n:], qkv[n:])


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
def test_append_of_a_long_prompt_in_place_and_apart(fmt):
    """4101 rows of two sequences, a workgroup to each four (with few rows the heads of
    a row are spread over several): the same bits in place and apart."""
    D, n_q, n_kv, P, rows = 64, 8, 4, 64, [4000, 101]
    T, w, kw = sum(rows), (n_q + 2 * n_kv) * D, n_kv * D
    gen = torch.Generator(device=dev).manual_seed(3)
    x0 = (2 * torch.randn(T, w, generator=gen, device=dev)).bfloat16()
    rope = q.moe_rope_freqs(q.MOE_ROPE_PLAIN, 64, 10000.0)
    got = []
    for in_place in (True, False):
        print("long append", FMT[fmt], in_place, flush=True)
        cache = q.KvCache(fmt, n_q, n_kv, D, P, 67, np.ones(D), np.ones(D), rope)
        cache.pool.fill_(0xff)
        buf = q.AttnBuffers(cache, 2, T, 64)
        buf.page_table[0, :63] = torch.arange(63, device=dev)
        buf.page_table[1, :2] = i32([66, 64])
        buf.row_start.copy_(i32([0, rows[0], T]))
        buf.kv_len.copy_(i32(rows))
        x = x0.clone()
        qo, ko = (x, x.data_ptr() + 2 * n_q * D) if in_place else (torch.empty(T, n_q * D, dtype=torch.bfloat16, device=dev),
                                                                  torch.empty(T, kw, dtype=torch.bfloat16, device=dev))
        qs, ks = (w, w) if in_place else (n_q * D, kw)
        q.moe_kv_append(cache.desc, cache.qkv_desc, buf.seqs, x, w, T, None, qo, qs, ko, ks)
        torch.cuda.synchronize()
        assert torch.equal(x[:, n_q * D + kw:], x0[:, n_q * D + kw:])
        got.append((x[:, :n_q * D], x[:, n_q * D:n_q * D + kw], cache.pool) if in_place else (qo, ko, cache.pool))
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
@pytest.mark.parametrize("length", [2 ** 31 - 1, 10 ** 9, "a token more", "a page more"])
def test_decode_lengths_past_the_page_table(fmt, length):
    """The rows that see a token past the table are NaN, at once (the tokens past it
    are not gone over one by one); those of the same sequence that end before it and
    other sequences are right, with the table's last page held or not."""
    print("past the table", FMT[fmt], length, flush=True)
    for rows, P, lens in (([1, 1, 3], 32, [700, 70, 96]), ([2, 1, 4], 64, [128, 1, 900])):
        s = Setup(fmt, 2, 64, P, lens, rows, seed=9)
        end = P * s.width  # tokens that the table has places for
        L = {"a token more": end + 1, "a page more": end + P}.get(length, length)
        s.lens[0] = L
        s.to_device()
        qv = ref.bf16_bits(s.rng.standard_normal((s.T, 4 * 64)))
        for m in (max(lens), 1 << 20):
            got = run_decode(s, 4, qv, max_len=m)
            seen = np.isnan(ref.bf16_val(got[:rows[0]]))
            assert seen.all(), (m, seen.all(1))  # (all see the places behind its own tokens)
            check_decode(s, 4, qv, got, skip=(0,))
        # the last row of a sequence sees past the table, the ones before it end inside
        full = Setup(fmt, 2, 64, P, [P * 3, 40], [3, 1], seed=10)
        full.table = full.table[:, :3]
        full.width, full.lens = 3, [P * 3 + 1, 40]
        full.table = np.ascontiguousarray(full.table)
        full.to_device()
        qv = ref.bf16_bits(full.rng.standard_normal((full.T, 4 * 64)))
        got = run_decode(full, 4, qv)
        assert np.isnan(ref.bf16_val(got[2])).all()
        full.lens, full.rows, full.start = [P * 3, 40], [2, 1], np.array([0, 2, 3])
        keep = got[[0, 1, 3]]
        check_decode(full, 4, qv[[0, 1, 3]], keep)


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
def test_rows_claimed_beyond_t_are_left_out(fmt):
    """The last sequence claims more rows than the step has: those inside are at the
    positions that its claim gives them, in appends and in decode steps with and
    without a split."""
    for L in (60, 900):
        print("rows beyond T", FMT[fmt], L, flush=True)
        s = Setup(fmt, 2, 64, 32, [33, L], [2, 20], seed=12, pad_rows=0)
        T, inside = 9, 7
        qv = ref.bf16_bits(s.rng.standard_normal((T, 4 * 64)))
        s.T = T
        got = run_decode(s, 4, qv)
        lens, rows, start = list(s.lens), list(s.rows), s.start
        # (row i of the claim sees up to token L - 20 + i: as if the sequence ended with the 7th)
        s.lens, s.rows, s.start = [33, L - 20 + inside], [2, inside], np.array([0, 2, T])
        check_decode(s, 4, qv, got)
        s.lens, s.rows, s.start = lens, rows, start
        qkv = append_inputs(s, 4, 9)
        freq, _ = q.moe_rope_freqs(q.MOE_ROPE_PLAIN, 32, 10000.0)
        norm = [np.ones(64, np.float32)] * 2
        got_q, got_k, _ = run_append(s, 4, qkv, norm, 32, 0, freq, 1.0)
        s.lens, s.rows, s.start = [33, L - 20 + inside], [2, inside], np.array([0, 2, T])
        check_append(s, 4, qkv, norm, 32, 0, freq, 1.0, got_q, got_k)
