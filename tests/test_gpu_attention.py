"""Key/value cache and attention operators (moe_kv_append, moe_kv_read,
moe_attn_decode, moe_attn_prompt) against the 64-bit reference in attn_ref.py:
every cache format and head size, lengths around the tile and page sizes,
sequences without rows or tokens, rows that see nothing, tokens that rows do not
see holding NaN or infinity, bad pages, strides, in-place outputs, padding rows
and captured graphs.

Bounds: cache contents are equal bit for bit (both sides compute the values to
be quantised in 64 bits); normed and rotated rows are within one rounding to
bf16, 2^-8 of the value; attention within attn_ref.attend_bound."""
import math

import numpy as np
import pytest
import torch

import attn_ref as ref
import quantized_expert_ffn_router_amd as q
from attn_ref import BF16, NVFP4, Q8_0

pytestmark = pytest.mark.gpu

dev = "cuda"
FMT = {NVFP4: "nvfp4", Q8_0: "q8_0", BF16: "bf16"}


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def to_dev(u16):
    return torch.from_numpy(np.ascontiguousarray(u16).view(np.int16)).to(dev).view(torch.bfloat16)


class Setup:
    """A cache with sequences of the given lengths, random contents, pages in
    random order; stale tokens and unused pages hold `stale` bytes."""

    def __init__(self, fmt, n_kv, D, P, lens, rows, seed=0, k_ts=1.0, v_ts=1.0, pad_rows=2,
                 stale=0xff, vary=None):
        rng = np.random.default_rng(seed)
        self.rng = rng
        self.fmt, self.n_kv, self.D, self.P = fmt, n_kv, D, P
        self.lens, self.rows = list(lens), list(rows)
        need = [max(-(-x // P), 0) for x in lens]
        n_pages, self.width = sum(need) + 2, max(need + [0]) + 1
        where = rng.permutation(n_pages)
        self.table = np.full((len(lens), self.width), -1, np.int64)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = where[at:at + n]
            at += n
        self.ref = ref.Cache(fmt, n_kv, D, P, n_pages, k_ts, v_ts, stale)
        self.kv = {}
        for b, L in enumerate(lens):
            for j in range(max(L, 0)):
                for h in range(n_kv):
                    for w in (0, 1):
                        x = rng.standard_normal(D) * (1.0 if vary is None else vary[w])
                        self.ref.put(w, self.table[b, j // P], j % P, h, ref.bf16_bits(x))
        self.start = np.concatenate([[0], np.cumsum(rows)])
        self.T = int(self.start[-1]) + pad_rows
        self.to_device()

    def to_device(self):
        self.pool = torch.empty(self.ref.pool.size + 256, dtype=torch.uint8, device=dev)
        off = (-self.pool.data_ptr()) % 256
        self.pool = self.pool[off:off + self.ref.pool.size]
        self.pool.copy_(torch.from_numpy(self.ref.pool))
        self.start_d, self.len_d, self.table_d = i32(self.start), i32(self.lens), i32(self.table)
        c = self.ref
        self.cache = q.KvCacheDesc(self.fmt, self.n_kv, self.D, self.P, c.n_pages, float(c.ts[0]),
                                   float(c.ts[1]), self.pool.data_ptr())
        self.seqs = q.SeqBatch(len(self.lens), self.width, self.start_d.data_ptr(),
                               self.len_d.data_ptr(), self.table_d.data_ptr())


def run_decode(s, n_q, qv, max_len=None, out=None, stride=None):
    """qv: bf16 bits [T, n_q * D]; returns bf16 bits."""
    w = n_q * s.D
    stride = stride or w
    qd = torch.zeros(s.T, stride, dtype=torch.bfloat16, device=dev)
    qd[:, :w] = to_dev(qv)
    out = torch.full((s.T, stride), 7.0, dtype=torch.bfloat16, device=dev) if out is None else qd
    m = max(s.lens + [1]) if max_len is None else max_len
    nb = q.moe_attn_workspace_bytes(s.cache, n_q, len(s.lens), s.T, m)
    ws = torch.full((max(nb, 1),), 0xff, dtype=torch.uint8, device=dev)
    q.moe_attn_decode(s.cache, s.seqs, n_q, qd, stride, s.T, m, 1 / math.sqrt(s.D), out, stride, ws, nb)
    torch.cuda.synchronize()
    return bits(out[:, :w])


def check_decode(s, n_q, qv, got, skip=()):
    G = n_q // s.n_kv
    scale = float(np.float32(1 / math.sqrt(s.D)))
    for b, (n, L) in enumerate(zip(s.rows, s.lens)):
        if b in skip:
            continue
        for h in range(s.n_kv):
            if n == 0:
                continue
            k, v = s.ref.tokens(s.table[b], L, h)
            for i in range(n):
                t = int(s.start[b]) + i
                lim = L - n + i
                for g in range(G):
                    c = slice((h * G + g) * s.D, (h * G + g + 1) * s.D)
                    qr = ref.bf16_val(qv[t, c])
                    want, pv, qk = ref.attend(qr, k, v, lim, scale)
                    have = ref.bf16_val(got[t, c])
                    fin = np.isfinite(want)
                    assert np.array_equal(np.isnan(want), np.isnan(have)), (b, i, h, g)
                    assert np.array_equal(want[~fin & ~np.isnan(want)], have[~fin & ~np.isnan(want)])
                    vm = np.abs(v[:lim + 1])[np.isfinite(v[:lim + 1])].max() if lim >= 0 else 0.0
                    bound = ref.attend_bound(want[fin], pv[fin], qk, max(lim + 1, 0), vm, s.D, s.fmt)
                    err = np.abs(have[fin] - want[fin])
                    assert (err <= bound).all(), (b, i, h, g, float((err / bound).max()))


CASES = [  # fmt, n_kv, G, D, P, lens, rows
    (NVFP4, 2, 8, 128, 64, [1, 31, 64, 65, 300], [1, 1, 1, 1, 1]),
    (NVFP4, 1, 1, 64, 32, [700, 0, 33], [1, 1, 2]),
    (NVFP4, 2, 5, 256, 128, [129, 1, 260], [1, 1, 1]),
    (Q8_0, 2, 8, 128, 32, [32, 97, 5], [4, 3, 1]),
    (Q8_0, 2, 1, 64, 256, [257, 20], [1, 5]),
    (Q8_0, 1, 4, 256, 32, [100, 31], [1, 2]),
    (BF16, 2, 8, 128, 64, [63, 130], [1, 4]),
    (BF16, 1, 5, 64, 32, [1, 600], [1, 1]),
    (BF16, 2, 2, 256, 64, [65, 40], [1, 3]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{FMT[c[0]]}-{c[1]}x{c[2]}-D{c[3]}-P{c[4]}")
def test_decode_matches_reference(case):
    fmt, n_kv, G, D, P, lens, rows = case
    print("decode", case, flush=True)
    s = Setup(fmt, n_kv, D, P, lens, rows, seed=len(lens) + D, k_ts=0.75, v_ts=1.3)
    qv = ref.bf16_bits(1.5 * s.rng.standard_normal((s.T, n_kv * G * D)))
    got = run_decode(s, n_kv * G, qv)
    check_decode(s, n_kv * G, qv, got)
    assert (got[int(s.start[-1]):] == ref.bf16_bits([7.0])[0]).all(), "rows behind the last sequence"
    # the split of the work: one workgroup for everything, and the finest one
    for m in (1, 1 << 20):
        check_decode(s, n_kv * G, qv, run_decode(s, n_kv * G, qv, max_len=m))


@pytest.mark.parametrize("fmt,n_kv,G,D,P,lens,rows", [
    (NVFP4, 1, 8, 128, 32, [2500, 3, 0, 700, 33, 1500], [1, 1, 1, 0, 1, 3]),
    (Q8_0, 2, 4, 64, 64, [1, 2049, 500, 64, 0, 1100], [2, 9, 0, 1, 1, 1]),
    (BF16, 1, 2, 256, 32, [1200, 31, 1000], [1, 12, 1]),
    (Q8_0, 1, 2, 64, 32, [1 + (37 * b) % 90 for b in range(75)] + [1500, 2, 900], [b % 3 for b in range(78)]),
], ids=["nvfp4", "q8_0", "bf16", "78 sequences"])
def test_decode_split_over_sequences_of_different_lengths(fmt, n_kv, G, D, P, lens, rows):
    """The same chunks for all sequences, whatever the longest cache is said to be
    (too short, right, far too long): same answers."""
    print("ragged", FMT[fmt], len(lens), flush=True)
    s = Setup(fmt, n_kv, D, P, lens, rows, seed=len(lens), k_ts=0.75, v_ts=1.3)
    qv = ref.bf16_bits(1.5 * s.rng.standard_normal((s.T, n_kv * G * D)))
    for m in (None, 32, 500, 1 << 20):
        print("  max_len", m, flush=True)
        got = run_decode(s, n_kv * G, qv, max_len=m)
        check_decode(s, n_kv * G, qv, got)
        assert (got[int(s.start[-1]):] == ref.bf16_bits([7.0])[0]).all(), "rows behind the last sequence"


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
def test_decode_many_rows_empty_rows_and_strides(fmt):
    """Rows before a sequence's first token (fewer tokens than rows) give zero,
    sequences without rows are passed over, row strides beyond the width, output
    in place of the queries; more rows than one tile."""
    s = Setup(fmt, 2, 64, 32, [3, 50, 9, 40, 0], [5, 0, 1, 37, 2], seed=3)
    n_q = 6
    qv = ref.bf16_bits(s.rng.standard_normal((s.T, n_q * 64)))
    print("decode rows", FMT[fmt], flush=True)
    got = run_decode(s, n_q, qv, out="q", stride=n_q * 64 + 24)
    check_decode(s, n_q, qv, got)
    assert (got[:2] == 0).all() and (got[int(s.start[4]):int(s.start[5])] == 0).all()
    assert (got[int(s.start[-1]):] == qv[int(s.start[-1]):]).all()


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
@pytest.mark.parametrize("val", [math.nan, math.inf])
def test_decode_unseen_tokens_have_no_influence(fmt, val):
    """The second of three rows' tokens is NaN or infinite, in keys or values:
    the row before it is as if it were not there; those after show it."""
    for which in (0, 1):
        s = Setup(fmt, 1, 128, 32, [70, 45], [3, 1], seed=5)
        x = s.rng.standard_normal(128)
        x[17] = val
        s.ref.put(which, s.table[0, 68 // 32], 68 % 32, 0, ref.bf16_bits(x))
        s.to_device()
        qv = ref.bf16_bits(s.rng.standard_normal((s.T, 4 * 128)))
        print("unseen", FMT[fmt], val, which, flush=True)
        got = run_decode(s, 4, qv)
        if which == 1:
            check_decode(s, 4, qv, got)
            assert np.isfinite(ref.bf16_val(got[0])).all()
        else:
            check_decode(s, 4, qv, got, skip=(0,))
            assert np.isfinite(ref.bf16_val(got[0])).all()
            assert np.isnan(ref.bf16_val(got[2])).any()


def test_decode_bad_pages_give_nan():
    """Pages outside the pool, and lengths past the page table, are not read:
    the rows that would need them are NaN, the others are right."""
    for page in (-1, 10 ** 6):
        s = Setup(NVFP4, 2, 128, 64, [200, 200, 64], [1, 1, 1], seed=7)
        qv = ref.bf16_bits(s.rng.standard_normal((s.T, 8 * 128)))
        s.table[0, 1] = page
        s.lens[2] = 64 * s.width + 1
        s.to_device()
        print("bad page", page, flush=True)
        got = run_decode(s, 8, qv, max_len=200)
        assert np.isnan(ref.bf16_val(got[0])).all() and np.isnan(ref.bf16_val(got[2])).all()
        check_decode(s, 8, qv, got, skip=(0, 2))


def test_decode_large_and_small_queries():
    """Query rows far from one in magnitude are scaled into fp16 exactly."""
    for mag in (1e-20, 1e-4, 3e5):
        s = Setup(NVFP4, 1, 128, 64, [90], [1], seed=9, vary=(1.0 / max(mag, 1.0), 1.0))
        qv = ref.bf16_bits(mag * s.rng.standard_normal((s.T, 4 * 128)))
        check_decode(s, 4, qv, run_decode(s, 4, qv))


def append_inputs(s, n_q, seed):
    rng = np.random.default_rng(seed)
    w = (n_q + 2 * s.n_kv) * s.D
    return ref.bf16_bits(rng.standard_normal((s.T, w)) * 2.0)


def run_append(s, n_q, qkv, norm, rot, inter, freq, scale, pos=None, in_place=False, k_out=True,
               eps=1e-6):
    D = s.D
    w, kw = (n_q + 2 * s.n_kv) * D, s.n_kv * D
    x = to_dev(qkv)
    nq, nk = (torch.from_numpy(n).to(dev) if n is not None else None for n in norm)
    f = torch.from_numpy(freq).to(dev)
    d = q.QkvDesc(n_q, eps, nq.data_ptr() if nq is not None else None,
                  nk.data_ptr() if nk is not None else None, rot, inter, f.data_ptr(), scale)
    p = i32(pos) if pos is not None else None
    if in_place:
        qo, ko, qs, ks = x, x.data_ptr() + 2 * n_q * D, w, w
    else:
        qo = torch.full((s.T, n_q * D), 7.0, dtype=torch.bfloat16, device=dev)
        ko = torch.full((s.T, kw), 7.0, dtype=torch.bfloat16, device=dev) if k_out else None
        qs, ks = n_q * D, kw
    q.moe_kv_append(s.cache, d, s.seqs, x, w, s.T, p, qo, qs, ko, ks)
    torch.cuda.synchronize()
    if in_place:
        y = bits(x)
        return y[:, :n_q * D], y[:, n_q * D:n_q * D + kw], y
    return bits(qo), (bits(ko) if k_out else None), bits(x)


def check_append(s, n_q, qkv, norm, rot, inter, freq, scale, got_q, got_k, pos=None, eps=1e-6):
    """Updates the reference pool and compares everything."""
    D, n_kv = s.D, s.n_kv
    for b, (n, L) in enumerate(zip(s.rows, s.lens)):
        for i in range(n):
            t, tok = int(s.start[b]) + i, L - n + i
            p = tok if pos is None else pos[t]
            for h in range(n_q + 2 * n_kv):
                x = qkv[t, h * D:(h + 1) * D]
                if h < n_q + n_kv:
                    y = ref.norm_rotate(ref.bf16_val(x), norm[0 if h < n_q else 1], eps, p, rot, inter, freq, scale)
                    have = got_q[t, h * D:(h + 1) * D] if h < n_q else got_k[t, (h - n_q) * D:(h - n_q + 1) * D]
                    err = np.abs(ref.bf16_val(have) - y)
                    assert (err <= 2.0 ** -8 * np.abs(y) + 1e-38).all(), (b, i, h)
                    x = ref.bf16_bits(y)
                if h >= n_q and tok >= 0:
                    kh = h - n_q if h < n_q + n_kv else h - n_q - n_kv
                    page = s.table[b, tok // s.P] if tok // s.P < s.width else -1
                    if 0 <= page < s.ref.n_pages:
                        s.ref.put(0 if h < n_q + n_kv else 1, page, tok % s.P, kh, x)
    assert np.array_equal(s.pool.cpu().numpy(), s.ref.pool)


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
@pytest.mark.parametrize("D,P,rot,inter,normed", [
    (128, 64, 128, 0, 1), (64, 32, 16, 1, 1), (256, 128, 96, 0, 0), (128, 32, 48, 0, 1),
    (128, 256, 0, 0, 1), (256, 32, 256, 1, 1)])
def test_append_matches_reference(fmt, D, P, rot, inter, normed):
    """Cache bytes equal to the reference's (tokens, stale places and unused
    pages alike), queries and keys within one rounding; sequences of one row,
    several, none, one that starts inside a page and crosses into the next."""
    n_q, n_kv = 6, 2
    s = Setup(fmt, n_kv, D, P, [1, P + 3, 40, 7], [1, 6, 0, 2], seed=D + P, k_ts=0.5, v_ts=1.7)
    qkv = append_inputs(s, n_q, 1)
    rng = np.random.default_rng(2)
    norm = [(1 + 0.2 * rng.standard_normal(D)).astype(np.float32) if normed else None for _ in range(2)]
    freq, _ = q.moe_rope_freqs(q.MOE_ROPE_PLAIN, max(rot, 16), 10000.0)
    print("append", FMT[fmt], D, P, rot, inter, normed, flush=True)
    got_q, got_k, _ = run_append(s, n_q, qkv, norm, rot, inter, freq, 1.0)
    check_append(s, n_q, qkv, norm, rot, inter, freq, 1.0, got_q, got_k)
    assert (got_q[int(s.start[-1]):] == ref.bf16_bits([7.0])[0]).all()
    assert (got_k[int(s.start[-1]):] == ref.bf16_bits([7.0])[0]).all()


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
@pytest.mark.parametrize("D,n_kv", [(64, 3), (64, 9), (128, 5), (256, 3)])
def test_append_whole_and_part_quads(fmt, D, n_kv):
    """Tokens are written four at a time where a call holds all four: prompts
    that start and end inside a quad and cross pages, more than 64 sequences
    before them, fewer tokens than rows."""
    n_q = n_kv
    lens = [1] * 66 + [13, 43, 3, 8]
    rows = [1] * 30 + [0] * 36 + [13, 38, 5, 8]
    s = Setup(fmt, n_kv, D, 32, lens, rows, seed=D + n_kv, v_ts=1.5, pad_rows=1)
    qkv = append_inputs(s, n_q, 6)
    norm = [np.ones(D, np.float32)] * 2
    freq, _ = q.moe_rope_freqs(q.MOE_ROPE_PLAIN, 32, 10000.0)
    print("append quads", FMT[fmt], D, n_kv, flush=True)
    got_q, got_k, _ = run_append(s, n_q, qkv, norm, 32, 0, freq, 1.0)
    check_append(s, n_q, qkv, norm, 32, 0, freq, 1.0, got_q, got_k)
    assert (got_q[int(s.start[-1]):] == ref.bf16_bits([7.0])[0]).all()


@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_append_norms_of_tiny_and_huge_heads(eps):
    """Heads whose squares lie outside fp32: the largest and the smallest bf16
    values, and some between."""
    n_q, D = 9, 64
    s = Setup(BF16, 1, D, 32, [9], [9], seed=12, pad_rows=0)
    qkv = append_inputs(s, n_q, 7)
    x = ref.bf16_val(qkv).reshape(s.T, n_q + 2, D)
    x = np.clip(x / 8, -0.99, 0.99)
    for t, m in enumerate([1e-37, 2.0 ** -120, 1e-25, 1e-19, 1.0, 1e18, 1e20, 1e30, 3e38]):
        x[t] *= m
    x[0, 3], x[0, 9] = 2.0 ** -133, -(2.0 ** -133)  # the smallest there is
    qkv = ref.bf16_bits(x.reshape(s.T, -1))
    norm = [np.full(D, 1.5, np.float32)] * 2
    freq, _ = q.moe_rope_freqs(q.MOE_ROPE_PLAIN, 64, 10000.0)
    print("append, tiny and huge", eps, flush=True)
    got_q, got_k, _ = run_append(s, n_q, qkv, norm, 64, 0, freq, 1.0, eps=eps)
    check_append(s, n_q, qkv, norm, 64, 0, freq, 1.0, got_q, got_k, eps=eps)


def test_append_far_positions_scaled_and_given():
    """Positions near 2^31 given by the caller, frequencies interpolated by
    parts with their factor on cosines and sines; queries and keys written in
    place, the values' part of the rows untouched."""
    n_q, n_kv, D = 5, 1, 128
    s = Setup(NVFP4, n_kv, D, 64, [9, 3], [4, 3], seed=1)
    qkv = append_inputs(s, n_q, 3)
    freq, scale = q.moe_rope_freqs(q.MOE_ROPE_PARTS, 128, 1e6, 32.0, 4096.0, 1.0, 32.0)
    pos = [2147483647, 1048575, 999999, 0, 262144, 5, 1 << 30, 0, 0]
    norm = [np.ones(D, np.float32)] * 2
    got_q, got_k, whole = run_append(s, n_q, qkv, norm, 128, 0, freq, scale, pos, in_place=True)
    check_append(s, n_q, qkv, norm, 128, 0, freq, scale, got_q, got_k, pos)
    assert np.array_equal(whole[:, -D:], qkv[:, -D:])


def test_append_special_values_and_bad_places():
    """Zero, tiny, huge, infinite and NaN blocks are held as stated; tokens
    without a page, or before the sequence's first token, are not stored."""
    for fmt in (NVFP4, Q8_0, BF16):
        D, n_kv = 128, 1
        s = Setup(fmt, n_kv, D, 32, [8, 3, 40], [8, 5, 2], seed=4, v_ts=2.0)
        s.table[2, 1] = -1
        s.to_device()
        qkv = append_inputs(s, 1, 5)
        v = qkv[:, 2 * D:].copy()
        v[0] = 0
        v[1, :16] = ref.bf16_bits(np.full(16, 1e-30))
        v[2] = ref.bf16_bits(np.full(D, 3e38) * np.where(np.arange(D) % 2, 1, -1))
        v[3, 5] = ref.bf16_bits([np.inf])[0]
        v[4, 70] = 0xffc0
        v[5] = ref.bf16_bits(np.linspace(-1, 1, D) * 1e-4)
        v[6] = ref.bf16_bits(np.full(D, 65000.0))
        v[7] = 0x8000
        qkv[:, 2 * D:] = v
        norm = [None, None]
        freq = np.zeros(8)
        print("append special", FMT[fmt], flush=True)
        got_q, got_k, _ = run_append(s, 1, qkv, norm, 0, 0, freq, 1.0)
        check_append(s, 1, qkv, norm, 0, 0, freq, 1.0, got_q, got_k)


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_read_matches_reference(fmt, D):
    """Ranges that start and end inside pages and 16-token units, room for
    fewer rows than tokens, pages that are not there (NaN), rows beyond."""
    s = Setup(fmt, 2, D, 32, [70, 1, 0, 33, 40], [0] * 5, seed=D, k_ts=0.3, v_ts=1.1)
    s.table[4, 1] = -5
    s.to_device()
    first = [5, 0, 0, 31, 30]
    count = [65, 1, 0, 2, 10]
    room = [65, 1, 0, 1, 10]
    start = np.concatenate([[0], np.cumsum(room)])
    R = int(start[-1]) + 3
    print("read", FMT[fmt], D, flush=True)
    st = 2 * D + 8
    ko = torch.full((R, st), 7.0, dtype=torch.bfloat16, device=dev)
    vo = torch.full((R, st), 7.0, dtype=torch.bfloat16, device=dev)
    q.moe_kv_read(s.cache, s.seqs, i32(first), i32(start), R, ko, st, vo, st)
    torch.cuda.synchronize()
    want = np.full((2, R, st), ref.bf16_bits([7.0])[0], np.uint16)
    nan = np.zeros((R, st), bool)
    for b in range(5):
        for j in range(min(count[b], room[b])):
            tok, row = first[b] + j, start[b] + j
            page = s.table[b, tok // 32]
            for h in range(2):
                c = slice(h * D, (h + 1) * D)
                if page < 0:
                    nan[row, c] = True
                    continue
                for w in (0, 1):
                    x = s.ref.get(w, page, tok % 32, h).astype(np.float64)
                    want[w, row, c] = ref.bf16_bits(x)
    for w, got in ((0, bits(ko)), (1, bits(vo))):
        assert np.isnan(ref.bf16_val(got[nan])).all()
        assert np.array_equal(ref.bf16_val(got[~nan]), ref.bf16_val(want[w][~nan])), w


def run_prompt(n_q, n_kv, D, qs, ks, T, Tk, qv, kv, vv, v_off=0, in_place=False):
    """qv [T, n_q D], kv, vv [Tk, n_kv D] bf16 bits; values inside wider rows."""
    kw = n_kv * D
    qd, kd = to_dev(qv), to_dev(kv)
    wide = torch.zeros(max(Tk, 1), kw + v_off + 8, dtype=torch.bfloat16, device=dev)
    wide[:Tk, v_off:v_off + kw] = to_dev(vv)
    out = qd if in_place else torch.full((T, n_q * D), 7.0, dtype=torch.bfloat16, device=dev)
    ksd = None if ks is None else i32(ks)
    q.moe_attn_prompt(n_q, n_kv, D, len(qs) - 1, i32(qs), ksd, T, Tk, qd, n_q * D, kd, kw,
                      wide.data_ptr() + 2 * v_off, kw + v_off + 8, 1 / math.sqrt(D), out, n_q * D)
    torch.cuda.synchronize()
    return bits(out)


def check_prompt(n_q, n_kv, D, qs, ks, qv, kv, vv, got, rows=None):
    ks = qs if ks is None else ks
    G = n_q // n_kv
    scale = float(np.float32(1 / math.sqrt(D)))
    for b in range(len(qs) - 1):
        n, L = qs[b + 1] - qs[b], ks[b + 1] - ks[b]
        for h in range(n_kv):
            c = slice(h * D, (h + 1) * D)
            k, v = ref.bf16_val(kv[ks[b]:ks[b + 1], c]), ref.bf16_val(vv[ks[b]:ks[b + 1], c])
            for i in (range(n) if rows is None else [x for x in rows if x < n]):
                lim = L - n + i
                for g in range(G):
                    e = slice((h * G + g) * D, (h * G + g + 1) * D)
                    want, pv, qk = ref.attend(ref.bf16_val(qv[qs[b] + i, e]), k, v, lim, scale)
                    have = ref.bf16_val(got[qs[b] + i, e])
                    fin = np.isfinite(want)
                    assert np.array_equal(np.isnan(want), np.isnan(have)), (b, i, h, g)
                    assert np.array_equal(want[~fin & ~np.isnan(want)], have[~fin & ~np.isnan(want)])
                    bound = ref.attend_bound(want[fin], pv[fin], qk, max(lim + 1, 0), 0.0, D, BF16)
                    err = np.abs(have[fin] - want[fin])
                    assert (err <= bound).all(), (b, i, h, g, float((err / bound).max()))


@pytest.mark.parametrize("n_q,n_kv,D,qlen,klen", [
    (8, 2, 128, [1, 63, 64, 65, 130], None),
    (2, 2, 64, [200, 1, 33], None),
    (5, 1, 256, [70, 129], None),
    (4, 1, 128, [5, 40, 0, 128], [200, 40, 17, 500]),   # chunks behind longer keys
    (6, 3, 64, [20, 9], [7, 0]),                        # fewer keys than rows: rows that see nothing
    (16, 2, 128, [300], None),
])
def test_prompt_matches_reference(n_q, n_kv, D, qlen, klen):
    rng = np.random.default_rng(D + len(qlen))
    qs = np.concatenate([[0], np.cumsum(qlen)]).tolist()
    ks = None if klen is None else np.concatenate([[0], np.cumsum(klen)]).tolist()
    T, Tk = qs[-1] + 2, (qs if ks is None else ks)[-1] + (2 if ks is None else 0)
    qv = ref.bf16_bits(1.5 * rng.standard_normal((T, n_q * D)))
    kv, vv = (ref.bf16_bits(rng.standard_normal((Tk, n_kv * D))) for _ in range(2))
    print("prompt", n_q, n_kv, D, qlen, klen, flush=True)
    got = run_prompt(n_q, n_kv, D, qs, ks, T, Tk, qv, kv, vv, v_off=16)
    check_prompt(n_q, n_kv, D, qs, ks, qv, kv, vv, got)
    assert (got[qs[-1]:] == ref.bf16_bits([7.0])[0]).all()
    assert np.array_equal(run_prompt(n_q, n_kv, D, qs, ks, T, Tk, qv, kv, vv, in_place=True)[:qs[-1]], got[:qs[-1]])


def test_prompt_many_sequences():
    """More sequences than lanes: empty ones, and prompts on both sides of 64 and 128 of them."""
    qlen = [(5 * b) % 7 for b in range(150)]
    qlen[62:66], qlen[127:130] = [70, 1, 0, 131], [0, 40, 66]
    klen = [n + (b % 3) * 40 for b, n in enumerate(qlen)]
    rng = np.random.default_rng(3)
    for D in (64, 128):
        qs, ks = (np.concatenate([[0], np.cumsum(x)]).tolist() for x in (qlen, klen))
        qv = ref.bf16_bits(1.5 * rng.standard_normal((qs[-1] + 2, 2 * D)))
        kv, vv = (ref.bf16_bits(rng.standard_normal((ks[-1], D))) for _ in range(2))
        print("prompt, 150 sequences", D, flush=True)
        got = run_prompt(2, 1, D, qs, ks, qs[-1] + 2, ks[-1], qv, kv, vv)
        check_prompt(2, 1, D, qs, ks, qv, kv, vv, got)
        assert (got[qs[-1]:] == ref.bf16_bits([7.0])[0]).all()


def test_prompt_long():
    """4200 rows behind 100 cached keys, the larger tile of rows: rows at tile ends and between,
    also with a value and a key that only later rows see being NaN."""
    n, L, D = 4200, 4300, 128
    rng = np.random.default_rng(4)
    qv = ref.bf16_bits(1.5 * rng.standard_normal((n, 2 * D)))
    kv, vv = (ref.bf16_bits(rng.standard_normal((L, D))) for _ in range(2))
    k, v, scale = ref.bf16_val(kv), ref.bf16_val(vv), float(np.float32(D ** -0.5))
    rows = sorted({0, 1, n - 1, n - 2} | set(range(255, n, 256)) | set(range(256, n, 256)) | set(range(31, n, 97)))
    for bad in (None, 2999, 3000):
        print("prompt, 4200 rows, NaN at", bad, flush=True)
        kb, vb = kv.copy(), vv.copy()
        if bad is not None:
            (kb if bad % 2 else vb)[bad, 7] = 0x7fc0
        got = run_prompt(2, 1, D, [0, n], [0, L], n, L, qv, kb, vb)
        for i in rows + [2898, 2899, 2900, 2901]:
            for h in range(2):
                c, lim = slice(h * D, (h + 1) * D), L - n + i
                have = ref.bf16_val(got[i, c])
                if bad is not None and lim >= bad:
                    assert np.isnan(have).all() if bad % 2 else np.isnan(have[7]), (bad, i, h)
                    continue
                want, pv, qk = ref.attend(ref.bf16_val(qv[i, c]), k, v, lim, scale)
                bound = ref.attend_bound(want, pv, qk, lim + 1, 0.0, D, BF16)
                assert (np.abs(have - want) <= bound).all(), (bad, i, h)


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
def test_pages_beyond_32_bit_offsets(fmt):
    """A pool of more than 4 GiB: tokens in its last pages as in the first pages of a small one."""
    n_kv, D, P, n_q = 8, 256, 256, 8
    pb = q.moe_kv_page_bytes(fmt, n_kv, D, P)
    far = (1 << 32) // pb + 3
    gen = torch.Generator(device=dev).manual_seed(6)
    qkv = torch.randn(600, (n_q + 2 * n_kv) * D, generator=gen, device=dev).bfloat16()
    got = []
    for n_pages, pages in ((3, [2, 0, 1]), (far, [far - 1, far - 3, far - 2])):
        print("pool", FMT[fmt], n_pages, flush=True)
        cache = q.KvCache(fmt, n_q, n_kv, D, P, n_pages)
        buf = q.AttnBuffers(cache, 1, 600, 3)
        buf.page_table.copy_(i32([pages]))
        buf.row_start.copy_(i32([0, 600]))
        buf.kv_len.copy_(i32([600]))
        kv = [torch.empty(600, n_kv * D, dtype=torch.bfloat16, device=dev) for _ in range(2)]
        one = q.attention_forward(cache, buf, qkv, 600, 1 / 16, (buf.row_start, 600, *kv)).clone()
        buf.row_start.copy_(i32([0, 1]))
        buf.kv_len.copy_(i32([601]))
        two = q.attention_forward(cache, buf, qkv, 1, 1 / 16)[:1].clone()
        torch.cuda.synchronize()
        got.append((one, two, *kv))
        del cache, buf
    assert all(torch.isfinite(a.float()).all() and torch.equal(a, b) for a, b in zip(*got))


def test_read_many_sequences():
    """Spans of more sequences than lanes."""
    lens = [(3 * b) % 8 for b in range(140)]
    lens[63], lens[64], lens[128] = 45, 0, 33
    s = Setup(Q8_0, 1, 64, 32, lens, [0] * 140, seed=8)
    start = np.concatenate([[0], np.cumsum(lens)])
    ko, vo = (torch.full((int(start[-1]), 64), 7.0, dtype=torch.bfloat16, device=dev) for _ in range(2))
    print("read, 140 sequences", flush=True)
    q.moe_kv_read(s.cache, s.seqs, None, i32(start), int(start[-1]), ko, 64, vo, 64)
    torch.cuda.synchronize()
    for w, got in ((0, bits(ko)), (1, bits(vo))):
        want = [s.ref.get(w, s.table[b, j // 32], j % 32, 0) for b, n in enumerate(lens) for j in range(n)]
        assert np.array_equal(got, ref.bf16_bits(np.array(want, np.float64)))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("val", [math.nan, math.inf])
def test_prompt_unseen_tokens_have_no_influence(D, val):
    """A NaN or an infinity in token 70's key or value: rows before it are as
    without it, rows from it on show it."""
    rng = np.random.default_rng(3)
    qs = [0, 100, 130]
    for which in (0, 1):
        qv = ref.bf16_bits(rng.standard_normal((130, 2 * D)))
        kv, vv = (ref.bf16_bits(rng.standard_normal((130, D))) for _ in range(2))
        (kv, vv)[which][70, 9] = ref.bf16_bits([val])[0]
        print("prompt unseen", D, val, which, flush=True)
        got = run_prompt(2, 1, D, qs, None, 130, 130, qv, kv, vv)
        assert np.isfinite(ref.bf16_val(got[:70])).all() and np.isfinite(ref.bf16_val(got[100:])).all()
        rows = [0, 5, 40, 63, 64, 69] + ([70, 71, 99] if which else [])
        check_prompt(2, 1, D, qs, None, qv, kv, vv, got, rows)
        if which == 0:
            assert np.isnan(ref.bf16_val(got[70])).any() or val == math.inf


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prompt_scores_far_above_the_first_keys(D):
    """The first tile's keys are small and later ones large: weights relative to
    the first tile's maximum leave every range, and the rows have to be done
    again with a running maximum; also keys that only get smaller."""
    rng = np.random.default_rng(D)
    for first, rest in ((0.01, 40.0), (0.01, 6.0), (20.0, 0.01)):
        mag = np.where(np.arange(190) < 64, first, rest)[:, None]
        qv = ref.bf16_bits(rng.standard_normal((190, 2 * D)))
        kv = ref.bf16_bits(rng.standard_normal((190, D)) * mag)
        vv = ref.bf16_bits(rng.standard_normal((190, D)))
        print("prompt far", D, first, rest, flush=True)
        got = run_prompt(2, 1, D, [0, 190], None, 190, 190, qv, kv, vv)
        check_prompt(2, 1, D, [0, 190], None, qv, kv, vv, got, [0, 63, 64, 65, 100, 127, 128, 189])


def test_prompt_bad_ranges_give_nan():
    """Keys that reach past Tk are not read: their sequence is NaN."""
    rng = np.random.default_rng(3)
    qv = ref.bf16_bits(rng.standard_normal((20, 128)))
    kv, vv = (ref.bf16_bits(rng.standard_normal((20, 128))) for _ in range(2))
    got = run_prompt(1, 1, 128, [0, 10, 20], [0, 10, 21], 20, 20, qv, kv, vv)
    check_prompt(1, 1, 128, [0, 10], [0, 10], qv, kv, vv, got)
    assert np.isnan(ref.bf16_val(got[10:])).all()


def test_prompt_rows_beyond_t_are_left_out():
    """The last sequence claims more rows than there are: those inside are answered, at the
    positions that its claim gives them."""
    rng = np.random.default_rng(4)
    T, L = 40, 1000
    qv = ref.bf16_bits(rng.standard_normal((T, 128)))
    kv, vv = (ref.bf16_bits(rng.standard_normal((20 + L, 128))) for _ in range(2))
    got = run_prompt(1, 1, 128, [0, 20, 920], [0, 20, 20 + L], T, 20 + L, qv, kv, vv)
    check_prompt(1, 1, 128, [0, 20, 920], [0, 20, 20 + L], qv, kv, vv, got, rows=range(20))


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
def test_prompt_chunk_then_decode_steps(fmt):
    """The operators together, as a server uses them: a prompt appended in two
    chunks (the second attends to the cached first through moe_kv_read), then
    decode steps of one and two rows; every output against the reference of the
    cache's own contents."""
    n_q, n_kv, D, P = 8, 2, 128, 32
    norm = [np.ones(D, np.float32), np.full(D, 0.9, np.float32)]
    freq, _ = q.moe_rope_freqs(q.MOE_ROPE_LINEAR, 64, 10000.0, 4.0)
    s = Setup(fmt, n_kv, D, P, [110, 75], [0, 0], seed=11)
    s.ref.pool[:] = 0xff
    kw = n_kv * D
    steps = [([40, 20], [40, 20]), ([37, 50], [77, 70]), ([1, 1], [78, 71]), ([2, 2], [80, 73])]
    for step, (rows, lens) in enumerate(steps):
        s.rows, s.lens = rows, lens
        s.start = np.concatenate([[0], np.cumsum(rows)])
        s.T = int(s.start[-1])
        keep = torch.from_numpy(s.ref.pool.copy())
        s.to_device()
        s.pool.copy_(keep)
        qkv = append_inputs(s, n_q, 20 + step)
        print("chunks", FMT[fmt], step, flush=True)
        got_q, got_k, _ = run_append(s, n_q, qkv, norm, 64, 1, freq, 1.0)
        check_append(s, n_q, qkv, norm, 64, 1, freq, 1.0, got_q, got_k)
        if step < 2:
            ks = np.concatenate([[0], np.cumsum(lens)])
            Tk = int(ks[-1])
            k, v = (torch.empty(Tk, kw, dtype=torch.bfloat16, device=dev) for _ in range(2))
            q.moe_kv_read(s.cache, s.seqs, None, i32(ks), Tk, k, kw, v, kw)
            torch.cuda.synchronize()
            got = run_prompt(n_q, n_kv, D, s.start, ks, s.T, Tk, got_q, bits(k), bits(v))
            check_prompt(n_q, n_kv, D, s.start.tolist(), ks.tolist(), got_q, bits(k), bits(v), got)
        else:
            check_decode(s, n_q, got_q, run_decode(s, n_q, got_q))


def test_step_in_a_graph_replays():
    """Append and attention of a decode step captured once; lengths, rows and
    inputs change between replays, with eager work in between."""
    n_q, n_kv, D, P = 8, 2, 128, 64
    s = Setup(NVFP4, n_kv, D, P, [700, 40, 3], [1, 1, 1], seed=2, pad_rows=0)
    w = (n_q + 2 * n_kv) * D
    x = torch.zeros(3, w, dtype=torch.bfloat16, device=dev)
    qo = torch.zeros(3, n_q * D, dtype=torch.bfloat16, device=dev)
    out = torch.zeros(3, n_q * D, dtype=torch.bfloat16, device=dev)
    f = torch.from_numpy(q.moe_rope_freqs(q.MOE_ROPE_PLAIN, 128, 10000.0)[0]).to(dev)
    nrm = torch.ones(D, device=dev)
    d = q.QkvDesc(n_q, 1e-6, nrm.data_ptr(), nrm.data_ptr(), 128, 0, f.data_ptr(), 1.0)
    nb = q.moe_attn_workspace_bytes(s.cache, n_q, 3, 3, 800)
    ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=dev)

    def step():
        q.moe_kv_append(s.cache, d, s.seqs, x, w, 3, None, qo, n_q * D)
        q.moe_attn_decode(s.cache, s.seqs, n_q, qo, n_q * D, 3, 800, 0.09, out, n_q * D, ws, nb)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        gen = torch.Generator(device=dev).manual_seed(i)
        x.copy_(torch.randn(3, w, generator=gen, device=dev).bfloat16())
        s.len_d.copy_(i32([700 - i, 40 + i % 2, 3 + i]))
        g.replay()
        torch.cuda.synchronize()
        a, pool = out.clone(), s.pool.clone()
        out.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(a.view(torch.int16), out.view(torch.int16)), i
        assert torch.equal(pool, s.pool)
        assert torch.isfinite(out.float()).all()


def test_two_streams_with_workspaces_of_their_own():
    s = Setup(Q8_0, 2, 128, 64, [500, 300], [1, 1], seed=8, pad_rows=0)
    n_q = 8
    nb = q.moe_attn_workspace_bytes(s.cache, n_q, 2, 2, 500)
    qs = [torch.randn(2, n_q * 128, device=dev).bfloat16() for _ in range(2)]
    want = []
    for x in qs:
        o, ws = torch.empty_like(x), torch.empty(max(nb, 1), dtype=torch.uint8, device=dev)
        q.moe_attn_decode(s.cache, s.seqs, n_q, x, n_q * 128, 2, 500, 0.1, o, n_q * 128, ws, nb)
        want.append(o)
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    got = [torch.empty_like(x) for x in qs]
    wss = [torch.empty(max(nb, 1), dtype=torch.uint8, device=dev) for _ in qs]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            q.moe_attn_decode(s.cache, s.seqs, n_q, qs[i], n_q * 128, 2, 500, 0.1, got[i], n_q * 128,
                              wss[i], nb, stream=st[i])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_attention_forward_then_layer_forward():
    """The binding's path: two layers of attention and experts over a prompt in
    two chunks and two decode steps give the rows of the same tokens taken in one
    chunk, up to roundings: every chunk attends to what the cache holds."""
    import moegen
    n_q, n_kv, D, P = 8, 2, 64, 32
    w = moegen.Workload(name="attn_stack", E=8, k=2, H=512, I=128, T=64)
    rope = q.moe_rope_freqs(q.MOE_ROPE_PLAIN, 64, 10000.0)
    layers = [q.DeviceLayer(moegen.make_layer(w)) for _ in range(2)]
    gen = torch.Generator(device=dev).manual_seed(1)
    proj = [torch.randn(512, (n_q + 2 * n_kv) * D, generator=gen, device=dev) / 20 for _ in range(2)]
    x_all = torch.randn(1, 60, 512, generator=gen, device=dev).bfloat16()

    def run(steps):
        caches = [q.KvCache(NVFP4, n_q, n_kv, D, P, 4, np.ones(D), np.ones(D), rope) for _ in layers]
        buf = q.AttnBuffers(caches[0], 1, 64, 2)
        sb = q.StepBuffers(layers[0], 64)
        buf.page_table.copy_(i32([[3, 1]]))
        out, at = [], 0
        for n, prompt in steps:
            buf.row_start.copy_(i32([0, n]))
            buf.kv_len.copy_(i32([at + n]))
            x = x_all[0, at:at + n].clone()
            at += n
            kv = [torch.empty(at, n_kv * D, dtype=torch.bfloat16, device=dev) for _ in range(2)]
            for cache, layer, pj in zip(caches, layers, proj):
                qkv = (x.float() @ pj).bfloat16()
                o = q.attention_forward(cache, buf, qkv, n, 0.125, (i32([0, at]), at, *kv) if prompt else None)
                x = (x.float() + o[:n].float()).bfloat16()
                x = q.layer_forward(layer, sb, x, n, x)[:n].view(torch.bfloat16).clone()
            out.append(x)
        torch.cuda.synchronize()
        return torch.cat(out), caches

    whole, c1 = run([(60, True)])
    parts, c2 = run([(37, True), (20, True), (1, False), (2, False)])
    assert torch.isfinite(whole.float()).all()
    err = (whole.float() - parts.float()).norm() / whole.float().norm()
    # a decode row's weights are fp16 and a prompt's bf16 (2^-8), the row itself
    # is rounded to bf16 a few times over in each of the two layers
    assert err < 8 * 2.0 ** -8, float(err)


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16], ids=FMT.get)
def test_buffers_for_long_prompts_serve_short_steps(fmt):
    """A prompt of 600 rows, then steps of 2 and 24 rows over long caches, in buffers made for 600
    rows: bit for bit what buffers of each step's own size give."""
    n_q, n_kv, D, P, pages = 8, 2, 128, 64, 40
    gen = torch.Generator(device=dev).manual_seed(5)
    rope = q.moe_rope_freqs(q.MOE_ROPE_LINEAR, 64, 10000.0, 4.0)
    table = i32(np.random.default_rng(2).permutation(2 * pages).reshape(2, pages))
    qkv = torch.randn(600, (n_q + 2 * n_kv) * D, generator=gen, device=dev).bfloat16()
    got = []
    for own in (False, True):
        cache = q.KvCache(fmt, n_q, n_kv, D, P, 2 * pages, rope=rope, interleaved=1)
        lens, outs, big = [0, 0], [], q.AttnBuffers(cache, 2, 600, pages)
        for rows in ([590, 10], [300, 300], [1, 1], [4, 20], [1, 1]):
            n = sum(rows)
            buf = q.AttnBuffers(cache, 2, n, pages) if own else big
            lens = [a + b for a, b in zip(lens, rows)]
            print("step", FMT[fmt], own, rows, flush=True)
            buf.page_table.copy_(table)
            buf.row_start.copy_(i32([0, rows[0], n]))
            buf.kv_len.copy_(i32(lens))
            prompt = None
            if n > 100:
                kv = [torch.empty(sum(lens), n_kv * D, dtype=torch.bfloat16, device=dev) for _ in range(2)]
                prompt = (i32([0, lens[0], sum(lens)]), sum(lens), *kv)
            outs.append(q.attention_forward(cache, buf, qkv[:n], n, D ** -0.5, prompt)[:n].clone())
        torch.cuda.synchronize()
        got.append(torch.cat(outs))
    assert torch.isfinite(got[0].float()).all() and torch.equal(got[0], got[1])
