"""Contract checks of the key/value cache and attention calls that need no GPU:
sizes, refusals on the host before any launch, calls without work, and the
rotary frequencies.  The reference of the GPU tests is checked here too, against
facts outside itself."""
import ctypes
import math

import numpy as np
import pytest
import torch

import attn_ref as ref
import quantized_expert_ffn_router_amd as q
from attn_ref import BF16, NVFP4, Q8_0

OK, BAD, UNSUP, WS = q.MOE_OK, q.MOE_ERR_INVALID_ARG, q.MOE_ERR_UNSUPPORTED, q.MOE_ERR_WORKSPACE
A = 0x1000  # a non-NULL, aligned address that must never be read


def cache(fmt=NVFP4, n_kv=2, D=128, P=64, n_pages=4, ks=1.0, vs=1.0, pool=A):
    return q.KvCacheDesc(fmt, n_kv, D, P, n_pages, ks, vs, pool)


def seqs(n=2, width=4, start=A, lens=A, table=A):
    return q.SeqBatch(n, width, start, lens, table)


def qkv(n_q=8, eps=1e-6, qn=A, kn=A, rot=128, inter=0, freq=A, scale=1.0):
    return q.QkvDesc(n_q, eps, qn, kn, rot, inter, freq, scale)


def append(c=None, p=None, s=None, x=A, xs=12 * 128, T=4, pos=None, qo=A, qs=1024, ko=None, ks=0):
    c, p, s = c or cache(), p or qkv(), s or seqs()
    return q.lib().moe_kv_append(ctypes.byref(c), ctypes.byref(p), ctypes.byref(s), x, xs, T, pos, qo,
                                 qs, ko, ks, None)


def read(c=None, s=None, first=None, start=A, R=4, ko=A, ks=256, vo=A, vs=256):
    c, s = c or cache(), s or seqs()
    return q.lib().moe_kv_read(ctypes.byref(c), ctypes.byref(s), first, start, R, ko, ks, vo, vs, None)


def decode(c=None, s=None, n_q=8, x=A, xs=1024, T=2, max_len=8192, scale=0.1, out=A, os=1024, ws=A,
           wb=1 << 30):
    c, s = c or cache(), s or seqs()
    return q.lib().moe_attn_decode(ctypes.byref(c), ctypes.byref(s), n_q, x, xs, T, max_len, scale, out,
                                   os, ws, wb, None)


def prompt(n_q=8, n_kv=2, D=128, n=2, qs=A, ks=None, T=4, Tk=4, x=A, xst=1024, k=A, kst=256, v=A,
           vst=256, scale=0.1, out=A, os=1024):
    return q.lib().moe_attn_prompt(n_q, n_kv, D, n, qs, ks, T, Tk, x, xst, k, kst, v, vst, scale, out,
                                   os, None)


def test_page_bytes():
    assert q.moe_kv_page_bytes(NVFP4, 4, 128, 64) == 4 * 64 * 2 * (64 + 8)
    assert q.moe_kv_page_bytes(Q8_0, 2, 64, 32) == 2 * 32 * 2 * (64 + 4)
    assert q.moe_kv_page_bytes(BF16, 1, 256, 256) == 256 * 2 * 512
    for fmt in (NVFP4, Q8_0, BF16):
        for D in (64, 128, 256):
            for P in (32, 64, 128, 256):
                assert q.moe_kv_page_bytes(fmt, 3, D, P) % 256 == 0
                assert q.moe_kv_page_bytes(fmt, 3, D, P) == 3 * ref.Cache(fmt, 3, D, P, 1).head
    assert q.moe_kv_page_bytes(2, 4, 128, 64) == 0 and "format" in q.last_error()
    assert q.moe_kv_page_bytes(NVFP4, 4, 96, 64) == 0 and "D=96" in q.last_error()
    assert q.moe_kv_page_bytes(NVFP4, 4, 128, 48) == 0 and "page_tokens" in q.last_error()
    assert q.moe_kv_page_bytes(NVFP4, 0, 128, 64) == 0


@pytest.mark.parametrize("call", [append, read, decode])
@pytest.mark.parametrize("kw,status,msg", [
    (dict(fmt=5), UNSUP, "cache format 5"), (dict(D=32), UNSUP, "D=32"), (dict(P=16), UNSUP, "page_tokens=16"),
    (dict(n_kv=0), UNSUP, "n_kv=0"), (dict(n_pages=0), BAD, "n_pages=0"), (dict(ks=0.0), BAD, "k_scale"),
    (dict(vs=math.inf), BAD, "v_scale"), (dict(ks=math.nan), BAD, "k_scale"), (dict(pool=None), BAD, "pool is NULL"),
    (dict(pool=A + 16), BAD, "256-byte")])
def test_cache_refusals(call, kw, status, msg):
    assert call(c=cache(**kw)) == status
    assert msg in q.last_error()


@pytest.mark.parametrize("call,rows", [(append, True), (read, False), (decode, True)])
def test_sequence_refusals(call, rows):
    for s, st, msg in ((seqs(n=-1), BAD, "n_seq"), (seqs(n=65536), UNSUP, "n_seq"), (seqs(width=0), BAD, "max_pages"),
                       (seqs(lens=None), BAD, "kv_len"), (seqs(table=None), BAD, "page_table")):
        assert call(s=s) == st and msg in q.last_error()
    if rows:
        assert call(s=seqs(start=None)) == BAD and "row_start" in q.last_error()


@pytest.mark.parametrize("kw,status,msg", [
    (dict(p=qkv(n_q=7)), BAD, "n_q=7"), (dict(p=qkv(n_q=2048)), UNSUP, "n_q=2048"), (dict(p=qkv(eps=-1.0)), BAD, "eps"),
    (dict(p=qkv(eps=math.nan)), BAD, "eps"), (dict(p=qkv(rot=24)), UNSUP, "rot_dim=24"), (dict(p=qkv(rot=144)), UNSUP, "rot_dim=144"),
    (dict(p=qkv(inter=2)), BAD, "interleaved"), (dict(p=qkv(freq=None)), BAD, "inv_freq"), (dict(p=qkv(scale=math.inf)), BAD, "rope_scale"),
    (dict(T=-1), BAD, "T=-1"), (dict(T=1 << 25), UNSUP, "too large"), (dict(x=None), BAD, "qkv is NULL"),
    (dict(xs=1528), BAD, "qkv stride"), (dict(xs=1540), BAD, "qkv stride"), (dict(x=A + 8), BAD, "qkv is not 16-byte"),
    (dict(qo=None), BAD, "q_out is NULL"), (dict(qs=1016), BAD, "q_out stride"), (dict(ko=A, ks=128), BAD, "k_out stride"),
    (dict(p=qkv(qn=A + 4)), BAD, "q_norm"), (dict(p=qkv(kn=A + 4)), BAD, "k_norm")])
def test_append_refusals(kw, status, msg):
    assert append(**kw) == status
    assert msg in q.last_error()


def test_read_decode_and_prompt_refusals():
    for call, kw, status, msg in [
            (read, dict(R=-1), BAD, "R=-1"), (read, dict(start=None), BAD, "out_start"), (read, dict(ks=128), BAD, "k_out stride"),
            (read, dict(vo=A + 2), BAD, "v_out is not"),
            (decode, dict(n_q=3), BAD, "n_q=3"), (decode, dict(scale=0.0), BAD, "scale"), (decode, dict(scale=math.nan), BAD, "scale"),
            (decode, dict(max_len=-5), BAD, "max_len"), (decode, dict(x=None), BAD, "q is NULL"), (decode, dict(os=1000), BAD, "out stride"),
            (decode, dict(ws=None), BAD, "ws is NULL"), (decode, dict(wb=64), WS, "workspace"), (decode, dict(ws=A + 8), BAD, "ws is not"),
            (prompt, dict(D=80), UNSUP, "D=80"), (prompt, dict(n=-2), BAD, "n_seq"), (prompt, dict(n=70000), UNSUP, "n_seq"),
            (prompt, dict(n_kv=0), BAD, "n_kv=0"), (prompt, dict(n_q=12, n_kv=5), BAD, "n_q=12"), (prompt, dict(scale=-1.0), BAD, "scale"),
            (prompt, dict(Tk=-1), BAD, "Tk=-1"), (prompt, dict(Tk=3), BAD, "without kv_start"), (prompt, dict(qs=None), BAD, "q_start"),
            (prompt, dict(x=None), BAD, "q is NULL"), (prompt, dict(k=None), BAD, "k is NULL"), (prompt, dict(vst=250), BAD, "v stride"),
            (prompt, dict(out=A + 4), BAD, "out is not"), (prompt, dict(kst=(1 << 24) + 8), UNSUP, "strides"), (prompt, dict(T=1 << 24), UNSUP, "too large")]:
        assert call(**kw) == status, (call.__name__, kw, q.last_error())
        assert msg in q.last_error(), (call.__name__, kw, q.last_error())
    c, p, s = cache(), qkv(), seqs()
    f = q.lib().moe_kv_append
    assert f(None, ctypes.byref(p), ctypes.byref(s), A, 1536, 4, None, A, 1024, None, 0, None) == BAD
    assert f(ctypes.byref(c), None, ctypes.byref(s), A, 1536, 4, None, A, 1024, None, 0, None) == BAD
    assert f(ctypes.byref(c), ctypes.byref(p), None, A, 1536, 4, None, A, 1024, None, 0, None) == BAD


def test_calls_without_work_launch_nothing():
    assert append(T=0, x=None, qo=None) == OK
    assert append(s=seqs(n=0, start=None, lens=None, table=None)) == OK
    assert read(R=0) == OK and read(ko=None, vo=None) == OK and read(s=seqs(n=0)) == OK
    assert decode(T=0, x=None, ws=None, wb=0) == OK and decode(s=seqs(n=0)) == OK
    assert prompt(T=0, x=None) == OK and prompt(n=0) == OK


def test_workspace_grows_with_the_longest_cache_only_as_far_as_it_helps():
    c = cache()
    one = q.moe_attn_workspace_bytes(c, 8, 1, 1, 64)
    sizes = [q.moe_attn_workspace_bytes(c, 8, 1, 1, n) for n in (64, 1000, 10000, 10 ** 6, 0)]
    assert one == 0 and sizes == sorted(sizes) and sizes[-1] == sizes[-2]
    assert q.moe_attn_workspace_bytes(c, 8, 1, 0, 64) == 0
    assert q.moe_attn_workspace_bytes(c, 7, 1, 1, 64) == 0 and "n_q=7" in q.last_error()


@pytest.mark.parametrize("fmt", [q.MOE_FMT_NVFP4, q.MOE_FMT_Q8_0, q.MOE_FMT_BF16])
@pytest.mark.parametrize("n_q,n_kv,D", [(32, 4, 128), (5, 5, 64), (16, 2, 256), (1, 1, 64)])
def test_workspace_serves_every_smaller_step(fmt, n_q, n_kv, D):
    """Buffers made for the largest step are used for all: bytes never fall as
    rows or the longest cache grow."""
    c = cache(fmt=fmt, n_kv=n_kv, D=D)
    for n_seq in (1, 8, 64, 300):
        for longest in (300, 5000, 10 ** 5):
            b = [q.moe_attn_workspace_bytes(c, n_q, n_seq, t, longest) for t in (*range(1, 600, 7), 5000, 60000)]
            assert b == sorted(b), (n_seq, longest)
        for t in (1, 9, 100, 600):
            b = [q.moe_attn_workspace_bytes(c, n_q, n_seq, t, n) for n in (1, 384, 385, 1000, 9999, 10 ** 7, 0)]
            assert b == sorted(b), (n_seq, t)


def test_attention_forward_refuses_what_its_buffers_cannot_hold():
    c = q.KvCache(NVFP4, 8, 2, 64, 32, 4, device="cpu")
    buf = q.AttnBuffers(c, 1, 6, 2, device="cpu")
    qkv = torch.zeros(7, 12 * 64, dtype=torch.bfloat16)
    with pytest.raises(q.MoeError, match="T_max=6"):
        q.attention_forward(c, buf, qkv, 7, 0.125)
    k, v = torch.zeros(40, 128, dtype=torch.bfloat16), torch.zeros(39, 128, dtype=torch.bfloat16)
    with pytest.raises(q.MoeError, match="Tk=40"):
        q.attention_forward(c, buf, qkv, 6, 0.125, prompt=(buf.kv_len, 40, k, v))


def test_rope_frequencies():
    f, s = q.moe_rope_freqs(q.MOE_ROPE_PLAIN, 64, 10000.0)
    i = np.arange(32)
    assert s == 1.0 and np.allclose(f, 10000.0 ** (-i / 32), rtol=1e-14)
    g, s = q.moe_rope_freqs(q.MOE_ROPE_LINEAR, 64, 10000.0, 8.0)
    assert s == 1.0 and np.allclose(g, f / 8, rtol=1e-15)
    g, s = q.moe_rope_freqs(q.MOE_ROPE_BASE, 64, 10000.0, 8.0)
    assert s == 1.0 and g[0] == 1.0 and math.isclose(g[-1], f[-1] / 8, rel_tol=1e-12)
    assert (np.diff(g / f) < 0).all()
    g, s = q.moe_rope_freqs(q.MOE_ROPE_PARTS, 64, 10000.0, 8.0, 4096.0, 1.0, 32.0)
    turns = 4096 * f / (2 * math.pi)
    assert math.isclose(s, 0.1 * math.log(8) + 1, rel_tol=1e-6)
    assert np.allclose(g[turns >= 32], f[turns >= 32], rtol=1e-14)
    assert np.allclose(g[turns <= 1], f[turns <= 1] / 8, rtol=1e-14)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (g[mid] < f[mid]).all() and (g[mid] > f[mid] / 8).all()
    # the share kept is linear in the index
    kept = (g - f / 8) / (f - f / 8)
    assert np.allclose(np.diff(kept[mid], 2), 0, atol=1e-12)
    for kw in (dict(kind=9), dict(kind=q.MOE_ROPE_LINEAR, factor=0.5), dict(kind=q.MOE_ROPE_PARTS, factor=2.0, orig_len=0.0),
               dict(kind=q.MOE_ROPE_PARTS, factor=2.0, orig_len=4096.0, turns_lo=40.0), dict(base=1.0), dict(rot_dim=24),
               dict(rot_dim=512)):
        with pytest.raises(q.MoeError):
            q.moe_rope_freqs(**{**dict(kind=q.MOE_ROPE_PLAIN, rot_dim=64, base=10000.0), **kw})


# ------------------------------------------------------- pins of the reference

def test_reference_e2m1_rounding_is_nearest_even():
    r = np.linspace(-7, 7, 4001).astype(np.float32)
    got = ref.E2M1[ref.e2m1_code(r)]
    best = np.abs(r[:, None].astype(np.float64) - ref.E2M1[None]).min(1)
    assert np.allclose(np.abs(r - got), best, atol=0)
    ties = {0.25: 0.0, 0.75: 1.0, 1.25: 1.0, 1.75: 2.0, 2.5: 2.0, 3.5: 4.0, 5.0: 4.0}
    for t, want in ties.items():
        assert ref.E2M1[ref.e2m1_code(np.float32([t, -t]))].tolist() == [want, -want]


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16])
def test_reference_cache_places_are_disjoint_and_values_near(fmt):
    """Every byte of a page is written by exactly the places that own it, and a
    stored value is within half a step of its block's grid."""
    for D, P in ((64, 32), (128, 64), (256, 32)):
        c = ref.Cache(fmt, 1, D, P, 1, fill=0)
        seen = np.zeros(c.head, np.int64)
        for w in (0, 1):
            for o in range(P):
                at, nib = c.code_at(w, o, np.arange(D))
                np.add.at(seen, at, 1 if fmt == NVFP4 else 2)
                if fmt == BF16:
                    np.add.at(seen, at + 1, 2)
                else:
                    n = D // (16 if fmt == NVFP4 else 32)
                    p = c.scale_at(w, o, np.arange(n))
                    np.add.at(seen, p, 2)
                    if fmt == Q8_0:
                        np.add.at(seen, p + 1, 2)
        assert (seen == 2).all()
        x = np.random.default_rng(D).standard_normal(D)
        u = ref.bf16_bits(x)
        c.put(1, 0, 5, 0, u)
        got, v = c.get(1, 0, 5, 0), ref.bf16_val(u)
        if fmt == BF16:
            assert np.array_equal(got, v)
        else:
            n = 16 if fmt == NVFP4 else 32
            top = np.abs(v).reshape(-1, n).max(1).repeat(n)
            # NVFP4: half of the widest gap (4..6 of 6) plus the scale's rounding, 2^-4
            step = top / 6 * (1 + 2 ** -4) + top * 2.0 ** -4 if fmt == NVFP4 else top / 254 * (1 + 2.0 ** -10)
            assert (np.abs(got - v) <= step).all()


def test_reference_attention_and_rotation_against_torch():
    rng = np.random.default_rng(0)
    qv, k, v = rng.standard_normal(64), rng.standard_normal((20, 64)), rng.standard_normal((20, 64))
    want = torch.softmax(torch.from_numpy(k[:12] @ qv) * 0.125, 0).numpy() @ v[:12]
    got, _, _ = ref.attend(qv, k, v, 11, 0.125)
    assert np.allclose(got, want, atol=1e-13)
    assert (ref.attend(qv, k, v, -1, 0.125)[0] == 0).all()
    f = 10000.0 ** (-np.arange(16) / 16)
    for inter in (0, 1):  # a rotation keeps lengths, and products of equal distances
        x, y = rng.standard_normal(64), rng.standard_normal(64)
        a = [ref.norm_rotate(x, None, 0, p, 32, inter, f, 1.0) for p in (7, 107)]
        b = [ref.norm_rotate(y, None, 0, p, 32, inter, f, 1.0) for p in (3, 103)]
        assert math.isclose(a[0] @ a[0], x @ x, rel_tol=1e-12)
        assert math.isclose(a[0] @ b[0], a[1] @ b[1], rel_tol=1e-9)
        assert np.array_equal(a[0][32:], x[32:])
    n = ref.norm_rotate(np.full(64, 3.0), np.ones(64), 0.0, 0, 0, 0, f, 1.0)
    assert np.allclose(n, 1.0)


# ------------------------------------------------- outputs in their inputs' place

def refused(call, **kw):
    return call(**kw) == BAD and "overlaps" in q.last_error()


def test_outputs_overlap_inputs_only_in_their_own_place():
    w = 12 * 128  # elements of a row: 8 query, 2 key and 2 value heads of 128
    behind = A + 2 * 4 * w  # the first address behind the 4 rows
    for kw in (dict(qs=w + 8), dict(qo=A + 16, qs=w), dict(qo=A - 16, qs=w), dict(qo=A + 2 * 1016, T=1),
               dict(qo=A + 2 * 3 * w + 16), dict(qs=w, ko=A, ks=w), dict(qs=w, ko=A + 2 * 1024, ks=w + 8),
               dict(qs=w, ko=A + 2 * 1024 + 16, ks=w), dict(qo=behind, ko=behind + 2 * 1016, ks=1024)):
        assert refused(append, **kw), (kw, q.last_error())
    for out, x, os, xs in ((A, A, 1032, 1024), (A, A + 16, 1024, 1024), (A + 16, A, 1024, 1024), (A + 16, A, 1200, 1200),
                           (A + 2 * 1104, A, 1200, 1200), (A + 2 * 1104, A, 1600, 1200)):
        assert refused(decode, out=out, x=x, os=os, xs=xs), (out, x, os, xs, q.last_error())
        assert refused(prompt, out=out, x=x, os=os, xst=xs, k=A << 9, v=A << 9), (out, x, os, xs, q.last_error())
    for kw in (dict(v=A + 2 * 1016), dict(v=A, vst=1024), dict(v=A + 2 * 3 * 1024, vst=1024), dict(k=A + 16), dict(k=A, kst=1024)):
        assert refused(prompt, **{"k": A << 9, "v": A << 9, **kw}), (kw, q.last_error())
    for kw in (dict(), dict(vo=A + 16), dict(vo=A + 2 * 3 * 256, vs=512), dict(ks=512, vs=512, vo=A + 2 * 248)):
        assert refused(read, **kw), (kw, q.last_error())


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16])
def test_pages_made_at_once_read_back_byte_by_byte(fmt):
    import attn_pages
    for n_kv, D, P in ((2, 64, 32), (1, 128, 64), (3, 256, 32)):
        gen = torch.Generator().manual_seed(D)
        lens = [70, 1, 33]
        pool, table, kv = attn_pages.make(fmt, n_kv, D, P, lens, gen, "cpu", 0.75, 1.5)
        c = ref.Cache(fmt, n_kv, D, P, pool.numel() // q.moe_kv_page_bytes(fmt, n_kv, D, P), 0.75, 1.5)
        c.pool = pool.numpy()
        for b, L in enumerate(lens):
            for h in range(n_kv):
                got = c.tokens(table[b].numpy(), L, h)
                for w in (0, 1):
                    assert np.array_equal(got[w], kv[b][w][:, h].numpy()), (D, b, h, w)
    x, k, v = (torch.randn(4, 64, dtype=torch.float64, generator=gen), *(torch.randn(20, 64, dtype=torch.float64, generator=gen) for _ in range(2)))
    want, _ = attn_pages.attend(x, k, v, torch.tensor([0, 5, 19, 11]), 0.2, fmt, 64)
    for i, lim in enumerate((0, 5, 19, 11)):
        assert np.allclose(want[i].numpy(), ref.attend(x[i].numpy(), k.numpy(), v.numpy(), lim, 0.2)[0], atol=1e-13)


@pytest.mark.parametrize("fmt", [NVFP4, Q8_0, BF16])
def test_a_part_of_a_long_sequence_left_out_is_outside_the_bounds(fmt):
    import attn_pages
    gen = torch.Generator().manual_seed(1)
    for D in (64, 128, 256):
        L = 1 << 14
        k, v = attn_pages.make(fmt, 1, D, 64, [L], gen, "cpu")[2][0]
        x = 1.5 * torch.randn(2, D, dtype=torch.float64, generator=gen)
        want, bound = attn_pages.attend(x, k[:, 0], v[:, 0], torch.tensor([L - 1, L - 1]), D ** -0.5, fmt, 4096)
        for part in (0, 100, 255):
            keep = torch.arange(L) * 256 // L != part
            less, _ = attn_pages.attend(x, k[keep, 0], v[keep, 0], torch.tensor([L, L]), D ** -0.5, fmt, 4096)
            assert (((less - want).abs() / bound).max(1).values > 8).all(), (D, part)


@pytest.mark.parametrize("fmt,n_seq,n_kv,G,D,rows,longest", [
    (BF16, 65, 4, 8, 128, 1, 131072), (Q8_0, 65, 4, 8, 128, 1, 131072), (BF16, 33, 8, 4, 128, 1, 262144),
    (NVFP4, 65, 8, 4, 128, 1, 131072), (Q8_0, 16, 8, 2, 256, 5, 150000), (NVFP4, 300, 4, 8, 128, 1, 40000)])
def test_long_sequences_are_split_however_many_others_there_are(fmt, n_seq, n_kv, G, D, rows, longest):
    """A workspace is asked for, so a long sequence among many does not stay with one
    workgroup a head; never more than 64 MB of partial sums, and none for steps of
    too many rows."""
    c = cache(fmt=fmt, n_kv=n_kv, D=D)
    T = n_seq * rows
    b = q.moe_attn_workspace_bytes(c, n_kv * G, n_seq, T, longest)
    # (8 of D + 2 values each, and the numbers of chunks; parts are aligned to 256 bytes)
    assert T * n_kv * G * 8 * (D + 2) * 4 <= b <= (64 << 20) * (1 + 2 / D) + T * n_kv * G * 4 + 768
    most = q.moe_attn_workspace_bytes(c, n_kv * G, n_seq, 1 << 16, 0)
    assert most <= (64 << 20) * (1 + 2 / D) + (1 << 14) * 4 + 768
    assert decode(c=c, s=seqs(n=n_seq, width=1 << 13), n_q=n_kv * G, T=T, max_len=longest, xs=n_kv * G * D, os=n_kv * G * D, ws=None) == BAD
    assert "ws is NULL" in q.last_error()
