"""The attention-side operators of the library, in plain form and as a user's program calls them.

moe_kv_append   per-head norms of queries and keys, rotary positions, and keys and values quantised
                into a paged cache
moe_kv_read     cached keys and values read back as bf16 rows
moe_attn_decode attention of each sequence's newest rows over the paged cache
moe_attn_prompt causal attention over whole prompts, packed sequences of different lengths

Where ``own`` is false, ``run`` computes the operators from elementary torch operations, in 32 bits
(64 for rotary angles, norms and whatever is then quantised, where the last bit decides a code).
"""
import math

import numpy as np
import torch

own = False

NVFP4, Q8_0, BF16 = 1, 3, 6
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    base = dict(n_q=32, n_kv=4, D=128, P=64, fmt=NVFP4, rot=128, inter=False)
    return [
        # One decode step of 8 request slots: one new token each, the smallest append.
        dict(base, name="append_step_8", kind="append", n_seq=8, rows=8, first=500, last=4000, all=False),
        # A chunk of a long prompt: 4096 new rows behind a cached prefix, and the whole
        # sequence read back for the prompt attention.
        dict(base, name="append_chunk_4096", kind="append", n_seq=1, rows=4096, first=12288, last=12288, all=True),
        # Prompts of different lengths in one batch; 64-wide heads, interleaved pairs, a
        # quarter of the head rotated, 8-bit cache, pages of 32.
        dict(base, name="append_ragged_q8", kind="append", n_seq=13, rows=6001, first=0, last=0, all=False,
             n_q=24, n_kv=8, D=64, P=32, fmt=Q8_0, rot=16, inter=True),
        # A whole prefill batch of 16384 tokens into the 16-bit cache.
        dict(base, name="append_prompt_16384", kind="append", n_seq=4, rows=16384, first=0, last=0, all=False, fmt=BF16, P=128),
        # Four long sequences read back, as a chunked prompt does before its attention.
        dict(base, name="read_65536", kind="read", n_seq=4, first=12000, last=16384),
        # One slot, short context: the latency of a single decode step.
        dict(base, name="decode_1x700", kind="decode", n_seq=1, rows=1, first=700, last=700),
        # All 8 slots in long conversations.
        dict(base, name="decode_8x32768", kind="decode", n_seq=8, rows=8, first=24576, last=32768),
        # Verification batches: 4 rows of each of 8 slots, lengths far apart, 8-bit cache.
        dict(base, name="decode_verify_q8", kind="decode", n_seq=8, rows=32, first=90, last=30001, fmt=Q8_0, P=32),
        # One slot that uses the whole context.
        dict(base, name="decode_1x262144", kind="decode", n_seq=1, rows=1, first=262144, last=262144, P=256),
        # A short single prompt.
        dict(base, name="prompt_1x333", kind="prompt", n_seq=1, rows=333, first=0, last=0),
        # The prefill batch, packed from prompts of different lengths.
        dict(base, name="prompt_ragged_16384", kind="prompt", n_seq=9, rows=16384, first=0, last=0),
        # One long prompt: its last 8192 rows as a chunk behind 8192 cached ones.
        dict(base, name="prompt_chunk_8192", kind="prompt", n_seq=1, rows=8192, first=8192, last=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    D = rng.choice([64, 128, 128, 128, 256])
    n_kv = rng.choice([1, 2, 4, 8])
    c = dict(n_q=n_kv * rng.choice([1, 4, 5, 8]), n_kv=n_kv, D=D, P=rng.choice([32, 64, 128, 256]),
             fmt=rng.choice([NVFP4, NVFP4, Q8_0, BF16]), rot=16 * rng.randint(1, D // 16), inter=rng.random() < 0.5,
             kind=rng.choice(["append", "append", "read", "decode", "decode", "decode", "prompt", "prompt"]))
    k, wide = c["kind"], n_kv * D  # what a token costs goes by its width: wide ones are drawn shorter
    if k == "append":
        rows = _log(rng, 1, min(9000, 80_000_000 // ((c["n_q"] + 2 * n_kv) * D)))
        c.update(rows=rows, n_seq=min(rows, rng.randint(1, 16)), all=rng.random() < 0.3)
        c["first"] = rng.choice([0, rng.randint(0, min(5000, 25_000_000 // (wide * c["n_seq"])))])
        c["last"] = c["first"] + rng.randint(0, min(1500, 8_000_000 // (wide * c["n_seq"])))
    elif k == "read":
        n = rng.randint(1, 8)
        c.update(n_seq=n, first=_log(rng, 1, min(6000, 25_000_000 // (wide * n))))
        c["last"] = c["first"] + rng.randint(0, min(1500, 8_000_000 // (wide * n)))
    elif k == "decode":
        n = rng.randint(1, 16)
        c.update(n_seq=n, rows=n * rng.choice([1, 1, 1, 2, 3, 5]), last=_log(rng, 1, min(150_000, 40_000_000 // (wide * n))))
        c["first"] = max(1, c["last"] // rng.choice([1, 2, 30]))
    else:
        rows = _log(rng, 1, 5000)
        c.update(rows=rows, n_seq=min(rows, rng.randint(1, 6)), first=rng.choice([0, 0, rng.randint(0, 2500)]))
        c["last"] = c["first"]
    return c


def _lengths(c):
    """Rows and cached tokens of each sequence: fixed by the case alone."""
    B = c["n_seq"]
    if c["kind"] == "decode":
        new = [c["rows"] // B] * B
    elif c["kind"] == "read":
        new = [0] * B
    else:  # packed rows: uneven shares, each at least one row
        w = [1.0 + (7 * b) % 5 for b in range(B)]
        new = [max(1, int(c["rows"] * x / sum(w))) for x in w]
        new[0] += c["rows"] - sum(new)
        if new[0] < 1:  # many sequences of few rows
            new = [c["rows"] // B + (b < c["rows"] % B) for b in range(B)]
    before = [c["first"] + (c["last"] - c["first"]) * b // max(1, B - 1) for b in range(B)]
    if c["kind"] == "decode":  # first..last are whole lengths, the new rows among them
        return new, [max(n, x) for n, x in zip(new, before)]
    return new, [x + n for x, n in zip(before, new)]


def _head_bytes(c):
    D, P = c["D"], c["P"]
    return P * {NVFP4: D // 2 + D // 16, Q8_0: D + D // 16, BF16: 2 * D}[c["fmt"]] * 2


# ------------------------------------------------------------------ the cache's bytes, plain

def _e2m1_code(r):
    a = r.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code | (torch.signbit(r).to(torch.uint8) << 3)


def _quantise(c, x):
    """x: bf16 [..., D] -> (codes, scales) of the cache format: NVFP4 one code (4 bits) a byte and
    E4M3 bytes [..., D/16]; Q8_0 int8 codes and fp16 [..., D/32]; bf16 as it is."""
    if c["fmt"] == BF16:
        return x, None
    if c["fmt"] == NVFP4:
        b = x.float().unflatten(-1, (-1, 16))
        s = (b.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
        d = s.float().unsqueeze(-1)
        r = torch.where(d > 0, b / d, torch.zeros_like(b))
        return _e2m1_code(r).flatten(-2), s.view(torch.uint8)
    b = x.float().unflatten(-1, (-1, 32))
    d = (b.abs().amax(-1).clamp(max=65024.0) / 127.0).half()
    f = d.float().unsqueeze(-1)
    r = torch.where(f > 0, b / f, torch.zeros_like(b))
    return r.round().clamp(-127, 127).to(torch.int8).flatten(-2), d


def _sections(c, pool):
    """Views of a pool's K codes [page, head, P, ...], K scales, V codes, V scales."""
    D, P = c["D"], c["P"]
    h = pool.view(pool.shape[0], c["n_kv"], _head_bytes(c))
    if c["fmt"] == BF16:
        n = P * D * 2
        return (h[..., :n].view(torch.bfloat16).unflatten(-1, (P, D)), None,
                h[..., n:].view(torch.bfloat16).unflatten(-1, (P // 4, D, 4)), None)
    n, s = (P * D // 2, P * D // 16) if c["fmt"] == NVFP4 else (P * D, P * D // 16)
    kq, ks, vq, vs = h[..., :n], h[..., n:n + s], h[..., n + s:2 * n + s], h[..., 2 * n + s:]
    if c["fmt"] == NVFP4:
        return (kq.unflatten(-1, (P, D // 2)), ks.unflatten(-1, (P, D // 16)),
                vq.unflatten(-1, (P // 4, 16, 4, D // 32)), vs.unflatten(-1, (D // 16, P)))
    return (kq.view(torch.int8).unflatten(-1, (P, D)), ks.view(torch.float16).unflatten(-1, (P, D // 32)),
            vq.view(torch.int8).unflatten(-1, (P // 4, D, 4)), vs.view(torch.float16).unflatten(-1, (D // 32, P)))


def _store(c, pool, page, off, k, v):
    """k, v: bf16 [n, n_kv, D] into the slots (page, off) of the pool."""
    kq, ks, vq, vs = _sections(c, pool)
    (ck, sk), (cv, sv) = _quantise(c, k), _quantise(c, v)
    if c["fmt"] == NVFP4:
        ck, cv = (x[..., 0::2] | (x[..., 1::2] << 4) for x in (ck, cv))
        vq[page, :, off // 4, :, off % 4] = cv.unflatten(-1, (16, -1))
    else:
        vq[page, :, off // 4, :, off % 4] = cv
    kq[page, :, off] = ck
    if sk is not None:
        ks[page, :, off] = sk
        vs[page, :, :, off] = sv


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _load(c, pages, dtype=torch.float32):
    """The values of whole pages: k, v [page, n_kv, P, D]."""
    kq, ks, vq, vs = _sections(c, pages)
    if c["fmt"] == BF16:
        return kq.to(dtype), vq.transpose(-1, -2).flatten(2, 3).to(dtype)
    if c["fmt"] == NVFP4:
        lut = torch.tensor(_E2M1, dtype=dtype, device=pages.device)
        val = lambda q: torch.stack((lut[(q & 15).int()], lut[(q >> 4).int()]), -1).flatten(-2)  # noqa: E731
        k = val(kq) * ks.contiguous().view(torch.float8_e4m3fn).to(dtype).repeat_interleave(16, -1)
        v = val(vq).transpose(3, 4).flatten(-2).flatten(2, 3)  # [page, head, quad, 16, 4, d] -> [.., P, D]
        v = v * vs.contiguous().view(torch.float8_e4m3fn).to(dtype).transpose(-1, -2).repeat_interleave(16, -1)
        return k, v
    k = kq.to(dtype) * ks.to(dtype).repeat_interleave(32, -1)
    v = vq.transpose(-1, -2).flatten(2, 3).to(dtype) * vs.to(dtype).transpose(-1, -2).repeat_interleave(32, -1)
    return k, v


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    new, lens = _lengths(c)
    T, D, n_q, n_kv, P = sum(new), c["D"], c["n_q"], c["n_kv"], c["P"]
    st = dict(case=c, seqs=len(new), T=T, longest=max(lens), most=max(max(new), 1), scale=1.0 / math.sqrt(D),
              row_start=i32(np.concatenate([[0], np.cumsum(new)])), kv_len=i32(lens))
    if c["kind"] == "prompt":  # queries and keys as the append leaves them, values in the projections' rows
        Tk = sum(lens)
        st.update(Tk=Tk, kv_start=i32(np.concatenate([[0], np.cumsum(lens)])),
                  q=(1.5 * rand(T, n_q * D)).bfloat16(), k=rand(Tk, n_kv * D).bfloat16(), v=rand(Tk, n_kv * D).bfloat16(),
                  out=torch.empty(T, n_q * D, dtype=torch.bfloat16, device="cuda"))
        return st
    need = [-(-x // P) for x in lens]
    n_pages, width = sum(need) + 3, max(need) + 1
    where = np.random.RandomState(seed % (1 << 31)).permutation(n_pages)
    table = np.full((len(lens), width), -1, np.int64)  # columns behind a sequence's pages: no page
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = where[at:at + n]
        at += n
    st.update(table=i32(table), n_pages=n_pages,
              pool=torch.zeros(n_pages, n_kv * _head_bytes(c), dtype=torch.uint8, device="cuda"))
    if c["kind"] != "append" or c["last"]:  # what earlier steps left in the pool
        page = torch.arange(n_pages, device="cuda").repeat_interleave(P)
        off = torch.arange(P, device="cuda").repeat(n_pages)
        step = max(P, (1 << 26) // (n_kv * D) // P * P)
        for a in range(0, len(page), step):
            n = len(page[a:a + step])
            _store(c, st["pool"], page[a:a + step], off[a:a + step], rand(n, n_kv, D).bfloat16(), rand(n, n_kv, D).bfloat16())
    if c["kind"] == "append":
        st.update(qkv=rand(T, (n_q + 2 * n_kv) * D).bfloat16(),
                  q_norm=1 + 0.1 * rand(D), k_norm=1 + 0.1 * rand(D),
                  inv_freq=torch.tensor(1e6 ** -(np.arange(c["rot"] // 2) / (c["rot"] / 2)), dtype=torch.float64, device="cuda"),
                  q_out=torch.empty(T, n_q * D, dtype=torch.bfloat16, device="cuda"),
                  k_out=torch.empty(T, n_kv * D, dtype=torch.bfloat16, device="cuda"))
    if c["kind"] == "decode":
        st.update(q=(1.5 * rand(T, n_q * D)).bfloat16(), out=torch.empty(T, n_q * D, dtype=torch.bfloat16, device="cuda"))
    else:  # what is read back: the new rows, or everything
        first = [x - n for n, x in zip(new, lens)] if c["kind"] == "append" and not c["all"] else [0] * len(lens)
        counts = [x - f for x, f in zip(lens, first)]
        R = sum(counts)
        st.update(R=R, first=i32(first), read_start=i32(np.concatenate([[0], np.cumsum(counts)])),
                  k_read=torch.empty(R, n_kv * D, dtype=torch.bfloat16, device="cuda"),
                  v_read=torch.empty(R, n_kv * D, dtype=torch.bfloat16, device="cuda"))
    return st


# ------------------------------------------------------------------ plain forms

def _owner(start, n):
    """Sequence and offset inside it of each of n packed rows."""
    t = torch.arange(n, device=start.device)
    b = torch.searchsorted(start[1:].long(), t, right=True)
    return b, t - start.long()[b]


def _norm_rotate(st, x, w, pos):
    """x: bf16 [T, heads, D] -> bf16, normed and rotated, computed in 64 bits."""
    c, x = st["case"], x.double()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.double()
    half = c["rot"] // 2
    angle = (pos.double()[:, None] * st["inv_freq"]).unsqueeze(1)
    cos, sin = angle.cos(), angle.sin()
    r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    a, b = (r[..., 0::2], r[..., 1::2]) if c["inter"] else (r[..., :half], r[..., half:])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((u, v), -1).flatten(-2) if c["inter"] else torch.cat((u, v), -1)
    return torch.cat((r, rest), -1).bfloat16()


def _plain_append(st):
    c = st["case"]
    n_q, n_kv, D, P = c["n_q"], c["n_kv"], c["D"], c["P"]
    x = st["qkv"].view(st["T"], n_q + 2 * n_kv, D)
    b, i = _owner(st["row_start"], st["T"])
    pos = (st["kv_len"] - st["row_start"][1:] + st["row_start"][:-1]).long()[b] + i
    q = _norm_rotate(st, x[:, :n_q], st["q_norm"], pos)
    k = _norm_rotate(st, x[:, n_q:n_q + n_kv], st["k_norm"], pos)
    _store(c, st["pool"], st["table"].long()[b, pos // P], pos % P, k, x[:, n_q + n_kv:])
    return q.flatten(1), k.flatten(1)


def _plain_read(st):
    c = st["case"]
    b, i = _owner(st["read_start"], st["R"])
    at = st["first"].long()[b] + i
    k, v = _load(c, st["pool"][st["table"].clamp(min=0).long()].flatten(0, 1))
    page = b * st["table"].shape[1] + at // c["P"]
    return k[page, :, at % c["P"]].bfloat16().flatten(1), v[page, :, at % c["P"]].bfloat16().flatten(1)


def _attend(q, k, v, sees, scale):
    """q [B, heads, rows, D], k and v [B, heads, keys, D], sees [B, 1, rows, keys]: softmax over the keys seen."""
    s = (q @ k.transpose(-1, -2).contiguous()).mul_(scale).masked_fill_(~sees, -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    return (s @ v) / s.sum(-1, keepdim=True).clamp(min=1e-30)


def _padded(st, x, start, n, most):
    """Packed rows x [n, ...] as [B, most, ...], and the packed rows' places in it."""
    b, i = _owner(start, n)
    p = torch.zeros(st["seqs"], most, *x.shape[1:], dtype=torch.float32, device=x.device)
    p[b, i] = x.float()
    return p, b, i


def _sees(st, keys):
    """[B, 1, rows, keys]: row i of the n rows of a sequence of L tokens sees tokens up to L - n + i."""
    n = st["row_start"][1:] - st["row_start"][:-1]
    last = (st["kv_len"] - n)[:, None] + torch.arange(st["most"], device="cuda")
    return (torch.arange(keys, device="cuda") <= last[..., None])[:, None]


def _plain_decode(st):
    c = st["case"]
    n_q, n_kv, D = c["n_q"], c["n_kv"], c["D"]
    B, G = st["seqs"], n_q // n_kv
    k, v = _load(c, st["pool"][st["table"].clamp(min=0).long()].flatten(0, 1))
    k, v = (x.unflatten(0, (B, -1)).transpose(1, 2).flatten(2, 3) for x in (k, v))  # [B, n_kv, keys, D]
    q, b, i = _padded(st, st["q"].view(-1, n_kv, G, D), st["row_start"], st["T"], st["most"])
    sees = _sees(st, k.shape[2]).repeat_interleave(G, 2)
    o = _attend(q.transpose(1, 2).flatten(2, 3).contiguous(), k, v, sees, st["scale"])
    return o.unflatten(2, (st["most"], G))[b, :, i].bfloat16().flatten(1)


def _plain_prompt(st):
    c = st["case"]
    n_q, n_kv, D = c["n_q"], c["n_kv"], c["D"]
    G = n_q // n_kv
    q, b, i = _padded(st, st["q"].view(-1, n_kv, G, D), st["row_start"], st["T"], st["most"])
    k, _, _ = _padded(st, st["k"].view(-1, n_kv, D), st["kv_start"], st["Tk"], st["longest"])
    v, _, _ = _padded(st, st["v"].view(-1, n_kv, D), st["kv_start"], st["Tk"], st["longest"])
    sees = _sees(st, st["longest"])
    out = torch.empty(st["T"], n_kv, G, D, dtype=torch.bfloat16, device=q.device)
    for h in range(n_kv):  # one key head at a time: the scores of all heads together do not fit
        kh, vh = k[:, None, :, h].contiguous(), v[:, None, :, h].contiguous()
        o = _attend(q[:, :, h].transpose(1, 2).contiguous(), kh, vh, sees, st["scale"])
        out[:, h] = o[b, :, i].bfloat16()
    return out.flatten(1)


# ------------------------------------------------------------------ the framework's calls

def _handles(st):
    """The descriptors and the workspace that a program keeps beside its buffers."""
    import quantized_expert_ffn_router_amd as m
    c = st["case"]
    h = dict(m=m)
    if c["kind"] != "prompt":
        h["cache"] = m.KvCacheDesc(c["fmt"], c["n_kv"], c["D"], c["P"], st["n_pages"], 1.0, 1.0, st["pool"].data_ptr())
        h["seqs"] = m.SeqBatch(st["seqs"], st["table"].shape[1], st["row_start"].data_ptr(), st["kv_len"].data_ptr(), st["table"].data_ptr())
    if c["kind"] == "append":
        h["qkv"] = m.QkvDesc(c["n_q"], EPS, st["q_norm"].data_ptr(), st["k_norm"].data_ptr(), c["rot"], int(c["inter"]), st["inv_freq"].data_ptr(), 1.0)
    if c["kind"] == "decode":
        h["ws_bytes"] = m.moe_attn_workspace_bytes(h["cache"], c["n_q"], st["seqs"], st["T"], st["longest"])
        h["ws"] = torch.empty(max(1, h["ws_bytes"]), dtype=torch.uint8, device="cuda")
    return h


def _own(st):
    c = st["case"]
    if "handles" not in st:
        st["handles"] = _handles(st)
    h, D = st["handles"], c["D"]
    m, q_w, kv_w = h["m"], c["n_q"] * D, c["n_kv"] * D
    if c["kind"] == "prompt":
        m.moe_attn_prompt(c["n_q"], c["n_kv"], D, st["seqs"], st["row_start"], st["kv_start"], st["T"], st["Tk"],
                          st["q"], q_w, st["k"], kv_w, st["v"], kv_w, st["scale"], st["out"], q_w)
        return st["out"]
    if c["kind"] == "decode":
        m.moe_attn_decode(h["cache"], h["seqs"], c["n_q"], st["q"], q_w, st["T"], st["longest"], st["scale"],
                          st["out"], q_w, h["ws"], h["ws_bytes"])
        return st["out"]
    if c["kind"] == "append":
        m.moe_kv_append(h["cache"], h["qkv"], h["seqs"], st["qkv"], q_w + 2 * kv_w, st["T"], None,
                        st["q_out"], q_w, st["k_out"], kv_w)
    m.moe_kv_read(h["cache"], h["seqs"], st["first"], st["read_start"], st["R"], st["k_read"], kv_w, st["v_read"], kv_w)
    if c["kind"] == "append":
        return st["q_out"], st["k_out"], st["k_read"], st["v_read"]
    return st["k_read"], st["v_read"]


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind == "prompt":
        return _plain_prompt(state)
    if kind == "decode":
        return _plain_decode(state)
    if kind == "append":
        return _plain_append(state) + _plain_read(state)
    return _plain_read(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    new, lens = _lengths(c)
    T, Tk, D, n_q, n_kv = sum(new), sum(lens), c["D"], c["n_q"], c["n_kv"]
    token = n_kv * _head_bytes(c) // c["P"]  # cache bytes of one token
    pairs = sum(n * x - n * (n - 1) // 2 for n, x in zip(new, lens))
    if c["kind"] == "prompt":
        return {"bytes": 2 * D * (2 * T * n_q + 2 * Tk * n_kv), "flops": 4 * D * n_q * pairs}
    if c["kind"] == "decode":
        return {"bytes": 2 * D * 2 * T * n_q + Tk * token, "flops": 4 * D * n_q * pairs}
    if c["kind"] == "read":
        return {"bytes": Tk * (token + 4 * n_kv * D), "flops": 2 * Tk * n_kv * D}
    R = Tk if c["all"] else T
    return {"bytes": T * (2 * D * (2 * n_q + 3 * n_kv) + token) + R * (token + 4 * n_kv * D),
            "flops": T * D * (n_q + 2 * n_kv) * 10}


# ------------------------------------------------------------------ the definition, in 64 bits

def _exact_codes(c, x):
    """bf16 values x (as float64 [..., D]) as the cache holds them."""
    if c["fmt"] == BF16:
        return x
    n = 16 if c["fmt"] == NVFP4 else 32
    b = x.reshape(*x.shape[:-1], -1, n)
    top = b.abs().max(-1).values
    if c["fmt"] == Q8_0:
        s = (top.clamp(max=65024.0) / 127.0).to(torch.float16).double()[..., None]
        return (torch.round(torch.nan_to_num(b / s)).clamp(-127, 127) * s).reshape(x.shape)
    s = (top / 6.0).clamp(max=448.0).float().to(torch.float8_e4m3fn).double()[..., None]
    r = torch.nan_to_num(b / s)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    edge = (grid[1:] + grid[:-1]) / 2
    lo, hi = torch.bucketize(r.abs(), edge, right=False), torch.bucketize(r.abs(), edge, right=True)
    code = torch.where(lo == hi, lo, torch.where(lo % 2 == 0, lo, hi))  # a tie goes to the even code
    return (grid[code] * r.sign() * s).reshape(x.shape)


def _exact_cached(st, pages, L):
    """Tokens 0..L-1 of a sequence with these pages, k and v float64 [L, n_kv, D]: each value from the
    place of its own byte in the pool."""
    c, pool = st["case"], st["pool"].flatten()
    D, P, n_kv = c["D"], c["P"], c["n_kv"]
    t = torch.arange(L, device="cuda")[:, None]
    d = torch.arange(D, device="cuda")
    got = torch.empty(2, L, n_kv, D, dtype=torch.float64, device="cuda")
    bits = {NVFP4: 4, Q8_0: 8, BF16: 16}[c["fmt"]]
    codes, scales = P * D * bits // 8, 0 if c["fmt"] == BF16 else P * D // 16
    two = lambda at: pool[at].int() | (pool[at + 1].int() << 8)  # noqa: E731
    half = lambda u: u.to(torch.int16).view(torch.float16).double()  # noqa: E731
    for h in range(n_kv):
        base = (pages[t // P] * n_kv + h) * _head_bytes(c)
        o = t % P
        for j in (0, 1):
            b = base + j * (codes + scales)
            if c["fmt"] == NVFP4:
                n = D // 16  # a value group of v: 16 of them over the head, each for 4 tokens in turn
                at = o * (D // 2) + d // 2 if j == 0 else ((o // 4 * 16 + d // n) * 4 + o % 4) * (n // 2) + d % n // 2
                q = (pool[b + at].int() >> (d % 2 * 4)) & 15
                e, m = (q >> 1) & 3, q & 1
                x = torch.where(e > 0, (1 + 0.5 * m) * torch.exp2(e.double() - 1), 0.5 * m) * (1 - 2 * (q >> 3))
                f = pool[b + codes + (o * (D // 16) + d // 16 if j == 0 else d // 16 * P + o)].int()
                e, m = (f >> 3) & 15, f & 7
                x = x * torch.where(e > 0, (1 + m / 8.0) * torch.exp2(e.double() - 7), m * 2.0 ** -9)
            elif c["fmt"] == Q8_0:
                at = o * D + d if j == 0 else (o // 4 * D + d) * 4 + o % 4
                q = pool[b + at].int()
                x = (q - 256 * (q >> 7)) * half(two(b + codes + 2 * (o * (D // 32) + d // 32 if j == 0 else d // 32 * P + o)))
            else:
                u = two(b + 2 * (o * D + d if j == 0 else (o // 4 * D + d) * 4 + o % 4))
                x = u.to(torch.int16).view(torch.bfloat16).double()
            got[j, :, h] = x
    return got[0], got[1]


def _exact_turned(st, x, w, pos):
    c, x = st["case"], x.double()
    z = x / (x.pow(2).sum(-1, keepdim=True) / c["D"] + EPS).sqrt() * w.double()
    y, n = z.clone(), c["rot"] // 2
    first = torch.arange(n, device="cuda") * 2 if c["inter"] else torch.arange(n, device="cuda")
    second = first + 1 if c["inter"] else first + n
    w = torch.polar(torch.ones(len(pos), 1, n, dtype=torch.float64, device="cuda"), (pos.double()[:, None] * st["inv_freq"])[:, None])
    turned = torch.complex(z[..., first], z[..., second]) * w
    y[..., first], y[..., second] = turned.real, turned.imag
    return y


def _exact_rows(q, k, v, last, scale):
    """q [heads, n, D] of one key head, k and v [L, D], all float64; row i sees keys up to last[i]."""
    out = torch.empty_like(q)
    for h in range(q.shape[0]):
        for a in range(0, q.shape[1], 2048):
            s = q[h, a:a + 2048] @ k.T.contiguous() * scale
            s.masked_fill_(torch.arange(k.shape[0], device="cuda") > last[a:a + 2048, None], -math.inf)
            out[h, a:a + 2048] = torch.softmax(s, -1) @ v
    return out


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    new, lens = _lengths(c)
    n_q, n_kv, D, P = c["n_q"], c["n_kv"], c["D"], c["P"]
    G = n_q // n_kv
    rows = np.concatenate([[0], np.cumsum(new)])
    if c["kind"] == "prompt":
        keys = np.concatenate([[0], np.cumsum(lens)])
        out = torch.zeros(st["T"], n_kv, G, D, dtype=torch.float64, device="cuda")
        q, k, v = st["q"].view(-1, n_kv, G, D), st["k"].view(-1, n_kv, D), st["v"].view(-1, n_kv, D)
        for b, (n, L) in enumerate(zip(new, lens)):
            r, s = slice(rows[b], rows[b] + n), slice(keys[b], keys[b] + L)
            last = torch.arange(L - n, L, device="cuda")
            for h in range(n_kv):
                out[r, h] = _exact_rows(q[r, h].double().transpose(0, 1).contiguous(), k[s, h].double(), v[s, h].double(), last, st["scale"]).transpose(0, 1)
        return out.flatten(1)
    table = st["table"].cpu().numpy()

    def cached(b):
        return _exact_cached(st, torch.from_numpy(table[b].astype(np.int64)).cuda(), lens[b])

    if c["kind"] == "decode":
        out = torch.zeros(st["T"], n_kv, G, D, dtype=torch.float64, device="cuda")
        for b, (n, L) in enumerate(zip(new, lens)):
            k, v = cached(b)
            r, last = slice(rows[b], rows[b] + n), torch.arange(L - n, L, device="cuda")
            for h in range(n_kv):
                q = st["q"].view(-1, n_kv, G, D)[r, h].double().transpose(0, 1).contiguous()
                out[r, h] = _exact_rows(q, k[:, h].contiguous(), v[:, h].contiguous(), last, st["scale"]).transpose(0, 1)
        return out.flatten(1)
    got = [cached(b) for b in range(len(lens))]
    if c["kind"] == "read":
        return tuple(torch.cat([x[j] for x in got]).flatten(1) for j in (0, 1))
    x = st["qkv"].view(st["T"], n_q + 2 * n_kv, D)
    pos = torch.cat([torch.arange(L - n, L) for n, L in zip(new, lens)]).cuda()
    q, k = _exact_turned(st, x[:, :n_q], st["q_norm"], pos), _exact_turned(st, x[:, n_q:n_q + n_kv], st["k_norm"], pos)
    held = _exact_codes(c, k.bfloat16().double()), _exact_codes(c, x[:, n_q + n_kv:].double())
    whole = []
    for j in (0, 1):
        parts = []
        for b, (n, L) in enumerate(zip(new, lens)):
            fresh = held[j][rows[b]:rows[b] + n]
            parts.append(torch.cat((got[b][j][:L - n], fresh)) if c["all"] else fresh)
        whole.append(torch.cat(parts).flatten(1))
    return q.flatten(1), k.flatten(1), whole[0], whole[1]
