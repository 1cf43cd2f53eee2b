"""What a decoder layer needs around its experts and its cache, in plain form and as a user's program
calls it.

moe_add_norm         the residual's addition and the root-mean-square norm, out in 16 bits and, for the
                     projections, in 8 bits with a power-of-two scale for each 32 values
moe_mx_quant         rows in the microscaled formats: 4-bit or 8-bit floating point, the same scales
moe_mx_linear        product of microscaled rows with a 4-bit microscaled matrix
moe_mx_linear_rows   the same from 16-bit rows, quantised on the way
moe_attn_chunk       attention of the new tokens of prompts' chunks over the paged cache

Where ``own`` is false, ``run`` computes the operators from elementary torch operations, in 32 bits
(64 for norms and whatever is then quantised, where the last bit decides a code).
"""
import math

import numpy as np
import torch

own = False

NVFP4, Q8_0, BF16, MXFP4, MXFP8 = 1, 3, 6, 7, 8
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    cache = dict(kind="chunk", n_q=32, n_kv=4, D=128, P=64, fmt=NVFP4)
    return [
        # The norm before a decode step's projections: 8 request slots.
        dict(name="norm_step_8", kind="norm", T=8, H=2048, res=True, out=True, fmt=MXFP8),
        # The same for a whole prefill batch.
        dict(name="norm_16384", kind="norm", T=16384, H=2048, res=True, out=True, fmt=MXFP8),
        # Attention outputs of 8 slots (32 heads of 128) in 8 bits.
        dict(name="quant_step_8", kind="quant", T=8, K=4096, fmt=MXFP8),
        # Those of a prefill batch.
        dict(name="quant_16384", kind="quant", T=16384, K=4096, fmt=MXFP8),
        # One slot's projection to 32 query and 2 * 4 key and value heads, from the norm's 8 bits.
        dict(name="linear_qkv_1", kind="linear", T=1, N=5120, K=2048, fmt=MXFP8, rows=False, bias=False),
        # 8 slots' projection from the attention's output back to the hidden size.
        dict(name="linear_out_8", kind="linear", T=8, N=2048, K=4096, fmt=MXFP4, rows=True, bias=False),
        # The scores of a vocabulary of odd size, for a verification batch.
        dict(name="linear_head_5", kind="linear", T=5, N=100003, K=2048, fmt=MXFP8, rows=True, bias=False),
        # A short ragged prompt, with a bias; every size ends inside a tile.
        dict(name="linear_777", kind="linear", T=777, N=4107, K=1152, fmt=MXFP4, rows=True, bias=True),
        # The prefill batch's projection.
        dict(name="linear_qkv_16384", kind="linear", T=16384, N=5120, K=2048, fmt=MXFP8, rows=False, bias=False),
        # One slot's follow-up question in a long conversation.
        dict(cache, name="chunk_1x64", n_seq=1, rows=64, uneven=0, first=32768, last=32768),
        # A mixed step: most of the rows are one slot's chunk, the other slots decode; 8-bit cache,
        # 64-wide heads, pages of 32.
        dict(cache, name="chunk_mixed_q8", n_seq=8, rows=512, uneven=2, first=300, last=16001, n_q=24, n_kv=8, D=64, P=32, fmt=Q8_0),
        # A chunk of a long prompt behind what is cached of it.
        dict(cache, name="chunk_4096", n_seq=1, rows=4096, uneven=0, first=12288, last=12288),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "quant", "linear", "linear", "linear", "linear", "chunk", "chunk", "chunk"])
    if kind == "norm":
        H = 128 * _log(rng, 1, 64)
        return dict(kind=kind, T=_log(rng, 1, 30_000_000 // H), H=H, res=rng.random() < 0.7, out=rng.random() < 0.7,
                    fmt=rng.choice([MXFP8, MXFP8, 0]))
    if kind == "quant":
        K = 128 * _log(rng, 1, 128)
        return dict(kind=kind, T=_log(rng, 1, 60_000_000 // K), K=K, fmt=MXFP8)
    if kind == "linear":
        K = 128 * _log(rng, 1, 64)
        N = _log(rng, 1, min(100_000, 200_000_000 // K))
        T = rng.choice([rng.randint(1, 16), _log(rng, 1, 16384)])
        return dict(kind=kind, T=max(1, min(T, 160_000_000_000 // (N * K), 80_000_000 // N)), N=N, K=K, fmt=rng.choice([MXFP4, MXFP8]),
                    rows=rng.random() < 0.5, bias=rng.random() < 0.3)
    D = rng.choice([64, 128, 128, 128, 256])
    n_kv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 4, 5, 8])
    n_seq = rng.randint(1, 8)
    rows = max(n_seq, _log(rng, 8, 2500))
    last = _log(rng, 1, min(60_000, 1_000_000_000 // (n_seq * rows * G), 40_000_000 // (n_kv * D * n_seq)))
    return dict(kind=kind, n_q=n_kv * G, n_kv=n_kv, D=D, P=rng.choice([32, 64, 128, 256]), fmt=rng.choice([NVFP4, NVFP4, Q8_0, BF16]),
                n_seq=n_seq, rows=rows, uneven=rng.randint(0, 2), first=last // rng.choice([1, 2, 30]), last=last)


def _lengths(c):
    """Rows of each sequence, and its tokens with those: fixed by the case alone. uneven 0: equal
    shares of the rows; 1: shares of different sizes; 2: one sequence's chunk, one row of the others."""
    B, R = c["n_seq"], c["rows"]
    if c["uneven"] == 0:
        new = [R // B + (b < R % B) for b in range(B)]
    elif c["uneven"] == 1:
        w = [1.0 + (7 * b) % 5 for b in range(B)]
        new = [1 + int((R - B) * x / sum(w)) for x in w]
        new[0] += R - sum(new)
    else:
        new = [1] * B
        new[B // 2] += R - B
    before = [c["first"] + (c["last"] - c["first"]) * b // max(1, B - 1) for b in range(B)]
    return new, [x + n for x, n in zip(before, new)]


# ------------------------------------------------------------------ microscaled values, plain

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _e2m1_code(r):
    a = r.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code | (torch.signbit(r).to(torch.uint8) << 3)


def _pow2(k):
    """2^k, float64, exactly (-1022 <= k <= 1023)."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _mx(fmt, x):
    """x: bf16 [.., K] -> codes (float8_e4m3fn, or one byte for each E2M1 code) and scale bytes
    [.., K/32]: 2^(s - 127) with s from the block's largest magnitude, so that this comes to lie in
    the format's highest binade; what is beyond the largest value is held to it."""
    b = x.float().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    s = torch.frexp(top).exponent - 1 - (2 if fmt == MXFP4 else 8)
    s = torch.where(top > 0, s.clamp(min=-127), torch.full_like(s, -127))
    r = b.double() * _pow2(-s)[..., None]
    most = 6.0 if fmt == MXFP4 else 448.0
    r = r.clamp(-most, most)
    scale = (s + 127).to(torch.uint8)
    if fmt == MXFP4:
        return _e2m1_code(r).flatten(-2), scale
    return r.float().to(torch.float8_e4m3fn).flatten(-2), scale


def _packed(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _factor(scale):
    """2^(s - 127) of scale bytes, float32 (0 stands for 2^-127, a subnormal number)."""
    return _pow2(scale.int() - 127).float()


def _mx_values(fmt, codes, scale):
    """What codes (MXFP4: two a byte) stand for, float32 [.., K]."""
    if fmt == MXFP4:
        lut = torch.tensor(_E2M1, dtype=torch.float32, device=codes.device)
        v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).flatten(-2)
    else:
        v = codes.float()
    return (v.unflatten(-1, (-1, 32)) * _factor(scale)[..., None]).flatten(-2)


# ------------------------------------------------------------------ the cache's bytes, plain

def _head_bytes(c):
    D, P = c["D"], c["P"]
    return P * {NVFP4: D // 2 + D // 16, Q8_0: D + D // 16, BF16: 2 * D}[c["fmt"]] * 2


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
        ck, cv = _packed(ck), _packed(cv)
        vq[page, :, off // 4, :, off % 4] = cv.unflatten(-1, (16, -1))
    else:
        vq[page, :, off // 4, :, off % 4] = cv
    kq[page, :, off] = ck
    if sk is not None:
        ks[page, :, off] = sk
        vs[page, :, :, off] = sv


def _load(c, pages):
    """The values of whole pages: k, v float32 [page, n_kv, P, D]."""
    kq, ks, vq, vs = _sections(c, pages)
    if c["fmt"] == BF16:
        return kq.float(), vq.transpose(-1, -2).flatten(2, 3).float()
    if c["fmt"] == NVFP4:
        lut = torch.tensor(_E2M1, dtype=torch.float32, device=pages.device)
        val = lambda q: torch.stack((lut[(q & 15).int()], lut[(q >> 4).int()]), -1).flatten(-2)  # noqa: E731
        k = val(kq) * ks.contiguous().view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)
        v = val(vq).transpose(3, 4).flatten(-2).flatten(2, 3)  # [page, head, quad, 16, 4, d] -> [.., P, D]
        v = v * vs.contiguous().view(torch.float8_e4m3fn).float().transpose(-1, -2).repeat_interleave(16, -1)
        return k, v
    k = kq.float() * ks.float().repeat_interleave(32, -1)
    v = vq.transpose(-1, -2).flatten(2, 3).float() * vs.float().transpose(-1, -2).repeat_interleave(32, -1)
    return k, v


# ------------------------------------------------------------------ inputs

def _rows(rand, T, W):
    """Activations as a layer meets them: some columns much larger than the others, rows of
    different size."""
    x = rand(T, W) * torch.exp(0.5 * rand(T, 1))
    x[:, :: 97] *= 8.0
    return x.bfloat16()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    bf16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    st = dict(case=c)
    if c["kind"] == "norm":
        T, H = c["T"], c["H"]
        st.update(x=rand(T, H).bfloat16(), residual=_rows(rand, T, H) if c["res"] else None, weight=1 + 0.1 * rand(H),
                  sum=bf16(T, H) if c["res"] else None, out=bf16(T, H) if c["out"] or not c["fmt"] else None,
                  codes=u8(T, H) if c["fmt"] else None, scales=u8(T, H // 32) if c["fmt"] else None)
        return st
    if c["kind"] == "quant":
        T, K = c["T"], c["K"]
        st.update(x=_rows(rand, T, K), codes=u8(T, K), scales=u8(T, K // 32))
        return st
    if c["kind"] == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        wq, ws = _mx(MXFP4, (0.02 * rand(N, K)).bfloat16())
        st.update(w_codes=_packed(wq), w_scales=ws, bias=0.1 * rand(N) if c["bias"] else None,
                  y=bf16(T, (N + 7) // 8 * 8)[:, :N])
        x = _rows(rand, T, K)
        if c["rows"]:
            st["x"] = x
        else:
            q, s = _mx(c["fmt"], x)
            st.update(codes=_packed(q) if c["fmt"] == MXFP4 else q, scales=s)
        return st
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    new, lens = _lengths(c)
    T, D, n_q, n_kv, P = sum(new), c["D"], c["n_q"], c["n_kv"], c["P"]
    need = [-(-x // P) for x in lens]
    n_pages, width = sum(need) + 3, max(need) + 1
    where = np.random.RandomState(seed % (1 << 31)).permutation(n_pages)
    table = np.full((len(lens), width), -1, np.int64)  # columns behind a sequence's pages: no page
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = where[at:at + n]
        at += n
    st.update(seqs=len(new), T=T, longest=max(lens), most=max(new), scale=1.0 / math.sqrt(D),
              row_start=i32(np.concatenate([[0], np.cumsum(new)])), kv_len=i32(lens), table=i32(table), n_pages=n_pages,
              pool=torch.zeros(n_pages, n_kv * _head_bytes(c), dtype=torch.uint8, device="cuda"),
              q=(1.5 * rand(T, n_q * D)).bfloat16(), out=bf16(T, n_q * D))
    page = torch.arange(n_pages, device="cuda").repeat_interleave(P)
    off = torch.arange(P, device="cuda").repeat(n_pages)
    step = max(P, (1 << 26) // (n_kv * D) // P * P)
    for a in range(0, len(page), step):  # what this and earlier steps appended
        n = len(page[a:a + step])
        _store(c, st["pool"], page[a:a + step], off[a:a + step], rand(n, n_kv, D).bfloat16(), rand(n, n_kv, D).bfloat16())
    return st


# ------------------------------------------------------------------ plain forms

def _plain_norm(st):
    c = st["case"]
    h = st["x"] if st["residual"] is None else (st["x"].float() + st["residual"].float()).bfloat16()
    z = h.double()
    z = (z * torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS) * st["weight"].double()).bfloat16()
    got = {}
    if c["res"]:
        got["sum"] = h
    if st["out"] is not None:
        got["out"] = z
    if c["fmt"]:
        got["codes"], s = _mx(c["fmt"], z)
        got["scales"] = s.view(torch.float8_e8m0fnu)
    return got


def _plain_quant(st):
    q, s = _mx(st["case"]["fmt"], st["x"])
    return q, s.view(torch.float8_e8m0fnu)


def _plain_linear(st):
    c = st["case"]
    if c["rows"]:
        q, s = _mx(c["fmt"], st["x"])
        q = _packed(q) if c["fmt"] == MXFP4 else q
    else:
        q, s = st["codes"], st["scales"]
    y = _mx_values(c["fmt"], q, s) @ _mx_values(MXFP4, st["w_codes"], st["w_scales"]).t()
    return (y if st["bias"] is None else y + st["bias"]).bfloat16()


def _plain_chunk(st):
    c = st["case"]
    n_q, n_kv, D = c["n_q"], c["n_kv"], c["D"]
    B, G, most = st["seqs"], n_q // n_kv, st["most"]
    k, v = _load(c, st["pool"][st["table"].clamp(min=0).long()].flatten(0, 1))
    k, v = (x.unflatten(0, (B, -1)).transpose(1, 2).flatten(2, 3) for x in (k, v))  # [B, n_kv, keys, D]
    t = torch.arange(st["T"], device="cuda")
    b = torch.searchsorted(st["row_start"][1:].long(), t, right=True)
    i = t - st["row_start"].long()[b]
    q = torch.zeros(B, most, n_kv, G, D, device="cuda")
    q[b, i] = st["q"].float().view(-1, n_kv, G, D)
    # row i of the n rows of a sequence of L tokens sees tokens up to L - n + i
    last = (st["kv_len"] - st["row_start"][1:] + st["row_start"][:-1])[:, None] + torch.arange(most, device="cuda")
    hidden = (torch.arange(k.shape[2], device="cuda") > last[..., None]).repeat_interleave(G, 1)
    out = torch.empty(st["T"], n_kv, G, D, dtype=torch.bfloat16, device="cuda")
    for h in range(n_kv):  # one key head at a time: the scores of all heads together do not fit
        s = (q[:, :, h].flatten(1, 2).contiguous() @ k[:, h].transpose(-1, -2).contiguous()).mul_(st["scale"])
        s = s.masked_fill_(hidden, -math.inf)
        s = s.sub_(s.amax(-1, keepdim=True)).exp_()
        o = (s @ v[:, h].contiguous()) / s.sum(-1, keepdim=True)
        out[:, h] = o.unflatten(1, (most, G))[b, i].bfloat16()
    return out.flatten(1)


# ------------------------------------------------------------------ the framework's calls

def _handles(st):
    """The packed matrix, the descriptors and the workspaces that a program keeps beside its buffers."""
    import quantized_expert_ffn_router_amd as m
    c = st["case"]
    h = dict(m=m)
    if c["kind"] == "linear":
        h["packed"] = torch.empty(m.moe_mx_matrix_bytes(c["N"], c["K"]), dtype=torch.uint8, device="cuda")
        m.moe_mx_pack(c["N"], c["K"], st["w_codes"], st["w_scales"], h["packed"])
        h["w"] = m.MxMatrix(c["N"], c["K"], h["packed"].data_ptr(), None if st["bias"] is None else st["bias"].data_ptr())
        h["ws_bytes"] = m.moe_mx_workspace_bytes(c["fmt"], c["K"], c["T"])
        h["ws"] = torch.empty(max(1, h["ws_bytes"]), dtype=torch.uint8, device="cuda")
    elif c["kind"] == "chunk":
        h["cache"] = m.KvCacheDesc(c["fmt"], c["n_kv"], c["D"], c["P"], st["n_pages"], 1.0, 1.0, st["pool"].data_ptr())
        h["seqs"] = m.SeqBatch(st["seqs"], st["table"].shape[1], st["row_start"].data_ptr(), st["kv_len"].data_ptr(), st["table"].data_ptr())
        h["ws_bytes"] = m.moe_attn_chunk_workspace_bytes(h["cache"], c["n_q"], st["seqs"], st["T"], st["longest"])
        h["ws"] = torch.empty(max(1, h["ws_bytes"]), dtype=torch.uint8, device="cuda")
    return h


def _own(st):
    c = st["case"]
    if "handles" not in st:
        st["handles"] = _handles(st)
    h = st["handles"]
    m = h["m"]
    if c["kind"] == "norm":
        m.moe_add_norm(c["H"], c["T"], st["x"], c["H"], st["residual"], c["H"], st["weight"], EPS, st["sum"], c["H"],
                       st["out"], c["H"], c["fmt"], st["codes"], st["scales"])
        got = {}
        if c["res"]:
            got["sum"] = st["sum"]
        if st["out"] is not None:
            got["out"] = st["out"]
        if c["fmt"]:
            got.update(codes=st["codes"].view(torch.float8_e4m3fn), scales=st["scales"].view(torch.float8_e8m0fnu))
        return got
    if c["kind"] == "quant":
        m.moe_mx_quant(c["fmt"], c["K"], c["T"], st["x"], c["K"], st["codes"], st["scales"])
        return st["codes"].view(torch.float8_e4m3fn), st["scales"].view(torch.float8_e8m0fnu)
    if c["kind"] == "linear":
        y = st["y"]
        if c["rows"]:
            m.moe_mx_linear_rows(h["w"], c["fmt"], st["x"], c["K"], c["T"], y, y.stride(0), m.MOE_DTYPE_BF16, h["ws"], h["ws_bytes"])
        else:
            m.moe_mx_linear(h["w"], c["fmt"], st["codes"], st["scales"], c["T"], y, y.stride(0), m.MOE_DTYPE_BF16)
        return y
    w = c["n_q"] * c["D"]
    m.moe_attn_chunk(h["cache"], h["seqs"], c["n_q"], st["q"], w, st["T"], st["longest"], st["scale"], st["out"], w, h["ws"], h["ws_bytes"])
    return st["out"]


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind == "norm":
        return _plain_norm(state)
    if kind == "quant":
        return _plain_quant(state)
    if kind == "linear":
        return _plain_linear(state)
    return _plain_chunk(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["kind"] == "norm":
        T, H = c["T"], c["H"]
        row = 2 * H * (1 + 2 * c["res"] + (c["out"] or not c["fmt"])) + (H + H // 32 if c["fmt"] else 0)
        return {"bytes": T * row + 4 * H, "flops": 6 * T * H}
    if c["kind"] == "quant":
        T, K = c["T"], c["K"]
        return {"bytes": T * (3 * K + K // 32), "flops": 2 * T * K}
    if c["kind"] == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        row = 2 * K if c["rows"] else K // 32 + (K // 2 if c["fmt"] == MXFP4 else K)
        return {"bytes": T * row + N * (K // 2 + K // 32) + 2 * T * N + 4 * N * c["bias"], "flops": 2 * T * N * K}
    new, lens = _lengths(c)
    T, Tk, D, n_q, n_kv = sum(new), sum(lens), c["D"], c["n_q"], c["n_kv"]
    pairs = sum(n * x - n * (n - 1) // 2 for n, x in zip(new, lens))
    return {"bytes": 2 * D * 2 * T * n_q + Tk * n_kv * _head_bytes(c) // c["P"], "flops": 4 * D * n_q * pairs}


# ------------------------------------------------------------------ the definition, in 64 bits

def _exact_mx(fmt, x):
    """x: float64 [T, K], 16-bit values -> codes and factors 2^e as numbers, float64."""
    b = x.view(x.shape[0], -1, 32)
    top = b.abs().max(-1, keepdim=True).values
    mant, drop, low, most = (1, 2, 0, 6.0) if fmt == MXFP4 else (3, 8, -6, 448.0)
    power = torch.tensor([2.0 ** k for k in range(-160, 161)], dtype=torch.float64, device=x.device)
    binade = lambda v: torch.frexp(v)[1].long() - 1  # noqa: E731
    e = torch.where(top == 0, -127, (binade(top) - drop).clamp(min=-127))
    r = b / power[e + 160]
    step = power[torch.where(r == 0, low, binade(r).clamp(min=low)) - mant + 160]
    r = (torch.round(r / step) * step).clamp(-most, most)  # round() takes ties to the even multiple
    return r.view(x.shape), power[e + 160].squeeze(-1)


def _exact_matrix(st):
    """The 4-bit matrix, float64 [N, K]."""
    q = st["w_codes"].view(-1, 1).int()
    q = torch.cat((q % 16, q // 16), 1).view(st["w_codes"].shape[0], -1)
    e, m = (q >> 1) & 3, (q & 1).double()
    v = torch.where(e > 0, (1 + 0.5 * m) * torch.exp2(e.double() - 1), 0.5 * m) * (1 - 2 * (q >> 3))
    return (v.view(v.shape[0], -1, 32) * _pow2(st["w_scales"].int() - 127)[..., None]).view(v.shape)


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


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    if c["kind"] == "norm":
        h, got = st["x"].double(), {}
        if c["res"]:
            got["sum"] = h + st["residual"].double()
            h = got["sum"].bfloat16().double()
        z = h / (h.pow(2).sum(-1, keepdim=True) / c["H"] + EPS).sqrt() * st["weight"].double()
        if st["out"] is not None:
            got["out"] = z
        if c["fmt"]:
            got["codes"], got["scales"] = _exact_mx(c["fmt"], z.bfloat16().double())
        return got
    if c["kind"] == "quant":
        return _exact_mx(c["fmt"], st["x"].double())
    if c["kind"] == "linear":
        if c["rows"]:
            r, f = _exact_mx(c["fmt"], st["x"].double())
        else:
            f = _pow2(st["scales"].int() - 127)
            if c["fmt"] == MXFP4:
                grid = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")
                r = grid[torch.stack((st["codes"] % 16, st["codes"] // 16), -1).long()].view(c["T"], -1)
            else:
                r = st["codes"].double()
        a = (r.view(c["T"], -1, 32) * f[..., None]).view(c["T"], -1)
        y = a @ _exact_matrix(st).t().contiguous()
        return y if st["bias"] is None else y + st["bias"].double()
    new, lens = _lengths(c)
    n_q, n_kv, D = c["n_q"], c["n_kv"], c["D"]
    G, table = n_q // n_kv, st["table"].cpu().numpy()
    out = torch.zeros(st["T"], n_kv, G, D, dtype=torch.float64, device="cuda")
    r0 = 0
    for b, (n, L) in enumerate(zip(new, lens)):
        k, v = _exact_cached(st, torch.from_numpy(table[b].astype(np.int64)).cuda(), L)
        for h in range(n_kv):
            kh, vh = k[:, h].t().contiguous(), v[:, h].contiguous()
            for g in range(G):
                for a in range(0, n, 2048):
                    i = torch.arange(a, min(a + 2048, n), device="cuda")
                    s = st["q"].view(-1, n_kv, G, D)[r0 + i, h, g].double() @ kh * st["scale"]
                    s.masked_fill_(torch.arange(L, device="cuda") > (L - n + i)[:, None], -math.inf)
                    out[r0 + i, h, g] = torch.softmax(s, -1) @ vh
        r0 += n
    return out.flatten(1)
