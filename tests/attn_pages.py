"""Caches of long sequences made at once with torch, on any device: random codes and
scales packed into pages after the layout stated in include/moe.h, and the values
that they stand for in float64.  Shares no code with the library or with attn_ref.py
(whose byte-by-byte reading checks the packing)."""
import math

import torch

NVFP4, Q8_0, BF16 = 1, 3, 6
E2M1 = [0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6]


def _bytes(t):
    return t.contiguous().view(torch.uint8)


def _pack_pairs(c):  # 4-bit codes, the even one in the low half
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8)


def pages_of(fmt, kc, ks, vc, vs):
    """Codes [N, n_kv, P, D] and scales [N, n_kv, P, blocks] of N pages -> uint8 [N, bytes]."""
    N, n_kv, P, D = kc.shape
    quads = vc.view(N, n_kv, P // 4, 4, D)
    if fmt == NVFP4:
        v = _pack_pairs(quads.view(N, n_kv, P // 4, 4, 16, D // 16).transpose(3, 4).contiguous())
        parts = [_pack_pairs(kc), ks, v, vs.transpose(2, 3)]
    elif fmt == Q8_0:
        parts = [kc, ks, quads.transpose(3, 4), vs.transpose(2, 3)]
    else:
        parts = [kc, quads.transpose(3, 4)]
    return torch.cat([_bytes(p).reshape(N, n_kv, -1) for p in parts], 2).reshape(N, -1)


def values_of(fmt, codes, scales, ts):
    """float64 values of codes [..., D] and scales [..., blocks]."""
    if fmt == BF16:
        return codes.double()
    n = 16 if fmt == NVFP4 else 32
    x = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)[codes.long()] if fmt == NVFP4 else codes.double()
    s = scales.view(torch.float8_e4m3fn).double() if fmt == NVFP4 else scales.double()
    return x * s.repeat_interleave(n, -1) * (ts if fmt == NVFP4 else 1.0)


def make(fmt, n_kv, D, P, lens, gen, device, k_ts=1.0, v_ts=1.0):
    """-> pool uint8, table int32 [n, width], per sequence (k, v) float64 [L, n_kv, D].
    Keys are random; a token's value is positive in one element, the one of its 256th
    of the sequence (modulo D), and zero in all others, so that an output element is
    the weight of a part of the sequence: a part left out or counted twice shows.
    Tokens behind the last one of a page are NaN (4 and 8 bits: by their scales)."""
    need = [-(-L // P) for L in lens]
    total = sum(need) + 1
    where = torch.randperm(total, generator=gen, device=device)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=device)
    rand = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=gen, device=device)  # noqa: E731
    pool, out, at = None, [], 0
    for b, (L, n) in enumerate(zip(lens, need)):
        T = n * P
        j = torch.arange(T, device=device)
        hot = torch.arange(D, device=device) == (j * 256 // max(L, 1) % D)[:, None]  # [T, D]
        hot = hot[:, None, :].expand(T, n_kv, D)
        if fmt == BF16:
            kc = torch.randn(T, n_kv, D, generator=gen, device=device).bfloat16()
            vc = torch.where(hot, 0.5 + torch.rand(T, n_kv, D, generator=gen, device=device), 0).bfloat16()
            kc[L:], vc[L:], ks, vs = math.nan, math.nan, None, None
        elif fmt == Q8_0:
            kc = rand(-127, 128, T, n_kv, D).to(torch.int8)
            vc = torch.where(hot, rand(20, 128, T, n_kv, D), 0).to(torch.int8)
            ks, vs = (((2 + torch.rand(T, n_kv, D // 32, generator=gen, device=device)) / 200).half() for _ in range(2))
            ks[L:], vs[L:] = math.nan, math.nan
        else:
            kc = rand(0, 16, T, n_kv, D).to(torch.uint8)
            vc = torch.where(hot, rand(1, 8, T, n_kv, D), 0).to(torch.uint8)
            # (scales 2^-2 to 2^-1 less a step)
            ks, vs = (rand(0x28, 0x30, T, n_kv, D // 16).to(torch.uint8) for _ in range(2))
            ks[L:], vs[L:] = 0x7f, 0x7f
        paged = lambda t: None if t is None else t.view(n, P, n_kv, -1).transpose(1, 2)  # noqa: E731
        bytes_ = pages_of(fmt, *(paged(t) if t is None else paged(t).contiguous() for t in (kc, ks, vc, vs)))
        if pool is None:
            pool = torch.full((total, bytes_.shape[1]), 0xff, dtype=torch.uint8, device=device)
        mine = where[at:at + n]
        at += n
        pool[mine] = bytes_
        table[b, :n] = mine.int()
        cut = lambda t: None if t is None else t[:L]  # noqa: E731
        out.append((values_of(fmt, kc[:L], cut(ks), k_ts), values_of(fmt, vc[:L], cut(vs), v_ts)))
    return pool.reshape(-1), table, out


def attend(q, k, v, limit, scale, fmt, depth):
    """Rows q [n, D] float64 of one head, row i seeing tokens 0..limit[i] of k, v [L, D].
    -> the outputs, and how far a result may be from them.  Half a step of bf16; a
    weight's rounding, 2^-11 (fp16) or 2^-8 (bf16), or 2^-32 of the largest weight
    where fp16 has no normal number (the largest is held as 2^7 or more); the error of
    a score, D 2^-24 of sum |q||k|, and for 8 bits 2^-11 of it (code * scale as fp16),
    in numerator and denominator; 2^-20 for exponentials and the division, and depth
    2^-24 for sums in which no chain of additions is longer than depth."""
    D, L = q.shape[1], k.shape[0]
    s = scale * (q @ k.T)
    s.masked_fill_(torch.arange(L, device=q.device) > limit[:, None], -math.inf)
    e = (s - s.max(1, keepdim=True).values).exp()
    total = e.sum(1, keepdim=True)
    want, pv = e @ v / total, e @ v.abs() / total
    qk = float((q.abs() @ k.abs().T).max()) * scale
    e_p, e_kv = (2.0 ** -8 if fmt == BF16 else 2.0 ** -11), (2.0 ** -11 if fmt == Q8_0 else 0.0)
    w = e_p + e_kv + 2 * math.expm1(qk * (D * 2.0 ** -24 + e_kv)) + 2.0 ** -20 + depth * 2.0 ** -24
    tiny = 0.0 if fmt == BF16 else (v.abs().sum(0) + L * want.abs()) * 2.0 ** -32 / total
    return want, want.abs() * 2.0 ** -8 * (1 + w) + pv * w * (1 + 2.0 ** -8) + tiny + 1e-30
