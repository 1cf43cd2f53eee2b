"""Plain 64-bit reference of the key/value cache and attention operators, on the
CPU, from the formulas and byte layout stated in include/moe.h.  Shares no code
with the library: values are found byte by byte, sums are float64."""
import math

import numpy as np
import torch

NVFP4, Q8_0, BF16 = 1, 3, 6
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6])


def bf16_bits(x):
    """float64/32 -> fp32 -> bf16 (each to nearest even) as uint16."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float64)).float().bfloat16().view(torch.int16).numpy().view(np.uint16)


def bf16_val(u):
    return (np.asarray(u, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def e4m3_byte(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def e4m3_val(b):
    return torch.from_numpy(np.ascontiguousarray(b, dtype=np.uint8)).view(torch.float8_e4m3fn).double().numpy()


def e2m1_code(r):
    """Nearest E2M1 code of float32 r, ties to the even code, saturating."""
    a = np.abs(r)
    code = np.zeros(a.shape, np.uint8)
    for i in range(7):
        mid = np.float32((E2M1[i] + E2M1[i + 1]) / 2)
        code += (a > mid) | ((a == mid) & (i % 2 == 1))
    return code | (np.signbit(r).astype(np.uint8) << 3)


class Cache:
    """A pool as bytes, read and written token by token."""

    def __init__(self, fmt, n_kv, D, P, n_pages, k_ts=1.0, v_ts=1.0, fill=0):
        self.fmt, self.n_kv, self.D, self.P, self.n_pages = fmt, n_kv, D, P, n_pages
        self.ts = (np.float32(k_ts), np.float32(v_ts)) if fmt == NVFP4 else (np.float32(1), np.float32(1))
        self.codes = P * D * {NVFP4: 4, Q8_0: 8, BF16: 16}[fmt] // 8
        self.scales = 0 if fmt == BF16 else P * D // 16
        self.head = 2 * (self.codes + self.scales)
        self.pool = np.full(n_pages * n_kv * self.head, fill, np.uint8)

    def code_at(self, which, o, d):
        """Byte offset (and nibble) of token o, elements d, inside a head block."""
        D, P = self.D, self.P
        base = which * (self.codes + self.scales)
        if self.fmt == NVFP4:
            if which == 0:
                return base + o * (D // 2) + d // 2, d & 1
            g = D // 16
            return base + ((o // 4 * 16 + d // g) * 4 + o % 4) * (g // 2) + (d % g) // 2, d & 1
        i = o * D + d if which == 0 else (o // 4 * D + d) * 4 + o % 4
        return base + i * (1 if self.fmt == Q8_0 else 2), None

    def scale_at(self, which, o, blk):
        D, P = self.D, self.P
        base = which * (self.codes + self.scales) + self.codes
        nb = D // (16 if self.fmt == NVFP4 else 32)
        i = o * nb + blk if which == 0 else blk * P + o
        return base + i * (1 if self.fmt == NVFP4 else 2)

    def quantise(self, which, x):
        """x: bf16 bits [D] -> (codes, scale bytes) as stored."""
        v = bf16_val(x).astype(np.float32)
        if self.fmt == BF16:
            return x, None
        n = 16 if self.fmt == NVFP4 else 32
        b = v.reshape(-1, n)
        bad = ~np.isfinite(b).all(-1)
        with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
            amax = np.abs(np.where(np.isfinite(b), b, 0)).max(-1)
            if self.fmt == NVFP4:
                ts = self.ts[which]
                s = e4m3_byte(np.minimum(amax / (np.float32(6) * ts), np.float32(448)))
                den = e4m3_val(s).astype(np.float32) * ts
                den = np.where(bad, np.float32(0), den)[:, None]
                q = e2m1_code(np.where(den > 0, b / den, np.float32(0)))
                q = np.where(den > 0, q, 0).astype(np.uint8)
                return q.reshape(-1), np.where(bad, 0x7f, s).astype(np.uint8)
            d = (np.minimum(amax, np.float32(65024)) / np.float32(127)).astype(np.float16)
            den = np.where(bad, np.float32(0), d.astype(np.float32))[:, None]
            q = np.clip(np.rint(np.where(den > 0, b / den, np.float32(0))), -127, 127).astype(np.int8)
            return q.reshape(-1), np.where(bad, np.float16(np.nan), d).astype(np.float16)

    def block(self, page, h):
        o = (page * self.n_kv + h) * self.head
        return self.pool[o:o + self.head]

    def put(self, which, page, o, h, x):
        blk, d = self.block(page, h), np.arange(self.D)
        q, s = self.quantise(which, np.asarray(x, np.uint16))
        at, nib = self.code_at(which, o, d)
        if self.fmt == NVFP4:
            for p, n, c in zip(at, nib, q):
                blk[p] = (blk[p] & (0xf0 if n == 0 else 0x0f)) | (int(c) << (4 * n))
            blk[self.scale_at(which, o, np.arange(len(s)))] = s
        elif self.fmt == Q8_0:
            blk[at] = q.view(np.uint8)
            p = self.scale_at(which, o, np.arange(len(s)))
            u = s.view(np.uint16)
            blk[p], blk[p + 1] = u & 255, u >> 8
        else:
            blk[at], blk[at + 1] = q & 255, q >> 8

    def get(self, which, page, o, h):
        """Values [D] float64 of one token."""
        blk, d = self.block(page, h), np.arange(self.D)
        at, nib = self.code_at(which, o, d)
        if self.fmt == NVFP4:
            x = E2M1[(blk[at] >> (4 * nib)) & 15]
            return x * e4m3_val(blk[self.scale_at(which, o, d // 16)]) * float(self.ts[which])
        if self.fmt == Q8_0:
            p = self.scale_at(which, o, d // 32)
            s = (blk[p].astype(np.uint16) | (blk[p + 1].astype(np.uint16) << 8)).view(np.float16)
            return blk[at].view(np.int8).astype(np.float64) * s.astype(np.float64)
        return bf16_val(blk[at].astype(np.uint16) | (blk[at + 1].astype(np.uint16) << 8))

    def tokens(self, table_row, L, h):
        """k, v [L, D] of a sequence."""
        out = np.empty((2, L, self.D))
        for j in range(L):
            for w in (0, 1):
                out[w, j] = self.get(w, table_row[j // self.P], j % self.P, h)
        return out


def norm_rotate(x, w, eps, pos, rot, interleaved, inv_freq, scale):
    """x [D] float64 -> float64 [D] (not yet rounded)."""
    x = np.asarray(x, np.float64)
    if w is not None:
        x = x / math.sqrt(np.mean(x * x) + float(np.float32(eps))) * np.asarray(w, np.float64)
    y = x.copy()
    for i in range(rot // 2):
        u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a = float(pos) * inv_freq[i]
        c, s = math.cos(a) * float(np.float32(scale)), math.sin(a) * float(np.float32(scale))
        y[u], y[v] = x[u] * c - x[v] * s, x[v] * c + x[u] * s
    return y


def attend(q, k, v, limit, scale):
    """One row: q [D], k, v [L, D]; sees tokens 0..limit.  Returns (out [D], bound
    terms): sum p |v| and the largest sum |q||k| scale over the tokens seen."""
    D = q.shape[0]
    if limit < 0:
        return np.zeros(D), np.zeros(D), 0.0
    k, v = k[:limit + 1], v[:limit + 1]
    with np.errstate(invalid="ignore"):
        s = scale * (k @ q)
        p = np.exp(s - s.max())
        p /= p.sum()
        return p @ v, p @ np.abs(v), float((np.abs(k) @ np.abs(q)).max()) * scale


def attend_bound(ref, pv, qk, n_tok, v_max, D, fmt):
    """How far a result may be from attend()'s, element by element.

    Output: half a bf16 step of the value, 2^-8.  Weights: each is off by its
    rounding, e_p = 2^-11 (fp16) or 2^-8 (bf16), by the error of the scores in
    it (twice, in numerator and denominator), and by 2^-20 for the fp32 sums,
    exponential and reciprocal (n_tok additions of 2^-24 at most, for the sizes
    used here below 2^-12 of the sum).  Scores: fp32 accumulation of D products,
    D 2^-24 of sum |q||k|, and for Q8_0 the rounding of code * scale to fp16,
    2^-11 of it; fp16 weights below 2^-14 round to steps of 2^-24."""
    e_p = 2.0 ** -8 if fmt == BF16 else 2.0 ** -11
    e_kv = 2.0 ** -11 if fmt == Q8_0 else 0.0
    ds = qk * (D * 2.0 ** -24 + e_kv)
    tiny = 0.0 if fmt == BF16 else n_tok * 2.0 ** -25 * v_max
    w = e_p + e_kv + 2 * math.expm1(min(ds, 1.0)) + 2.0 ** -20 + n_tok * 2.0 ** -24
    return np.abs(ref) * 2.0 ** -8 * (1 + w) + pv * w * (1 + 2.0 ** -8) + tiny + 1e-30
