"""The 8-bit KV cache in 64 bits on the host: quantisation, attention and page choice from their definitions.

Shares no code with the library.  A cache is held as numpy arrays in the library's layout; rows are float64.
"""

import math

import numpy as np

TOP = {"int8": 127.0, "e4m3": 448.0}
LOW = 16
FLT_MAX = float(np.finfo(np.float32).max)


def e4m3_values():
    """Value of each e4m3 byte (S.1111.111 read as 480, as the library does)."""
    out = np.empty(256)
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        out[b] = (-1) ** (b >> 7) * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return out


E4M3 = e4m3_values()
_POS = E4M3[:127]  # 0 .. 448, increasing


def decode(codes, exps, fmt):
    """codes [..., 16 k, D], exps [..., k] -> float64."""
    x = codes.view(np.int8).astype(np.float64) if fmt == "int8" else E4M3[codes]
    return x * np.repeat(2.0 ** (exps.astype(np.float64) - 127), 16, axis=-1)[..., None]


def exponent(amax, top):
    if amax == 0:
        return LOW
    e = math.frexp(amax)[1] + 127 - 12
    while amax > top * 2.0 ** (e - 127):
        e += 1
    return max(e, LOW)


def quantise(x, fmt):
    """One block [16, D] (NaN counts as 0, infinities do not count for amax) -> codes, exponent."""
    x = np.where(np.isnan(x), 0.0, x)
    fin = np.where(np.isinf(x), 0.0, np.abs(x))
    e = exponent(float(fin.max(initial=0.0)), TOP[fmt])
    y = np.clip(x / 2.0 ** (e - 127), -TOP[fmt], TOP[fmt])
    if fmt == "int8":
        return np.rint(y).astype(np.int8).view(np.uint8), e
    a = np.abs(y)
    hi = np.searchsorted(_POS, a).clip(0, 126)  # first value >= a
    lo = np.maximum(hi - 1, 0)
    up, dn = _POS[hi] - a, a - _POS[lo]
    pick = np.where((up < dn) | ((up == dn) & (hi % 2 == 0)) | (_POS[hi] == a), hi, lo)  # nearest, ties to the even code
    return (pick | np.where(np.signbit(y), 128, 0)).astype(np.uint8), e


class Cache:
    """k, v uint8 [pages, H, PT, D]; k_exp, v_exp uint8 [pages, H, PT / 16]; table int32 [batch, max_pages]."""

    def __init__(self, fmt, pages, heads, page_tokens, dim, table, rng, summaries=True):
        self.fmt, self.H, self.PT, self.D = fmt, heads, page_tokens, dim
        self.table = np.asarray(table, dtype=np.int32)
        shape = (pages, heads, page_tokens, dim)
        # whatever was there before: any byte, NaN patterns and extreme exponents among them
        self.k, self.v = (rng.integers(0, 256, shape, dtype=np.uint8) for _ in range(2))
        self.k_exp, self.v_exp = (rng.choice(np.array([0, 1, 100, 127, 254, 255], np.uint8), shape[:2] + (page_tokens // 16,)) for _ in range(2))
        self.k_min, self.k_max, self.k_sexp = None, None, None
        if summaries:
            self.k_min, self.k_max = (rng.integers(-128, 128, (pages, heads, dim), dtype=np.int8) for _ in range(2))
            self.k_sexp = rng.integers(0, 256, (pages, heads), dtype=np.uint8)

    def append(self, s, start, k, v):
        """k, v float64 [n, H, D] at positions start .. of sequence s."""
        n = len(k)
        if n == 0:
            return
        end = start + n
        for b in range(start // 16, (end + 15) // 16):
            page, sub = self.table[s, b * 16 // self.PT], b * 16 % self.PT // 16
            lo, hi = b * 16, min(b * 16 + 16, end)
            for codes, exps, rows in ((self.k, self.k_exp, k), (self.v, self.v_exp, v)):
                for h in range(self.H):
                    x = np.zeros((16, self.D))
                    old = codes[page, h, sub * 16:sub * 16 + 16]
                    if lo < start:
                        x[:start - lo] = decode(old, exps[page, h, sub:sub + 1], self.fmt)[:start - lo]
                        x = np.where(np.abs(x) > FLT_MAX, np.copysign(np.inf, x), x)  # read back in fp32
                    x[max(start - lo, 0):hi - lo] = rows[max(lo, start) - start:hi - start, h]
                    q, e = quantise(x, self.fmt)
                    old[:hi - lo] = q[:hi - lo]
                    exps[page, h, sub] = e
        if self.k_min is None:
            return
        for pi in range(start // self.PT, (end + self.PT - 1) // self.PT):
            page, held = self.table[s, pi], min(end - pi * self.PT, self.PT)
            x = decode(self.k[page], self.k_exp[page], self.fmt)[:, :held].clip(-FLT_MAX, FLT_MAX)
            for h in range(self.H):
                mn, mx = x[h].min(0), x[h].max(0)
                e = exponent(max(np.abs(mn).max(), np.abs(mx).max()), 127.0)
                self.k_min[page, h] = np.rint(mn / 2.0 ** (e - 127))
                self.k_max[page, h] = np.rint(mx / 2.0 ** (e - 127))
                self.k_sexp[page, h] = e

    def keys(self, s, pages):
        """float64 keys and values [H, len(pages) * PT, D] of pages (indices into the table row)."""
        ids = self.table[s, pages]
        out = []
        for codes, exps in ((self.k, self.k_exp), (self.v, self.v_exp)):
            x = decode(codes[ids], exps[ids], self.fmt)  # [n, H, PT, D]
            out.append(x.transpose(1, 0, 2, 3).reshape(self.H, -1, self.D))
        return out

    def attend(self, s, q, limit, scale, pages=None, mantissa=22, planes=22):
        """q float64 [Hq, D] of one row -> out [Hq, D], lse [Hq], and error bounds of both for a kernel that sums in
        fp32 with q used to `mantissa` bits and weights to `planes` bits (relative errors 2^-mantissa and 2^-planes), both
        through f16 after a scaling that puts the largest at 2^14 or above, so that f16's least step (2^-24) is 2^-38 of
        it.  pages: list per key/value head, or None.

        A score is a sum of D products taken in fp32 (at most D + 4 roundings, each of at most 2^-23 of the sum of
        magnitudes: the tensor core may cut instead of round) from a q off by 2^-mantissa of itself or by half of f16's
        least step; all scores off by d move each weight by a factor exp(+-2 d).  An output is a sum of L weighted values:
        weights off by 2^-planes, the exponential and its argument's rounding (2^-22 (1 + |score|)), and at most L / 4 + 64
        roundings of 2^-23.  Weights times their block's scale are taken relative to 1 times the largest scale and 2^8 at
        least: off by half of f16's least step, 2^-33, each times a code of at most top."""
        Hq = len(q)
        G = Hq // self.H
        out, lse = np.zeros((Hq, self.D)), np.full(Hq, -np.inf)
        eo, el = np.zeros((Hq, self.D)), np.zeros(Hq)
        for h in range(Hq):
            kv = h // G
            mine = list(range((limit + self.PT - 1) // self.PT)) if pages is None else list(pages[kv])
            if limit <= 0 or not mine:
                continue
            k, v = (x[kv] for x in self.keys(s, mine))
            pos = np.concatenate([p * self.PT + np.arange(self.PT) for p in mine])
            see = pos < limit
            if not see.any():
                continue
            k, v = k[see], v[see]
            z = scale * (k @ q[h])
            m = z.max()
            w = np.exp(z - m)
            lse[h] = m + np.log(w.sum())
            p = w / w.sum()
            out[h] = p @ v
            mag = float((abs(scale) * (np.abs(k) @ np.abs(q[h]))).max())
            d = mag * ((self.D + 4) * 2.0 ** -23 + 2.0 ** -mantissa) + 2.0 ** -22 * (1 + np.abs(z).max())
            d += 2.0 ** -39 * float(abs(scale) * np.abs(q[h]).max() * np.abs(k).sum(1).max())
            top = TOP[self.fmt] * 2.0 ** (float(self.v_exp[self.table[s, mine], kv].reshape(-1)[see.reshape(-1, 16).any(1)].max()) - 127)
            n = (len(z) / 4 + 64) * 2.0 ** -23
            eo[h] = (p @ np.abs(v)) * (2 * d + n + 2.0 ** -planes) + 2.0 ** -33 * len(z) * top
            el[h] = d + n + 2.0 ** -22 * (1 + abs(lse[h]))
        return out, lse, eo, el

    def select(self, s, q, limit, n_select, n_sink, n_local):
        """Pages chosen for one row, per key/value head."""
        nb = max(0, -(-limit // self.PT))
        out = []
        G = len(q) // self.H
        for h in range(self.H):
            if nb <= n_select:
                out.append(list(range(nb)))
                continue
            score = np.full(nb, -np.inf)
            for g in range(G):
                x = np.where(np.isnan(q[h * G + g]), 0.0, q[h * G + g])
                e = exponent(float(np.where(np.isinf(x), 0.0, np.abs(x)).max()), 127.0)
                qi = np.clip(np.rint(x / 2.0 ** (e - 127)), -127, 127)
                for p in range(nb):
                    page = self.table[s, p]
                    dot = np.maximum(qi * self.k_min[page, h].astype(np.float64), qi * self.k_max[page, h].astype(np.float64)).sum()
                    score[p] = max(score[p], dot * 2.0 ** (e - 127) * 2.0 ** (float(self.k_sexp[page, h]) - 127))
            must = [p for p in range(nb) if p < n_sink or p >= nb - n_local]
            rest = sorted((p for p in range(nb) if p not in must), key=lambda p: (-score[p], p))
            out.append(sorted(must + rest[:n_select - len(must)]))
        return out
