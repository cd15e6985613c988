"""The operators of the products held in few bits, from their definitions, in
64 bits on the CPU: numpy only, one sequence, head and row at a time. Nothing
here is shared with the library."""

from __future__ import annotations

import numpy as np


# ------------------------------------------------------------------ W4


def codes_of(packed: np.ndarray, K: int) -> np.ndarray:
    q = np.empty((packed.shape[0], 2 * packed.shape[1]), np.int64)
    q[:, 0::2], q[:, 1::2] = packed & 15, packed >> 4
    return q[:, :K]


def w4_matrix(packed, scales, zeros, K, group) -> np.ndarray:
    """N x K doubles."""
    g = np.arange(K) // group
    z = 8 if zeros is None else (zeros.astype(np.int64) & 15)[:, g]
    return (codes_of(packed, K) - z) * scales.astype(np.float64)[:, g]


def round_half_even(x):
    return np.rint(x)


def w4_quantize(W: np.ndarray, group: int, zeros: bool, to_stype):
    """(codes N x K, scales, zeros or None); W float64 holding values of the
    input's type, to_stype a rounding of float32 values to the scales' type."""
    N, K = W.shape
    G = -(-K // group)
    q = np.empty((N, K), np.int64)
    S = np.empty((N, G), np.float64)
    Z = np.full((N, G), 8, np.int64)
    for n in range(N):
        for g in range(G):
            w = W[n, g * group:(g + 1) * group]
            if not np.isfinite(w).all():
                S[n, g], q[n, g * group:(g + 1) * group] = np.nan, 8
                continue
            if zeros:
                lo, hi = min(0.0, w.min()), max(0.0, w.max())
                span = np.float64(np.float32(hi) - np.float32(lo)) / 15
            else:
                lo, span = 0.0, np.abs(w).max() / 7
            s = np.float64(to_stype(np.float32(span)))
            S[n, g] = s
            if s == 0:
                q[n, g * group:(g + 1) * group] = 8
                continue
            if zeros:
                Z[n, g] = min(15, max(0, int(round_half_even(-lo / s))))
            q[n, g * group:(g + 1) * group] = np.clip(round_half_even(w / s) + Z[n, g], 0, 15)
    return q, S, (Z if zeros else None)


# ------------------------------------------------------------------ KV8

E4M3 = np.empty(256)
for _c in range(256):
    _e, _f = (_c >> 3) & 15, _c & 7
    _v = _f * 2.0**-9 if _e == 0 else (1 + _f / 8) * 2.0**(_e - 7)
    if _e == 15 and _f == 7:
        _v = np.nan
    E4M3[_c] = -_v if _c & 0x80 else _v


def e4m3(x: np.ndarray) -> np.ndarray:
    """Codes of doubles (|x| <= 448 or NaN), to nearest, ties to even; the
    sign of zeros is kept."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    with np.errstate(all="ignore"):
        e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6)
        n = np.rint(a / 2.0**(e - 3))          # in 8..16 for normal numbers, 0..8 below
        up = n >= 16
        e, n = np.where(up, e + 1, e), np.where(up, 8, n)
        code = np.where(n >= 8, ((e + 7) * 8 + (n - 8)), n)
    code = np.where(np.isnan(a), 0x7F, code).astype(np.int64)
    return np.where(np.signbit(x) & ~np.isnan(x), code | 0x80, code).astype(np.uint8)


def scale_for(x: np.ndarray) -> float:
    a = np.abs(x[np.isfinite(x)])
    top = a.max() if a.size else 0.0
    if top == 0:
        return 0.0
    s = 2.0**-126
    while top / s > 448:
        s *= 2
    return s


class Cache:
    """Codes (pages, heads, block, dim uint8) and scales (pages, heads)."""

    def __init__(self, K, V, Ks, Vs):
        self.codes = [K.copy(), V.copy()]
        self.scales = [Ks.astype(np.float64).copy(), Vs.astype(np.float64).copy()]
        self.pages, self.heads, self.block, self.dim = K.shape

    def page(self, table, b, p):
        if p >= table.shape[1]:
            return -1
        page = int(table[b, p])
        return page if 0 <= page < self.pages else -1

    def write(self, new, table, lens, starts):
        """new: [K, V], rows x heads x dim doubles."""
        rows = new[0].shape[0]
        for b in range(len(lens)):
            first, end = (min(max(int(s), 0), rows) for s in starts[b:b + 2])
            n, length = max(0, end - first), max(0, int(lens[b]))
            start = length - n
            for p in range(max(start, 0) // self.block, -(-length // self.block)):
                t0 = p * self.block
                lo, hi = max(start, t0), min(length, t0 + self.block)
                page = self.page(table, b, p)
                if page < 0 or hi <= lo:
                    continue
                for i in range(2):
                    for h in range(self.heads):
                        x = new[i][first + lo - start:first + hi - start, h]
                        codes = self.codes[i][page, h]
                        old = self.scales[i][page, h] if lo > t0 else 0.0
                        s = max(scale_for(x), old)
                        if lo > t0 and s != old:
                            codes[:lo - t0] = e4m3(E4M3[codes[:lo - t0]] * (old / s))
                        with np.errstate(all="ignore"):
                            v = np.where(np.isfinite(x), x / s if s > 0 else 0.0 * np.sign(x), np.nan)
                        codes[lo - t0:hi - t0] = e4m3(v)
                        self.scales[i][page, h] = s

    def tokens(self, table, b, count, i):
        """count x heads x dim values of sequence b's first tokens; NaN on
        pages that are not the cache's."""
        out = np.full((count, self.heads, self.dim), np.nan)
        for p in range(-(-count // self.block)):
            page = self.page(table, b, p)
            hi = min(count, (p + 1) * self.block)
            if page >= 0:
                v = E4M3[self.codes[i][page]] * self.scales[i][page][:, None, None]
                out[p * self.block:hi] = v.transpose(1, 0, 2)[:hi - p * self.block]
        return out

    def attend(self, Q, table, lens, starts, scale, causal, window):
        """(O, bound): O rows x heads_q x dim doubles (NaN rows outside the
        sequences), and a bound on a float32 evaluation's error."""
        rows, heads_q, dim = Q.shape
        O, bound = np.full(Q.shape, np.nan), np.zeros(Q.shape)
        u = 2.0**-24
        for b in range(len(lens)):
            first, end = (min(max(int(s), 0), rows) for s in starts[b:b + 2])
            n, length = max(0, end - first), max(0, int(lens[b]))
            if n == 0:
                continue
            named = table.shape[1] * self.block  # a row that sees a token behind them is NaN
            K, V = (self.tokens(table, b, min(length, named), i) for i in range(2))
            for i in range(n):
                p = length - n + i
                hi = min(length, p + 1) if causal else length
                lo = max(0, p + 1 - window) if window else 0
                for h in range(heads_q):
                    if hi > named:
                        continue  # NaN
                    if hi <= lo:
                        O[first + i, h] = 0.0
                        continue
                    k, v, q = K[lo:hi, h // (heads_q // self.heads)], V[lo:hi, h // (heads_q // self.heads)], Q[first + i, h]
                    z = k @ q * scale
                    w = np.exp(z - z.max())
                    w /= w.sum()
                    O[first + i, h] = w @ v
                    # z: dim products, their float32 sum and two multiplications, each rounding at most u
                    # of the sum of magnitudes; an error d of z moves its weight by d and the normaliser by
                    # at most the largest d. 2^x is good to 2 units; weights and V's scale are rounded once
                    # each, the two sums have hi - lo terms and a few rescalings.
                    d = (dim + 4) * u * np.abs(scale) * (np.abs(k) @ np.abs(q)).max() + 4 * u
                    bound[first + i, h] = (2 * d + (2 * (hi - lo) + 64) * u) * (w @ np.abs(v)) + 1e-30
        return O, bound
