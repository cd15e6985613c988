"""The operators of a serving step in numpy doubles, from their definitions in
include/sgemm.h, for the tests: the 4-bit cache and attention over it, rotary
positions, page tables."""

import numpy as np

from tests import lowbit_ref

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
# Half way between neighbouring levels. A tie goes to the even code: to the
# lower one at the first, third, .. of them.
MIDPOINTS = (LEVELS[1:] + LEVELS[:-1]) / 2


def e2m1(x: np.ndarray) -> np.ndarray:
    """Codes of doubles, to nearest, ties to even, at most 6 in size."""
    a = np.abs(np.asarray(x, np.float64))
    code = np.zeros(a.shape, np.int64)
    for i, m in enumerate(MIDPOINTS):
        code += (a >= m) if i % 2 else (a > m)
    return np.where(np.signbit(x) & (code > 0), code | 8, code).astype(np.uint8)


def values(packed: np.ndarray) -> np.ndarray:
    """What packed codes stand for, the lower half of a byte first."""
    code = np.stack([packed & 15, packed >> 4], axis=-1).reshape(*packed.shape[:-1], -1)
    return np.where(code & 8, -1.0, 1.0) * LEVELS[code & 7]


def pack(code: np.ndarray) -> np.ndarray:
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def bf16(x) -> np.ndarray:
    """float32 values rounded to bfloat16 (ties to even), as doubles."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)
    return r.view(np.float32).astype(np.float64)


def scale_of(x: np.ndarray) -> np.ndarray:
    """The scale of each row (last dimension), NaN where a value is not finite."""
    with np.errstate(invalid="ignore"):
        top = np.abs(x).max(axis=-1)
    fine = np.isfinite(x).all(axis=-1)
    s = bf16(np.where(fine, top, 1).astype(np.float32) / np.float32(6))
    s = np.where(top > 0, np.maximum(s, 2.0**-100), 0.0)
    return np.where(fine, s, np.nan)


class Cache(lowbit_ref.Cache):
    """Codes (pages, heads, block, dim / 2 bytes) and scales (pages, heads, block)."""

    def __init__(self, K, V, Ks, Vs):
        self.codes = [K.copy(), V.copy()]
        self.scales = [Ks.astype(np.float64).copy(), Vs.astype(np.float64).copy()]
        self.pages, self.heads, self.block = K.shape[:3]
        self.dim = 2 * K.shape[3]

    def write(self, new, table, lens, starts):
        """new: [K, V], rows x heads x dim doubles."""
        rows = new[0].shape[0]
        for b in range(len(lens)):
            first, end = (min(max(int(s), 0), rows) for s in starts[b:b + 2])
            n, length = max(0, end - first), max(0, int(lens[b]))
            for i in range(n):
                t = length - n + i
                page = self.page(table, b, t // self.block) if t >= 0 else -1
                if page < 0:
                    continue
                for j in range(2):
                    x = new[j][first + i]
                    s = scale_of(x)
                    safe = np.where(s > 0, s, 1.0)[:, None]
                    code = np.where(np.isfinite(s)[:, None], e2m1(np.where(np.isfinite(x), x, 0) / safe), 0)
                    self.codes[j][page, :, t % self.block] = pack(code.astype(np.uint8))
                    self.scales[j][page, :, t % self.block] = s

    def tokens(self, table, b, count, i):
        """count x heads x dim values of sequence b's first tokens; NaN on
        pages that are not the cache's, and where a scale is not finite."""
        out = np.full((count, self.heads, self.dim), np.nan)
        for p in range(-(-count // self.block)):
            page = self.page(table, b, p)
            hi = min(count, (p + 1) * self.block)
            if page >= 0:
                s = np.where(np.isfinite(self.scales[i][page]), self.scales[i][page], np.nan)
                v = values(self.codes[i][page]) * s[:, :, None]
                out[p * self.block:hi] = v.transpose(1, 0, 2)[:hi - p * self.block]
        return out

    def attend(self, Q, table, lens, starts, scale, causal, window):
        """(O, bound) as lowbit_ref.Cache.attend, whose reasoning holds here:
        the codes enter the products exactly and the scales in float32. The
        kernel may hold a weight to 2^-22 of itself or 2^-38 of the largest
        value's scale, whichever is more: the first is within the 64 units of
        that bound, the second is added for each token seen (codes up to 6)."""
        O, bound = super().attend(Q, table, lens, starts, scale, causal, window)
        top = max([np.abs(s[np.isfinite(s)]).max(initial=0.0) for s in self.scales[1:]])
        most = max([0] + [int(l) for l in lens if l < 2**30])
        return O, bound + min(most, table.shape[1] * self.block) * 2.0**-38 * 6 * top


def rope(x, positions, freqs, interleaved=False, amplitude=1.0, inverse=False):
    """rows x heads x dim doubles turned; angles in extended precision."""
    half = len(freqs)
    angle = positions.astype(np.longdouble)[:, None] * freqs.astype(np.longdouble)[None, :]
    c, s = np.cos(angle).astype(np.float64)[:, None] * amplitude, np.sin(angle).astype(np.float64)[:, None] * amplitude
    s = -s if inverse else s
    y = x.astype(np.float64).copy()
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


def tables(table, lens, new, pool, taken, block, rows):
    """(starts, positions, slots, taken_after, table), in Python integers."""
    table = table.copy()
    columns, starts, positions, slots = table.shape[1], [0], [], []
    at = int(taken)
    for b in range(len(lens)):
        length = max(0, int(lens[b]))
        n = min(max(0, int(new[b])), length)
        starts.append(min(starts[-1] + n, 2**31 - 1))
        for column in range(-(-(length - n) // block), min(-(-length // block), columns)):
            table[b, column] = pool[at] if 0 <= at < len(pool) else -1
            at += 1
        for t in range(length - n, length):
            if len(positions) == rows:
                break
            page = int(table[b, t // block]) if t // block < columns else -1
            positions.append(t)
            slots.append(page * block + t % block if page >= 0 else -1)
    return np.array(starts), np.array(positions, np.int64), np.array(slots, np.int64), min(at, 2**31 - 1), table
