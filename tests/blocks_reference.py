"""Plain 64-bit reference of the block-scaled 8-bit cache (write_kv and what reads it) and of
update_pages. Loops over definitions; shares no code with the library."""
import math

import numpy as np

GROUPS = [(0, 128), (128, 256), (256, 384), (384, 512), (512, 576)]
LEAST = -110
NAN_CODE = 0x7F


def _table():
    """The value of every e4m3 code."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = (math.nan if (c & 0x7F) == 0x7F else x) * (-1 if c & 0x80 else 1)
    return v


VALUE = _table()
_UP = VALUE[:127]                         # codes of the magnitudes, ascending
_MID = (_UP[1:] + _UP[:-1]) / 2


def power(top):
    """The smallest e >= LEAST with top <= 448 * 2^e."""
    if top == 0:
        return LEAST
    f, x = math.frexp(top)  # top = f * 2^x, 0.5 <= f < 1; 448 = 0.875 * 2^9
    return max(LEAST, x - 9 + (1 if f > 0.875 else 0))


def codes(x):
    """Nearest e4m3 codes of an array, ties to the even code; NaN for what is not finite."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.abs(np.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0))
    lo = np.searchsorted(_MID, mag, side="left")    # a tie goes to the lower code
    hi = np.searchsorted(_MID, mag, side="right")   # ... or to the upper one
    c = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi)).astype(np.uint8)
    c |= np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(np.isfinite(x), c, NAN_CODE).astype(np.uint8)


def write(cache, entries, rows, table, lens, new, page, block):
    """write_kv on numpy arrays in place: cache [pages, page, 576] and entries [pages, page // block, 8] uint8,
    rows [T, 576] float64, table a list of lists, lens and new lists."""
    at = 0
    for b, (L, n) in enumerate(zip(lens, new)):
        p0 = L - n
        for k in range(p0 // block, -(-L // block)) if n else ():
            lo, hi = max(k * block, p0), min(k * block + block, L)
            pg, off = table[b][k * block // page], k * block % page
            entry = entries[pg, off // block]
            for g, (c0, c1) in enumerate(GROUPS):
                x = rows[at + lo - p0:at + hi - p0, c0:c1]
                e = power(np.abs(np.where(np.isfinite(x), x, 0)).max())
                older = slice(off, off + lo - k * block)
                if lo > k * block:
                    before = int(entry[g]) - 127
                    if e > before:
                        cache[pg, older, c0:c1] = codes(np.ldexp(VALUE[cache[pg, older, c0:c1]], before - e))
                    e = max(e, before)
                entry[g] = e + 127
                cache[pg, off + lo - k * block:off + hi - k * block, c0:c1] = codes(np.ldexp(x, -e))
            entry[5:] = 0
        at += n


def values(cache, entries):
    """The values that a cache holds, float64 [pages, page, 576]."""
    page = cache.shape[1]
    e = np.repeat(entries[:, :, :5].astype(np.int64) - 127, page // entries.shape[1], axis=1)
    out = VALUE[cache]
    for g, (c0, c1) in enumerate(GROUPS):
        out[:, :, c0:c1] = np.ldexp(out[:, :, c0:c1], e[:, :, g:g + 1])
    return out


class Pages:
    """update_pages on Python lists."""

    def __init__(self, table, held, free, page):
        self.table, self.held, self.free, self.page = [list(r) for r in table], list(held), list(free), page
        self.refused = []

    def update(self, lens, new=None, n_rows=0):
        """Returns the slots; self.refused tells the sequences that were not served."""
        need = [-(-L // self.page) for L in lens]
        back = []
        for b, n in enumerate(need):
            for j in range(n, self.held[b]):
                back.append(self.table[b][j])
                self.table[b][j] = -1
        self.free += reversed(back)
        self.refused, room = [], len(self.free)
        for b, n in enumerate(need):
            missing = max(0, n - self.held[b])
            room -= missing
            if missing and room < 0:
                self.refused.append(b)
                continue
            for j in range(self.held[b], n):
                self.table[b][j] = self.free.pop()
            self.held[b] = n
        if new is None:
            return None
        slots = []
        for b, (L, n) in enumerate(zip(lens, new)):
            for pos in range(L - n, L):
                slots.append(-1 if b in self.refused else self.table[b][pos // self.page] * self.page + pos % self.page)
        return slots + [-1] * (n_rows - len(slots))
