"""Plain forms of the paged K/V cache operators in 64 bits (numpy), and helpers of their tests."""
from __future__ import annotations

import math

import numpy as np


def pages_of(n, page):
    return -(-n // page)


class Ring:
    """The free pages as lists: what il_kv_extend does, one sequence after the other."""

    def __init__(self, size, free, head=0):
        self.size, self.free, self.head = size, list(free), head
        self.tail = head + len(self.free)

    def extend(self, lens, tables, adds, page, width, max_slots):
        """(code, slots, positions, first, info); changes lens, tables (lists of pages) and the ring if code is 0."""
        new = [max(0, max(n, 0) + a) for n, a in zip(lens, adds)]
        had, has = [pages_of(max(n, 0), page) for n in lens], [pages_of(n, page) for n in new]
        take, give = sum(max(0, b - a) for a, b in zip(had, has)), sum(max(0, a - b) for a, b in zip(had, has))
        grow = sum(max(0, a) for a in adds)
        code = ((take > len(self.free)) | 2 * any(x > width or y > width or n >= 2**31 for x, y, n in zip(had, has, new))
                | 4 * (grow > max_slots) | 8 * (len(self.free) + give > self.size))
        info = [code, grow, take, give]
        if code:
            return code, [-1] * max_slots, [-1] * max_slots, [0] * (len(lens) + 1), info
        slots, positions, first, back = [], [], [0], []
        for r in range(len(lens)):
            while len(tables[r]) < has[r]:
                tables[r].append(self.free.pop(0))
            back += tables[r][has[r]:]
            del tables[r][has[r]:]
            for p in range(max(lens[r], 0), new[r]):
                slots.append(tables[r][p // page] * page + p % page)
                positions.append(p)
            first.append(len(slots))
            lens[r] = new[r]
        self.free += back
        self.head += take
        self.tail += give
        pad = [-1] * (max_slots - len(slots))
        return 0, slots + pad, positions + pad, first, info


def quantise(x):
    """Q8 of fp32 rows [..., dim]: (int8, fp32 scales), the definition in IEEE single precision."""
    b = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, 32)
    with np.errstate(all="ignore"):
        d = (np.max(np.abs(b), -1) / np.float32(127)).astype(np.float32)  # max propagates NaN
        usable = (d > 0) & np.isfinite(d)
        q = np.rint(b / np.where(usable, d, np.float32(1))[..., None]).clip(-127, 127)
        q = np.where(usable[..., None], q, 0).astype(np.int8)
    return q.reshape(x.shape), d


def attend(q, keys, values, scale, window):
    """One sequence: q [H][D], keys, values [len][Hk][D] in 64 bits -> out, lse and bounds of their error.

    The bounds, with u = 2^-23 (fp32 spacing): a logit is D products summed in fp32 in any order, its
    operands rounded to no fewer than 21 bits: off by at most delta = (D + 32) u sum|q k| scale.  A weight
    p / sum p is then off by a factor e^(2 delta); the exponential, the rounding of p and the
    division add 16 u; the sums over the tokens run over at most len/16 steps in each part and a
    few dozen joins: (len/16 + 64) u.  All of it times sum p |v|.
    """
    H, D = q.shape
    n = keys.shape[0]
    u = 2.0 ** -23
    out, lse = np.zeros((H, D)), np.full(H, -np.inf)
    out_tol, lse_tol = np.full((H, D), 1e-30), np.zeros(H)
    begin = max(0, n - window) if window else 0
    if n == 0:
        return out, lse, out_tol, lse_tol
    k, v = keys[begin:].astype(np.float64), values[begin:].astype(np.float64)
    G = H // k.shape[1]
    for h in range(H):
        kh, vh = k[:, h // G], v[:, h // G]
        s = scale * (kh @ q[h].astype(np.float64))
        m = s.max()
        e = np.exp(s - m)
        p = e / e.sum()
        out[h] = p @ vh
        lse[h] = m + math.log(e.sum())
        delta = (D + 32) * u * abs(scale) * (np.abs(kh) @ np.abs(q[h].astype(np.float64))).max()
        steps = (len(k) / 16 + 64) * u
        out_tol[h] += (math.expm1(2 * delta) + 16 * u + steps) * (p @ np.abs(vh))
        lse_tol[h] = delta + 16 * u + steps + 4 * u * abs(lse[h])
    return out, lse, out_tol, lse_tol
