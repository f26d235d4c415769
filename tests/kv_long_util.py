"""Plain forms in 64 bits (numpy) of the K/V cache operators for long contexts -- the 4-bit format, capped, biased and masked
scores, collected weights, eviction -- and what their tests share."""
from __future__ import annotations

import math

import numpy as np

import kv_util

U = 2.0 ** -23  # spacing of fp32 at 1


def _toward(x, up):
    """bf16 at or beyond fp32 x, as fp32."""
    bits = np.asarray(x, np.float32).view(np.uint32)
    head = bits & np.uint32(0xffff0000)
    short = (bits != head) & (((bits >> 31) == 0) if up else ((bits >> 31) == 1))
    return (head + (short.astype(np.uint32) << np.uint32(16))).view(np.float32)


def quantise(x):
    """IL_A4 of fp32 rows [..., dim]: (u of 0 .. 15 [..., dim], fp32 pairs d, m [..., dim / 32]), in IEEE single precision."""
    b = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, 32)
    with np.errstate(all="ignore"):
        least, most = np.min(b, -1), np.max(b, -1)  # both propagate NaN
        m = _toward(least, False)
        d = _toward(((most - m) / np.float32(15)).astype(np.float32), True)
        good = np.isfinite(least) & np.isfinite(d)
        usable = good & (d > 0)
        u = np.rint((b - m[..., None]) / np.where(usable, d, np.float32(1))[..., None]).clip(0, 15)
        u = np.where(usable[..., None], u, 0).astype(np.uint8)
    return u.reshape(x.shape), np.where(good, d, np.float32(0)), np.where(good, m, np.float32(np.nan))


def values(u, d, m):
    """What IL_A4 stands for, in 64 bits (no rounding)."""
    rep = lambda t: np.repeat(t.astype(np.float64), 32, -1)  # noqa: E731
    return u * rep(d) + rep(m)


def pack(u):
    return u[..., 0::2] | (u[..., 1::2] << 4)


def pool(fmt, x, place):
    """A cache's tensors of fp32 rows x [..][dim]: ([k or v, scale or None], values, magnitudes of the terms that make them)."""
    import torch
    if fmt == "bf16":
        t = torch.from_numpy(x).bfloat16()
        f = t.double().numpy()
        return [place(t), None], f, np.abs(f)
    if fmt == "q8":
        q, s = kv_util.quantise(x)
        f = q * np.repeat(s, 32, -1).astype(np.float64)
        return [place(torch.from_numpy(q)), place(torch.from_numpy(s))], f, np.abs(f)
    u, d, m = quantise(x)
    pairs = torch.from_numpy(np.stack([d, m], -1)).bfloat16()
    return [place(torch.from_numpy(pack(u))), place(pairs)], values(u, d, m), u * np.repeat(np.abs(d), 32, -1) + np.repeat(np.abs(m), 32, -1)


def begin_of(n, window, start):
    return min(n, max(max(0, n - window) if window else 0, start, 0))


def logits(q, keys, kmag, scale, cap=0.0, slopes=None, far=None):
    """Logits [H][T] of q [H][D] over keys [T][Hk][D], and a bound of their error in fp32.

    A product's D terms are summed in any order, their operands rounded to no fewer than 21 bits: (D + 32) u of the sum of the
    terms' magnitudes.  tanh has slope at most 1; tanhf, the multiplications and the bias's rounding add 8 u of what they give.
    """
    H, D = q.shape
    G = H // keys.shape[1]
    q = q.astype(np.float64)
    s, tol = np.empty((H, keys.shape[0])), np.empty((H, keys.shape[0]))
    for h in range(H):
        s[h] = scale * (keys[:, h // G] @ q[h])
        tol[h] = (D + 32) * U * abs(scale) * (kmag[:, h // G] @ np.abs(q[h]))
    if cap:
        s = cap * np.tanh(s / cap)
        tol = tol + 8 * U * np.abs(s)
    if slopes is not None:
        bias = slopes.astype(np.float64)[:, None] * far[None, :].astype(np.float64)
        s = s + bias
        tol = tol + 8 * U * (np.abs(bias) + np.abs(s))
    return s, tol


def attend(q, keys, values_, kmag, vmag, scale, floor=0.0, **score):
    """One sequence's seen tokens: q [H][D], keys, values [T][Hk][D] -> out, lse and bounds of their error (see
    kv_util.attend): a weight is off by a factor e^(2 tol), the sum of the weights by the mean of those; the exponential, the
    rounding of p and the division add 16 u, the sums over the tokens (T / 16 + 64) u.  floor: what every weight may be off by
    beside that, of the largest."""
    H, D = q.shape
    T = keys.shape[0]
    out, lse = np.zeros((H, D)), np.full(H, -np.inf)
    out_tol, lse_tol = np.full((H, D), 1e-30), np.zeros(H)
    if T == 0:
        return out, lse, out_tol, lse_tol
    s, tol = logits(q, keys, kmag, scale, **score)
    G = H // keys.shape[1]
    steps = (T / 16 + 64) * U
    for h in range(H):
        m = s[h].max()
        e = np.exp(s[h] - m)
        p = e / e.sum()
        off = p * np.expm1(2 * tol[h])
        out[h] = p @ values_[:, h // G]
        lse[h] = m + math.log(e.sum())
        mag = p @ vmag[:, h // G]
        out_tol[h] += off @ vmag[:, h // G] + (off.sum() + 16 * U + steps) * mag + floor * p.max() * vmag[:, h // G].sum(0)
        lse_tol[h] = off.sum() + 16 * U + steps + 4 * U * abs(lse[h])
    return out, lse, out_tol, lse_tol


def weigh(q, keys, kmag, scale, lse, **score):
    """What one token's attention adds to each of the seen tokens, and a bound of the error: each head's weight as above,
    the heads' sum in any order."""
    s, tol = logits(q, keys, kmag, scale, **score)
    # s - lse in fp32, in units of log2: their rounding is of their own sizes
    tol = tol + 4 * U * (np.abs(s) + np.abs(lse)[:, None])
    p = np.exp(s - lse[:, None])
    return p.sum(0), (p * (np.expm1(2 * tol) + (16 + len(q)) * U)).sum(0) + 1e-30


def evict(weights, positions, n, keep, first, recent):
    """Entries of one sequence after an eviction: the old index of each of the min(n, keep) that are left."""
    if n <= keep:
        return list(range(n))
    newest = int(positions[n - 1])
    def key(i):
        w = float(weights[i])
        always = positions[i] < first or positions[i] > newest - recent
        return (0 if always else 1, 1 if math.isnan(w) else 0, 0.0 if math.isnan(w) else -w, i)
    stay = sorted(range(n), key=key)[:keep]
    movers = iter(sorted(i for i in stay if i >= keep))
    kept = set(stay)
    return [i if i in kept else next(movers) for i in range(keep)]


class Case:
    """A cache in which only the seen tokens hold numbers: everything else, the other pages included, is NaN (or, of 4-bit
    elements, has NaN steps), and the table names pages that do not exist behind each sequence's own."""

    def __init__(self, sil, fmt, heads, kv, dim, page, lens, order="head", seed=0, window=0, spread=1.0, cap=0.0, slopes=None,
                 starts=None, positions=False, lopsided=0.0):
        import torch
        rng = np.random.default_rng(seed)
        self.sil, self.fmt, self.lens, self.page, self.heads, self.dim, self.window = sil, fmt, list(lens), page, heads, dim, window
        self.cap, self.slopes, self.starts = cap, slopes, starts
        held = [kv_util.pages_of(n, page) for n in lens]
        n_pages, width = sum(held) + 3, max(held + [1]) + 2
        perm = rng.permutation(n_pages)
        self.table = np.full((len(lens), width), 2**31 - 1, np.int32)
        self.table[:, -1] = -7
        k = np.full((n_pages, page, kv, dim), np.nan, np.float32)
        v = k.copy()
        self.begins = [begin_of(n, window, 0 if starts is None else starts[r]) for r, n in enumerate(lens)]
        offset = lopsided * rng.standard_normal((kv, dim))  # channels that do not lie about 0
        at = 0
        for r, n in enumerate(lens):
            mine = perm[at:at + held[r]]
            at += held[r]
            self.table[r, :held[r]] = mine
            p = np.arange(self.begins[r], n)
            k[mine[p // page], p % page] = spread * rng.standard_normal((len(p), kv, dim)) + offset
            v[mine[p // page], p % page] = rng.standard_normal((len(p), kv, dim)) + offset

        def place(t):
            if order == "head":
                return t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
            if order == "padded":  # rows apart, pages not next to each other; of 16 bytes, and of 4 where they are scales
                size = t.element_size() * (2 if t.dim() == 5 else 1)
                wide = torch.zeros((t.shape[0], t.shape[1] + 1, t.shape[2] + 1,
                                    t.shape[3] + (1 if t.dim() == 5 or t.dtype == torch.float32 else 16 // size), *t.shape[4:]), dtype=t.dtype)
                wide[:, :t.shape[1], :t.shape[2], :t.shape[3]] = t
                return wide.cuda()[:, :t.shape[1], :t.shape[2], :t.shape[3]]
            return t.contiguous().cuda()

        (kt, ks), kd, km = pool(fmt, k, place)
        (vt, vs), vd, vm = pool(fmt, v, place)
        self.cache = sil.KVCache(kt, vt, ks, vs)
        self.rows = []
        for r, n in enumerate(lens):
            p = np.arange(self.begins[r], n)
            rows = self.table[r, p // page], p % page
            self.rows.append((kd[rows], vd[rows], km[rows], vm[rows]))
        self.q = rng.standard_normal((len(lens), heads, dim)).astype(np.float32)
        most = max(list(lens) + [1])
        self.positions = None
        if positions:  # any order, the last the newest; a row is wider than any sequence
            self.positions = np.stack([rng.permutation(2 * most)[:most + 3] for _ in lens]).astype(np.int32)
            for r, n in enumerate(lens):
                if n:
                    self.positions[r, n - 1] = 2 * most

    def score(self):
        """Keyword arguments of the entry points."""
        import torch
        to = lambda x, dtype: None if x is None else torch.from_numpy(np.asarray(x, dtype)).cuda()  # noqa: E731
        return {"window": self.window, "cap": self.cap, "slopes": to(self.slopes, np.float32), "starts": to(self.starts, np.int32),
                "positions": to(self.positions, np.int32)}

    def plain_score(self, r):
        if self.slopes is None:
            return {"cap": self.cap}
        n = self.lens[r]
        pos = np.arange(n) if self.positions is None else self.positions[r, :n].astype(np.int64)
        return {"cap": self.cap, "slopes": np.asarray(self.slopes, np.float32), "far": (pos - pos[-1])[self.begins[r]:] if n else pos}

    def device(self):
        import torch
        return torch.from_numpy(self.q).cuda(), torch.from_numpy(self.table).cuda(), torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def run(self, stream=None, scale=None, q=None, out=None):
        import torch
        own, table, lens = self.device()
        out = torch.full((len(self.lens), self.heads, self.dim), float("nan"), device="cuda") if out is None else out
        lse = torch.full((len(self.lens), self.heads), float("nan"), device="cuda")
        more = self.score()
        torch.cuda.synchronize()
        self.sil.kv_attend(self.cache, own if q is None else q, table, lens, out, lse=lse, scale=scale, stream=stream, **more)
        torch.cuda.synchronize()
        return out, lse

    def check(self, out, lse, scale=None, rows=None):
        out, lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        scale = self.dim ** -0.5 if scale is None else scale
        for r in range(len(self.lens)) if rows is None else rows:
            k, v, km, vm = self.rows[r]
            # of Q8 the header states that p d is kept to 2^-26 d where 22 bits of it are less, p relative to the largest: a token's
            # part of out is off by 2^-26 d |q| = 2^-26 |v| of the largest weight then, which counts where a V of exactly 0 is in the
            # largest one's place.
            # (With scores the header promises more.)
            plain = self.cap == 0 and self.slopes is None and self.starts is None
            o, l, ot, lt = attend(self.q[r], k, v, km, vm, scale, floor=2.0**-26 if self.fmt == "q8" and plain else 0.0, **self.plain_score(r))
            assert np.all(np.isfinite(out[r])), (r, self.lens[r])
            worst = float(np.max(np.abs(out[r] - o) / ot))
            assert worst <= 1, f"sequence {r} of length {self.lens[r]}: out is {worst:.3g} x its bound"
            if len(k) == 0:
                assert np.all(np.isneginf(lse[r])) and np.all(out[r] == 0)
            else:
                worst = float(np.max(np.abs(lse[r] - l) / lt))
                assert worst <= 1, f"sequence {r} of length {self.lens[r]}: lse is {worst:.3g} x its bound"
