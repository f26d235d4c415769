"""How many bits of q and of the weights the K/V operators keep: bounds that a lost part of a split operand fails.

One token seen, its lse is its logit.  One element of q other than 0, the logit is one product, and nothing but the operands' parts
and a few roundings is left of its error; that bound takes all positions of the element.  With every element, the sums' errors count, which
are bounded by their rms.
"""
import math

import numpy as np
import pytest

import kv_long_util as kl

U = 2.0 ** -24  # half a spacing of fp32 at 1: a rounding


def terms(fmt, keys, kmag):
    """What a product's operands may be as large as in the sums: K; of 8 bits, which enter as q + 128, 256 steps.  A block's step is
    at least its largest element / 127."""
    if fmt != "q8":
        return kmag
    blocks = np.abs(keys).reshape(*keys.shape[:-1], -1, 32)
    return np.repeat(blocks.max(-1), 32, -1) * 256 / 127


def one_product(fmt, q, keys, kmag, scale):
    """Logits [H] of q [H][D], one element each, over one token, and their bound: 22 bits (2^-22) of q, and 8 roundings -- scale log2(e)
    and q times it (3), the block's sum, its step, the unit's two factors, ln 2 -- of the logit, 2 of the terms that its sum is made of."""
    g = q.shape[0] // keys.shape[0]
    k, m, t = (np.repeat(x.astype(np.float64), g, 0) for x in (keys, kmag, terms(fmt, keys, kmag)))
    a = np.abs(scale * q.astype(np.float64))
    return scale * (k * q.astype(np.float64)).sum(-1), (a * m).sum(-1) * (2.0 ** -22 + 8 * U) + (a * t).sum(-1) * 2 * U


# Of all elements: the rms of the error over that of one term times sqrt(D).  Sums of 16 products are cut 25 bits below the exponent of their
# largest operands; 4-bit and 8-bit K are subnormals there, 2 u or u of 2^-10 at most: a cut of up to 2^-17 (2^-15) steps a
# product of the largest q, 2.6 times its rms, evenly spread (rms 1 / sqrt 3): 2^-16.4 (2^-14.4) steps of K of 15 (60) steps, 2^-20.3.
# bf16: 16 steps of the sum, each cut by 2^-24 of it, 2^-20.  The other parts are less than as much again.
DENSE = 2.0 ** -19


def dense(q, keys, kmag, scale):
    """Logits [H] of one token, and what the rms of their errors is relative to."""
    g = q.shape[0] // keys.shape[0]
    k, m = (np.repeat(x.astype(np.float64), g, 0) for x in (keys, kmag))
    return scale * (k * q.astype(np.float64)).sum(-1), scale * np.sqrt(((m * q) ** 2).sum(-1))


def rms(x, axis=None):
    return np.sqrt(np.mean(np.square(x), axis))


def few_tokens(fmt, q, keys, values, kmag, vmag, scale, plain):
    """out [H][D] of one-element q over a few tokens, and its bound: a weight and the sum of the weights are off by their logits' errors, by
    22 bits and 8 roundings; the sums over T tokens and of V's parts, T + 16 roundings.  Plain Q8: 2^-26 of the largest weight's too."""
    H, D = q.shape
    g, T = H // keys.shape[1], len(keys)
    out, tol = np.zeros((H, D)), np.full((H, D), 1e-30)
    s, ds = (np.stack(x) for x in zip(*(one_product(fmt, q, keys[t], kmag[t], scale) for t in range(T))))
    for h in range(H):
        p = np.exp(s[:, h] - s[:, h].max())
        p /= p.sum()
        v, m = values[:, h // g].astype(np.float64), vmag[:, h // g].astype(np.float64)
        off = p * (ds[:, h] + (p @ ds[:, h]) + 2.0 ** -21 + 16 * U)
        out[h] = p @ v
        tol[h] += off @ m + (T + 16) * U * (p @ m) + (2.0 ** -26 * p.max() * m.sum(0) if plain and fmt == "q8" else 0.0)
    return out, tol


def one_element(rng, n, heads, dim):
    """q [n][heads][dim] of one element each, every place in turn."""
    q = np.zeros((n, heads, dim), np.float32)
    r, h = np.mgrid[:n, :heads]
    q[r, h, (7 * r + 13 * h + r // dim) % dim] = rng.uniform(1, 2, (n, heads)) * rng.choice([-1, 1], (n, heads))
    return q


FORMATS = ["bf16", "q8", "a4"]
LAYOUTS = [(8, 2, 128), (16, 2, 64), (5, 1, 256), (3, 3, 96)]


def _pool(fmt, x):
    _, f, mag = kl.pool(fmt, x, lambda t: t)
    return f, mag


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heads,kv,dim", LAYOUTS)
def test_the_bounds_tell_lost_bits(fmt, heads, kv, dim):
    """The definitions with operands of fewer bits: 22 pass, 11 (the lo part of two lost) do not, nor 16 (of three) of one product."""
    rng = np.random.default_rng(dim)
    n = 64
    keys, kmag = _pool(fmt, rng.standard_normal((n, kv, dim)).astype(np.float32))
    def bits(x, b):
        m, e = np.frexp(x)
        return np.ldexp(np.rint(np.ldexp(m, b)), e - b)
    q1, q = one_element(rng, n, heads, dim), rng.standard_normal((n, heads, dim)).astype(np.float32)
    scale = dim ** -0.5
    for b, fine in ((22, True), (16, False), (11, False)):
        worst, errors = 0.0, []
        for r in range(n):
            s, tol = one_product(fmt, q1[r], keys[r], kmag[r], scale)
            k = np.repeat(keys[r].astype(np.float64), heads // kv, 0)
            worst = max(worst, np.max(np.abs(scale * (k * bits(q1[r].astype(np.float64), b)).sum(-1) - s) / tol))
            s, unit = dense(q[r], keys[r], kmag[r], scale)
            errors.append((scale * (k * bits(q[r].astype(np.float64), b)).sum(-1) - s) / unit)
        assert (worst <= 1) == fine, (b, worst)
        if b != 16:
            assert (rms(np.array(errors), 0).max() <= DENSE) == fine == (rms(np.array(errors)) <= DENSE)
    values, vmag = _pool(fmt, rng.standard_normal((n, kv, dim)).astype(np.float32))
    out, tol = few_tokens(fmt, q1[0], keys[:3], values[:3], kmag[:3], vmag[:3], scale, True)
    for b, fine in ((22, True), (11, False)):
        worst = 0.0
        for h in range(heads):
            p = np.exp(np.array([scale * keys[t, h // (heads // kv)] @ q1[0, h].astype(np.float64) for t in range(3)]))
            p = bits(p / p.max(), b) / np.sum(p / p.max())
            worst = max(worst, np.max(np.abs(p @ values[:3, h // (heads // kv)] - out[h]) / tol[h]))
        assert (worst <= 1) == fine, (b, worst)


@pytest.fixture(scope="module")
def sil():
    import torch
    from gpu_util import lib
    torch.cuda.set_device(0)
    return lib()


def _case(sil, fmt, heads, kv, dim, scored, window, lens, seed):
    return kl.Case(sil, fmt, heads, kv, dim, 16, lens, window=window, starts=[0] * len(lens) if scored else None, seed=seed)


LENS = [1 + i % 64 for i in range(320)]  # the token seen in every place of a tile


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heads,kv,dim", LAYOUTS)
@pytest.mark.parametrize("scored", [False, True])
def test_logits(sil, fmt, heads, kv, dim, scored):
    c = _case(sil, fmt, heads, kv, dim, scored, 1, LENS, dim)
    rng = np.random.default_rng(dim + heads)
    scale = dim ** -0.5
    c.q = one_element(rng, len(LENS), heads, dim)
    lse = c.run()[1].double().cpu().numpy()
    for r, (k, _, m, _) in enumerate(c.rows):
        s, tol = one_product(fmt, c.q[r], k[0], m[0], scale)
        assert np.all(np.abs(lse[r] - s) <= tol), (r, np.max(np.abs(lse[r] - s) / tol))
    c.q = rng.standard_normal(c.q.shape).astype(np.float32)
    lse = c.run()[1].double().cpu().numpy()
    s, unit = (np.stack(x) for x in zip(*(dense(c.q[r], k[0], m[0], scale) for r, (k, _, m, _) in enumerate(c.rows))))
    off = (lse - s) / unit
    assert rms(off, 0).max() <= DENSE, np.log2(rms(off, 0))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heads,kv,dim", LAYOUTS)
@pytest.mark.parametrize("scored", [False, True])
def test_collected_weights(sil, fmt, heads, kv, dim, scored):
    """A head's weight of a token whose lse is its logit is 1 and the logit's error; the other heads' lse is beyond reach."""
    import torch
    c = _case(sil, fmt, heads, kv, dim, scored, 1, LENS, dim + 1)
    rng = np.random.default_rng(dim + heads)
    scale = dim ** -0.5
    last = torch.tensor(LENS, device="cuda")[:, None] - 1
    for one in (True, False):
        c.q = one_element(rng, len(LENS), heads, dim) if one else rng.standard_normal(c.q.shape).astype(np.float32)
        s, bound = (np.stack(x) for x in zip(*(one_product(fmt, c.q[r], k[0], m[0], scale) if one else dense(c.q[r], k[0], m[0], scale)
                                              for r, (k, _, m, _) in enumerate(c.rows))))
        q, table, lens = c.device()
        for h in range(heads):
            lse = torch.full((len(LENS), heads), 1000.0, device="cuda")
            lse[:, h] = torch.from_numpy(s[:, h]).float()
            weights = torch.zeros((len(LENS), 64), device="cuda")
            sil.kv_weigh(c.cache, q, table, lens, lse, weights, **c.score())
            w = weights.gather(1, last)[:, 0].double().cpu().numpy()
            exact = s[:, h] - lse[:, h].double().cpu().numpy()
            off = np.log(w) - exact
            # beside the logit's error: lse times log2(e) and the difference, 4 roundings of them; exp2, 2^-22, and a rounding
            more = 4 * U * np.abs(s[:, h]) + 2.0 ** -22 + 2 * U
            if one:
                assert np.all(np.abs(off) <= bound[:, h] + more), (h, np.max(np.abs(off) / (bound[:, h] + more)))
            else:
                assert rms(off / bound[:, h]) <= DENSE + rms(more / bound[:, h]), (h, math.log2(rms(off / bound[:, h])))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heads,kv,dim", LAYOUTS)
@pytest.mark.parametrize("scored", [False, True])
def test_weights_of_a_few_tokens(sil, fmt, heads, kv, dim, scored):
    lens = [1, 2, 3, 5, 16, 17, 33, 40] * 8
    c = _case(sil, fmt, heads, kv, dim, scored, 3, lens, dim + 2)
    c.q = one_element(np.random.default_rng(dim), len(lens), heads, dim)
    scale = 2.0
    out = c.run(scale=scale)[0].double().cpu().numpy()
    for r, (k, v, km, vm) in enumerate(c.rows):
        o, tol = few_tokens(fmt, c.q[r], k, v, km, vm, scale, not scored)
        assert np.all(np.abs(out[r] - o) <= tol), (r, np.max(np.abs(out[r] - o) / tol))
