"""il_kv_attend over a Q8 cache whose scales, weights and queries lie far apart or far from 1."""
import numpy as np
import pytest

import kv_util
from gpu_util import lib
from test_gpu_kv_attend import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sil():
    import torch
    torch.cuda.set_device(0)
    return lib()


def _bound(c, r, scale):
    """out, lse and their bounds (kv_util.attend) without its floor of 1e-30, for values of any size."""
    o, l, ot, lt = kv_util.attend(c.q[r], c.keys[r], c.values[r], scale, c.window)
    return o, l, ot - 1e-30, lt


def _scale_values(c, factor):
    """V's scales times `factor` [dim / 32], on the device and in the plain values."""
    import torch
    c.cache.v_scale.mul_(torch.from_numpy(np.asarray(factor, np.float32)).cuda())
    c.values = [v * np.repeat(np.asarray(factor, np.float64), 32) for v in c.values]


@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 128), (8, 2, 64), (16, 1, 128), (16, 1, 64), (4, 1, 256), (9, 1, 256), (4, 1, 96)])
@pytest.mark.parametrize("apart", [20, 27, 40, 70])
def test_blocks_of_columns_do_not_share_their_bits(sil, heads, kv, dim, apart):
    # each block of 32 columns is 2^-apart of one beside it: as accurate as the other
    c = Case(sil, "q8", heads, kv, dim, 16, [1, 40, 333, 1500], seed=apart)
    _scale_values(c, 2.0 ** (-apart * (np.arange(dim // 32) % 2)))
    out, lse = c.run()
    got = out.double().cpu().numpy()
    for r in range(len(c.lens)):
        o, _, ot, _ = _bound(c, r, dim ** -0.5)
        assert np.all(np.abs(got[r] - o) <= ot), f"sequence {r}"
    c.check(out, lse)


def test_blocks_may_grow_along_a_sequence(sil):
    # scales that rise by 2^40 from token to token and back, in another order in each block: what came before keeps its size
    c = Case(sil, "q8", 8, 2, 128, 16, [700], seed=5)
    t, b = np.arange(700)[:, None], np.arange(4)
    f = np.exp2(np.rint(np.minimum(t * (b + 1) / 40.0, 40.0)))
    import torch
    rows = torch.from_numpy(c.table[0, np.arange(700) // 16].astype(np.int64)).cuda(), torch.arange(700).cuda() % 16
    c.cache.v_scale[rows] *= torch.from_numpy(f.astype(np.float32)).cuda()[:, None]
    c.values[0] = c.values[0] * np.repeat(f, 32, -1)[:, None]
    out, _ = c.run()
    o, _, ot, _ = _bound(c, 0, 128 ** -0.5)
    assert np.all(np.abs(out[0].double().cpu().numpy() - o) <= ot)


def _levels(c, level):
    """K's column 0 becomes `level` (nats, at q's 8 and a scale of 1/8) along sequence 0."""
    import torch
    n = c.lens[0]
    t = np.arange(n)
    c.q[:, :, 0] = 8.0
    kd = c.keys[0].copy()
    kd[:, :, 0] = level[:, None]
    rows = torch.from_numpy(c.table[0, t // 16].astype(np.int64)).cuda(), torch.from_numpy(t % 16).cuda()
    kq, ks = kv_util.quantise(kd.astype(np.float32))
    c.cache.k[rows], c.cache.k_scale[rows] = torch.from_numpy(kq).cuda(), torch.from_numpy(ks).cuda()
    c.keys[0] = kq * np.repeat(ks, 32, -1).astype(np.float64)


@pytest.mark.parametrize("heads,dim,n", [(8, 64, 250000), (16, 64, 160000)])
@pytest.mark.parametrize("shape", ["first", "fall"])
def test_small_values_behind_a_peak(sil, heads, dim, n, shape):
    # every row of a product is a head's; runs of several tiles a warp in which the first tokens outweigh the others by 60 nats and more: the sums stay what they
    # are however small V is, to the bit, because V's scales are multiplied by powers of two
    import torch
    c = Case(sil, "q8", heads, 1, dim, 16, [n], seed=11)
    t = np.arange(n)
    _levels(c, {"first": np.where(t == 0, 60.0, 0.0), "fall": np.maximum(-t * 1.25, -65.0)}[shape])
    out, lse = c.run(scale=0.125)
    c.check(out, lse, scale=0.125)
    for k in (40, 70, 90):
        _scale_values(c, [2.0 ** -k] * (dim // 32))
        small, same = c.run(scale=0.125)
        off = (small.double() * 2.0 ** k - out.double()).abs()
        # 0, but where single precision ends: a few hundred parts, each rounded to 2^-150
        assert bool(((off == 0) | ((out.abs() < 2.0 ** -30) & (off <= 2.0 ** (k - 140)))).all()), k
        assert torch.equal(same, lse)
        _scale_values(c, [2.0 ** k] * (dim // 32))


@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 64), (16, 1, 128), (4, 1, 256)])
def test_large_queries_on_small_keys(sil, heads, kv, dim):
    # |scale * q| of 2^117 and more, logits of ordinary size
    c = Case(sil, "q8", heads, kv, dim, 16, [5, 130, 700], seed=13, spread=2.0 ** -119)
    c.q *= np.float32(2.0 ** 62)
    scale = 2.0 ** 57 * dim ** -0.5
    c.check(*c.run(scale=scale), scale=scale)
