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


def _scale_values(c, factor):
    """V's scales times `factor` [dim / 32], on the device and in the plain values."""
    import torch
    c.cache.v_scale.mul_(torch.from_numpy(np.asarray(factor, np.float32)).cuda())
    c.values = [v * np.repeat(np.asarray(factor, np.float64), 32) for v in c.values]


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
