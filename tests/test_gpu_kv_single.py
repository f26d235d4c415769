"""Dimensions of one entry: their strides mean nothing and are not compared."""
import pytest

from gpu_util import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sil():
    import torch
    torch.cuda.set_device(0)
    return lib()


@pytest.mark.parametrize("fmt", ["bf16", "q8"])
@pytest.mark.parametrize("pages,page,kv", [(5, 16, 1), (5, 1, 2), (1, 16, 2), (1, 1, 1)])
def test_k_and_v_of_other_strides_there(sil, fmt, pages, page, kv):
    import torch
    shape = (pages, page, kv)
    odd = tuple(7777 if n == 1 else st for n, st in zip((*shape, 64), (page * kv * 64, kv * 64, 64, 1)))
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((2, *shape, 64), generator=gen, device="cuda")
    if fmt == "bf16":
        k, v, ks, vs = x[0].bfloat16(), x[1].bfloat16(), None, None
    else:
        k, v = (40 * x).round().clamp(-127, 127).to(torch.int8).unbind()
        ks, vs = (0.01 + 0.02 * torch.rand((2, *shape, 2), generator=gen, device="cuda")).unbind()
    n = pages * page
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    q = torch.randn((1, 4, 64), generator=gen, device="cuda")
    want, got = torch.empty_like(q), torch.empty_like(q)
    sil.kv_attend(sil.KVCache(k, v, ks, vs), q, table, lens, want)
    other = torch.as_strided(v, v.shape, odd)
    other_s = None if vs is None else torch.as_strided(vs, vs.shape, tuple(
        9999 if m == 1 else st for m, st in zip(vs.shape, (page * kv * 2, kv * 2, 2, 1))))
    assert torch.equal(other, v)
    sil.kv_attend(sil.KVCache(k, other, ks, other_s), q, table, lens, got)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_a_table_of_one_column(sil):
    import torch
    cache = sil.kv_cache("bf16", 4, 16, 1, 64)
    cache.k.normal_()
    cache.v.normal_()
    q = torch.randn((3, 2, 64), device="cuda")
    lens = torch.tensor([5, 16, 0], dtype=torch.int32, device="cuda")
    want, got = torch.empty_like(q), torch.empty_like(q)
    table = torch.tensor([[2], [0], [3]], dtype=torch.int32, device="cuda")
    sil.kv_attend(cache, q, table, lens, want)
    sil.kv_attend(cache, q, table.as_strided((3, 1), (1, 40)), lens, got)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
