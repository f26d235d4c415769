"""Pages that no cache has, in the ring or the table that il_kv_extend reads: their tokens' slots are flagged by
il_kv_append and il_kv_read and reach nobody's rows."""
import pytest

from gpu_util import lib

pytestmark = pytest.mark.gpu

WILD = [-1, -2**31, 1 << 27, 1 << 28, (1 << 28) + 3, 2**31 - 1]  # with 16 tokens a page, 2^27 and more pass 31 bits


@pytest.fixture(scope="module")
def sil():
    import torch
    torch.cuda.set_device(0)
    return lib()


@pytest.mark.parametrize("wild", WILD)
@pytest.mark.parametrize("where", ["ring", "table"])
def test_wild_pages_give_slots_that_are_flagged(sil, wild, where):
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = sil.kv_cache("bf16", 6, 16, 2, 64)
    cache.k.fill_(77)
    cache.v.fill_(77)
    # sequence 0: page 0 and, of the ring, page 4; sequence 1: the wild page, from the ring or in its table
    lens = torch.tensor([16, 0 if where == "ring" else 3], **i32)
    table = torch.tensor([[0, -1], [-1 if where == "ring" else wild, -1]], **i32)
    ring = torch.tensor([4, wild if where == "ring" else 5, 5, 1, 2, 3], **i32)
    cursor = torch.tensor([0, 3], dtype=torch.int64, device="cuda")
    slots, positions, info = torch.empty(9, **i32), torch.empty(9, **i32), torch.zeros(4, dtype=torch.int64, device="cuda")
    sil.check_device_status()
    sil.kv_extend(lens, torch.tensor([2, 5], **i32), table, ring, cursor, 16, slots, positions=positions, info=info)
    torch.cuda.synchronize()
    assert info.tolist()[0] == 0 and table[0].tolist() == [0, 4] and int(table[1, 0]) == wild
    got = slots.tolist()
    assert got[:2] == [64, 65] and got[2:7] == [2**31 - 1] * 5 and got[7:] == [-1, -1]
    assert positions.tolist() == [16, 17] + [p + int(where == "table") * 3 for p in range(5)] + [-1, -1]
    x = torch.randn((9, 2, 64), device="cuda")
    sil.kv_append(cache, x, x.clone(), slots)
    with pytest.raises(sil.ILError) as ei:
        sil.check_device_status()
    assert ei.value.code == -1
    page4 = cache.k[4, :2].float()
    assert torch.equal(page4, x[:2].bfloat16().float())
    cache.k[4, :2] = 77
    assert bool((cache.k == 77).all())
    k, v = torch.full_like(x, 5.0), torch.full_like(x, 5.0)
    sil.kv_read(cache, slots, k, v)
    with pytest.raises(sil.ILError):
        sil.check_device_status()
    assert bool((k[2:] == 0).all()) and bool((v[2:] == 0).all())


def test_the_last_slots_of_31_bits(sil):
    # one below and one at the limit: page p of one token a page is slot p
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    slots = torch.empty(3, **i32)
    sil.kv_extend(torch.zeros(3, **i32), torch.ones(3, **i32), torch.full((3, 1), -1, **i32),
                  torch.tensor([2**31 - 2, 2**31 - 1, 7], **i32), torch.tensor([0, 3], dtype=torch.int64, device="cuda"), 1, slots)
    assert slots.tolist() == [2**31 - 2, 2**31 - 1, 7]
