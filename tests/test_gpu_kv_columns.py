"""il_kv_attend with q and out as columns of one buffer; what does overlap is refused."""
import pytest

from gpu_util import lib
from test_gpu_kv_attend import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sil():
    import torch
    torch.cuda.set_device(0)
    return lib()


@pytest.mark.parametrize("at_q,at_out", [(0, 2), (2, 0), (1, 2), (3, 0)])
def test_q_and_out_in_one_buffer(sil, at_q, at_out):
    import torch
    c = Case(sil, "bf16", 8, 2, 64, 16, [70, 3, 0, 128], seed=4)
    wide = torch.full((4, 4, 8, 64), 5.5, device="cuda")
    wide[:, at_q] = torch.from_numpy(c.q).cuda()
    out, lse = c.run(q=wide[:, at_q], out=wide[:, at_out])
    c.check(out, lse)
    for i in range(4):
        if i != at_out:
            assert torch.equal(wide[:, i], torch.from_numpy(c.q).cuda() if i == at_q else torch.full_like(wide[:, i], 5.5))


def test_overlaps_are_refused(sil):
    import torch
    c = Case(sil, "bf16", 8, 2, 64, 16, [70, 3, 0, 128], seed=4)
    table, lens = torch.from_numpy(c.table).cuda(), torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    flat = torch.full((4 * 4 * 512 + 64,), 3.0, device="cuda")

    def rows(first, stride=2048):
        return flat.as_strided((4, 8, 64), (stride, 64, 1), first)

    for q, out in ((rows(0), rows(0)), (rows(0), rows(508)), (rows(508), rows(0)), (rows(0), rows(1540)), (rows(0), rows(512, 1540)),
                   (rows(0, 512), rows(1024, 512)), (rows(8), rows(1548))):
        with pytest.raises(sil.ILError) as ei:
            sil.kv_attend(c.cache, q, table, lens, out)
        assert ei.value.code == -1
    one = rows(0)[:1]
    with pytest.raises(sil.ILError):
        sil.kv_attend(c.cache, one, table[:1], lens[:1], rows(256)[:1])
    torch.cuda.synchronize()
    assert bool((flat == 3.0).all())
