"""il_kv_attend gives equal bits for equal calls: the order in which parts of a row are added up follows from
the lengths, not from which CTA arrives last."""
import numpy as np
import pytest

from gpu_util import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sil():
    import torch
    torch.cuda.set_device(0)
    return lib()


# 32 heads on 8 of 128 and 14 on 2 of 64: a CTA has more threads than a row has float4s, as it has for 2 on 1 of 256;
# 18 on 2 of 128: fewer
@pytest.mark.parametrize("fmt", ["bf16", "q8"])
@pytest.mark.parametrize("heads,kv,dim,n_seq", [(32, 8, 128, 21), (2, 1, 256, 90), (14, 2, 64, 60), (18, 2, 128, 40)])
def test_equal_calls_give_equal_bits(sil, fmt, heads, kv, dim, n_seq):
    import torch
    page = 16
    lens = np.random.default_rng(dim).integers(2000, 9000, n_seq)  # rows of several CTAs whose ends fall anywhere
    held = -(-lens // page)
    gen = torch.Generator(device="cuda").manual_seed(dim)
    table = torch.randint(0, 600, (n_seq, int(held.max())), generator=gen, device="cuda").int()  # pages may be shared
    pool = [torch.randn((600, page, kv, dim), generator=gen, device="cuda") for _ in range(2)]
    if fmt == "bf16":
        cache = sil.KVCache(*(t.bfloat16() for t in pool))
    else:
        scales = [0.01 + 0.02 * torch.rand((600, page, kv, dim // 32), generator=gen, device="cuda") for _ in range(2)]
        cache = sil.KVCache(*((40 * t).round().clamp(-127, 127).to(torch.int8) for t in pool), *scales)
    q = torch.randn((n_seq, heads, dim), generator=gen, device="cuda")
    d_lens = torch.from_numpy(lens.astype(np.int32)).cuda()
    first, first_lse = torch.empty_like(q), torch.empty((n_seq, heads), device="cuda")
    sil.kv_attend(cache, q, table, d_lens, first, lse=first_lse)
    changed = torch.zeros((), dtype=torch.int64, device="cuda")
    out, lse = torch.empty_like(first), torch.empty_like(first_lse)
    for i in range(400):
        if i % 3 == 0:
            out.fill_(float("nan"))  # and now and then a launch that does not follow its like
        sil.kv_attend(cache, q, table, d_lens, out, lse=lse)
        changed += ((out.view(torch.int32) != first.view(torch.int32)).any()
                    | (lse.view(torch.int32) != first_lse.view(torch.int32)).any())
    assert int(changed) == 0, f"{int(changed)} of 400 calls gave other bits"
