"""il_kv_attend and il_kv_attend_scored over 4- and 8-bit caches: steps of V that are 0 beside large ones, or that are no numbers."""
import numpy as np
import pytest

import kv_long_util as kl
from gpu_util import lib

pytestmark = pytest.mark.gpu
LAYOUTS = [("q8", False), ("q8", True), ("a4", False), ("a4", True)]


@pytest.fixture(scope="module")
def sil():
    import torch
    torch.cuda.set_device(0)
    return lib()


@pytest.mark.parametrize("fmt,scored", LAYOUTS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("exponent", [-20, 13, 14, 15, 16, 17, 60])
def test_a_block_of_zeros_beside_large_steps(sil, fmt, scored, dim, exponent):
    """In each half of a head the largest step of a block is 2^exponent to 2^(exponent + 1) or 1, that of another is 0 in all tokens, of
    others 2^-40 and 1, in tiles with weights below 2^-26: every block as accurate as its own values allow."""
    import torch
    low = -np.linspace(17.0, 97.0, 32)
    logits = np.concatenate([np.zeros(64), low, np.zeros(32), low[::-1], np.full(32, -20.0), np.zeros(8)]).astype(np.float32)
    n, n_seq = len(logits), 200
    pages = (n + 15) // 16
    cache = sil.kv_cache(fmt, pages, 16, 1, dim)
    g = torch.Generator().manual_seed(dim + exponent)
    k = torch.from_numpy(np.repeat(logits / dim, dim).reshape(n, 1, dim).astype(np.float32)).cuda()  # every element of a token the same
    v = torch.rand(n, 1, dim // 32, 32, generator=g, dtype=torch.float64) - 0.5
    v[..., 0], v[..., 1] = -0.5, 0.5  # a block's steps: its range over 15, or its largest over 127
    unit = {"q8": 127 / 0.5, "a4": 15.0}[fmt] * 1.01
    sizes = {64: [exponent, None], 128: [exponent, None, -40, 0], 256: [exponent, None, -40, 0, 0, None, 0, -40]}[dim]
    for b, e in enumerate(sizes):
        v[:, :, b] *= 0.0 if e is None else unit * 2.0 ** e
    v = v.view(n, 1, dim).float().cuda()
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    sil.kv_append(cache, k, v, slots)
    sil.kv_read(cache, slots, k, v)
    q = torch.ones(n_seq, 1, dim, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(n_seq, 1, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(n_seq, 1)
    lens = torch.full((n_seq,), n, dtype=torch.int32, device="cuda")
    starts = torch.zeros(n_seq, dtype=torch.int32, device="cuda") if scored else None
    sil.kv_attend(cache, q, table, lens, out, lse=lse, scale=1.0, starts=starts)
    s = k.double().sum(-1)[:, 0]
    want = (torch.softmax(s, 0) @ v.double()[:, 0]).view(-1, 32)
    most = v.double().abs().view(n, -1, 32).amax((0, 2))[:, None]
    # q and p in 21 bits or more, roundings of sums of 8 tiles and of their joins, all of numbers of up to 2 `most` (4 bits: u - 8 and m + 8 d)
    off = (out.double().view(n_seq, -1, 32) - want).abs()
    assert bool((off <= 2 * most * (2 * 2**-21 + 64 * 2**-24)).all()), (off / most.clamp(min=1e-300)).amax((0, 2)).tolist()
    assert (lse.double() - torch.logsumexp(s, 0)).abs().max() <= 1e-5


@pytest.mark.parametrize("fmt,scored", LAYOUTS)
@pytest.mark.parametrize("heads,kv,dim", [(8, 4, 64), (8, 4, 128), (32, 4, 128), (8, 4, 256)])
@pytest.mark.parametrize("what", ["nan", "inf", "nan in a wide tile"])
def test_a_step_that_is_no_number_stays_in_its_columns(sil, fmt, scored, heads, kv, dim, what):
    """The heads that read it give no number in the 32 columns of the step and what they should in all others."""
    import torch
    c = kl.Case(sil, fmt, heads, kv, dim, 16, [700, 90, 33], starts=[0, 0, 0] if scored else None, seed=9,
                spread=40.0 if "wide" in what else 1.0)
    c.check(*c.run())
    bad = float(what[:3])
    tokens, head, block = {0: [83, 84, 600], 1: [0]}, 2, dim // 32 - 1 if dim != 128 else 1
    for r, ts in tokens.items():
        for t in ts:
            scales = c.cache.v_scale[int(c.table[r][t // 16]), t % 16, head]
            scales[block, ...][0 if fmt == "a4" else ...] = bad
    out, lse = c.run()
    hs = slice(head * heads // kv, (head + 1) * heads // kv)
    columns = slice(32 * block, 32 * block + 32)
    for r in (0, 1):
        assert bool((~torch.isfinite(out[r, hs, columns])).all())
    out[:, hs, columns] = 0.0
    for row in c.rows:  # the other columns against the same bounds
        row[1][:, head, columns] = 0.0
    c.check(out, lse)


@pytest.mark.parametrize("fmt", ["bf16", "q8", "a4"])
@pytest.mark.parametrize("scored", [False, True])
def test_an_appended_infinity_of_v_stays_in_its_columns(sil, fmt, scored):
    """As kv_append leaves it: of bf16 in one column, else in 32.  Rows enough for several tiles a warp before and behind it."""
    import torch
    n, dim, n_seq = 600, 128, 400
    pages = (n + 15) // 16
    g = torch.Generator().manual_seed(3)
    cache = sil.kv_cache(fmt, pages, 16, 1, dim)
    k, v = (torch.randn(n, 1, dim, generator=g).cuda() for _ in range(2))
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    v[301, 0, 40] = float("inf")
    sil.kv_append(cache, k, v, slots)
    sil.kv_read(cache, slots, k, v)
    q = torch.randn(1, 4, dim, generator=g).cuda().repeat(n_seq, 1, 1)
    out, lse = torch.empty_like(q), torch.empty(n_seq, 4, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(n_seq, 1)
    lens = torch.full((n_seq,), n, dtype=torch.int32, device="cuda")
    sil.kv_attend(cache, q, table, lens, out, lse=lse, starts=torch.zeros_like(lens) if scored else None)
    s = q[0].double() @ k[:, 0].double().T / dim ** 0.5
    want = torch.softmax(s, 1) @ v[:, 0].double()
    good = torch.isfinite(v[:, 0]).all(0)
    assert int((~good).sum()) == (1 if fmt == "bf16" else 32)
    assert not torch.isfinite(out[:, :, ~good]).any()
    # a logit: 22 bits of q, up to 40 in sum |q k| / 11; p: 21 bits; roundings of sums of 19 tiles and two joins, of numbers of up to 5
    assert (out.double() - want)[:, :, good].abs().max() <= 5 * (40 * 2**-22 + 2**-21 + 32 * 2**-24)
