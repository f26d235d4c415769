"""il_kv_attend_scored: capped logits, a bias by distance, sequences that begin later, against 64 bits."""
import math

import numpy as np
import pytest

import kv_long_util as kl
from gpu_util import lib

pytestmark = pytest.mark.gpu
FORMATS = ["bf16", "q8", "a4"]


@pytest.fixture(scope="module")
def sil():
    import torch
    torch.cuda.set_device(0)
    return lib()


def _slopes(heads):
    return np.exp2(-8 * np.arange(1, heads + 1) / heads).astype(np.float32)


def _check(sil, *args, **kw):
    c = kl.Case(sil, *args, **kw)
    out, lse = c.run()
    c.check(out, lse)
    sil.check_device_status()
    return c, out, lse


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heads,kv,dim", [(32, 8, 128), (4, 4, 64), (8, 1, 256), (16, 8, 256), (18, 2, 64), (16, 1, 128), (40, 1, 96), (34, 2, 256)])
@pytest.mark.parametrize("what", ["cap", "slopes", "starts", "all"])
def test_forms_and_layouts(sil, fmt, heads, kv, dim, what):
    lens = [1, 0, 37, 300, 16, 129, 64]
    kw = {}
    if what in ("cap", "all"):
        kw["cap"] = 5.0 if what == "cap" else 30.0
    if what in ("slopes", "all"):
        kw["slopes"] = _slopes(heads)
    if what in ("starts", "all"):
        kw["starts"] = [0, 0, 36, 5, 16, 64, -3]
    if what == "all":
        kw.update(window=100, positions=True)
    _check(sil, fmt, heads, kv, dim, 16, lens, seed=heads + dim, spread=4.0, **kw)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("cap", [1e-3, 1.0, 50.0, 1e4, 1e30])
def test_caps(sil, fmt, cap):
    """From logits that all lie at the cap to a cap that does nothing."""
    _check(sil, fmt, 8, 2, 128, 16, [5, 77, 600], cap=cap, spread=6.0, seed=3)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("slopes", [[0.0] * 8, [1.0, 0.5, 0.0, -0.001, 3.0, 1e-6, 20.0, 1e3], [-0.01] * 8])
def test_slopes(sil, fmt, slopes):
    """Of any size and sign; steep ones leave little but the newest tokens."""
    _check(sil, fmt, 8, 2, 128, 16, [5, 77, 1200, 0, 1], slopes=np.float32(slopes), seed=4)
    _check(sil, fmt, 8, 2, 128, 24, [5, 77, 1200, 0, 1], slopes=np.float32(slopes), positions=True, seed=5)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window", [0, 20])
def test_starts(sil, fmt, window):
    """Inside and at the ends of tiles and pages, behind the last token, below 0 and beyond 31 bits of the length."""
    lens = [64] * 10 + [0, 1, 1]
    starts = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 5, 1, -2**31]
    c, out, lse = _check(sil, fmt, 8, 2, 64, 16, lens, starts=starts, window=window, seed=window)
    assert bool((out[9] == 0).all()) and bool(lse[9].isneginf().all()) and bool((out[11] == 0).all())
    c.starts = [2**31 - 1] * 13
    out, lse = c.run()
    assert bool((out == 0).all()) and bool(lse.isneginf().all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_long_sequences_split_and_join(sil, fmt):
    c, out, lse = _check(sil, fmt, 16, 4, 128, 64, [20011, 9, 4096], cap=20.0, slopes=_slopes(16), starts=[777, 0, 4000], seed=1)
    again = c.run()
    assert bool((again[0] == out).all()) and bool((again[1] == lse).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_nothing_set_is_the_plain_call(sil, fmt):
    c = kl.Case(sil, fmt, 8, 2, 128, 16, [70, 3, 0, 128], seed=2)
    plain = c.run()
    c.positions = np.zeros((4, 128), np.int32)  # nothing that a logit depends on
    same = c.run()
    assert bool((plain[0] == same[0]).all()) and bool((plain[1] == same[1]).all())
    c.starts, c.positions = [0] * 4, None  # the scored kernel, which shares the work out in another way
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("slope", [0.05, 0.5, 5.0])
def test_long_sequences_behind_a_steep_bias(sil, fmt, slope):
    """Most tiles give nothing beside the newest, but each part of a row is first taken by itself; of positions in any order, any tile may count."""
    for positions in (False, True):
        _check(sil, fmt, 8, 2, 128, 64, [9001, 40, 3000], slopes=np.full(8, slope, np.float32), positions=positions, seed=7)
        _check(sil, fmt, 9, 1, 256, 16, [2000], slopes=np.linspace(0, slope, 9, dtype=np.float32), positions=positions, seed=8)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_wide_tile_far_below_a_heavy_peak(sil, fmt, scored, dim):
    """1024 equal logits, and before and behind them tiles of logits from 2^-24 to 2^-140 of them: no sum leaves fp32 on the way.
    As many sequences (of the same pages) as leave a warp tiles of both."""
    import torch
    low = -np.linspace(17.0, 97.0, 32)
    logits = np.concatenate([low, np.zeros(1024), low[::-1], low, np.full(32, -60.0), [-80.0]]).astype(np.float32)
    n, n_seq = len(logits), 600
    pages = (n + 15) // 16
    cache = sil.kv_cache(fmt, pages, 16, 1, dim)
    k = torch.from_numpy(np.repeat(logits / dim, dim).reshape(n, 1, dim).astype(np.float32)).cuda()  # every element of a token the same
    v = torch.zeros(n, 1, dim, device="cuda")
    v[..., ::2] = 100.0
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
    want = torch.softmax(s, 0) @ v.double()[:, 0]
    # q and p in 21 bits or more, and roundings of sums of 32 tiles and of their joins, all of numbers of up to 101
    assert (out[:, 0].double() - want).abs().max() <= 101 * (2 * 2**-21 + 64 * 2**-24)
    assert (lse.double() - torch.logsumexp(s, 0)).abs().max() <= 1e-5  # 8 times a rounding of 2^4, in exp2's units


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("half", [0, 1])
def test_v_of_two_sizes_in_one_half_of_a_wide_head(sil, fmt, scored, half):
    """The warps of a head above 128 elements see V of different ranges; their parts are joined across CTAs by one maximum."""
    import torch
    n, dim, heads = 100003, 256, 3
    g = torch.Generator().manual_seed(5)
    pages = (n + 63) // 64
    cache = sil.kv_cache(fmt, pages, 64, 1, dim)
    k, v = (torch.randn(n, 1, dim, generator=g).cuda() for _ in range(2))
    v[::2, :, 128 * half:128 * half + 128] *= 2.0**-20
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    sil.kv_append(cache, k, v, slots)
    sil.kv_read(cache, slots, k, v)
    q = torch.randn(1, heads, dim, generator=g).cuda()
    out, lse = torch.empty_like(q), torch.empty(1, heads, device="cuda")
    table, lens = torch.arange(pages, dtype=torch.int32, device="cuda")[None], torch.tensor([n], dtype=torch.int32, device="cuda")
    starts = torch.zeros(1, dtype=torch.int32, device="cuda") if scored else None
    sil.kv_attend(cache, q, table, lens, out, lse=lse, starts=starts)
    s = q[0].double() @ k[:, 0].double().T / 16
    want = torch.softmax(s, 1) @ v[:, 0].double()
    # a logit: 22 bits of q, up to 40 in sum |q k| / 16; p: 21 bits; roundings of sums of 5 tiles and two joins, of numbers of up to 5
    assert (out[0].double() - want).abs().max() <= 5 * (40 * 2**-22 + 2**-21 + 32 * 2**-24)
    assert (lse[0].double() - torch.logsumexp(s, 1)).abs().max() <= 40 * 2**-22 + 8 * 2**-20


@pytest.mark.parametrize("fmt", ["q8", "a4"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("where", ["k", "v"])
def test_a_nan_far_behind_a_steep_bias_is_seen(sil, fmt, dim, where):
    """In a tile that weighs nothing beside the newest, as anywhere: the heads that read it give no number, the others what they gave."""
    import torch
    c = kl.Case(sil, fmt, 8, 4, dim, 16, [700, 90], slopes=np.full(8, 4.0, np.float32), seed=9)
    c.check(*c.run())
    before = c.run()
    pools = {"k": c.cache.k_scale, "v": c.cache.v_scale}[where]
    page = c.table[0][5]
    pools[int(page), 3, 2].view(-1)[-1 if fmt == "q8" else -2] = float("nan")  # d of the last block of token 83's K/V head 2
    out, lse = c.run()
    assert torch.isnan(out[0, 4:6, dim - 32:]).all() and (where == "v" or torch.isnan(lse[0, 4:6]).all())
    keep = torch.ones(2, 8, dtype=torch.bool, device=out.device)
    keep[0, 4:6] = False
    assert torch.equal(out[keep], before[0][keep]) and torch.equal(lse[keep], before[1][keep])


def test_a_length_is_cut_to_the_positions(sil):
    import torch
    c = kl.Case(sil, "bf16", 4, 1, 64, 16, [40, 40], slopes=_slopes(4), positions=True, seed=2)
    q, table, lens = c.device()
    out = torch.empty_like(q)
    more = c.score()
    more["positions"] = more["positions"][:, :25]  # rows stay apart
    sil.kv_attend(c.cache, q, table, lens, out, **more)
    c.lens = [25, 25]
    c.rows = [tuple(x[:25] for x in r) for r in c.rows]
    o, _ = c.run()
    assert torch.equal(out, o)


def test_refusals(sil):
    import torch
    c = kl.Case(sil, "bf16", 8, 2, 64, 16, [70, 3], seed=2)
    q, table, lens = c.device()
    out = torch.full_like(q, 9.0)
    f32, i32 = (lambda *s: torch.zeros(s, device="cuda")), (lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda"))

    def no(code, **kw):
        with pytest.raises(sil.ILError) as e:
            sil.kv_attend(c.cache, q, table, lens, kw.pop("out", out), **kw)
        assert e.value.code == code

    no(-1, cap=-1.0)
    no(-1, cap=math.inf)
    no(-1, cap=math.nan)
    no(-1, cap=1e-30, scale=1e30)
    no(-1, slopes=f32(7))
    no(-1, slopes=f32(8).double())
    no(-1, starts=i32(3))
    no(-1, starts=f32(2))
    no(-1, starts=i32(2), positions=i32(3, 80))
    no(-1, starts=i32(2), positions=i32(80))
    no(-2, starts=i32(2), positions=i32(2, 80).as_strided((2, 80), (40, 1)))
    no(-1, starts=i32(2).cpu())
    flat = torch.zeros(2 * 8 * 64, device="cuda")
    no(-1, slopes=flat[:8], out=flat.view(2, 8, 64))
    no(-1, starts=flat[8:10].view(torch.int32), out=flat.view(2, 8, 64))
    no(-1, starts=i32(2), positions=flat[:160].view(torch.int32).view(2, 80), out=flat.view(2, 8, 64))
    torch.cuda.synchronize()
    assert bool((out == 9.0).all()) and bool((flat == 0).all())
