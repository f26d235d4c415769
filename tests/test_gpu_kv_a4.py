"""The 4-bit K/V cache: what il_kv_append writes is the definition's bit for bit, il_kv_read gives its values, and
il_kv_attend over it is softmax attention in 64 bits."""
import math

import numpy as np
import pytest

import kv_long_util as kl
from gpu_util import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sil():
    import torch
    torch.cuda.set_device(0)
    return lib()


def _round_trip(sil, x, page=16, n_pages=None, order="head", slots=None, fused=False):
    """Appends rows x = (k, v) [n][heads][dim]; the cache's bytes and steps at the slots, and the values read back."""
    import torch
    n, heads, dim = x[0].shape
    n_pages = (n + page - 1) // page + 1 if n_pages is None else n_pages
    cache = sil.kv_cache("a4", n_pages, page, heads, dim)
    if order == "token":
        cache = sil.KVCache(*(t.contiguous() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
    slots = torch.randperm(n_pages * page, device="cuda")[:n].to(torch.int32) if slots is None else slots
    k, v = (torch.from_numpy(t).cuda() for t in x)
    if fused:
        wide = torch.zeros((n, 3, heads, dim), device="cuda")
        wide[:, 1], wide[:, 2] = k, v
        k, v = wide[:, 1], wide[:, 2]
    out = [torch.full((n, heads, dim), 7.0, device="cuda") for _ in range(2)]
    sil.kv_append(cache, k, v, slots)
    sil.kv_read(cache, slots, *out)
    sil.check_device_status()
    at = slots.long().clamp(min=0)
    held = [t[at // page, at % page].cpu() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    return cache, held, [o.cpu().numpy() for o in out]


def _same(x, held, back):
    for rows, u8, steps, got in zip(x, held[:2], held[2:], back):
        u, d, m = kl.quantise(rows)
        good = np.isfinite(m)
        assert np.array_equal(u8.numpy(), kl.pack(u))
        assert np.array_equal(np.where(good, steps.float().numpy()[..., 0], 0), d)
        assert np.array_equal(np.isnan(steps.float().numpy()[..., 1]), ~good)
        assert np.array_equal(steps.float().numpy()[..., 1][good], m[good])
        want = kl.values(u, d, m).astype(np.float32)  # one rounding
        assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("n,heads,dim,order", [(1, 1, 32, "head"), (7, 8, 128, "token"), (33, 3, 96, "head"), (300, 2, 256, "token"),
                                               (4097, 1, 64, "head"), (129, 5, 160, "token")])
def test_append_and_read_are_the_definition(sil, n, heads, dim, order):
    rng = np.random.default_rng(n)
    x = [(rng.standard_normal((n, heads, dim)) * 10.0 ** rng.integers(-3, 3, (n, heads, 1)) + rng.standard_normal((1, heads, dim))).astype(np.float32)
         for _ in range(2)]
    _, held, back = _round_trip(sil, x, order=order, fused=n % 2 == 1)
    _same(x, held, back)
    for rows, got in zip(x, back):  # the bound that the header states
        b = rows.reshape(n, heads, -1, 32).astype(np.float64)
        lo, hi = b.min(-1), b.max(-1)
        d = (1 + 2.0**-7) * ((hi - lo) + 2.0**-7 * np.abs(lo)) / 15
        assert np.all(np.abs(got.reshape(b.shape) - b) <= (d / 2 * (1 + 1e-6) + 2.0**-23 * np.maximum(np.abs(lo), np.abs(hi)))[..., None])


def test_append_at_the_edges_of_fp32(sil):
    """Constant blocks, zeros of both signs, subnormals, halves between steps, the largest numbers, ranges beyond bf16."""
    rng = np.random.default_rng(3)
    rows = [np.zeros(32), np.full(32, -0.0), np.full(32, 3.7), np.full(32, -1.00390625), rng.standard_normal(32) * 1e-40,
            np.full(32, 1e-45), np.linspace(0, 15, 32), np.repeat(np.arange(16) + 0.5, 2) - 0.5, np.arange(32) * 0.5, -np.arange(32) / 3,
            rng.standard_normal(32) * 1e37, np.r_[-3e38, np.zeros(30), 3e38], np.r_[3.4e38, np.zeros(31)], np.r_[-3.4e38, np.zeros(31)],
            np.r_[np.nan, np.zeros(31)], np.r_[np.inf, np.zeros(31)], np.r_[np.zeros(31), -np.inf], np.r_[0.0, np.full(31, 1e-44)],
            np.full(32, 3.4028235e38), np.full(32, -3.4028235e38), np.r_[1e-38, np.full(31, 1.1e-38)], np.r_[-1e-30, np.full(31, 1e30)]]
    x = np.stack(rows).astype(np.float32).reshape(-1, 1, 32)
    _, held, back = _round_trip(sil, (x, x[::-1].copy()), page=4)
    _same((x, x[::-1]), held, back)


def test_append_random_bits(sil):
    bits = np.random.default_rng(5).integers(0, 2**32, (500, 2, 64), dtype=np.uint32)
    x = [bits.view(np.float32).copy(), (np.roll(bits, 1, 0) & np.uint32(0xbfffffff)).view(np.float32).copy()]
    _, held, back = _round_trip(sil, x)
    _same(x, held, back)


def test_slots_outside_are_skipped_and_flagged(sil):
    import torch
    x = np.random.default_rng(1).standard_normal((6, 2, 64)).astype(np.float32)
    cache = sil.kv_cache("a4", 3, 4, 2, 64)
    slots = torch.tensor([0, -1, 11, 12, 5, 2**31 - 1], dtype=torch.int32, device="cuda")
    t = torch.from_numpy(x).cuda()
    before = [p.clone() for p in (cache.k, cache.k_scale)]
    sil.kv_append(cache, t, t, slots)
    with pytest.raises(sil.ILError) as e:
        sil.check_device_status()
    assert e.value.code == -1
    touched = torch.zeros(12, dtype=torch.bool)
    touched[[0, 11, 5]] = True
    same = (cache.k.flatten(0, 1) == before[0].flatten(0, 1)).flatten(1).all(1).cpu()
    assert torch.equal(same, ~touched)
    out = [torch.full((6, 2, 64), 3.0, device="cuda") for _ in range(2)]
    sil.kv_read(cache, slots, *out)
    with pytest.raises(sil.ILError):
        sil.check_device_status()
    u, d, m = kl.quantise(x)
    want = kl.values(u, d, m).astype(np.float32)
    want[[1, 3, 5]] = 0
    assert np.array_equal(out[0].cpu().numpy(), want)


# ---------------------------------------------------------------------------
# il_kv_attend
# ---------------------------------------------------------------------------
def _check(sil, *args, **kw):
    c = kl.Case(sil, "a4", *args, **kw)
    c.check(*c.run())
    sil.check_device_status()
    return c


@pytest.mark.parametrize("heads,kv,dim", [(4, 1, 128), (32, 8, 128), (4, 4, 64), (8, 1, 256), (1, 1, 32), (7, 1, 128), (18, 2, 64), (16, 1, 128),
                                          (40, 1, 96), (12, 2, 160), (34, 2, 256), (9, 3, 224), (3, 1, 64), (16, 1, 64), (5, 1, 192)])
def test_head_layouts(sil, heads, kv, dim):
    _check(sil, heads, kv, dim, 16, [1, 0, 37, 300, 16, 129], seed=heads + dim)


@pytest.mark.parametrize("page", [1, 3, 8, 16, 20, 32, 100, 512])
@pytest.mark.parametrize("order", ["head", "token", "padded"])
def test_pages_and_orders(sil, page, order):
    _check(sil, 8, 2, 128, page, [1, 15, 16, 17, 31, 100, 203, 0], order=order, seed=page, lopsided=2.0)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 31, 32, 33, 100, 1000])
def test_windows(sil, window):
    _check(sil, 8, 2, 64, 16, [0, 1, 2, 16, 17, 33, 150, 401], window=window, seed=window)


@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 128), (8, 1, 128), (2, 1, 256), (32, 2, 64), (16, 1, 256)])
@pytest.mark.parametrize("lens", [[20011], [4096, 3, 0, 9000], [2048] * 5])
def test_long_sequences_split_and_join(sil, heads, kv, dim, lens):
    c = kl.Case(sil, "a4", heads, kv, dim, 64, lens, seed=len(lens))
    out, lse = c.run()
    c.check(out, lse)
    again = c.run()
    assert bool((again[0] == out).all()) and bool((again[1] == lse).all())  # the same bits


@pytest.mark.parametrize("spread", [1e-3, 8.0, 40.0])
def test_flat_and_sharp_softmax(sil, spread):
    _check(sil, 8, 2, 128, 16, [5, 77, 1300], spread=spread, seed=int(spread) + 1)


@pytest.mark.parametrize("size", [2.0**-110, 2.0**-60, 2.0**60, 2.0**118])
@pytest.mark.parametrize("against", ["scale", "keys"])
def test_large_and_small_queries(sil, size, against):
    """Logits of ordinary size from queries that are not."""
    scale = 0.125 / size if against == "scale" else 0.125
    c = kl.Case(sil, "a4", 8, 2, 128, 16, [5, 77, 300], seed=9, spread=1.0 if against == "scale" else 1.0 / size)
    c.q *= np.float32(size)
    out, lse = c.run(scale=scale)
    c.check(out, lse, scale=scale)


def _steps(c, rows, d=None, m=None):
    """Sets the V steps of (sequence, token) rows and their part of the plain form."""
    import torch
    for r, t in rows:
        page, at = int(c.table[r, t // c.page]), t % c.page
        s = c.cache.v_scale[page, at]
        if d is not None:
            s[..., 0] = torch.as_tensor(d).to(s)
        if m is not None:
            s[..., 1] = torch.as_tensor(m).to(s)
        b = c.cache.v[page, at].cpu().numpy()
        u = np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1)
        f = s.float().cpu().numpy()
        c.rows[r][1][t] = kl.values(u, f[..., 0], f[..., 1])
        c.rows[r][3][t] = u * np.repeat(np.abs(f[..., 0]), 32, -1) + np.repeat(np.abs(f[..., 1]), 32, -1)


@pytest.mark.parametrize("gap", [10, 20, 30, 60, 85])
@pytest.mark.parametrize("heads", [2, 6, 12])
def test_small_values_behind_a_peak(sil, gap, heads):
    """One token takes nearly all the weight and its V is 0: what is left are weights of 2^-gap, to fp32's accuracy."""
    c = kl.Case(sil, "a4", heads, 1, 64, 16, [100], seed=gap)
    # keys 0 but for the peak's, which every head meets with the logit gap ln 2
    k = c.cache.k_scale
    k[..., 0], k[..., 1] = 0.0, 0.0
    page, at = int(c.table[0, 3]), 50 % 16
    k[page, at, :, :, 1] = 1.0
    c.rows[0][0][:], c.rows[0][2][:] = 0, 0
    c.rows[0][0][50], c.rows[0][2][50] = 1, 1
    c.q = np.zeros_like(c.q)
    c.q[..., 0] = np.float32(gap * math.log(2))
    _steps(c, [(0, 50)], d=0.0, m=0.0)
    out, lse = c.run(scale=1.0)
    c.check(out, lse, scale=1.0)
    assert float(out.abs().max()) > 2.0**-gap * 0.1


@pytest.mark.parametrize("heads", [2, 6, 12])
def test_steps_of_unlike_sizes(sil, heads):
    """V whose blocks lie up to 2^60 apart, between tokens and between columns, and negative steps."""
    c = kl.Case(sil, "a4", heads, 1, 128, 16, [70, 33], seed=heads)
    rng = np.random.default_rng(7)
    for r, n in enumerate(c.lens):
        for t in range(n):
            e = rng.integers(-30, 31, (1, 4)) if t % 3 else np.full((1, 4), 5 * (t % 7))
            d = (np.ldexp(1.0, e) * rng.choice([1, -1], (1, 4))).astype(np.float32)
            _steps(c, [(r, t)], d=d, m=-8 * d * (t % 2))
    out, lse = c.run()
    for r in range(2):  # column by column: the bound's V is that of the column
        k, v, km, vm = c.rows[r]
        o, _, ot, _ = kl.attend(c.q[r], k, v, km, vm, c.dim ** -0.5)
        assert np.all(np.abs(out[r].cpu().numpy() - o) <= ot)


def test_far_pages(sil):
    """Offsets past 32 bits: pages of a pool of more than 2^31 bytes."""
    import torch
    page, heads, dim = 1024, 8, 128
    n_pages = 5000  # 512 KB of K each
    cache = sil.KVCache(*(torch.zeros((n_pages, page, heads, dim // 2), dtype=torch.uint8, device="cuda") for _ in range(2)),
                        *(torch.zeros((n_pages, page, heads, dim // 32, 2), dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    n = 70
    x = [np.random.default_rng(s).standard_normal((n, heads, dim)).astype(np.float32) for s in (1, 2)]
    table = torch.tensor([[n_pages - 1]], dtype=torch.int32, device="cuda")
    slots = ((n_pages - 1) * page + torch.arange(n, device="cuda")).to(torch.int32)
    sil.kv_append(cache, *(torch.from_numpy(t).cuda() for t in x), slots)
    q = torch.randn((1, 32, dim), device="cuda")
    out = torch.empty_like(q)
    sil.kv_attend(cache, q, table, torch.tensor([n], dtype=torch.int32, device="cuda"), out)
    sil.check_device_status()
    k, v = (kl.values(*kl.quantise(t)) for t in x)
    mag = [kl.quantise(t) for t in x]
    km, vm = (u * np.repeat(d, 32, -1) + np.repeat(np.abs(m), 32, -1) for u, d, m in mag)
    o, _, ot, _ = kl.attend(q[0].cpu().numpy(), k, v, km, vm, dim ** -0.5)
    assert np.all(np.abs(out[0].cpu().numpy() - o) <= ot)


def test_bad_pages_are_skipped_and_flagged(sil):
    c = kl.Case(sil, "a4", 8, 2, 128, 16, [50, 100], seed=2)
    page = int(c.table[1, 2])
    c.table[1, 2] = 10**6  # tokens 32 .. 47 are no longer there
    out, lse = c.run()
    with pytest.raises(sil.ILError) as e:
        sil.check_device_status()
    assert e.value.code == -1 and page >= 0
    c.rows[1] = tuple(np.delete(x, slice(32, 48), 0) for x in c.rows[1])
    c.check(out, lse)


def test_graph_and_streams(sil):
    import torch
    c = kl.Case(sil, "a4", 32, 8, 128, 16, [900, 1, 0, 333], seed=1)
    q, table, lens = c.device()
    out, stream = torch.empty_like(q), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        sil.kv_attend(c.cache, q, table, lens, out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            sil.kv_attend(c.cache, q, table, lens, out)
    for seed in range(3):
        c.q = np.random.default_rng(seed).standard_normal(c.q.shape).astype(np.float32)
        q.copy_(torch.from_numpy(c.q))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        again, lse = c.run()
        c.check(out, lse)
        assert torch.equal(again, out)


def test_refusals(sil):
    import torch
    z = lambda *s, dtype=torch.uint8: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    k, s = z(4, 16, 2, 32), z(4, 16, 2, 2, 2, dtype=torch.bfloat16)
    sil.KVCache(k, k.clone(), s, s.clone())
    for make in (lambda: sil.KVCache(k, k), lambda: sil.KVCache(k, k, s, None), lambda: sil.KVCache(k, k, s.float(), s.float()),
                 lambda: sil.KVCache(k, k, s[..., :1, :], s[..., :1, :]), lambda: sil.KVCache(k, k, s[..., 0], s[..., 0]),
                 lambda: sil.KVCache(k, k, s.transpose(3, 4), s.transpose(3, 4)), lambda: sil.KVCache(k, k, s, s.cpu()),
                 lambda: sil.kv_cache("q4", 4, 16, 2, 64), lambda: sil.kv_cache("a8", 4, 16, 2, 64),
                 lambda: sil.kv_cache("a4", 4, 16, 2, 33), lambda: sil.kv_cache("a4", 4, 16, 2, 48)):
        with pytest.raises(sil.ILError):
            make()
    odd = z(4 * 16 * 2 * 5 + 8, dtype=torch.bfloat16).as_strided((4, 16, 2, 2, 2), (160, 10, 5, 2, 1))
    with pytest.raises(sil.ILError):
        sil.KVCache(k, k, odd, odd)  # pairs off 4 bytes
    x = torch.zeros((1, 2, 40), device="cuda")
    short = sil.KVCache(z(4, 16, 2, 20), z(4, 16, 2, 20), z(4, 16, 2, 1, 2, dtype=torch.bfloat16), z(4, 16, 2, 1, 2, dtype=torch.bfloat16))
    with pytest.raises(sil.ILError) as e:
        sil.kv_append(short, x, x, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert e.value.code == -2
