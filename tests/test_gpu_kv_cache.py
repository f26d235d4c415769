"""il_kv_extend, il_kv_append and il_kv_read: whole numbers and cache bytes equal the definition's,
and the decode path of all of them with the matmul batches."""
import numpy as np
import pytest

import kv_util
from gpu_util import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sil():
    import torch
    torch.cuda.set_device(0)
    return lib()


# ---------------------------------------------------------------------------
# il_kv_extend
# ---------------------------------------------------------------------------
class Server:
    """The device state beside its plain form."""

    def __init__(self, sil, n_seq, page, n_pages, width, max_slots, head=0, spare=0, seed=0):
        import torch
        self.sil, self.n, self.page, self.width, self.most = sil, n_seq, page, width, max_slots
        perm = np.random.default_rng(seed).permutation(n_pages).astype(np.int32)
        size = n_pages + spare
        ring = np.full(size, -9, np.int32)
        ring[(head + np.arange(n_pages)) % size] = perm
        self.plain = kv_util.Ring(size, perm.tolist(), head)
        self.lens, self.tables = [0] * n_seq, [[] for _ in range(n_seq)]
        i32 = lambda *s: torch.full(s, -5, dtype=torch.int32, device="cuda")  # noqa: E731
        self.d_lens = torch.zeros(n_seq, dtype=torch.int32, device="cuda")
        self.table, self.ring = i32(n_seq, width), torch.from_numpy(ring).cuda()
        self.cursor = torch.tensor([head, head + n_pages], dtype=torch.int64, device="cuda")
        self.slots, self.positions, self.first = i32(max_slots), i32(max_slots), i32(n_seq + 1)
        self.info = torch.full((4,), -5, dtype=torch.int64, device="cuda")

    def step(self, adds, in_place=True, optional=True, stream=None):
        import torch
        before = self.table.clone(), self.ring.clone()
        add = torch.tensor(adds, dtype=torch.int32, device="cuda")
        lens_out, cursor_out = (self.d_lens, self.cursor) if in_place else (self.d_lens.clone(), self.cursor.clone())
        torch.cuda.synchronize()
        self.sil.kv_extend(self.d_lens, add, self.table, self.ring, self.cursor, self.page, self.slots,
                           lens_out=None if in_place else lens_out, cursor_out=None if in_place else cursor_out,
                           positions=self.positions if optional else None, first=self.first if optional else None,
                           info=self.info if optional else None, stream=stream)
        torch.cuda.synchronize()
        was = list(self.lens)
        code, slots, positions, first, info = self.plain.extend(self.lens, self.tables, adds, self.page, self.width, self.most)
        assert self.slots.tolist() == slots
        if optional:
            assert self.info.tolist() == info and self.first.tolist() == first and self.positions.tolist() == positions
        assert lens_out.tolist() == self.lens
        assert cursor_out.tolist() == [self.plain.head, self.plain.tail]
        if not in_place:
            assert self.d_lens.tolist() == was
        table, ring = self.table.cpu().numpy(), self.ring.cpu().numpy()
        for r, pages in enumerate(self.tables):
            assert table[r, :len(pages)].tolist() == pages
        live = (self.plain.head + np.arange(len(self.plain.free))) % self.plain.size
        assert ring[live].tolist() == self.plain.free
        if code:
            assert torch.equal(self.table, before[0]) and torch.equal(self.ring, before[1])
        self.d_lens, self.cursor = lens_out, cursor_out
        return code


def _adds(rng, lens, most):
    got = []
    for n in lens:
        u = rng.random()
        got.append(int(rng.integers(1, most)) if u < 0.2 else 1 if u < 0.6 else 0 if u < 0.7
                   else -int(rng.integers(0, 6)) if u < 0.9 else -n - int(rng.integers(0, 2)))
    return got


@pytest.mark.parametrize("n_seq", [1, 2, 31, 512, 513, 1500])
@pytest.mark.parametrize("page", [1, 16, 24])
def test_extend_random_steps(sil, n_seq, page):
    rng = np.random.default_rng(n_seq * 100 + page)
    s = Server(sil, n_seq, page, n_pages=kv_util.pages_of(120, page) * n_seq, width=kv_util.pages_of(150, page),
               max_slots=12 * n_seq + 30, head=int(rng.integers(0, 1 << 40)), spare=int(rng.integers(0, 5)), seed=n_seq)
    codes = {s.step(_adds(rng, s.lens, 20), in_place=i % 2 == 0, optional=i % 3 != 2) for i in range(12)}
    assert 0 in codes


@pytest.mark.parametrize("in_place", [True, False])
def test_extend_long_prompts_over_many_ctas(sil, in_place):
    s = Server(sil, 5, 16, n_pages=20000, width=10000, max_slots=150001, head=7)
    assert s.step([100003, 1, 0, 33000, 7], in_place=in_place) == 0
    assert s.step([1, -1, 5, -33000, 40001], in_place=in_place) == 0
    assert s.step([-100004, 1, 1, 1, 1], in_place=in_place) == 0


def test_extend_refuses_as_a_whole(sil):
    s = Server(sil, 4, 8, n_pages=10, width=6, max_slots=40, spare=1)
    assert s.step([8, 9, 0, 16]) == 0       # 5 pages
    assert s.step([40, 40, 1, 1]) == 1 | 2 | 4
    assert s.step([0, 0, 41, 0]) == 1 | 4
    assert s.step([1, 1, 1, 30]) == 1
    assert s.step([0, 40, 0, 0]) == 2
    assert s.step([16, 16, 16, 0], in_place=False) == 1 | 4
    assert s.step([1, 1, 1, 1]) == 0
    assert s.step([-100, -1, -1, -17], in_place=False) == 0
    assert s.step([0, 0, 0, 0]) == 0


def test_extend_impossible_ring_is_refused(sil):
    import torch
    s = Server(sil, 2, 8, n_pages=4, width=6, max_slots=8)
    for cursor in ([-1, 2], [5, 4], [0, 99]):
        c = torch.tensor(cursor, dtype=torch.int64, device="cuda")
        sil.kv_extend(s.d_lens, torch.ones(2, dtype=torch.int32, device="cuda"), s.table, s.ring, c, 8, s.slots, info=s.info)
        assert int(s.info[0]) & 8 and s.d_lens.tolist() == [0, 0] and c.tolist() == cursor
        assert s.slots.tolist() == [-1] * 8


def test_extend_extreme_numbers(sil):
    s = Server(sil, 3, 16, n_pages=8, width=8, max_slots=20)
    assert s.step([2**31 - 1, 1, 1]) == 1 | 2 | 4
    assert s.step([1, 2, 3]) == 0
    assert s.step([-2**31, 2**31 - 1, 0]) & 2
    assert s.step([-2**31, 1, 0]) == 0


def test_extend_negative_lengths_count_as_zero(sil):
    import torch
    s = Server(sil, 2, 8, n_pages=4, width=3, max_slots=6)
    s.d_lens.copy_(torch.tensor([-4, 0], dtype=torch.int32))
    s.lens = [-4, 0]
    assert s.step([3, 2]) == 0


def test_extend_table_columns_of_a_wider_one_and_stream(sil):
    import torch
    s = Server(sil, 40, 4, n_pages=400, width=10, max_slots=200)
    wide = torch.full((40, 25), -3, dtype=torch.int32, device="cuda")
    s.table = wide[:, 4:14]
    st = torch.cuda.Stream()
    assert s.step([5] * 40, stream=st) == 0
    assert s.step([-2] * 20 + [4] * 20, stream=st) == 0
    assert bool((wide[:, :4] == -3).all()) and bool((wide[:, 14:] == -3).all())


def test_extend_refusals(sil):
    import torch
    s = Server(sil, 3, 8, n_pages=6, width=4, max_slots=9)
    add = torch.ones(3, dtype=torch.int32, device="cuda")

    def no(code, **kw):
        a = dict(lens=s.d_lens, add=add, table=s.table, ring=s.ring, cursor=s.cursor, page_size=8, slots=s.slots)
        a.update(kw)
        with pytest.raises(sil.ILError) as ei:
            sil.kv_extend(**a)
        assert ei.value.code == code, str(ei.value)

    no(-2, page_size=0)
    no(-2, page_size=2**21)
    no(-1, add=add[:2])
    no(-1, add=add.long())
    no(-1, cursor=s.cursor.int())
    no(-1, table=s.table[:2])
    no(-1, first=s.first[:3])
    no(-1, info=s.info.int())
    no(-1, positions=s.slots)
    no(-1, lens_out=add)
    no(-1, slots=s.ring)
    no(-1, cursor_out=torch.zeros(3, dtype=torch.int64, device="cuda"))
    assert s.d_lens.tolist() == [0, 0, 0] and s.cursor.tolist() == [0, 6]
    assert s.step([1, 1, 1]) == 0


# ---------------------------------------------------------------------------
# il_kv_append / il_kv_read
# ---------------------------------------------------------------------------
def _cache(sil, fmt, n_pages, page, heads, dim, order):
    import torch
    if order == "head":
        c = sil.kv_cache(fmt, n_pages, page, heads, dim)
    else:
        dtype = torch.bfloat16 if fmt == "bf16" else torch.int8
        kv = [torch.zeros((n_pages, page, heads, dim), dtype=dtype, device="cuda") for _ in range(2)]
        c = sil.KVCache(*kv, *([torch.zeros((n_pages, page, heads, dim // 32), device="cuda") for _ in range(2)]
                               if fmt == "q8" else []))
    for t in (c.k, c.v):
        t.fill_(77)
    for t in (c.k_scale, c.v_scale):
        if t is not None:
            t.fill_(-3.0)
    return c


def _rows(rng, n, heads, dim):
    x = rng.standard_normal((n, heads, dim)).astype(np.float32) * np.exp(rng.uniform(-20, 20, (n, heads, 1))).astype(np.float32)
    flat = x.reshape(-1, dim)
    flat[0] = 0.0
    if len(flat) > 4:
        flat[1] = 1e-45      # scale underflows to 0
        flat[2, 0] = np.nan
        flat[3, dim - 1] = np.inf
        flat[4] = (np.arange(dim) - dim // 2) * 0.5 + 0.25  # ties
        flat[4, ::32] = 127.0
    return x


def _same(a, b):
    return np.array_equal(np.asarray(a), np.asarray(b), equal_nan=True)


@pytest.mark.parametrize("fmt,heads,dim", [("bf16", 8, 128), ("q8", 8, 128), ("bf16", 1, 8), ("bf16", 3, 72), ("q8", 1, 32),
                                           ("q8", 2, 96), ("bf16", 2, 256), ("q8", 2, 256)])
@pytest.mark.parametrize("n", [1, 5, 1000])
@pytest.mark.parametrize("order", ["head", "token"])
def test_append_and_read(sil, fmt, heads, dim, n, order):
    import torch
    rng = np.random.default_rng(n + dim)
    page = 16 if n > 5 else 3
    n_pages = kv_util.pages_of(n, page) + 2
    cache = _cache(sil, fmt, n_pages, page, heads, dim, order)
    slots = rng.permutation(n_pages * page)[:n].astype(np.int32)
    if n > 4:
        slots[3] = -1
    x = {w: _rows(rng, n, heads, dim) for w in "kv"}
    # K and V as columns of one wider buffer
    wide = torch.full((n, 4, heads, dim), 3.0, device="cuda")
    wide[:, 1], wide[:, 3] = torch.from_numpy(x["k"]).cuda(), torch.from_numpy(x["v"]).cuda()
    ds = torch.from_numpy(slots).cuda()
    sil.kv_append(cache, wide[:, 1], wide[:, 3], ds)
    torch.cuda.synchronize()
    used = slots[slots >= 0]
    rows = used // page, used % page
    rest = np.ones((n_pages, page), bool)
    rest[rows] = False
    values = {}
    for w, pool, scale in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale)):
        got = pool.float().cpu().numpy()
        live = x[w][slots >= 0]
        if fmt == "bf16":
            want = torch.from_numpy(live).bfloat16().float().numpy()
            assert _same(got[rows], want)
            values[w] = want
        else:
            q, d = kv_util.quantise(live)
            assert np.array_equal(got[rows], q) and _same(scale.cpu().numpy()[rows], d)
            assert bool((scale.cpu()[torch.from_numpy(rest)] == -3.0).all())
            with np.errstate(invalid="ignore"):
                values[w] = q.astype(np.float32) * np.repeat(d, 32, -1)
        assert np.all(got[rest] == 77)
    # read back into columns of a wider buffer
    back = torch.full((n, 2, heads, dim), 8.0, device="cuda")
    sil.kv_read(cache, ds, back[:, 1], back[:, 0])
    torch.cuda.synchronize()
    for w, i in (("k", 1), ("v", 0)):
        got = back[:, i].cpu().numpy()
        assert _same(got[slots >= 0], values[w]) and np.all(got[slots < 0] == 0)
    sil.check_device_status()


@pytest.mark.parametrize("fmt", ["bf16", "q8"])
def test_slots_outside_the_cache_are_skipped_and_flagged(sil, fmt):
    import torch
    cache = _cache(sil, fmt, 2, 4, 2, 64, "head")
    x = torch.randn((4, 2, 64), device="cuda")
    slots = torch.tensor([1, 8, 2**31 - 1, -1], dtype=torch.int32, device="cuda")
    sil.kv_append(cache, x, x.clone(), slots)
    with pytest.raises(sil.ILError) as ei:
        sil.check_device_status()
    assert ei.value.code == -1
    k, v = torch.full_like(x, 5.0), torch.full_like(x, 5.0)
    sil.kv_read(cache, slots, k, v)
    with pytest.raises(sil.ILError):
        sil.check_device_status()
    assert bool((k[1:] == 0).all()) and bool((v[1:] == 0).all())
    assert torch.allclose(k[0], x[0], atol=0.05) and torch.equal(k[0], v[0])
    assert int((cache.k != 77).any(-1).sum()) == 2  # one token of two heads
    sil.check_device_status()


@pytest.mark.parametrize("fmt", ["bf16", "q8"])
def test_append_offsets_beyond_31_bits(sil, fmt):
    import torch
    page, kv, dim = 16, 2, 64
    row = page * kv * dim
    far = (2**31 + 2**20) // row * row
    dtype = torch.bfloat16 if fmt == "bf16" else torch.int8
    pools = [torch.empty(far + row, dtype=dtype, device="cuda").as_strided((2, page, kv, dim), (far, kv * dim, dim, 1)) for _ in range(2)]
    sc = [torch.zeros((2, page, kv, 2), device="cuda") for _ in range(2)] if fmt == "q8" else []
    cache = sil.KVCache(*pools, *sc)
    x = torch.randn((2, kv, dim), device="cuda")
    slots = torch.tensor([16 + 3, 2], dtype=torch.int32, device="cuda")
    sil.kv_append(cache, x, -x, slots)
    k, v = torch.empty_like(x), torch.empty_like(x)
    sil.kv_read(cache, slots, k, v)
    torch.cuda.synchronize()
    assert torch.equal(k, -v) and torch.allclose(k, x, atol=0.03, rtol=0.01)
    if fmt == "bf16":
        assert torch.equal(pools[0][1, 3].float(), x[0].bfloat16().float())


def test_append_read_refusals(sil):
    import torch
    cache = _cache(sil, "bf16", 2, 4, 2, 64, "head")
    x = torch.randn((3, 2, 64), device="cuda")
    y, slots = x.clone(), torch.arange(3, dtype=torch.int32, device="cuda")

    def no(code, fn, *a):
        with pytest.raises(sil.ILError) as ei:
            fn(*a)
        assert ei.value.code == code, str(ei.value)

    no(-1, sil.kv_append, cache, x.half(), y, slots)
    no(-1, sil.kv_append, cache, x[:, :1], y, slots)
    no(-2, sil.kv_append, cache, x[:2], y, slots)
    no(-1, sil.kv_append, cache, x, y, slots.long())
    no(-1, sil.kv_append, cache, x[:, :, :32], y, slots)
    no(-1, sil.kv_read, cache, slots, x, x)                     # one buffer for both
    no(-1, sil.kv_read, cache, slots, x.cpu(), y)
    flat = torch.zeros(400, device="cuda")
    no(-1, sil.kv_append, cache, flat[1:385].view(3, 2, 64), y, slots)   # not 16-byte aligned
    no(-2, sil.kv_append, cache, flat[:390].as_strided((3, 2, 64), (130, 64, 1)), y, slots)  # row stride not a multiple of 4
    into = cache.k.view(torch.float32) if cache.k.is_contiguous() else cache.k.transpose(1, 2).view(torch.float32)
    no(-1, sil.kv_read, cache, slots[:1], into.reshape(-1)[:128].view(1, 2, 64), y[:1])      # into the cache itself
    assert bool((cache.k == 77).all())
    sil.kv_append(cache, x[:0], y[:0], slots[:0])               # empty: a no-op
    assert bool((cache.k == 77).all())
