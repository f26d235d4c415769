"""il_kv_attend against softmax attention in 64 bits: formats, head layouts, lengths, pages that end
inside a tile, windows, strides, garbage outside the attended range, streams, graphs, refusals."""
import math

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


class Case:
    """A cache in which only the attended tokens hold numbers: everything else, the other pages
    included, is NaN, and the table names pages that do not exist behind each sequence's own."""

    def __init__(self, sil, fmt, heads, kv, dim, page, lens, order="head", seed=0, window=0, spread=1.0, pad=0):
        import torch
        rng = np.random.default_rng(seed)
        self.sil, self.lens, self.page, self.heads, self.dim, self.window = sil, list(lens), page, heads, dim, window
        held = [kv_util.pages_of(n, page) for n in lens]
        n_pages = sum(held) + 3
        width = max(held + [1]) + 2
        perm = rng.permutation(n_pages)
        self.table = np.full((len(lens), width), 2**31 - 1, np.int32)
        self.table[:, -1] = -7
        k = np.full((n_pages, page, kv, dim), np.nan, np.float32)
        v = k.copy()
        self.keys, self.values = [], []
        at = 0
        for r, n in enumerate(lens):
            mine = perm[at:at + held[r]]
            at += held[r]
            self.table[r, :held[r]] = mine
            begin = max(0, n - window) if window else 0
            for p in range(begin, n):
                k[mine[p // page], p % page] = spread * rng.standard_normal((kv, dim))
                v[mine[p // page], p % page] = rng.standard_normal((kv, dim))

        def place(x, dtype):  # onto the device in the wanted order of dimensions
            t = torch.from_numpy(x).to(dtype)
            if order == "head":
                return t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
            if order == "padded":  # rows apart, pages not next to each other
                wide = torch.zeros((t.shape[0], t.shape[1] + 1, t.shape[2] + 1, t.shape[3] + (16 if dtype == torch.int8 else 8)
                                    if t.shape[3] >= 8 else t.shape[3] + 1), dtype=dtype)
                wide[:, :t.shape[1], :t.shape[2], :t.shape[3]] = t
                return wide.cuda()[:, :t.shape[1], :t.shape[2], :t.shape[3]]
            return t.contiguous().cuda()

        if fmt == "bf16":
            kt, vt = place(k, torch.bfloat16), place(v, torch.bfloat16)
            self.cache = sil.KVCache(kt, vt)
            kd, vd = (t.float().cpu().numpy() for t in (kt, vt))
        else:
            (kq, ks), (vq, vs) = kv_util.quantise(k), kv_util.quantise(v)  # NaN blocks: q 0, scale NaN
            self.cache = sil.KVCache(place(kq, torch.int8), place(vq, torch.int8), place(ks, torch.float32),
                                     place(vs, torch.float32))
            kd = kq * np.repeat(ks, 32, -1).astype(np.float64)
            vd = vq * np.repeat(vs, 32, -1).astype(np.float64)
        for r, n in enumerate(lens):
            p = np.arange(n)
            rows = self.table[r, p // page], p % page
            self.keys.append(kd[rows])
            self.values.append(vd[rows])
        self.q = rng.standard_normal((len(lens), heads, dim)).astype(np.float32)

    def run(self, stream=None, scale=None, q=None, out=None):
        import torch
        n = len(self.lens)
        q = torch.from_numpy(self.q).cuda() if q is None else q
        out = torch.full((n, self.heads, self.dim), float("nan"), device="cuda") if out is None else out
        lse = torch.full((n, self.heads), float("nan"), device="cuda")
        table, lens = torch.from_numpy(self.table).cuda(), torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        self.sil.kv_attend(self.cache, q, table, lens, out, lse=lse, scale=scale, window=self.window, stream=stream)
        torch.cuda.synchronize()
        return out, lse

    def check(self, out, lse, scale=None, rows=None):
        out, lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        scale = self.dim ** -0.5 if scale is None else scale
        for r in range(len(self.lens)) if rows is None else rows:
            o, l, ot, lt = kv_util.attend(self.q[r], self.keys[r], self.values[r], scale, self.window)
            assert np.all(np.isfinite(out[r])), (r, self.lens[r])
            worst = float(np.max(np.abs(out[r] - o) / ot))
            assert worst <= 1, f"sequence {r} of length {self.lens[r]}: out is {worst:.3g} x its bound"
            if self.lens[r] == 0:
                assert np.all(np.isneginf(lse[r])) and np.all(out[r] == 0)
            else:
                worst = float(np.max(np.abs(lse[r] - l) / lt))
                assert worst <= 1, f"sequence {r} of length {self.lens[r]}: lse is {worst:.3g} x its bound"


@pytest.mark.parametrize("fmt", ["bf16", "q8"])
@pytest.mark.parametrize("heads,kv,dim", [(32, 8, 128), (4, 4, 64), (8, 1, 256), (1, 1, 32), (7, 1, 128), (18, 2, 64),
                                          (16, 1, 128), (40, 1, 96), (12, 2, 160), (34, 2, 256), (9, 3, 224)])
def test_head_layouts(sil, fmt, heads, kv, dim):
    c = Case(sil, fmt, heads, kv, dim, 16, [1, 0, 37, 300, 16, 129], seed=heads + dim)
    c.check(*c.run())
    sil.check_device_status()


@pytest.mark.parametrize("dim", [8, 16, 24, 40, 72, 80, 120, 136, 200, 248])
def test_odd_head_dims_bf16(sil, dim):
    c = Case(sil, "bf16", 6, 2, dim, 16, [5, 33, 0, 70], seed=dim, order="token" if dim % 16 else "head")
    c.check(*c.run())


@pytest.mark.parametrize("fmt", ["bf16", "q8"])
@pytest.mark.parametrize("page", [1, 3, 8, 16, 20, 32, 100, 512])
@pytest.mark.parametrize("order", ["head", "token", "padded"])
def test_pages_and_orders(sil, fmt, page, order):
    c = Case(sil, fmt, 8, 2, 128, page, [1, 15, 16, 17, 31, 100, 203, 0], order=order, seed=page)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", ["bf16", "q8"])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 1000])
def test_windows(sil, fmt, window):
    c = Case(sil, fmt, 8, 2, 64, 16, [0, 1, 2, 16, 17, 33, 150, 401], window=window, seed=window)
    c.check(*c.run())


@pytest.mark.parametrize("fmt,heads,kv,dim", [("bf16", 8, 1, 128), ("q8", 8, 1, 128), ("bf16", 2, 1, 256), ("q8", 32, 2, 64)])
@pytest.mark.parametrize("lens", [[20011], [4096, 3, 0, 9000], [2048] * 5])
def test_long_sequences_split_and_join(sil, fmt, heads, kv, dim, lens):
    c = Case(sil, fmt, heads, kv, dim, 64, lens, seed=len(lens))
    out, lse = c.run()
    c.check(out, lse)
    again = c.run()
    assert bool((again[0] == out).all()) and bool((again[1] == lse).all())  # the same bits


@pytest.mark.parametrize("fmt", ["bf16", "q8"])
@pytest.mark.parametrize("n_seq", [150, 700, 1300])
def test_many_sequences(sil, fmt, n_seq):
    rng = np.random.default_rng(n_seq)
    lens = rng.integers(0, 40, n_seq).tolist()
    lens[0] = 0
    lens[-1] = 0
    lens[5] = 700
    c = Case(sil, fmt, 4, 2, 32, 16, lens, seed=n_seq)
    c.check(*c.run())


def test_all_sequences_empty(sil):
    c = Case(sil, "bf16", 4, 2, 64, 16, [0, 0, 0])
    c.check(*c.run())


def test_no_sequences_is_a_no_op(sil):
    import torch
    c = Case(sil, "bf16", 4, 2, 64, 16, [3])
    e = torch.empty((0, 4, 64), device="cuda")
    sil.kv_attend(c.cache, e, torch.empty((0, 1), dtype=torch.int32, device="cuda"),
                  torch.empty(0, dtype=torch.int32, device="cuda"), e.clone())


@pytest.mark.parametrize("fmt", ["bf16", "q8"])
@pytest.mark.parametrize("spread,scale", [(20.0, 1.0), (1.0, -0.7), (1.0, 0.0), (1e-20, 1e18), (1e4, 1e-3)])
def test_peaked_flat_and_odd_logits(sil, fmt, spread, scale):
    c = Case(sil, fmt, 8, 2, 64, 16, [1, 50, 333], spread=spread, seed=3)
    c.check(*c.run(scale=scale), scale=scale)


def test_q8_scales_of_all_sizes(sil):
    import torch
    c = Case(sil, "q8", 8, 2, 128, 16, [40, 200], seed=9)
    rng = np.random.default_rng(1)
    # values of very unlike magnitude from token to token and block to block, and blocks of zeros
    vs = c.cache.v_scale
    f = np.exp(rng.uniform(-40, 40, tuple(vs.shape))) * rng.integers(0, 2, tuple(vs.shape))
    f = torch.from_numpy(f.astype(np.float32)).cuda()
    vs.copy_(torch.where(torch.isnan(vs), vs, f))
    vd = c.cache.v.double().cpu().numpy() * np.repeat(vs.double().cpu().numpy(), 32, -1)
    for r, n in enumerate(c.lens):
        p = np.arange(n)
        c.values[r] = vd[c.table[r, p // 16], p % 16]
    out, lse = c.run()
    # a part's V scales share one power of two: a weight is kept to 2^-30 of the largest p|v| beside it
    o = out.double().cpu().numpy()
    for r in range(2):
        ref, _, tol, _ = kv_util.attend(c.q[r], c.keys[r], c.values[r], 128 ** -0.5, 0)
        top = np.abs(c.values[r]).max()
        assert np.all(np.abs(o[r] - ref) <= tol + 2.0 ** -30 * top)


def test_strided_q_out_and_table(sil):
    import torch
    c = Case(sil, "bf16", 8, 2, 64, 16, [70, 3, 0, 128], seed=4)
    wide_q = torch.zeros((4, 3, 8, 64), device="cuda")
    wide_q[:, 1] = torch.from_numpy(c.q).cuda()
    wide_o = torch.full((4, 2, 8, 64), 5.5, device="cuda")
    out, lse = c.run(q=wide_q[:, 1], out=wide_o[:, 1])
    c.check(out, lse)
    assert bool((wide_o[:, 0] == 5.5).all())
    # a table that is columns of a wider one
    wide = torch.full((4, c.table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, 2:-3] = torch.from_numpy(c.table).cuda()
    out2 = torch.empty_like(wide_q[:, 1].contiguous())
    sil.kv_attend(c.cache, wide_q[:, 1], wide[:, 2:-3], torch.tensor(c.lens, dtype=torch.int32, device="cuda"), out2)
    torch.cuda.synchronize()
    assert torch.equal(out2, out)


def test_length_beyond_the_table_is_cut(sil):
    import torch
    c = Case(sil, "bf16", 4, 2, 64, 16, [64, 20], seed=5)
    lens = torch.tensor([10**9, -5], dtype=torch.int32, device="cuda")
    out, lse = torch.empty((2, 4, 64), device="cuda"), torch.empty((2, 4), device="cuda")
    sil.kv_attend(c.cache, torch.from_numpy(c.q).cuda(), torch.from_numpy(c.table[:, :4].copy()).cuda(), lens, out, lse=lse)
    torch.cuda.synchronize()
    c.lens[1], c.keys[1], c.values[1] = 0, c.keys[1][:0], c.values[1][:0]
    c.check(out, lse)


@pytest.mark.parametrize("fmt", ["bf16", "q8"])
def test_bad_pages_are_skipped_and_flagged(sil, fmt):
    c = Case(sil, fmt, 4, 2, 64, 16, [100, 60, 40], seed=6)
    good = c.table.copy()
    c.table[1, 1] = -1
    c.table[1, 2] = 10**6
    out, lse = c.run()
    c.check(out, lse, rows=[0, 2])
    with pytest.raises(sil.ILError) as ei:
        sil.check_device_status()
    assert ei.value.code == -1
    sil.check_device_status()  # cleared
    c.table = good
    c.check(*c.run())


@pytest.mark.parametrize("fmt", ["bf16", "q8"])
def test_offsets_beyond_31_bits(sil, fmt):
    # one page far behind the other: its elements lie beyond 2^31 elements from the base
    import torch
    page, kv, dim = 16, 2, 64
    row = page * kv * dim
    far = (2**31 + 2**20) // row * row
    dtype = torch.bfloat16 if fmt == "bf16" else torch.int8
    base = torch.empty(far + row, dtype=dtype, device="cuda")
    pool = base.as_strided((2, page, kv, dim), (far, kv * dim, dim, 1))
    g = torch.Generator(device="cuda").manual_seed(0)
    sc = []
    if fmt == "q8":
        pool.copy_(torch.randint(-127, 128, (2, page, kv, dim), generator=g, device="cuda").to(dtype))
        sc = [torch.rand((2, page, kv, 2), generator=g, device="cuda") * 0.02 for _ in range(2)]
    else:
        pool.copy_(torch.randn((2, page, kv, dim), generator=g, device="cuda").to(dtype))
    cache = sil.KVCache(pool, pool, *sc)  # K and V may be the same elements when they are only read
    q = torch.randn((1, 4, dim), generator=g, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((1, 4), device="cuda")
    sil.kv_attend(cache, q, torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"),
                  torch.tensor([31], dtype=torch.int32, device="cuda"), out, lse=lse)
    torch.cuda.synchronize()
    tok = pool[[1, 0]].reshape(32, kv, dim)[:31].double().cpu().numpy()
    k, v = (tok * (np.repeat(s[[1, 0]].reshape(32, kv, 2)[:31].double().cpu().numpy(), 32, -1)) for s in sc) if sc else (tok, tok)
    o, l, ot, lt = kv_util.attend(q[0].cpu().numpy(), k, v, dim ** -0.5, 0)
    assert np.all(np.abs(out[0].cpu().numpy() - o) <= ot) and np.all(np.abs(lse[0].cpu().numpy() - l) <= lt)


def test_other_stream_and_graph_with_changing_lengths(sil):
    import torch
    c = Case(sil, "bf16", 8, 2, 128, 16, [300, 40, 0, 90], seed=7)
    s = torch.cuda.Stream()
    out, lse = c.run(stream=s)
    c.check(out, lse)
    q, table = torch.from_numpy(c.q).cuda(), torch.from_numpy(c.table).cuda()
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((4, 8), device="cuda")
    with torch.cuda.stream(s):
        sil.kv_attend(c.cache, q, table, lens, out, lse=lse)  # the workspace exists before the capture
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            sil.kv_attend(c.cache, q, table, lens, out, lse=lse)
    for new in ([300, 40, 0, 90], [1, 0, 0, 33], [17, 16, 0, 15]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        keep = c.lens, c.keys, c.values
        c.lens = new
        c.keys, c.values = [k[:n] for k, n in zip(c.keys, new)], [v[:n] for v, n in zip(c.values, new)]
        c.check(out, lse)
        c.lens, c.keys, c.values = keep


def test_refusals(sil):
    import torch
    c = Case(sil, "bf16", 8, 2, 64, 16, [20, 4], seed=8)
    q, table = torch.from_numpy(c.q).cuda(), torch.from_numpy(c.table).cuda()
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 9.0)

    def no(code, cache=c.cache, q=q, table=table, lens=lens, out=out, **kw):
        with pytest.raises(sil.ILError) as ei:
            sil.kv_attend(cache, q, table, lens, out, **kw)
        assert ei.value.code == code, str(ei.value)

    no(-1, q=q.double())
    no(-1, q=q[:, :, ::2])
    no(-2, q=q[:, :7], out=torch.empty((2, 7, 64), device="cuda"))   # 7 query heads, 2 K/V heads
    no(-1, table=table.long())
    no(-1, table=table[:1])
    no(-1, lens=lens[:1])
    no(-1, lens=lens.long())
    no(-1, out=out[:, :, :32])
    no(-2, out=torch.empty((3, 8, 64), device="cuda"))
    no(-1, out=q)                                                     # in place
    no(-1, window=-1)
    no(-1, scale=math.inf)
    no(-1, scale=math.nan)
    no(-1, lse=torch.empty((2, 7), device="cuda"))
    flat = torch.zeros(2 * 8 * 64 + 4, device="cuda")
    no(-1, q=flat[1:1 + 1024].view(2, 8, 64))                         # not 16-byte aligned
    assert bool((out == 9.0).all())
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    for make in (lambda: sil.KVCache(k, k.float()), lambda: sil.KVCache(k.float(), k.float()),
                 lambda: sil.KVCache(k, k[:3]), lambda: sil.KVCache(k.transpose(2, 3), k.transpose(2, 3)),
                 lambda: sil.KVCache(k.to(torch.int8), k.to(torch.int8)),
                 lambda: sil.KVCache(k, k, torch.zeros((4, 16, 2, 2), device="cuda"), torch.zeros((4, 16, 2, 2), device="cuda")),
                 lambda: sil.kv_cache("q4", 4, 16, 2, 64)):
        with pytest.raises(sil.ILError):
            make()
    for shape, dtype in (((4, 16, 2, 264), torch.bfloat16), ((4, 16, 2, 12), torch.bfloat16), ((4, 16, 2, 48), torch.int8)):
        t = torch.zeros(shape, dtype=dtype, device="cuda")
        s = torch.zeros((*shape[:3], shape[3] // 32), device="cuda") if dtype == torch.int8 else None
        qq = torch.zeros((2, 8, shape[3]), device="cuda")
        no(-2, cache=sil.KVCache(t, t, s, s), q=qq, out=torch.empty_like(qq))
    no(-2, cache=sil.KVCache(k[..., :60], k[..., :60]), q=torch.zeros((2, 8, 60), device="cuda"), out=torch.empty((2, 8, 60), device="cuda"))
    odd = torch.zeros(4 * 16 * 2 * 65 + 8, dtype=torch.bfloat16, device="cuda").as_strided((4, 16, 2, 64), (16 * 2 * 65, 130, 65, 1))
    no(-2, cache=sil.KVCache(odd, odd))                               # rows not 16-byte aligned
    assert bool((out == 9.0).all())
    sil.check_device_status()


def test_the_most_sequences(sil):
    import torch
    n = 65536
    lens = torch.zeros(n, dtype=torch.int32)
    live = [0, 1, 255, 256, 30000, 65000, n - 1]
    lens[live] = torch.tensor([1, 40, 16, 17, 33, 2, 20], dtype=torch.int32)
    kv = torch.randn((9, 16, 1, 32), device="cuda").bfloat16()
    cache = sil.KVCache(kv, kv)
    q = torch.randn((n, 2, 32), device="cuda")
    table = torch.full((n, 3), -1, dtype=torch.int32, device="cuda")
    table[live] = torch.tensor([[1, 5, 8]], dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((n, 2), 7.0, device="cuda")
    sil.kv_attend(cache, q, table, lens.cuda(), out, lse=lse)
    torch.cuda.synchronize()
    tok = kv[[1, 5, 8]].reshape(48, 1, 32).float().cpu().numpy()
    for r in live:
        o, l, ot, lt = kv_util.attend(q[r].cpu().numpy(), tok[:int(lens[r])], tok[:int(lens[r])], 32 ** -0.5, 0)
        assert np.all(np.abs(out[r].cpu().numpy() - o) <= ot) and np.all(np.abs(lse[r].cpu().numpy() - l) <= lt)
    rest = torch.ones(n, dtype=torch.bool)
    rest[live] = False
    assert bool((out[rest] == 0).all()) and bool(torch.isneginf(lse[rest]).all())
    e = torch.empty((n + 1, 2, 32), device="cuda")
    with pytest.raises(sil.ILError):
        sil.kv_attend(cache, e, torch.empty((n + 1, 1), dtype=torch.int32, device="cuda"),
                      torch.empty(n + 1, dtype=torch.int32, device="cuda"), e.clone())


@pytest.mark.parametrize("fmt", ["bf16", "q8"])
def test_logits_that_rise_and_fall_along_a_sequence(sil, fmt):
    # a token far above the others first, then in the middle, and slopes of a few units a token: what came before is
    # scaled up and down, and tiles span more than fp16 does
    import torch
    for shape in ("first", "middle", "rise", "fall"):
        n, dim = 400, 64
        c = Case(sil, fmt, 8, 2, dim, 16, [n], seed=21)
        t = np.arange(n)
        level = {"first": np.where(t == 0, 60.0, 0.0), "middle": np.where(t == 200, 45.0, 0.0), "rise": t * 1.5 - 300,
                 "fall": 300 - t * 1.5}[shape]
        # K's first block becomes level / sqrt(dim) * sign(q0): adds `level` to every head whose q starts with that sign
        c.q[:, :, 0] = 8.0
        kd = c.keys[0].copy()
        kd[:, :, 0] = level[:, None]
        rows = torch.from_numpy(c.table[0, t // 16].astype(np.int64)).cuda(), torch.from_numpy(t % 16).cuda()
        if fmt == "bf16":
            c.cache.k[rows] = torch.from_numpy(kd).float().cuda().bfloat16()
            c.keys[0] = c.cache.k[rows].double().cpu().numpy()
        else:
            kq, ks = kv_util.quantise(kd.astype(np.float32))
            c.cache.k[rows] = torch.from_numpy(kq).cuda()
            c.cache.k_scale[rows] = torch.from_numpy(ks).cuda()
            c.keys[0] = kq * np.repeat(ks, 32, -1).astype(np.float64)
        c.check(*c.run())
