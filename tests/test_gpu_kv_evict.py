"""il_kv_evict against its definition: which tokens stay, where they go, the rows' bytes, and a server that runs with it."""
import numpy as np
import pytest

import kv_long_util as kl
import kv_util
from gpu_util import lib

pytestmark = pytest.mark.gpu
FORMATS = ["bf16", "q8", "a4"]


@pytest.fixture(scope="module")
def sil():
    import torch
    torch.cuda.set_device(0)
    return lib()


class Cut:
    """A cache of random bytes, its weights and positions."""

    def __init__(self, sil, fmt, lens, page=16, kv=2, dim=64, order="head", seed=0, positions=False, weights=None, extra=4, width=None):
        import torch
        rng = np.random.default_rng(seed)
        self.sil, self.lens, self.page = sil, list(lens), page
        held = [kv_util.pages_of(n, page) for n in lens]
        n_pages, cols = sum(held) + 2, max(held + [1]) + 1
        perm = rng.permutation(n_pages)
        self.table = np.full((len(lens), cols), -5, np.int32)
        at = 0
        for r, h in enumerate(held):
            self.table[r, :h] = perm[at:at + h]
            at += h
        cache = sil.kv_cache(fmt, n_pages, page, kv, dim)
        if order == "token":
            cache = sil.KVCache(*(t if t is None else t.contiguous() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
        self.cache = cache
        self.pools = [t for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]
        for t in self.pools:
            raw = torch.from_numpy(rng.integers(1, 100, tuple(t.shape)).astype(np.float32)).cuda()
            t.copy_(raw.to(t.dtype))
        width = max(self.lens + [1]) + extra if width is None else width
        self.weights = rng.choice([0, 1, 2, 3.5, 1e-3, 7], (len(lens), width)).astype(np.float32) if weights is None else weights
        self.positions = None
        if positions:
            self.positions = np.stack([rng.permutation(3 * width)[:width] for _ in lens]).astype(np.int32)
            for r, n in enumerate(lens):
                if n:
                    self.positions[r, n - 1] = 3 * width

    def run(self, keep, first=0, recent=0, in_place=False, stream=None):
        """Evicts, and checks every byte of every output; returns (kept, drop)."""
        import torch
        n, width = self.weights.shape
        before = [t.clone() for t in self.pools]
        w = torch.from_numpy(self.weights).cuda()
        p = None if self.positions is None else torch.from_numpy(self.positions).cuda()
        wo = w if in_place else torch.full_like(w, -3.0)
        po = p if in_place or p is None else torch.full_like(p, -3)
        kept = torch.full((n, keep + 2), -9, dtype=torch.int32, device="cuda")
        drop = torch.full((n,), -9, dtype=torch.int32, device="cuda")
        table, lens = torch.from_numpy(self.table).cuda(), torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        self.sil.kv_evict(self.cache, table, lens, w, kept[:, :keep], drop, first=first, recent=recent, weights_out=None if in_place else wo,
                          positions=p, positions_out=None if in_place else po, stream=stream)
        torch.cuda.synchronize()
        self.sil.check_device_status()
        got, got_w = kept.cpu().numpy(), wo.cpu().numpy()
        assert np.all(got[:, keep:] == -9) and torch.equal(lens.cpu(), torch.tensor(self.lens, dtype=torch.int32))
        want = [t.cpu().numpy() if t.dtype != torch.bfloat16 else t.view(torch.int16).cpu().numpy() for t in before]
        for r, length in enumerate(self.lens):
            full, length = max(length, 0), min(max(length, 0), width)
            pos = np.arange(width) if self.positions is None else self.positions[r]
            entries = kl.evict(self.weights[r], pos, length, keep, first, recent)
            m = len(entries)
            assert got[r, :m].tolist() == entries and np.all(got[r, m:keep] == -1)
            assert int(drop[r]) == m - full
            expect = (self.weights[r] if in_place else np.full(width, -3, np.float32)).copy()
            expect[:m] = self.weights[r][entries]
            assert np.array_equal(got_w[r], expect, equal_nan=True)
            if p is not None:
                expect = (self.positions[r] if in_place else np.full(width, -3, np.int32)).copy()
                expect[:m] = self.positions[r][entries]
                assert np.array_equal(po[r].cpu().numpy(), expect)
            for i, j in enumerate(entries):
                if i != j:
                    a, b = self.table[r, i // self.page], self.table[r, j // self.page]
                    for t in want:
                        t[a, i % self.page] = t[b, j % self.page]
        for t, x in zip(self.pools, want):
            t = t.view(torch.int16) if t.dtype == torch.bfloat16 else t
            assert np.array_equal(t.cpu().numpy(), x)
        return got[:, :keep], drop.tolist()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("order", ["head", "token"])
@pytest.mark.parametrize("keep,first,recent", [(1, 0, 0), (1, 0, 1), (7, 2, 3), (32, 0, 32), (64, 64, 0), (100, 4, 50), (1000, 1, 1)])
def test_choice_and_rows(sil, fmt, order, keep, first, recent):
    lens = [0, 1, 7, 8, 31, 32, 33, 63, 64, 65, 100, 101, 257, 1030]
    Cut(sil, fmt, lens, order=order, seed=keep).run(keep, first, recent)
    Cut(sil, fmt, lens, order=order, seed=keep, positions=True).run(keep, first, recent, in_place=True)


@pytest.mark.parametrize("fmt,kv,dim", [("bf16", 1, 8), ("bf16", 3, 72), ("bf16", 1, 256), ("q8", 5, 96), ("a4", 3, 32), ("a4", 9, 160), ("q8", 33, 256),
                                        ("bf16", 64, 128), ("a4", 100, 128)])
@pytest.mark.parametrize("page", [1, 5, 16, 128])
def test_row_shapes(sil, fmt, kv, dim, page):
    Cut(sil, fmt, [90, 3, 40], page=page, kv=kv, dim=dim, seed=dim, positions=True).run(29, 2, 5)


@pytest.mark.parametrize("kind", ["equal", "ascending", "descending", "zeros of both signs", "extremes", "negative", "nan", "random bits"])
@pytest.mark.parametrize("keep", [1, 33, 500, 2047])
def test_orders_of_weights(sil, kind, keep):
    rng = np.random.default_rng(keep)
    n, rows = 2048, 2
    w = {"equal": lambda: np.full((rows, n), 0.25), "ascending": lambda: np.arange(rows * n).reshape(rows, n),
         "descending": lambda: -np.arange(rows * n).reshape(rows, n), "zeros of both signs": lambda: rng.choice([0.0, -0.0], (rows, n)),
         "extremes": lambda: rng.choice([np.inf, -np.inf, 3e38, -3e38, 1e-45, -1e-45, 0], (rows, n)), "negative": lambda: -rng.random((rows, n)),
         "nan": lambda: rng.choice([np.nan, 1, 2, -np.inf], (rows, n)),
         "random bits": lambda: rng.integers(0, 2**32, (rows, n), dtype=np.uint32).view(np.float32)}[kind]().astype(np.float32)
    for in_place in (False, True):
        Cut(sil, "bf16", [n, n - 1], kv=1, dim=8, weights=w, seed=keep).run(keep, 0, 1, in_place=in_place)


@pytest.mark.parametrize("n,keep", [(5000, 4999), (20000, 1), (20000, 19000), (40000, 20000), (131072, 4096), (100001, 70000),
                                    (400000, 300), (400000, 250000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_long(sil, n, keep, in_place):
    w = np.random.default_rng(n).random((2, n)).astype(np.float32) ** 8
    w[1, ::3] = 0.5
    first, recent = (4, min(64, keep - 4)) if keep > 4 else (0, 0)
    Cut(sil, "bf16", [n, n // 2], page=64, kv=1, dim=8, weights=w, seed=keep).run(keep, first, recent, in_place=in_place)


@pytest.mark.parametrize("n_seq", [1, 7, 19, 30, 60, 100])
def test_numbers_of_sequences(sil, n_seq):
    """The CTAs that share a sequence go by the number of sequences and the rows' width."""
    rng = np.random.default_rng(n_seq)
    lens = [9000] + rng.integers(1, 9001, n_seq - 1).tolist()
    w = rng.choice(np.float32([0, 0.5, 1, 2]), (n_seq, 9004)) * rng.choice(np.float32([1, 1, 1, 0.999]), (n_seq, 9004))
    Cut(sil, "q8", lens, page=32, kv=1, dim=32, weights=w, seed=n_seq, positions=True).run(1777, 4, 100, in_place=n_seq % 2 == 0)


def test_many_sequences(sil):
    rng = np.random.default_rng(2)
    Cut(sil, "bf16", rng.integers(0, 40, 2000).tolist(), kv=1, dim=8, page=8, seed=1).run(16, 1, 4)


def test_lengths_are_cut(sil):
    """To the weights' width, and to the table's; negative ones count as 0."""
    import torch
    c = Cut(sil, "bf16", [50, 20], width=30, seed=3)
    c.run(10, 1, 2)
    c = Cut(sil, "bf16", [50, 0], seed=3, extra=200)
    kept, drop = torch.zeros((2, 8), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    lens = torch.tensor([2**31 - 1, -7], dtype=torch.int32, device="cuda")
    w = torch.from_numpy(c.weights).cuda()
    w[0, 60:] = -1
    sil.kv_evict(c.cache, torch.from_numpy(c.table).cuda(), lens, w, kept, drop)
    cap = c.table.shape[1] * 16
    assert drop.tolist() == [8 - (2**31 - 1), 0] and kept[1].tolist() == [-1] * 8 and 8 <= max(kept[0].tolist()) < cap


def test_bad_pages_are_skipped_and_flagged(sil):
    import torch
    w = np.tile(np.arange(64, dtype=np.float32), (1, 1))  # the last 16 stay: they move to the first page
    c = Cut(sil, "bf16", [64], weights=w, seed=3)
    before = [t.clone() for t in c.pools]
    c.table[0, 3] = 77
    kept, drop = torch.zeros((1, 16), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    sil.kv_evict(c.cache, torch.from_numpy(c.table).cuda(), torch.tensor([64], dtype=torch.int32, device="cuda"), torch.from_numpy(w).cuda(), kept, drop)
    with pytest.raises(sil.ILError) as e:
        sil.check_device_status()
    assert e.value.code == -1 and kept[0].tolist() == list(range(48, 64))
    assert all(torch.equal(t, b) for t, b in zip(c.pools, before))


def test_graph(sil):
    import torch
    c = Cut(sil, "q8", [300, 5, 90], seed=4, positions=True)
    w, p = torch.from_numpy(c.weights).cuda(), torch.from_numpy(c.positions).cuda()
    wo, po = torch.zeros_like(w), torch.zeros_like(p)
    kept, drop = torch.zeros((3, 40), dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    table, lens = torch.from_numpy(c.table).cuda(), torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        sil.kv_evict(c.cache, table, lens, w, kept, drop, first=2, recent=9, weights_out=wo, positions=p, positions_out=po)
    for _ in range(2):  # sources stay: a second call gives the same
        graph.replay()
        torch.cuda.synchronize()
        for r, n in enumerate(c.lens):
            entries = kl.evict(c.weights[r], c.positions[r], n, 40, 2, 9)
            assert kept[r, :len(entries)].tolist() == entries


def test_refusals(sil):
    import torch
    c = Cut(sil, "bf16", [50, 20], seed=3)
    w, table = torch.from_numpy(c.weights).cuda(), torch.from_numpy(c.table).cuda()
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    i32 = lambda *s: torch.full(s, 5, dtype=torch.int32, device="cuda")  # noqa: E731
    kept, drop = i32(2, 8), i32(2)

    def no(code, w=w, kept=kept, drop=drop, **kw):
        with pytest.raises(sil.ILError) as e:
            sil.kv_evict(c.cache, table, lens, w, kept, drop, **kw)
        assert e.value.code == code, str(e.value)

    no(-1, first=5, recent=4)
    no(-1, first=-1)
    no(-1, kept=i32(2, 0))
    no(-1, kept=i32(3, 8))
    no(-1, drop=i32(3))
    no(-1, w=w.double())
    no(-2, weights_out=w[:, :-1])
    no(-1, positions=w)
    no(-1, positions_out=i32(2, 60))
    no(-1, kept=w.view(torch.int32)[:, :8])
    wide = i32(2, 130)
    no(-1, positions=wide[:, :60], positions_out=wide[:, 30:90])
    torch.cuda.synchronize()
    assert bool((kept == 5).all()) and bool((drop == 5).all())


# ---------------------------------------------------------------------------
# All of them together: a decode loop at a fixed cache size
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", FORMATS)
def test_a_server_at_a_fixed_cache_size(sil, fmt):
    """Tokens arrive, are attended with a bias by position, weighed, and above `keep` evicted; beside it lists of the tokens that
    are left, their weights and positions.  The choice is taken from the device (weights that lie within their error of
    one another may change places) and checked against the device's own weights."""
    import torch
    rng = np.random.default_rng(11)
    n_seq, heads, kv, dim, page, keep, first, recent = 3, 8, 2, 64, 16, 40, 2, 8
    width = 128
    cache = sil.kv_cache(fmt, 32, page, kv, dim)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, table, ring = i32(n_seq), i32(n_seq, 9), torch.arange(32, dtype=torch.int32, device="cuda")
    cursor, slots, info = torch.tensor([0, 32], device="cuda"), i32(256), torch.zeros(4, dtype=torch.int64, device="cuda")
    weights, positions = torch.zeros((n_seq, width), device="cuda"), i32(n_seq, width)
    kept, drop, total = i32(n_seq, keep), i32(n_seq), [0] * n_seq
    slopes = np.exp2(-8 * np.arange(1, heads + 1) / heads).astype(np.float32)
    dev_slopes = torch.from_numpy(slopes).cuda()
    held = [[] for _ in range(n_seq)]  # (k, kmag, v, vmag, position)
    for step in range(30):
        add = [int(rng.integers(20, 60)) if step == 0 else int(rng.integers(0, 7)) for _ in range(n_seq)]
        dev_add = torch.tensor(add, dtype=torch.int32, device="cuda")
        sil.kv_extend(lens, dev_add, table, ring, cursor, page, slots, info=info)
        n = sum(add)
        x = [rng.standard_normal((n, kv, dim)).astype(np.float32) for _ in range(2)]
        if n:
            sil.kv_append(cache, *(torch.from_numpy(t).cuda() for t in x), slots[:n])
        (_, kd, km), (_, vd, vm) = (kl.pool(fmt, t, lambda t: t) for t in x)
        at = 0
        host = positions.cpu().numpy()
        for r, a in enumerate(add):
            for _ in range(a):
                host[r, len(held[r])] = total[r]
                held[r].append((kd[at], km[at], vd[at], vm[at], total[r]))
                total[r] += 1
                at += 1
        positions.copy_(torch.from_numpy(host))
        q = rng.standard_normal((n_seq, heads, dim)).astype(np.float32)
        dq, out, lse = torch.from_numpy(q).cuda(), torch.empty((n_seq, heads, dim), device="cuda"), torch.empty((n_seq, heads), device="cuda")
        score = dict(slopes=dev_slopes, positions=positions, cap=20.0)
        sil.kv_attend(cache, dq, table, lens, out, lse=lse, **score)
        before = weights.cpu().numpy()
        sil.kv_weigh(cache, dq, table, lens, lse, weights, add=dev_add, **score)
        after = weights.cpu().numpy()
        pos = positions.cpu().numpy()
        for r in range(n_seq):
            m = len(held[r])
            k, kmg, v, vmg = (np.stack([h[i] for h in held[r]]) for i in range(4))
            far = np.array([h[4] for h in held[r]])
            assert pos[r, :m].tolist() == far.tolist()
            plain = dict(cap=20.0, slopes=slopes, far=far - far[-1])
            o, l, ot, lt = kl.attend(q[r], k, v, kmg, vmg, dim ** -0.5, **plain)
            assert np.all(np.abs(out[r].cpu().numpy() - o) <= ot) and np.all(np.abs(lse[r].cpu().numpy() - l) <= lt)
            p, pt = kl.weigh(q[r], k, kmg, dim ** -0.5, lse[r].cpu().numpy().astype(np.float64), **plain)
            was = before[r, :m].copy()
            was[m - add[r]:] = 0
            assert np.all(np.abs(after[r, :m] - (was + p)) <= pt + kl.U * (np.abs(was) + p))
        sil.kv_evict(cache, table, lens, weights, kept, drop, first=first, recent=recent, positions=positions)
        sil.kv_extend(lens, drop, table, ring, cursor, page, slots, info=info)
        for r in range(n_seq):
            entries = kl.evict(after[r], pos[r], len(held[r]), keep, first, recent)
            assert kept[r, :len(entries)].tolist() == entries
            held[r] = [held[r][j] for j in entries]
        assert lens.tolist() == [len(h) for h in held] and int(info[0]) == 0
    assert max(total) > 100 and int(cursor[1] - cursor[0]) == 32 - sum(-(-len(h) // page) for h in held)
    sil.check_device_status()
