"""il_kv_weigh against 64 bits: what each cached token collects, over formats, layouts, masks and splits."""
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


def _weigh(c, add=None, in_place=False, extra=5, seed=0, stream=None):
    """Runs the operator after the attention that gives lse; checks every entry and returns the weights."""
    import torch
    sil = c.sil
    q, table, lens = c.device()
    _, lse = c.run()
    rng = np.random.default_rng(seed)
    width = max(c.lens + [1]) + extra
    w = (rng.random((len(c.lens), width)) * 3).astype(np.float32)
    if add is not None:
        for r, n in enumerate(c.lens):
            w[r, max(0, n - max(0, add[r])):n] = np.nan  # new: nothing of it may be used
    weights = torch.from_numpy(w).cuda()
    out = weights if in_place else torch.full_like(weights, 9.0)
    dev_add = None if add is None else torch.tensor(add, dtype=torch.int32, device="cuda")
    more = c.score()
    torch.cuda.synchronize()
    sil.kv_weigh(c.cache, q, table, lens, lse, weights, weights_out=None if in_place else out, add=dev_add, stream=stream, **more)
    torch.cuda.synchronize()
    got = out.cpu().numpy().astype(np.float64)
    lse = lse.cpu().numpy().astype(np.float64)
    for r, n in enumerate(c.lens):
        want = w[r].astype(np.float64) if in_place else np.full(width, 9.0)
        want[:n] = w[r, :n]
        if add is not None:
            want[max(0, n - max(0, add[r])):n] = 0
        tol = np.zeros(width)
        k, _, km, _ = c.rows[r]
        if len(k):
            p, pt = kl.weigh(c.q[r], k, km, c.dim ** -0.5, lse[r], **c.plain_score(r))
            tol[c.begins[r]:n] = pt + kl.U * (np.abs(want[c.begins[r]:n]) + p)
            want[c.begins[r]:n] += p
        off = np.abs(got[r] - want)
        assert np.all(off <= tol), (r, n, float(np.max(off / np.maximum(tol, 1e-30))), int(np.argmax(off - tol)))
    return out


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heads,kv,dim", [(32, 8, 128), (4, 4, 64), (8, 1, 256), (1, 1, 32), (7, 1, 128), (18, 2, 64), (16, 1, 128), (40, 1, 96),
                                          (12, 2, 160), (34, 2, 256), (9, 3, 224), (64, 64, 64), (33, 33, 128)])
def test_head_layouts(sil, fmt, heads, kv, dim):
    c = kl.Case(sil, fmt, heads, kv, dim, 16, [1, 0, 37, 300, 16, 129], seed=heads + dim)
    _weigh(c, add=[1] * 6)
    sil.check_device_status()


@pytest.mark.parametrize("dim", [8, 16, 24, 40, 72, 80, 120, 136, 200, 248])
def test_odd_head_dims_bf16(sil, dim):
    _weigh(kl.Case(sil, "bf16", 6, 2, dim, 16, [5, 33, 0, 70], seed=dim, order="token"))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heads,kv,dim", [(512, 128, 64), (320, 1, 128), (1024, 1, 256), (600, 150, 32)])
def test_more_heads_than_shared_memory_holds(sil, fmt, heads, kv, dim):
    _weigh(kl.Case(sil, fmt, heads, kv, dim, 16, [3, 70, 0, 300], seed=heads), add=[3, 1, 0, 2])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page", [1, 3, 8, 16, 20, 32, 100, 512])
@pytest.mark.parametrize("order", ["head", "token", "padded"])
def test_pages_and_orders(sil, fmt, page, order):
    _weigh(kl.Case(sil, fmt, 8, 2, 128, page, [1, 15, 16, 17, 31, 100, 203, 0], order=order, seed=page, lopsided=1.0))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("what", ["window", "starts", "cap", "slopes", "all"])
def test_masks_and_scores(sil, fmt, in_place, what):
    lens = [0, 1, 2, 16, 17, 33, 150, 401, 64, 64, 1000]
    kw = {}
    if what in ("window", "all"):
        kw["window"] = 40
    if what in ("starts", "all"):
        kw["starts"] = [0, 1, 1, 15, 17, -4, 100, 390, 64, 32, 999]
    if what in ("cap", "all"):
        kw["cap"] = 7.0
    if what in ("slopes", "all"):
        kw.update(slopes=_slopes(8), positions=what == "all")
    c = kl.Case(sil, fmt, 8, 2, 64, 16, lens, seed=5, spread=3.0, **kw)
    _weigh(c, in_place=in_place)
    _weigh(c, in_place=in_place, add=[0, 1, 1, 20, 17, -5, 150, 3, 2**31 - 1, 1, 500])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lens", [[20011], [4096, 3, 0, 9000], [2048] * 5, [100] * 400, [0] * 300 + [40000]])
def test_long_and_many(sil, fmt, lens):
    c = kl.Case(sil, fmt, 8, 2, 64, 64, lens, seed=len(lens))
    first = _weigh(c, add=[1] * len(lens))
    again = _weigh(c, add=[1] * len(lens))
    assert bool((first == again).all())  # the same bits


def test_collects_to_the_number_of_heads(sil):
    """Steps in place: after n tokens the weights of a sequence sum to n times the heads."""
    import torch
    c = kl.Case(sil, "bf16", 8, 2, 64, 16, [5, 90], seed=3)
    q, table, lens = c.device()
    weights = torch.zeros((2, 100), device="cuda")
    out, lse = torch.empty_like(q), torch.empty((2, 8), device="cuda")
    for _ in range(3):
        sil.kv_attend(c.cache, q, table, lens, out, lse=lse)
        sil.kv_weigh(c.cache, q, table, lens, lse, weights)
    assert torch.allclose(weights.sum(1), torch.full((2,), 24.0, device="cuda"), rtol=1e-5)


def test_bad_pages_are_skipped_and_flagged(sil):
    import torch
    c = kl.Case(sil, "bf16", 8, 2, 128, 16, [50, 100], seed=2)
    c.table[1, 2] = 10**6
    q, table, lens = c.device()
    _, lse = c.run()
    with pytest.raises(sil.ILError):
        sil.check_device_status()
    weights = torch.ones((2, 100), device="cuda")
    sil.kv_weigh(c.cache, q, table, lens, lse, weights)
    with pytest.raises(sil.ILError) as e:
        sil.check_device_status()
    assert e.value.code == -1
    assert bool((weights[1, 32:48] == 1).all()) and bool((weights[1, :32] > 1).all()) and bool((weights[1, 48:] > 1).all())


def test_rows_apart_and_lengths_cut_to_them(sil):
    import torch
    c = kl.Case(sil, "bf16", 4, 1, 64, 16, [40, 40], seed=2)
    q, table, lens = c.device()
    _, lse = c.run()
    wide = torch.full((2, 3, 33), 2.0, device="cuda")
    sil.kv_weigh(c.cache, q, table, lens, lse, wide[:, 1])
    full = torch.full((2, 64), 2.0, device="cuda")
    sil.kv_weigh(c.cache, q, table, lens, lse, full)
    assert torch.equal(wide[:, 1], full[:, :33]) and bool((wide[:, 0] == 2).all()) and bool((wide[:, 2] == 2).all())


def test_graph_and_stream(sil):
    import torch
    c = kl.Case(sil, "a4", 32, 8, 128, 16, [900, 1, 0, 333], seed=1)
    q, table, lens = c.device()
    _, lse = c.run()
    weights, out = torch.rand((4, 900), device="cuda"), torch.zeros((4, 900), device="cuda")
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        sil.kv_weigh(c.cache, q, table, lens, lse, weights, weights_out=out)
    graph.replay()
    torch.cuda.synchronize()
    want = torch.zeros_like(out)
    sil.kv_weigh(c.cache, q, table, lens, lse, weights, weights_out=want)
    torch.cuda.synchronize()
    assert torch.equal(want, out) and float(want.sum()) > 0


def test_refusals(sil):
    import torch
    c = kl.Case(sil, "bf16", 8, 2, 64, 16, [20, 4], seed=8)
    q, table, lens = c.device()
    lse, weights = torch.zeros((2, 8), device="cuda"), torch.ones((2, 30), device="cuda")

    def no(code, lse=lse, weights=weights, **kw):
        with pytest.raises(sil.ILError) as e:
            sil.kv_weigh(c.cache, q, table, lens, lse, weights, **kw)
        assert e.value.code == code, str(e.value)

    no(-1, lse=None)
    no(-1, lse=lse[:, :7])
    no(-1, weights=None)
    no(-1, weights=weights.double())
    no(-1, weights=weights[:1])
    no(-1, weights=weights[:, ::2])
    no(-2, weights_out=torch.ones((2, 31), device="cuda"))
    no(-1, weights_out=torch.as_strided(weights, (2, 30), (30, 1), 0)[:1])
    no(-1, add=torch.zeros(3, dtype=torch.int32, device="cuda"))
    wide = torch.ones((2, 61), device="cuda")
    no(-1, weights=wide[:, :30], weights_out=wide[:, 1:31])
    no(-1, lse=weights.flatten()[:16].view(2, 8))
    torch.cuda.synchronize()
    assert bool((weights == 1).all())
