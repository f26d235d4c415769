"""Host side of the 4-bit cache, scored attention, collected weights and eviction without a GPU: structs, refusals before a
device is touched, and the plain forms of the tests."""
import ctypes
import os
import re

import numpy as np
import pytest

import kv_long_util as kl

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def libil():
    import shared_input_linear_gb300 as sil
    sil.build()
    return sil.load()


def _kv(**kw):
    import shared_input_linear_gb300 as sil
    a = dict(format=3, page_size=16, n_pages=4, n_heads=2, head_dim=64, k=1 << 20, v=1 << 21, k_scale=1 << 22, v_scale=1 << 23,
             page_stride=1024, token_stride=64, head_stride=32, scale_page_stride=64, scale_token_stride=4, scale_head_stride=2)
    a.update(kw)
    return sil._KV(*[a[n] for n, _ in sil._KV._fields_])


def test_score_mirrors_the_header():
    import shared_input_linear_gb300 as sil
    text = open(os.path.join(ROOT, "include", "il.h")).read()
    body = re.findall(r"typedef struct \{([^}]*)\} il_kv_score;", text)[0]
    names = [n.strip(" *") for line in body.split(";") if line.strip() for n in re.sub(r"^\s*(const )?\w+", "", line).split(",")]
    assert names == [n for n, _ in sil._Score._fields_]
    assert ctypes.sizeof(sil._Score) == 48
    assert re.search(r"IL_A4 = 3\b", text) and sil.IL_A4 == 3 and sil.KV_FORMATS["a4"] == 3


@pytest.mark.parametrize("code,change", [
    (-3, dict(format=4)), (-3, dict(format=2)), (-2, dict(head_dim=40)), (-2, dict(head_dim=288)), (-2, dict(head_stride=24)),
    (-2, dict(head_stride=16)), (-2, dict(token_stride=40)), (-1, dict(k_scale=None)), (-1, dict(v_scale=None)),
    (-1, dict(k_scale=(1 << 22) + 2)), (-2, dict(scale_head_stride=1)), (-2, dict(scale_page_stride=1)), (-1, dict(k=(1 << 20) + 8)),
])
def test_bad_caches_are_refused_before_the_device(libil, code, change):
    kv = _kv(**change)
    p = ctypes.addressof(kv)
    W = 1 << 25
    for rc in (libil.il_kv_append(p, 16, 128, 16, 128, 4, 1, None), libil.il_kv_read(p, 4, 1, 16, 128, 16, 128, None),
               libil.il_kv_attend(p, 16, 128, 4, 1, 1, 4, 1, 2, 1.0, 0, 1 << 16, 128, None, None),
               libil.il_kv_attend_scored(p, 16, 128, 4, 1, 1, 4, 1, 2, 1.0, 0, None, 1 << 16, 128, None, None),
               libil.il_kv_weigh(p, 16, 128, 4, 1, 1, 4, 1, 2, 1.0, 0, None, 4, None, W, W, 64, 64, None),
               libil.il_kv_evict(p, 4, 1, 1, 4, 1, 8, 0, 0, W, W, 64, 64, None, None, 0, 0, W + 4096, 8, W + 8192, None)):
        assert rc == code, libil.il_last_error()


def test_scores_are_refused(libil):
    import shared_input_linear_gb300 as sil
    kv = _kv()
    p = ctypes.addressof(kv)

    def call(scale=1.0, n=2, **kw):
        a = dict(cap=0.0, slopes=None, starts=None, positions=None, positions_stride=0, positions_width=0)
        a.update(kw)
        score = sil._Score(*[a[x] for x, _ in sil._Score._fields_])
        return {libil.il_kv_attend_scored(p, 16, 128, 4, 1, 1, 4, n, 2, scale, 0, ctypes.addressof(score), 1 << 16, 128, None, None),
                libil.il_kv_weigh(p, 16, 128, 4, 1, 1, 4, n, 2, scale, 0, ctypes.addressof(score), 4, None, 1 << 25, 1 << 25, 64, 64, None)}

    inf, nan = float("inf"), float("nan")
    for kw in (dict(cap=-1.0), dict(cap=inf), dict(cap=nan), dict(cap=1e-30, scale=1e30), dict(slopes=6), dict(starts=6), dict(positions=6)):
        assert call(**kw) == {-1}, kw
    for kw in (dict(positions=8), dict(positions=8, positions_width=8, positions_stride=7), dict(positions=8, positions_width=1 << 32, positions_stride=1 << 32)):
        assert call(**kw) == {-2}, kw
    assert call(n=0, cap=2.0) == {0}   # a no-op


@pytest.mark.parametrize("cap,scale", [(1e31, 1.0), (3e38, 1.0), (3e38, 1e30), (7e-31, 1.0), (1e-45, 1e-45)])
def test_caps_beyond_fp32_are_refused(libil, cap, scale):
    """cap log2(e), or q scale / cap, would be infinite or lose bits where the logit is an ordinary number."""
    import shared_input_linear_gb300 as sil
    kv, score = _kv(), sil._Score(cap, None, None, None, 0, 0)
    p, c = ctypes.addressof(kv), ctypes.addressof(score)
    assert libil.il_kv_attend_scored(p, 16, 128, 4, 1, 1, 4, 2, 2, scale, 0, c, 1 << 16, 128, None, None) == -1
    assert libil.il_kv_weigh(p, 16, 128, 4, 1, 1, 4, 2, 2, scale, 0, c, 4, None, 1 << 25, 1 << 25, 64, 64, None) == -1
    assert b"cap" in libil.il_last_error()


def test_weigh_and_evict_are_refused(libil):
    kv = _kv()
    p = ctypes.addressof(kv)
    W = 1 << 25
    w = lambda **k: libil.il_kv_weigh(*[{**dict(  # noqa: E731
        kv=p, q=16, qs=128, t=4, ts=1, tw=1, lens=4, n=2, h=2, sc=1.0, win=0, score=None, lse=4, add=None, w=W, wo=W, ws=64, ww=64, st=None), **k}[x]
        for x in ("kv", "q", "qs", "t", "ts", "tw", "lens", "n", "h", "sc", "win", "score", "lse", "add", "w", "wo", "ws", "ww", "st")])
    assert w(n=0) == 0 and w(kv=None) == -1 and w(n=-1) == -1 and w(h=3) == -2 and w(win=-1) == -1 and w(lse=None) == -1 and w(lse=6) == -1
    assert w(w=None) == -1 and w(wo=None) == -1 and w(w=W + 2) == -1 and w(ww=0) == -2 and w(ws=63) == -2 and w(ww=1 << 31, ws=1 << 31) == -2
    assert w(wo=W + 4) == -1 and w(wo=W + 64) == -1 and w(wo=16) == -1 and w(lse=W) == -1 and w(add=W + 8) == -1 and w(t=W, ts=4) == -1
    e = lambda **k: libil.il_kv_evict(*[{**dict(  # noqa: E731
        kv=p, t=4, ts=1, tw=1, lens=4, n=2, keep=8, first=1, recent=2, w=W, wo=W, ws=64, ww=64, p=None, po=None, ps=0, pw=0, kept=W + 4096, ks=8,
        drop=W + 8192, st=None), **k}[x] for x in
        ("kv", "t", "ts", "tw", "lens", "n", "keep", "first", "recent", "w", "wo", "ws", "ww", "p", "po", "ps", "pw", "kept", "ks", "drop", "st")])
    assert e(n=0) == 0 and e(kv=None) == -1 and e(n=-1) == -1 and e(keep=0) == -1 and e(keep=1 << 31, ks=1 << 31) == -1
    assert e(first=-1) == -1 and e(recent=-1) == -1 and e(first=7) == -1 and e(first=1 << 62, recent=1 << 62) == -1 and e(recent=7, first=1) == e()
    assert e(kept=None) == -1 and e(drop=None) == -1 and e(t=None) == -1 and e(lens=None) == -1 and e(ks=7) == -2 and e(w=None) == -1
    assert e(p=1 << 26) == -1 and e(po=1 << 26) == -1 and e(p=1 << 26, po=1 << 26) == -2 and e(p=1 << 26, po=1 << 26, ps=8, pw=9) == -2
    assert e(kept=W) == -1 and e(drop=W + 4096) == -1 and e(wo=W + 4) == -1 and e(wo=1 << 20) == -1 and e(kept=1 << 23) == -1
    assert e(p=1 << 26, po=(1 << 26) + 4, ps=64, pw=64) == -1 and e(lens=W + 8192) == -1


def test_plain_a4():
    x = np.random.default_rng(0).standard_normal((9, 3, 96)).astype(np.float32)
    u, d, m = kl.quantise(x)
    back = kl.values(u, d, m)
    assert np.all(np.abs(back - x) <= np.repeat(d, 32, -1) * 0.5001)
    assert np.all(m <= x.reshape(9, 3, 3, 32).min(-1)) and u.max() == 15 and u.min() == 0
    assert np.array_equal(kl.pack(u)[..., 0], u[..., 0] + 16 * u[..., 1])
    u, d, m = kl.quantise(np.full((1, 32), -0.3, np.float32))
    assert abs(kl.values(u, d, m)[0, 0] + 0.3) <= d[0, 0] / 2 <= 1e-4


def test_plain_scores():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 8)), rng.standard_normal((5, 1, 8))
    s, _ = kl.logits(q, k, np.abs(k), 0.5, cap=2.0, slopes=np.float32([0.25, 0]), far=np.arange(5) - 4)
    for h in range(2):
        for t in range(5):
            assert np.isclose(s[h, t], 2 * np.tanh(0.25 * (q[h] @ k[t, 0])) + (0.25 * (t - 4) if h == 0 else 0))
    assert kl.begin_of(10, 4, 3) == 6 and kl.begin_of(10, 0, 12) == 10 and kl.begin_of(10, 0, -5) == 0
    lse = np.log(np.exp(s).sum(1))
    p, _ = kl.weigh(q, k, np.abs(k), 0.5, lse, cap=2.0, slopes=np.float32([0.25, 0]), far=np.arange(5) - 4)
    assert np.isclose(p.sum(), 2)


def test_plain_evict():
    w = [5, 1, 1, 9, 1, float("nan"), 2, 0]
    assert kl.evict(w, range(8), 8, 8, 0, 0) == list(range(8)) and kl.evict(w, range(8), 3, 8, 0, 0) == [0, 1, 2]
    assert kl.evict(w, range(8), 8, 4, 0, 0) == [0, 1, 6, 3]       # 5 9 2 1: of the ones the first
    assert kl.evict(w, range(8), 8, 4, 2, 1) == [0, 1, 7, 3]       # 0, 1 and 7 whatever their weight
    assert kl.evict(w, range(8), 8, 7, 0, 0) == [0, 1, 2, 3, 4, 7, 6]
    assert kl.evict(w, [9, 8, 0, 1, 2, 3, 4, 10], 8, 3, 1, 2) == [0, 7, 2]
