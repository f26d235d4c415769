"""Host side of the paged K/V cache without a GPU: the binding's struct mirrors the header's, arguments are
refused before a device is touched, and the plain forms of the tests hold their own invariants."""
import ctypes
import os
import re

import numpy as np
import pytest

import kv_util

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def libil():
    import shared_input_linear_gb300 as sil
    sil.build()
    return sil.load()


def test_struct_mirrors_the_header():
    import shared_input_linear_gb300 as sil
    text = open(os.path.join(ROOT, "include", "il.h")).read()
    body = re.search(r"typedef struct \{([^}]*)\} il_kv;", text).group(1)
    names = [n.strip(" *") for line in body.split(";") if line.strip() for n in re.sub(r"^\s*\w+", "", line).split(",")]
    assert names == [n for n, _ in sil._KV._fields_]
    assert ctypes.sizeof(sil._KV) == 104


def _kv(sil, **kw):
    a = dict(format=0, page_size=16, n_pages=4, n_heads=2, head_dim=64, k=1 << 20, v=1 << 21, k_scale=None, v_scale=None,
             page_stride=2048, token_stride=128, head_stride=64, scale_page_stride=0, scale_token_stride=0, scale_head_stride=0)
    a.update(kw)
    return sil._KV(*[a[n] for n, _ in sil._KV._fields_])


@pytest.mark.parametrize("code,change", [
    (-3, dict(format=2)), (-3, dict(format=9)), (-2, dict(page_size=0)), (-2, dict(page_size=1 << 21)), (-2, dict(n_pages=0)),
    (-2, dict(n_pages=1 << 40)), (-2, dict(n_heads=0)), (-2, dict(head_dim=0)), (-2, dict(head_dim=12)), (-2, dict(head_dim=264)),
    (-1, dict(k=None)), (-1, dict(v=None)), (-1, dict(k=(1 << 20) + 8)), (-2, dict(head_stride=60)), (-2, dict(token_stride=32)),
    (-2, dict(page_stride=-2048)), (-2, dict(page_stride=1 << 62)), (-1, dict(format=1)), (-2, dict(format=1, head_dim=40)),
    (-1, dict(k_scale=1 << 22, v_scale=1 << 23)),
    (-1, dict(format=1, k_scale=(1 << 22) + 2, v_scale=1 << 23, scale_page_stride=64, scale_token_stride=4, scale_head_stride=2)),
    (-2, dict(format=1, k_scale=1 << 22, v_scale=1 << 23, scale_page_stride=64, scale_token_stride=4, scale_head_stride=1)),
])
def test_bad_caches_are_refused_before_the_device(libil, code, change):
    import shared_input_linear_gb300 as sil
    kv = _kv(sil, **change)
    for rc in (libil.il_kv_append(ctypes.addressof(kv), 16, 128, 16, 128, 4, 1, None),
               libil.il_kv_read(ctypes.addressof(kv), 4, 1, 16, 128, 16, 128, None),
               libil.il_kv_attend(ctypes.addressof(kv), 16, 128, 4, 1, 1, 4, 1, 2, 1.0, 0, 1 << 16, 128, None, None)):
        assert rc == code, libil.il_last_error()


def test_null_and_range_checks(libil):
    import shared_input_linear_gb300 as sil
    kv = _kv(sil)
    p = ctypes.addressof(kv)
    assert libil.il_kv_append(None, 16, 128, 16, 128, 4, 1, None) == -1
    assert libil.il_kv_append(p, 16, 128, 16, 128, 4, -1, None) == -1
    assert libil.il_kv_append(p, None, 128, 16, 128, 4, 1, None) == -1
    assert libil.il_kv_append(p, 16, 128, 16, 128, None, 1, None) == -1
    assert libil.il_kv_append(p, 16, 127, 16, 128, 4, 2, None) == -2
    assert libil.il_kv_append(p, 16, 128, 16, 128, 4, 0, None) == 0    # a no-op
    assert libil.il_kv_attend(p, 16, 128, 4, 1, 1, 4, 0, 2, 1.0, 0, 1 << 16, 128, None, None) == 0
    assert libil.il_kv_attend(p, 16, 128, 4, 1, 1, 4, 1, 3, 1.0, 0, 1 << 16, 128, None, None) == -2   # 3 heads over 2
    assert libil.il_kv_attend(p, 16, 128, 4, 1, 0, 4, 1, 2, 1.0, 0, 1 << 16, 128, None, None) == -2
    assert libil.il_kv_attend(p, 16, 128, 4, 1, 1, 4, 1 << 20, 2, 1.0, 0, 1 << 16, 128, None, None) == -1
    e = lambda **k: libil.il_kv_extend(*[{**dict(  # noqa: E731
        n=2, P=16, lens=4096, add=8192, table=12288, ts=4, tw=4, ring=16384, rs=8, cur=20480, lo=4096, co=20480, slots=24576,
        ms=4, pos=None, first=None, info=None, st=None), **k}[x] for x in
        ("n", "P", "lens", "add", "table", "ts", "tw", "ring", "rs", "cur", "lo", "co", "slots", "ms", "pos", "first", "info", "st")])
    assert e(n=0) == 0 and e(n=-1) == -1 and e(P=0) == -2 and e(lens=None) == -1 and e(tw=0) == -2 and e(ts=3) == -2
    assert e(rs=0) == -2 and e(ms=-1) == -1 and e(cur=20484) == -1 and e(lens=4098) == -1 and e(slots=16384) == -1
    assert e(lo=4100) == -1 and e(info=24576) == -1 and e(add=4096) == -1


def test_plain_extend_conserves_pages():
    rng = np.random.default_rng(0)
    ring, lens, tables = kv_util.Ring(50, range(50)), [0] * 6, [[] for _ in range(6)]
    done = 0
    for _ in range(200):
        adds = [int(rng.integers(-20, 24)) for _ in lens]
        code, slots, positions, first, info = ring.extend(lens, tables, adds, 4, 12, 60)
        done += code == 0
        assert sorted(ring.free + [p for t in tables for p in t]) == list(range(50))
        assert [len(t) for t in tables] == [kv_util.pages_of(n, 4) for n in lens]
        live = [s for s in slots if s >= 0]
        assert len(set(live)) == len(live) == (0 if code else info[1])
    assert 20 < done < 200


def test_plain_attend_is_softmax_attention():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    out, lse, _, _ = kv_util.attend(q, k, v, 0.5, 3)
    for h in range(4):
        s = 0.5 * k[6:, h // 2] @ q[h]
        assert np.allclose(out[h], np.exp(s) @ v[6:, h // 2] / np.exp(s).sum()) and np.isclose(lse[h], np.log(np.exp(s).sum()))


def test_plain_quantise_round_trip():
    x = np.random.default_rng(2).standard_normal((3, 64)).astype(np.float32)
    q, d = kv_util.quantise(x)
    assert np.all(np.abs(q * np.repeat(d, 32, -1) - x) <= np.repeat(d, 32, -1) * 0.5001)
    z, dz = kv_util.quantise(np.zeros((1, 32), np.float32))
    assert not z.any() and dz[0, 0] == 0
