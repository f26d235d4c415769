"""cudaStreamPerThread is one handle for a stream of each thread: the library's per-stream scratch is the thread's own."""
import threading

import numpy as np
import pytest

import workloads as wl
from gpu_util import lib, upload

pytestmark = pytest.mark.gpu

PER_THREAD = 2  # cudaStreamPerThread


@pytest.fixture(scope="module")
def sil():
    import torch
    torch.cuda.set_device(0)
    return lib()


def _on_threads(n, work):
    """work(i) on n threads at once; what each raised or returned."""
    got = [None] * n

    def call(i):
        import torch
        torch.cuda.set_device(0)
        try:
            got[i] = work(i)
        except Exception as e:  # noqa: BLE001
            got[i] = e
    threads = [threading.Thread(target=call, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return got


def _attend_case(sil, seed):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pool = [torch.randn((300, 16, 8, 128), generator=gen, device="cuda").bfloat16() for _ in range(2)]
    lens = torch.from_numpy(np.random.default_rng(seed).integers(500, 4000, 19).astype(np.int32)).cuda()
    table = torch.randint(0, 300, (19, 250), generator=gen, device="cuda").int()
    q = torch.randn((19, 32, 128), generator=gen, device="cuda")
    cache = sil.KVCache(*pool)

    def call(out, stream=None):
        sil.kv_attend(cache, q, table, lens, out, stream=stream)
    want = torch.empty_like(q)
    call(want)
    return call, want


def test_a_thread_has_its_own_workspace(sil, monkeypatch):
    # one thread after the other, nothing runs beside anything: with device allocations failing, a thread that is new to
    # the stream has no workspace yet, whatever the others have
    import torch
    call, want = _attend_case(sil, 1)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    assert _on_threads(1, lambda i: call(out, PER_THREAD)) == [None]
    monkeypatch.setenv("IL_FAULT_ALLOC_FAIL_AFTER", "0")
    got = _on_threads(1, lambda i: call(out, PER_THREAD))[0]
    monkeypatch.delenv("IL_FAULT_ALLOC_FAIL_AFTER")
    assert isinstance(got, sil.ILError) and got.code == -5, got

    def whole(i):
        out.fill_(7.0)
        torch.cuda.synchronize()
        call(out, PER_THREAD)
        torch.cuda.synchronize()
        same = torch.equal(out, want)
        sil.release_scratch(PER_THREAD)
        return same
    assert _on_threads(1, whole) == [True]


def test_a_thread_has_its_own_copy_of_x(sil, monkeypatch):
    # the tensor-core path's scratch likewise
    import torch
    b = wl.make_batch(256, (64,), 40, "bf16", seed=3)
    w = upload(sil, b)[0]
    x, y = torch.from_numpy(b.x).cuda(), torch.empty((40, 64), device="cuda")
    torch.cuda.synchronize()
    assert _on_threads(1, lambda i: sil.matmul_batch(x, [(w, y)], stream=PER_THREAD)) == [None]
    monkeypatch.setenv("IL_FAULT_ALLOC_FAIL_AFTER", "0")
    got = _on_threads(1, lambda i: sil.matmul_batch(x, [(w, y)], stream=PER_THREAD))[0]
    monkeypatch.delenv("IL_FAULT_ALLOC_FAIL_AFTER")
    assert isinstance(got, sil.ILError) and got.code == -5, got
    w.free()


def test_threads_at_once_on_their_streams(sil):
    import torch
    cases = [_attend_case(sil, seed) for seed in range(4)]
    torch.cuda.synchronize()

    def work(i):
        call, want = cases[i]
        outs = [torch.empty_like(want) for _ in range(30)]
        torch.cuda.synchronize()
        for o in outs:
            call(o, PER_THREAD)
        torch.cuda.synchronize()
        same = all(torch.equal(o, want) for o in outs)
        sil.release_scratch(PER_THREAD)
        return same
    assert _on_threads(4, work) == [True] * 4


def _graph(call, out, stream):
    import torch
    with torch.cuda.stream(stream):
        call(out, stream)  # the workspace exists before the capture
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            for _ in range(10):
                call(out, stream)
    return graph


def test_graphs_of_streams_of_their_own_side_by_side(sil):
    # a graph uses the workspace of its capture stream, wherever it is replayed
    import torch
    cases = [_attend_case(sil, seed) for seed in (5, 6)]
    outs = [torch.empty_like(want) for _, want in cases]
    captured_on = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    graphs = [_graph(call, out, s) for (call, _), out, s in zip(cases, outs, captured_on)]
    for o in outs:
        o.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(5):
        for g in graphs:
            with torch.cuda.stream(torch.cuda.Stream()):
                g.replay()
        torch.cuda.synchronize()
        for (_, want), o in zip(cases, outs):
            assert torch.equal(o, want)
            o.fill_(7.0)
        torch.cuda.synchronize()


def test_graphs_of_one_stream_one_after_the_other(sil):
    import torch
    cases = [_attend_case(sil, seed) for seed in (7, 8)]
    outs = [torch.empty_like(want) for _, want in cases]
    stream, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs = [_graph(call, out, stream) for (call, _), out in zip(cases, outs)]
    for _ in range(5):
        for o in outs:
            o.fill_(7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graphs[0].replay()
        other.wait_stream(stream)
        with torch.cuda.stream(other):
            graphs[1].replay()
        torch.cuda.synchronize()
        for (_, want), o in zip(cases, outs):
            assert torch.equal(o, want)
