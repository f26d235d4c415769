"""examples/decode_attention.py at a fixed cache size: sequences that end, and prompts that come, after tokens were evicted."""
import importlib.util
import os

import pytest

from gpu_util import lib

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KEEP, FIRST, RECENT = 24, 2, 6


@pytest.fixture(scope="module")
def example():
    import torch
    torch.cuda.set_device(0)
    lib()
    spec = importlib.util.spec_from_file_location("decode_attention", os.path.join(ROOT, "examples", "decode_attention.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


class Run:
    """A block, and on the host which positions of each sequence the cache may and must hold."""

    def __init__(self, example, pages=60, n_seq=3):
        import torch
        self.block = example.AttentionBlock(n_in=256, heads=8, kv_heads=2, dim=64, n_seq=n_seq, page=16, pages=pages, cache="bf16", keep=KEEP,
                                            first=FIRST, recent=RECENT)
        self.gen = torch.Generator(device="cuda").manual_seed(7)
        self.held, self.seen = [[] for _ in range(n_seq)], [0] * n_seq

    def rows(self, n):
        import torch
        return torch.randn((n, 256), generator=self.gen, device="cuda")

    def prompt(self, lens):
        self.block.prompt(self.rows(sum(lens)), lens)
        for r, n in enumerate(lens):
            self.held[r] += range(self.seen[r], self.seen[r] + n)
            self.seen[r] += n
        self.check()

    def step(self, replay=None):
        import torch
        self.block.x.copy_(self.rows(len(self.held)))
        torch.cuda.synchronize()
        (replay or self.block.step)()
        torch.cuda.synchronize()
        for r, had in enumerate(self.held):
            had.append(self.seen[r])
            self.seen[r] += 1
            now = self.block.positions[r, :int(self.block.lens[r])].tolist()
            assert len(now) == len(set(now)) == min(KEEP, len(had)) and set(now) <= set(had)
            stay = [p for p in had if p < FIRST or p > had[-1] - RECENT]
            assert set(stay) <= set(now), (r, stay, now)
            had[:] = sorted(now)
        self.check()

    def finish(self, which):
        self.block.finish(which)
        for r in which:
            self.held[r], self.seen[r] = [], 0
        self.check()

    def check(self):
        b = self.block
        assert b.lens.tolist() == [len(h) for h in self.held] and b.seen.tolist() == self.seen
        for r, had in enumerate(self.held):
            assert sorted(b.positions[r, :len(had)].tolist()) == had


@pytest.mark.parametrize("graph", [False, True])
def test_a_prompt_that_comes_after_an_eviction(example, graph):
    """Into the row of a sequence that has ended, and behind one that runs on: the others' positions and weights stay theirs."""
    import torch
    run = Run(example)
    run.prompt([23, 1, 17])
    replay = None
    if graph:
        run.step()  # (capture() runs one of its own, with the x that is there)
        replay = run.block.capture().replay
        for r, had in enumerate(run.held):
            had.append(run.seen[r])
            run.seen[r] += 1
            had[:] = sorted(run.block.positions[r, :int(run.block.lens[r])].tolist())
        run.check()
    for _ in range(30):
        run.step(replay)
    run.finish([1])
    weights = run.block.weights.clone()
    run.prompt([0, 40, 5])
    lens = run.block.lens.tolist()
    assert lens == [KEEP, 40, KEEP + 5]
    assert torch.equal(run.block.weights[0, :KEEP], weights[0, :KEEP]) and torch.equal(run.block.weights[2, :KEEP], weights[2, :KEEP])
    assert not run.block.weights[1, :40].any() and not run.block.weights[2, KEEP:KEEP + 5].any()
    for _ in range(12):
        run.step(replay)
    run.finish([0, 2])
    for _ in range(40):  # rows whose first token is a step's
        run.step(replay)


def test_a_step_without_room(example):
    """No free page: no token is added or counted, also where a sequence has none yet."""
    run = Run(example, pages=9)
    run.prompt([48, 0, 48])
    run.block.cursor[1] = run.block.cursor[0]  # someone else has the pages that were free
    run.block.step()
    assert int(run.block.info[0]) != 0
    assert run.block.lens.tolist() == [KEEP, 0, KEEP] and run.block.seen.tolist() == [48, 0, 48]
    for r in (0, 2):
        now = run.block.positions[r, :KEEP].tolist()
        assert len(set(now)) == KEEP and set(now) <= set(range(48)) and {0, 1, *range(48 - RECENT, 48)} <= set(now)
    example.sil.check_device_status()
