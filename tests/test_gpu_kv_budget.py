"""The decode step of examples/decode_attention.py over a 4-bit cache, and at a fixed cache size: against the tokens that are left
in 64 bits, directly and as a replayed graph."""
import importlib.util
import os

import numpy as np
import pytest

import kv_long_util as kl
from gpu_util import lib

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import torch
    torch.cuda.set_device(0)
    lib()
    spec = importlib.util.spec_from_file_location("decode_attention", os.path.join(ROOT, "examples", "decode_attention.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("cache", ["bf16", "q8", "a4"])
@pytest.mark.parametrize("graph", [False, True])
def test_a_fixed_cache_size(example, cache, graph):
    """Attention over what the device's cache holds (read back), and the choice from the device's weights."""
    import torch
    sil = example.sil
    keep = 24
    block = example.AttentionBlock(n_in=256, heads=8, kv_heads=2, dim=64, n_seq=3, page=16, pages=60, cache=cache, keep=keep, first=2, recent=6)
    gen = torch.Generator(device="cuda").manual_seed(5)
    lens = [23, 1, 17]
    block.prompt(torch.randn((sum(lens), 256), generator=gen, device="cuda"), lens)
    replay = block.capture().replay if graph else block.step
    seen = [n + graph for n in lens]  # capture() runs a step that stays
    free = 60 - sum(-(-min(n, keep) // 16) for n in seen)
    assert block.lens.tolist() == [min(n, keep) for n in seen] and int(block.cursor[1] - block.cursor[0]) == free
    for _ in range(30):
        block.x.copy_(torch.randn((3, 256), generator=gen, device="cuda"))
        before, weights = block.lens.tolist(), block.weights.clone()
        positions = block.positions.cpu().numpy()
        torch.cuda.synchronize()
        replay()
        torch.cuda.synchronize()
        for r in range(3):
            n, pos = before[r] + 1, positions[r].copy()
            pos[n - 1] = seen[r]
            seen[r] += 1
            # the weights after this step's attention, where their tokens were: back from where they went
            kept = block.kept[r].tolist()
            after = np.full(n, np.nan)
            new = block.weights[r].cpu().numpy()
            for i, j in enumerate(kept):
                if j >= 0:
                    after[j] = new[i]
            left = [j for j in kept if j >= 0]
            assert len(left) == min(n, keep) == block.lens[r].item() and len(set(left)) == len(left)
            was = weights[r, :n].cpu().numpy()
            was[n - 1] = 0
            got = ~np.isnan(after)
            assert np.all(after[got] >= was[got] * (1 - 1e-6))  # tokens only collect
            gone = [j for j in range(n) if j not in left]
            assert all(2 <= pos[j] <= pos[n - 1] - 6 for j in gone)
            assert block.positions[r, :len(left)].tolist() == pos[left].tolist()
            # nobody that went had collected more before this step than a stayer has now, but for those that stay anyway
            bar = min([after[j] for j in left if 2 <= pos[j] <= pos[n - 1] - 6], default=np.inf)
            assert all(was[j] <= bar for j in gone)
    assert block.lens.tolist() == [keep, min(keep, seen[1]), keep] and min(seen) > keep
    sil.check_device_status()


@pytest.mark.parametrize("args", [["--cache", "a4"], ["--cache", "a4", "--keep", "40"], ["--keep", "64", "--cache", "bf16"]])
def test_main_runs(example, capsys, args):
    got = example.main(["--seqs", "4", "--prompt", "70", "--steps", "5", *args])
    assert got["us"] > 0 and "tokens/s" in capsys.readouterr().out


def test_decode_block_a4(example):
    """As test_gpu_kv_decode.py has it for the other formats; k and v are cached in steps of a fifteenth of a 32-element range."""
    import torch
    block = example.AttentionBlock(n_in=256, heads=8, kv_heads=2, dim=64, n_seq=3, page=16, pages=60, cache="a4")
    gen = torch.Generator(device="cuda").manual_seed(5)
    history = [torch.randn((n, 256), generator=gen, device="cuda") for n in (40, 1, 17)]
    block.prompt(torch.cat(history), [len(h) for h in history])
    wq, wk, wv = (w.double() for w in block.host)
    for _ in range(5):
        block.x.copy_(torch.randn((3, 256), generator=gen, device="cuda"))
        torch.cuda.synchronize()
        block.step()
        torch.cuda.synchronize()
        for r in range(3):
            seq = history[r] = torch.cat([history[r], block.x[r:r + 1]])
            # q, k, v as the batch gives them (x rounded to bf16 or better), k and v as the cache stands for them
            q, k, v = (sil_batch(example.sil, block, seq, i) for i in range(3))
            (ku, kd, km), (vu, vd, vm) = (kl.quantise(t.reshape(len(seq), 2, 64)) for t in (k, v))
            mags = [u * np.repeat(d, 32, -1) + np.repeat(np.abs(m), 32, -1) for u, d, m in ((ku, kd, km), (vu, vd, vm))]
            o, _, ot, _ = kl.attend(q[-1].reshape(8, 64), kl.values(ku, kd, km), kl.values(vu, vd, vm), *mags, 64 ** -0.5)
            got = block.attention[r].cpu().numpy()
            # q, k and v of other batch sizes differ in their last bits, by 2^-8 of their size at most (x as bf16): a few steps of 1/15
            # may fall to the other side; a tenth of the result's rms is far below what a wrong token or element would do
            assert np.max(np.abs(got - o)) <= 0.1 * np.sqrt(np.mean(o ** 2)) * 3 + np.max(ot), r


def sil_batch(sil, block, x, i):
    import torch
    y = torch.empty((len(x), block.host[i].shape[0]), device="cuda")
    sil.matmul_batch(x, [(block.dev[i], y)])
    torch.cuda.synchronize()
    return y.cpu().numpy()
