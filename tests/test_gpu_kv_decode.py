"""The cache operators together with the matmul batches, as a decode step uses them
(examples/decode_attention.py): against the same block in 64 bits, directly and as a replayed graph."""
import importlib.util
import os

import numpy as np
import pytest

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


def _reference(block, xs, x):
    """out [n_in] of token x after the tokens xs of one sequence, in 64 bits."""
    import torch
    wq, wk, wv = (w.double() for w in block.host)
    seq = torch.cat([xs, x[None]]).double().cpu()
    q = (wq @ seq[-1]).view(block.heads, block.dim)
    k, v = ((seq @ w.T).view(len(seq), block.kv_heads, block.dim) for w in (wk, wv))
    g = block.heads // block.kv_heads
    s = torch.einsum("hd,thd->ht", q, k.repeat_interleave(g, 1)) * block.dim ** -0.5
    o = torch.einsum("ht,thd->hd", s.softmax(-1), v.repeat_interleave(g, 1))
    return block.host_o.double() @ o.reshape(-1)


@pytest.mark.parametrize("cache", ["bf16", "q8"])
@pytest.mark.parametrize("graph", [False, True])
def test_decode_block(example, cache, graph):
    import torch
    block = example.AttentionBlock(n_in=256, heads=8, kv_heads=2, dim=64, n_seq=3, page=16, pages=60, cache=cache)
    gen = torch.Generator(device="cuda").manual_seed(5)
    history = [torch.randn((n, 256), generator=gen, device="cuda") for n in (40, 1, 17)]
    block.prompt(torch.cat(history), [len(h) for h in history])
    replay = block.capture().replay if graph else block.step
    for _ in range(20):  # past the ends of pages
        block.x.copy_(torch.randn((3, 256), generator=gen, device="cuda"))
        torch.cuda.synchronize()
        replay()
        torch.cuda.synchronize()
        for r in range(3):
            want = _reference(block, history[r], block.x[r]).numpy()
            got = block.out[r].double().cpu().numpy()
            # x enters the batches as bf16 (2^-9), k and v are cached as bf16 (2^-9) or Q8 (at most 1/254 of a 32-element
            # maximum, itself 3 to 4 times the rms): each moves the result by about 1 % of its rms; six times their sum
            assert np.max(np.abs(got - want)) <= 0.06 * np.sqrt(np.mean(want ** 2)) * 3, (r, len(history[r]))
            history[r] = torch.cat([history[r], block.x[r:r + 1]])
        assert block.info.tolist()[0] == 0
    assert block.lens.tolist() == [60, 21, 37]
    free = int(block.cursor[1] - block.cursor[0])
    block.finish([0, 2])
    assert block.lens.tolist() == [0, 21, 0] and int(block.cursor[1] - block.cursor[0]) == free + 4 + 3


def test_main_runs(example, capsys):
    got = example.main(["--seqs", "4", "--prompt", "70", "--steps", "5"])
    assert got["us"] > 0 and "tokens/s" in capsys.readouterr().out
