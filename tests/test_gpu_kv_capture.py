"""The example's capture() runs its first step behind what the caller's stream still has to do."""
import pytest

from test_gpu_kv_decode import example  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "q8"])
def test_capture_waits_for_the_current_stream(example, cache):  # noqa: F811
    import torch
    block = example.AttentionBlock(n_in=256, heads=8, kv_heads=2, dim=64, n_seq=3, page=16, pages=60, cache=cache)
    gen = torch.Generator(device="cuda").manual_seed(2)
    block.prompt(torch.randn((58, 256), generator=gen, device="cuda"), [40, 1, 17])
    x = torch.randn((3, 256), generator=gen, device="cuda")
    block.x.copy_(x)
    block.step()  # the step that capture() runs first, and takes back
    want = block.out.clone()
    import shared_input_linear_gb300 as sil
    sil.kv_extend(block.lens, -block.one, block.table, block.ring, block.cursor, block.page, block.slots)
    block.x.zero_()
    block.out.zero_()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # some 10 ms
    block.x.copy_(x)
    graph = block.capture()
    assert torch.equal(block.out, want)
    assert block.lens.tolist() == [40, 1, 17]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(block.out, want) and block.lens.tolist() == [41, 2, 18]
