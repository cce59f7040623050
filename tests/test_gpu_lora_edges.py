"""lora_add where its parts meet: formula, tolerance and helpers are those of
test_gpu_lora.py."""
import pytest
import torch

from test_gpu_lora import DEV, case, check, mxg  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R", [16, 32, 64, 128])
@pytest.mark.parametrize("sizes", [(5, 20, 3, 17, 1, 18), (20, 5, 39), (1, 63), (40, 1, 23),
                                   (16, 17, 16, 15)])
def test_lora_groups_of_few_and_of_many_tokens_in_turn(mxg, sizes, R):
    """So many blocks that a cluster takes several of a block's groups: their
    activations come by 16-byte copies (up to 16 tokens) and by boxes or
    gathers (more), one behind the other through the same slots."""
    M, K, N, L = 1024, 4104, 136, 7
    g = torch.Generator().manual_seed(len(sizes) + R)
    one = torch.cat([torch.full((n,), i) for i, n in enumerate(sizes)])
    for order in ("runs", "scattered"):
        index = torch.cat([(one if order == "runs" else one[torch.randperm(64, generator=g)])
                           for _ in range(M // 64)])
        x, a, b, index, y, s = case(M, K, N, R, L, seed=R, index=index)
        want = mxg.lora_add(x, a, b, index, y, scales=s)
        check(want, x, a, b, index, y, s)
        for _ in range(5):
            assert torch.equal(mxg.lora_add(x, a, b, index, y, scales=s), want)
