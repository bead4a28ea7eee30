"""Prepared contexts over and over: every block of the launch that forms them decides alike whether it
does, and forms all of its steps, so calls that alternate between two batches in one workspace give
each batch its own bits (bounds of test_gpu_attn.py)."""
import pytest

from test_gpu_attn import Setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 2, 256), (32, 8, 128), (32, 4, 64)])
@pytest.mark.parametrize("B", [1, 33, 511, 512])
def test_batches_that_take_turns_in_the_workspace(Hq, Hkv, D, B):
    # the number of requests sets which of the block's threads holds the batch's total
    import torch
    rows = 8 * 128 * Hkv // Hq  # of new tokens: eight row tiles
    both = []
    for seed in (1, 2):
        new = [2 * rows + 40 * seed] + [0] * (B - 1)
        s = Setup(Hq, Hkv, D, 64, new, [new[0] + 700 * seed] + [0] * (B - 1), seed=seed, n_pages=64)
        both.append(s)
    both[1].attn = both[0].attn
    want = [s.forward() for s in both]
    for s, w in zip(both, want):
        s.check(w)
    for _ in range(40):
        got = [s.forward() for s in both]
        for g, w in zip(got, want):
            assert torch.equal(g, w)
    assert both[0].attn.device_error() == 0
