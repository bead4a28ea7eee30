"""Many short prompts: row tiles of one or two steps each, several to a block, whose softmax runs ahead
of the writing of the outputs (bounds of test_gpu_attn.py)."""
import numpy as np
import pytest

from test_gpu_attn import Setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 2, 256), (32, 8, 128), (32, 4, 64)])
@pytest.mark.parametrize("B,longest", [(330, 64), (1024, 16), (500, 140)])
def test_row_tiles_of_few_steps(Hq, Hkv, D, B, longest):
    import torch
    rng = np.random.default_rng(B)
    new = rng.integers(1, 17, B).tolist()  # a row tile each
    kv = [int(n + rng.integers(0, longest - 16 + 1)) for n in new]
    new[0], kv[0] = 16, longest
    s = Setup(Hq, Hkv, D, 16, new, kv, seed=B)
    got = s.forward()
    s.check(got)
    for _ in range(20):
        assert torch.equal(s.forward(), got)
    assert s.attn.device_error() == 0
