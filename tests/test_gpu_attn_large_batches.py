"""Batches of more requests than the launches that cut the work have threads (384, 512 and 768), up to the
1024 of a call: tokens cut into even shares, batches that a longer request sends to the prompt kernel,
prepared and not (bounds of test_gpu_attn.py)."""
import numpy as np
import pytest

from test_gpu_attn import Setup

pytestmark = pytest.mark.gpu


def batch(B, seed, longest):
    rng = np.random.default_rng(seed)
    new = rng.integers(0, 3, B).tolist()
    kv = [int(n + x) for n, x in zip(new, np.exp(rng.uniform(0, np.log(longest), B)))]
    new[-1], kv[-1] = 2, longest
    return new, kv


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 256), (8, 2, 128), (4, 4, 64)])
@pytest.mark.parametrize("B", [385, 513, 769, 1024])
def test_tokens(Hq, Hkv, D, B):
    new, kv = batch(B, B, 3000)
    s = Setup(Hq, Hkv, D, 16, new, kv, seed=B)
    s.check(s.forward())
    s.check(s.forward(max_kv_len=1 << 17))


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 256), (8, 2, 128), (4, 4, 64)])
@pytest.mark.parametrize("B", [385, 513, 769, 1024])
@pytest.mark.parametrize("at", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("prepared", [False, True])
def test_prompts(Hq, Hkv, D, B, at, prepared):
    new, kv = batch(B, B, 60)
    b = int(at * (B - 1))
    n = -(-128 * Hkv // Hq) * (40 if prepared else 3) + 3
    if prepared:  # few contexts beside it, so that row tiles to a context are many
        new = [0] * B
        new[b // 2], kv[b // 2] = 1, 50
    new[b], kv[b] = n, n + 700
    s = Setup(Hq, Hkv, D, 16, new, kv, seed=B)
    s.check(s.forward())
