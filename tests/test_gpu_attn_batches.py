"""Batches of single tokens and drafts at the sizes where the way contexts are spread over the SMs
changes: a block per context (short ones, and many of like lengths), shares of equal work (the bounds
of test_gpu_attn.py)."""
import pytest

from test_gpu_attn import Setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 2, 256), (32, 8, 128), (8, 4, 64)])
@pytest.mark.parametrize("B,lo,hi", [(16, 1800, 2000), (16, 100, 2000), (19, 1990, 2000),
                                     (70, 1500, 1537), (3, 769, 900), (100, 700, 1200)])
def test_contexts_of_like_and_unlike_lengths(Hq, Hkv, D, B, lo, hi):
    kv = [lo + (hi - lo) * b // (B - 1) for b in range(B)]
    new = [1 + (b % 3 == 1) for b in range(B)]
    new[B // 2] = 0
    s = Setup(Hq, Hkv, D, 64, new, kv, seed=B + D)
    got = s.forward()
    s.check(got)
    import torch
    assert torch.equal(got, s.forward())
    # the lengths' bound is a capacity: with a large one the lengths alone decide
    s.check(s.forward(max_kv_len=1 << 17))


def test_one_long_context_among_many():
    kv = [5000] + [1600] * 60
    s = Setup(16, 2, 256, 32, [1] * 61, kv, seed=8)
    s.check(s.forward())
    s = Setup(16, 2, 256, 32, [1] * 61, kv[::-1], seed=9)
    s.check(s.forward())
