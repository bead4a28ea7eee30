"""The same call gives the same bits, whatever ran before it: single tokens, drafts, trees and chunks, with
windows and without, on blocks that share contexts."""
import random

import pytest

from test_gpu_attn_masked import View, drafted

pytestmark = pytest.mark.gpu

HEADS = [(16, 2, 256), (32, 8, 128), (32, 4, 64)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 4)])
@pytest.mark.parametrize("form", ["tokens", "drafts", "small trees", "wide trees", "chunks"])
def test_calls_repeat(Hq, Hkv, D, window, sinks, form):
    import torch
    rng = random.Random(5)
    most = {"tokens": 1, "drafts": 4, "small trees": 4, "wide trees": 60, "chunks": 200}[form]
    new = [most] + [rng.randint(1, most) for _ in range(6)]
    kv = [n + rng.randint(0, 3000) for n in new]
    seen = [drafted(n, rng) for n in new] if "trees" in form else None
    s = View(Hq, Hkv, D, 32, new, kv, seed=1, window=window, sinks=sinks, seen=seen)
    # the same object's other call, of other lengths, leaves its own partial results and parts
    q, offsets, lens = s.q[:3], s.q_offsets[:4].clamp(max=3), s.kv_lens[:3]
    first = s.forward()
    s.check(first)
    for _ in range(3):
        s.attn.forward(q, s.cache, s.table[:3], offsets, lens, 3, max(kv))
        assert torch.equal(s.forward(), first)
