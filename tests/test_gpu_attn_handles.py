"""Handles side by side: one made later, of fewer requests and another head size, changes nothing for
one made before (bounds of test_gpu_attn.py)."""
import pytest

import sparse_moe_02_gb300 as moe
from test_gpu_attn import Setup, check_plan, plan_reference, run_plan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 2, 256), (32, 8, 128), (32, 4, 64)])
@pytest.mark.parametrize("B", [64, 1024])
def test_a_small_handle_leaves_a_large_one_alone(Hq, Hkv, D, B):
    import numpy as np
    rows = -(-9 * 128 * Hkv // Hq)
    forms = {"cut": ([1] * B, [2000 + b % 7 for b in range(40)] + [5] * (B - 40)),
             "chunk": ([40] + [1] * (B - 1), [900] + [1 + b % 70 for b in range(B - 1)]),
             "prepared": ([rows] + [0] * (B - 1), [rows + 300] + [0] * (B - 1))}
    large = [Setup(Hq, Hkv, D, 64, new, kv, seed=B + i) for i, (new, kv) in enumerate(forms.values())]
    small = [moe.PagedAttention(1, 1, d, 16, 1, 1) for d in (64, 128, 256)]
    for s, form in zip(large, forms):
        s.check(s.forward(max_kv_len=1 << 17) if form == "cut" else s.forward())
    table, free = np.full((B, 3), -1, np.int32), list(range(2 * B))
    new = [1 + b % 100 for b in range(B)]
    T = sum(new)
    check_plan(run_plan(large[0].attn, table, [0] * B, new, free, 0, T),
               plan_reference(table, [0] * B, new, free, 0, T, 64))
    for a in small:
        a.close()
