"""The attention step as it is used: examples/attention_step.py, prompts and single tokens through one
layer, against the same rows as one prompt."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("prompts,tokens", [([3], 1), ([70, 1, 130], 4)])
def test_steps_equal_one_prompt(prompts, tokens):
    """The same cached rows and queries through different kernels and splits.  Each side lies
    within 2^-8 |o| + 2^-10 max|v| of the formula (one bf16 rounding, f16 values and weights), and
    cached values, projections of unit rows by weights of variance 1 / hidden, stay below 8."""
    import torch
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import attention_step
    finally:
        sys.path.pop(0)
    lines = []
    steps, replay, us = attention_step.run(prompts, tokens, hidden=512, inner=128,
                                           report=lines.append)
    assert len(lines) == 2 and (tokens == 1 or us > 0)
    for n, s, r in zip(prompts, steps, replay):
        assert s.shape == r.shape == (n + tokens, 16, 256)
        assert torch.isfinite(r).all() and r.abs().max() > 0.1
        bound = 2 * (2.0 ** -8 * r.double().abs() + 2.0 ** -10 * 8)
        assert ((s.double() - r.double()).abs() <= bound).all()


def test_a_cache_of_another_shape_is_refused():
    import torch
    import sparse_moe_02_gb300 as moe
    a = moe.PagedAttention(16, 2, 256, 64, 4, max_requests=1)
    small = moe.PagedAttention(16, 2, 256, 64, 3, max_requests=1).new_cache()
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = torch.zeros(1, 2, 256, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, 16, 256, dtype=torch.bfloat16, device="cuda")
    offs = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for call in (lambda: a.append(kv, kv, slots, small), lambda: a.read(slots, small),
                 lambda: a.forward(q, small, slots.view(1, 1), offs, offs[1:], 1, 64)):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == moe.MOE_ERR_INVALID_ARG
    assert a.device_error() == moe.MOE_OK
