"""MoE layers side by side: one made later, with a smaller inner size, changes nothing for one made
before."""
import pytest

import sparse_moe_02_gb300 as moe

pytestmark = pytest.mark.gpu


def layer(d, f, seed):
    import torch
    g = torch.Generator("cuda").manual_seed(seed)
    shapes = dict(w_router=(256, d), w_gate=(256, f, d), w_up=(256, f, d), w_down=(256, d, f),
                  ws_gate=(f, d), ws_up=(f, d), ws_down=(d, f))
    w = {}
    for name, s in shapes.items():
        w[name] = torch.empty(s, dtype=torch.bfloat16, device="cuda")
        w[name].normal_(0, s[-1] ** -0.5, generator=g)
    return moe.MoeLayer(w, 8)


def test_a_smaller_layer_leaves_a_larger_one_alone():
    # hidden sizes that the streamed launch of one token does not take
    import torch
    large = layer(2176, 2048, 1)
    x = torch.randn(1, 2176, generator=torch.Generator("cuda").manual_seed(2),
                    device="cuda").bfloat16()
    want = large.forward(x)
    assert large.device_error() == moe.MOE_OK and bool(want.isfinite().all())
    small = layer(2176, 1408, 3)  # both need more shared memory than a kernel has unasked
    small.forward(x)
    assert torch.equal(large.forward(x), want)
    assert large.device_error() == moe.MOE_OK and small.device_error() == moe.MOE_OK
    small.close()
    large.close()
