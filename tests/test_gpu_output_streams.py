"""Outputs that a call allocates belong to the stream that it works on: memory that earlier work of
another stream still uses is not among them, and once freed they go back to that stream."""
import pytest

import sparse_moe_02_gb300 as moe
from test_gpu_attn import Setup, ints

pytestmark = pytest.mark.gpu


def stream_of(t):
    """The stream that the allocator keeps t's memory for."""
    import torch
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's memory")


@pytest.fixture
def side():
    import torch
    torch.cuda.synchronize()
    yield torch.cuda.Stream()
    torch.cuda.synchronize()


def outputs(s, stream):
    import torch
    a, n = s.attn, len(s.new)
    w = torch.ones(s.D, dtype=torch.bfloat16, device="cuda")
    ctx, new, free, cur = ints([0] * n), ints([1] * n), ints([0, 1]), ints([0])
    k = s.k[:s.T].contiguous()
    torch.cuda.synchronize()
    out = [*a.plan(s.table.clone(), ctx, new, free, cur, T=n, stream=stream),
           *a.qk_norm_rope(s.q, k, None, w, w, None, stream=stream),
           *a.read(s.slots, s.cache, stream=stream), s.forward(stream=stream)]
    torch.cuda.synchronize()
    return out


def test_attention_outputs(side):
    import torch
    s = Setup(16, 2, 256, 64, [1, 1], [100, 70], seed=1)
    here = outputs(s, None)
    there = outputs(s, side)
    own = torch.cuda.current_stream().cuda_stream
    assert [stream_of(t) for t in here] == [own] * len(here)
    assert [stream_of(t) for t in there] == [side.cuda_stream] * len(there)
    for a, b in zip(here, there):
        assert torch.equal(a, b)
    # under a current stream of their own they need no argument
    with torch.cuda.stream(side):
        inside = outputs(s, None)
    assert [stream_of(t) for t in inside] == [side.cuda_stream] * len(inside)
    # given ones are used as they are
    o = torch.empty_like(s.q)
    torch.cuda.synchronize()
    assert s.forward(out=o, stream=side) is o
    torch.cuda.synchronize()
    assert torch.equal(o, here[-1])


def test_ffn_outputs(side):
    import torch
    g = torch.Generator("cuda").manual_seed(0)
    d, f = 512, 128
    shapes = dict(w_router=(256, d), w_gate=(256, f, d), w_up=(256, f, d), w_down=(256, d, f),
                  ws_gate=(f, d), ws_up=(f, d), ws_down=(d, f))
    layer = moe.MoeLayer({k: (torch.randn(*v, generator=g, device="cuda") * v[-1] ** -0.5).bfloat16()
                          for k, v in shapes.items()}, 16)
    x = torch.randn(16, d, generator=g, device="cuda").bfloat16()
    torch.cuda.synchronize()
    y, r = layer.forward(x), layer.route(x)
    torch.cuda.synchronize()
    y2, r2 = layer.forward(x, stream=side), layer.route(x, stream=side)
    torch.cuda.synchronize()
    assert stream_of(y2) == side.cuda_stream and torch.equal(y, y2)
    for name, t in r2.items():
        assert stream_of(t) == side.cuda_stream and torch.equal(t, r[name]), name
    layer.close()
