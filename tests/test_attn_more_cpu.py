"""What PagedAttention's calls for windows and drafted trees refuse before they call the library, with the
stand-ins of test_attn_binding_cpu.py (no GPU)."""
import types

import pytest
import torch

import sparse_moe_02_gb300 as moe
from test_attn_binding_cpu import (B, D, HKV, HQ, T, W, Tensor, attn, bf16, cache, i32,  # noqa: F401
                                   refused)

WORDS = 2


def arguments():
    """The calls, every tensor given."""
    q, k, w = (lambda: bf16(T, HQ, D)), (lambda: bf16(T, HKV, D)), (lambda: bf16(D))
    return {
        "tree_plan": dict(parents=i32(T), q_offsets=i32(B + 1), kv_lens=i32(B), max_q_len=2,
                          positions=i32(T), masks=i32(T, WORDS)),
        "qk_norm_rope_append": dict(q=q(), k=k(), v=k(), positions=i32(T), slots=i32(T),
                                    q_weight=w(), k_weight=w(),
                                    cos_sin=Tensor(torch.float32, 10, 32), cache=cache(),
                                    q_out=q()),
        "forward": dict(q=q(), cache=cache(), block_table=i32(B, W), q_offsets=i32(B + 1),
                        kv_lens=i32(B), max_q_len=2, max_kv_len=20, out=q(), window=8, sinks=2,
                        masks=i32(T, WORDS)),
        "accept": dict(cache=cache(), block_table=i32(B, W), ctx_lens=i32(B), paths=i32(B, 3),
                       path_lens=i32(B)),
    }


TENSORS = [(call, name) for call, args in arguments().items() for name in args
           if not name.startswith("max") and name not in ("window", "sinks")]


def test_calls_in_order_reach_the_library(attn):  # noqa: F811
    for call, args in arguments().items():
        getattr(attn, call)(**args)
    assert attn._lib.calls == ["attn_tree_plan", "attn_qk_norm_rope_append",
                               "attn_kv4_forward_masked", "attn_kv4_accept"]


@pytest.mark.parametrize("more,name", [
    (dict(window=0, sinks=0, masks=None), "attn_kv4_forward"),
    (dict(window=0, sinks=3, masks=None), "attn_kv4_forward_masked"),
    (dict(window=5, sinks=0, masks=None), "attn_kv4_forward_masked"),
    (dict(window=-5, sinks=0, masks=None), "attn_kv4_forward_masked"),  # (refused there)
    (dict(window=0, sinks=0), "attn_kv4_forward_masked"),
])
def test_views_choose_the_call(attn, more, name):  # noqa: F811
    attn.forward(**dict(arguments()["forward"], **more))
    assert attn._lib.calls == [name]


@pytest.mark.parametrize("call,name", TENSORS)
def test_tensors_of_another_device_are_refused(attn, call, name):  # noqa: F811
    args = arguments()[call]
    t = args[name].data if name == "cache" else args[name]
    t.index, t.device = 1, torch.device("cuda", 1)
    refused(attn, call, args)


@pytest.mark.parametrize("call,name", TENSORS)
def test_tensors_of_another_type_or_size_are_refused(attn, call, name):  # noqa: F811
    if name == "cache":
        args = arguments()[call]
        args[name].layout = (1, 2, 3, 4)
        refused(attn, call, args)
        return
    for dtype, shape in ((torch.float64, None), (None, (7,)), (None, (1, 1, 1, 1))):
        args = arguments()[call]
        t = args[name]
        if name == "cos_sin" and dtype is None and len(shape) == 2:
            continue
        args[name] = Tensor(dtype or t.dtype, *(shape or t.shape))
        with pytest.raises((moe.MoeError, ValueError, IndexError)):
            getattr(attn, call)(**args)
        assert not attn._lib.calls


@pytest.mark.parametrize("call", arguments())
def test_calls_with_another_device_or_stream_are_refused(attn, call):  # noqa: F811
    attn.now = 1
    refused(attn, call, arguments()[call])
    attn.now = 0
    stream = types.SimpleNamespace(cuda_stream=0, device_index=1)
    refused(attn, call, dict(arguments()[call], stream=stream))


@pytest.mark.parametrize("call,name", [(c, n) for c, n in TENSORS
                                       if n not in ("out", "q_out", "cos_sin", "masks")
                                       and (c, n) != ("tree_plan", "positions")])
def test_missing_tensors_are_refused(attn, call, name):  # noqa: F811
    # (outputs that are None are allocated, no masks and no rotation are forms of the calls)
    refused(attn, call, dict(arguments()[call], **{name: None}))


def test_the_norm_and_the_rotation_may_be_left_out(attn):  # noqa: F811
    args = arguments()["qk_norm_rope_append"]
    attn.qk_norm_rope_append(**dict(args, q_weight=None, k_weight=None))
    attn.qk_norm_rope_append(**dict(args, positions=None, cos_sin=None))
    assert attn._lib.calls == ["attn_qk_norm_rope_append"] * 2


def test_null_handles_are_refused():
    A = 0x100000  # never dereferenced
    bad = moe.MOE_ERR_INVALID_ARG
    assert moe.attn_tree_plan(None, A, A, A, 1, 1, 1, A, A, 1, None) == bad
    assert moe.attn_qk_norm_rope_append(None, A, 4096, A, 512, A, 512, A, A, A, A, 1e-6, A, 8, 64, 0,
                                        1, A, 4096, A, None) == bad
    assert moe.attn_kv4_forward_masked(None, A, 4096, A, A, 4, A, A, 1, 1, 1, 1, 8, 1, A, 1, A, 4096,
                                       None) == bad
    assert moe.attn_kv4_accept(None, A, A, 4, A, A, 1, A, 1, None) == bad
