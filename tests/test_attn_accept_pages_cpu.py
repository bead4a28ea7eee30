"""What PagedAttention.accept refuses where it puts pages back, before it calls the library, with the
stand-ins of test_attn_binding_cpu.py (no GPU)."""
import types

import pytest
import torch

import sparse_moe_02_gb300 as moe
from test_attn_binding_cpu import B, W, Tensor, attn, cache, i32, refused  # noqa: F401

BACK = ("kv_lens", "free_pages", "cursor")


def arguments():
    return dict(cache=cache(), block_table=i32(B, W), ctx_lens=i32(B), paths=i32(B, 3),
                path_lens=i32(B), kv_lens=i32(B), free_pages=i32(9), cursor=i32(1))


def test_pages_choose_the_call(attn):  # noqa: F811
    attn.accept(**arguments())
    attn.accept(**dict(arguments(), **{name: None for name in BACK}))
    assert attn._lib.calls == ["attn_kv4_accept_pages", "attn_kv4_accept"]


@pytest.mark.parametrize("names", [BACK[:1], BACK[1:2], BACK[2:], BACK[:2], BACK[1:]])
def test_some_of_the_plans_tensors_are_refused(attn, names):  # noqa: F811
    refused(attn, "accept", dict(arguments(), **{name: None for name in names}))


@pytest.mark.parametrize("name", BACK)
def test_tensors_of_another_device_type_or_size_are_refused(attn, name):  # noqa: F811
    args = arguments()
    args[name].index, args[name].device = 1, torch.device("cuda", 1)
    refused(attn, "accept", args)
    refused(attn, "accept", dict(arguments(), **{name: Tensor(torch.int64, *args[name].shape)}))
    if name != "free_pages":  # (a list of any length)
        refused(attn, "accept", dict(arguments(), **{name: i32(7)}))


def test_calls_with_another_device_or_stream_are_refused(attn):  # noqa: F811
    attn.now = 1
    refused(attn, "accept", arguments())
    attn.now = 0
    stream = types.SimpleNamespace(cuda_stream=0, device_index=1)
    refused(attn, "accept", dict(arguments(), stream=stream))


def test_null_handles_are_refused():
    A = 0x100000  # never dereferenced
    assert moe.attn_kv4_accept_pages(None, A, A, 4, A, A, 1, A, 1, A, A, 9, A, None) == \
        moe.MOE_ERR_INVALID_ARG
