"""Host-side checks of the attention step's C ABI that need no GPU: every function of
include/attn.h is exported and bound, and invalid arguments are refused before any CUDA call."""
import ctypes
import os
import re

import pytest

import sparse_moe_02_gb300 as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_library_exports_every_declared_function():
    src = open(os.path.join(ROOT, "include", "attn.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    declared = set(re.findall(r"^\s*int\s+(attn_\w+)\s*\(", src, re.M))
    assert declared == set(moe.ATTN_EXPORTS)
    for fn in declared:
        assert hasattr(moe.lib(), fn) and callable(getattr(moe, fn))


def _cfg(**kw):
    base = dict(n_q_heads=16, n_kv_heads=2, head_dim=256, page_size=64, n_pages=10,
                max_requests=8, scale=0.0)
    base.update(kw)
    return moe.attn_config(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(n_q_heads=0), moe.MOE_ERR_INVALID_ARG),
    (dict(n_kv_heads=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(n_pages=0), moe.MOE_ERR_INVALID_ARG),
    (dict(max_requests=0), moe.MOE_ERR_INVALID_ARG),
    (dict(scale=-1.0), moe.MOE_ERR_INVALID_ARG),
    (dict(scale=float("nan")), moe.MOE_ERR_INVALID_ARG),
    (dict(scale=float("inf")), moe.MOE_ERR_INVALID_ARG),
    (dict(n_q_heads=15), moe.MOE_ERR_UNSUPPORTED),
    (dict(n_q_heads=34), moe.MOE_ERR_UNSUPPORTED),
    (dict(n_q_heads=256, n_kv_heads=256), moe.MOE_ERR_UNSUPPORTED),
    (dict(head_dim=96), moe.MOE_ERR_UNSUPPORTED),
    (dict(page_size=48), moe.MOE_ERR_UNSUPPORTED),
    (dict(page_size=8), moe.MOE_ERR_UNSUPPORTED),
    (dict(n_pages=1 << 25), moe.MOE_ERR_UNSUPPORTED),
    (dict(max_requests=4097), moe.MOE_ERR_UNSUPPORTED),
])
def test_create_refuses_bad_config(kw, status):
    st, h = moe.attn_create(_cfg(**kw))
    assert st == status and not h.value


def test_null_handles_are_refused():
    L = moe.lib()
    assert L.attn_create(None, None) == moe.MOE_ERR_INVALID_ARG
    assert L.attn_create(ctypes.byref(_cfg()), None) == moe.MOE_ERR_INVALID_ARG
    A = 0x100000  # never dereferenced
    c = A
    assert moe.attn_destroy(None) == moe.MOE_OK
    assert moe.attn_get_device_error(None, None) == moe.MOE_ERR_INVALID_ARG
    assert moe.attn_plan(None, A, 4, A, A, 1, A, 1, A, 1, A, A, A, A, A, None) == \
        moe.MOE_ERR_INVALID_ARG
    assert moe.attn_qk_norm_rope(None, A, 4096, A, 512, A, A, A, 1e-6, A, 8, 64, 0, 1, A, 4096, A,
                                 512, None) == moe.MOE_ERR_INVALID_ARG
    assert moe.attn_kv4_append(None, A, 512, A, 512, A, 1, c, None) == moe.MOE_ERR_INVALID_ARG
    assert moe.attn_kv4_read(None, c, A, 1, A, 512, A, 512, None) == moe.MOE_ERR_INVALID_ARG
    assert moe.attn_kv4_forward(None, A, 4096, c, A, 4, A, A, 1, 1, 1, 1, A, 4096, None) == \
        moe.MOE_ERR_INVALID_ARG


def test_create_without_gpu_reports_cuda_error():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    st, h = moe.attn_create(_cfg())
    assert st == moe.MOE_ERR_CUDA and not h.value
    with pytest.raises(moe.MoeError):
        moe.PagedAttention(16, 2, 256, 64, 10, 8)
