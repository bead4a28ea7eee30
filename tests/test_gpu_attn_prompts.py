"""Prompts long enough that their contexts are formed into operands first (from eight row tiles of 128
per context on), against the plain implementation in 64 bits and the bounds of test_gpu_attn.py, and
the same contexts where they are too many to be formed."""
import math

import pytest

import sparse_moe_02_gb300 as moe
from test_gpu_attn import DEV, Setup, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,D,P", [(16, 2, 256, 64), (32, 8, 128, 16), (28, 4, 128, 32),
                                        (32, 4, 64, 256), (6, 2, 256, 16), (8, 8, 64, 64)])
def test_ragged_prompts(Hq, Hkv, D, P):
    # whole prompts, chunks behind a context, one token, none, an empty context, odd ends
    new = [1300, 1, 0, 1025, 1100, 16]
    kv = [1300, 130, 64, 1500, 2049, 0]
    s = Setup(Hq, Hkv, D, P, new, kv, seed=D + P)
    got = s.forward()
    s.check(got)
    import torch
    assert torch.equal(got, s.forward())


@pytest.mark.parametrize("n,L", [(1024, 1024), (513, 640), (700, 300), (2000, 17)])
def test_lengths_around_a_step(n, L):
    # (more queries than cached tokens: the first ones see nothing)
    s = Setup(16, 2, 256, 32, [n], [L], seed=n)
    got = s.forward()
    s.check(got)
    assert not got[:max(0, n - L)].any()


@pytest.mark.parametrize("v_gain", [1e-20, 3e3, 1e30])
def test_values_of_any_size(v_gain):
    s = Setup(16, 2, 256, 32, [600], [900], seed=3, v_gain=v_gain)
    s.check(s.forward())


def test_a_poisoned_token_reaches_exactly_the_queries_that_see_it():
    import torch

    def alive(s):
        s.k[620, 1, 3] = math.nan
        s.v[317, 0, 200] = math.inf
    n = 600
    s = Setup(16, 2, 256, 16, [n], [700], seed=4, alive=alive)
    nan = s.forward().isnan()
    assert torch.equal(nan.any(-1), nan.all(-1))
    pos = 100 + torch.arange(n, device=DEV)
    nan = nan.any(-1)
    assert torch.equal(nan[:, :8], (pos >= 317)[:, None].expand(n, 8))
    assert torch.equal(nan[:, 8:], (pos >= 620)[:, None].expand(n, 8))


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 2, 256), (32, 8, 128), (16, 4, 64)])
def test_requests_that_share_pages_beyond_the_workspace(Hq, Hkv, D):
    # twelve requests over the pages of one: more contexts than the cache's pages hold
    import torch
    n, L, B = 530, 900, 12
    s = Setup(Hq, Hkv, D, 64, [n], [L], seed=5)
    ref = s.reference()
    one = s.forward()
    s.check(one, ref)
    wide = moe.PagedAttention(Hq, Hkv, D, 64, s.n_pages, B)
    got = wide.forward(s.q.repeat(B, 1, 1), s.cache, s.table.repeat(B, 1),
                       ints([n * b for b in range(B + 1)]), ints([L] * B), n, L)
    assert wide.device_error() == moe.MOE_OK
    for b in range(B):
        s.close_to(got[n * b:n * b + n], ref)
    # and after it a batch that fits again
    assert torch.equal(s.forward(), one)


def test_pages_out_of_range_are_recorded_and_harmless():
    new, kv = [700, 600], [700, 800]
    s = Setup(16, 2, 256, 64, new, kv, seed=6)
    ref = s.reference()
    s.table[1, 3] = s.n_pages
    got = s.forward()
    assert s.attn.device_error() == moe.MOE_ERR_DEVICE
    s.close_to(got[:700], ref[:700])
    s.table[1, 3] = -7
    s.forward()
    assert s.attn.device_error() == moe.MOE_ERR_DEVICE
    s.kv_lens = ints([700, 1 << 30])  # longer than the table
    s.forward()
    assert s.attn.device_error() == moe.MOE_ERR_DEVICE
    s.kv_lens = ints([700, 0])
    got = s.forward()
    assert s.attn.device_error() == moe.MOE_OK
    s.close_to(got[:700], ref[:700])
    assert not got[700:].any()
