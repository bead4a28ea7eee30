"""What PagedAttention refuses before it calls the library, with stand-ins for CUDA tensors (no GPU): every
tensor there and on the handle's device, every call with that device current."""
import types

import pytest
import torch

import sparse_moe_02_gb300 as moe

HQ, HKV, D, P, PAGES, T, B, W = 4, 2, 64, 16, 8, 3, 2, 4


class Tensor:
    """What the binding asks of a CUDA tensor."""

    def __init__(self, dtype, *shape, device=0):
        self.dtype, self.shape, self.index = dtype, torch.Size(shape), device
        self.device = torch.device("cuda", device)
        self.is_cuda = True

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 0x100000

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def stride(self, i=None):
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s) if i is None else s[i]


class Library:
    """Notes the calls that reach it."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def attn():
    a = object.__new__(moe.PagedAttention)
    a.handle, a._lib, a._device, a._torch = None, Library(), 0, torch
    a.n_q_heads, a.n_kv_heads, a.head_dim, a.page_size, a.n_pages = HQ, HKV, D, P, PAGES
    a._layout = (PAGES, HKV, P, D)
    a._bf16, a._i32, a._f32 = torch.bfloat16, torch.int32, torch.float32
    a._raw_stream = lambda device: 0
    a.now = 0
    a._current_device = lambda: a.now
    return a


def bf16(*shape):
    return Tensor(torch.bfloat16, *shape)


def i32(*shape):
    return Tensor(torch.int32, *shape)


def cache():
    c = types.SimpleNamespace(layout=(PAGES, HKV, P, D), ptr=0x100000)
    c.data = Tensor(torch.uint8, PAGES, HKV, P // 16, 18 * D)
    return c


def arguments():
    """The calls, every tensor given."""
    q, k, w = (lambda: bf16(T, HQ, D)), (lambda: bf16(T, HKV, D)), (lambda: bf16(D))
    return {
        "plan": dict(block_table=i32(B, W), ctx_lens=i32(B), new_lens=i32(B), free_pages=i32(5),
                     cursor=i32(1), q_offsets=i32(B + 1), kv_lens=i32(B), positions=i32(T),
                     slots=i32(T), cursor_out=i32(1)),
        "qk_norm_rope": dict(q=q(), k=k(), positions=i32(T), q_weight=w(), k_weight=w(),
                             cos_sin=Tensor(torch.float32, 10, 32), q_out=q(), k_out=k()),
        "append": dict(k=k(), v=k(), slots=i32(T), cache=cache()),
        "read": dict(slots=i32(T), cache=cache(), k_out=k(), v_out=k()),
        "forward": dict(q=q(), cache=cache(), block_table=i32(B, W), q_offsets=i32(B + 1),
                        kv_lens=i32(B), max_q_len=2, max_kv_len=20, out=q()),
    }


TENSORS = [(call, name) for call, args in arguments().items() for name in args
           if not name.startswith("max")]


def refused(attn, call, args):
    with pytest.raises(moe.MoeError) as e:
        getattr(attn, call)(**args)
    assert e.value.status == moe.MOE_ERR_INVALID_ARG and not attn._lib.calls


def test_calls_in_order_reach_the_library(attn):
    for call, args in arguments().items():
        getattr(attn, call)(**args)
    assert attn._lib.calls == ["attn_plan", "attn_qk_norm_rope", "attn_kv4_append",
                               "attn_kv4_read", "attn_kv4_forward"]


@pytest.mark.parametrize("call,name", TENSORS)
def test_tensors_of_another_device_are_refused(attn, call, name):
    args = arguments()[call]
    t = args[name].data if name == "cache" else args[name]
    t.index, t.device = 1, torch.device("cuda", 1)
    refused(attn, call, args)


@pytest.mark.parametrize("call", arguments())
def test_calls_with_another_device_current_are_refused(attn, call):
    attn.now = 1
    refused(attn, call, arguments()[call])
    stream = types.SimpleNamespace(cuda_stream=0, device_index=0)
    refused(attn, call, dict(arguments()[call], stream=stream))


@pytest.mark.parametrize("call", arguments())
def test_streams_of_another_device_are_refused(attn, call):
    stream = types.SimpleNamespace(cuda_stream=0, device_index=1)
    refused(attn, call, dict(arguments()[call], stream=stream))


@pytest.mark.parametrize("call,name", [(c, n) for c, n in TENSORS
                                       if not n.endswith("out") and (c, n) not in (
                                           ("qk_norm_rope", "cos_sin"), ("plan", "q_offsets"),
                                           ("plan", "kv_lens"), ("plan", "positions"),
                                           ("plan", "slots"))])
def test_missing_tensors_are_refused(attn, call, name):
    # (positions are needed for a rotation only; outputs that are None are allocated)
    refused(attn, call, dict(arguments()[call], **{name: None}))


def test_positions_may_be_missing_without_a_rotation(attn):
    attn.qk_norm_rope(**dict(arguments()["qk_norm_rope"], positions=None, cos_sin=None))
    assert attn._lib.calls == ["attn_qk_norm_rope"]


def test_a_cache_is_where_its_tensor_is():
    c = moe.Kv4Cache(2, HKV, P, D, device="cpu")
    assert c.ptr == c.data.data_ptr()
    c.data = c.data.clone()  # as after a trip to the host and back
    assert c.ptr == c.data.data_ptr()
