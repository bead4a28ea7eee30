"""Prompt rows against the size of their own outputs, which over long contexts are far smaller than the
values: the root of the mean square error of each row (of a token and head) stays below 2^-8 of the
row's.  One bf16 rounding takes 2^-9 at most; the f16 roundings of a weight and a value are 2^-12 of its
own share each and do not add up in sign, and a sum in tensor memory over 100000 tokens (6250 additions
that truncate 2^-23 of it) drifts by less than 2^-10."""
import pytest

from test_gpu_attn import Setup

pytestmark = pytest.mark.gpu

HEADS = [(16, 2, 256), (32, 8, 128), (32, 4, 64)]


def check_rows(s):
    got, ref = s.forward().double(), s.reference()
    rel = ((got - ref).square().sum(-1) / ref.square().sum(-1)).sqrt()
    assert bool((rel < 2.0 ** -8).all()), rel.max().item()
    assert s.attn.device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("n,L", [(1500, 1500), (700, 5000), (96, 12000), (33, 3000)])
@pytest.mark.parametrize("q_gain", [0.0, 1.5])
def test_prompts(Hq, Hkv, D, n, L, q_gain):
    check_rows(Setup(Hq, Hkv, D, 64, [n], [L], seed=n, q_gain=q_gain))


@pytest.mark.parametrize("Hq,Hkv,D,n", [(16, 2, 256, 20), (16, 2, 256, 150), (8, 2, 128, 300),
                                        (8, 1, 64, 150), (4, 2, 64, 40)])
@pytest.mark.parametrize("q_gain", [0.0, 1.5])
@pytest.mark.parametrize("positive", [False, True])
def test_chunks_over_100000_tokens(Hq, Hkv, D, n, q_gain, positive):
    def alive(s):
        if positive:
            s.v.abs_()
    check_rows(Setup(Hq, Hkv, D, 64, [n], [100000], seed=n, q_gain=q_gain, alive=alive))
