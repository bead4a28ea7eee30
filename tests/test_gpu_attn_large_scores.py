"""Scores far beyond what a softmax tells apart.  Below 2^23 (in units of log 2) outputs are the
definition's; larger ones may read NaN, and from 2^28 on they do: never zeros, never something else
(bounds of test_gpu_attn.py).  Rows and keys are constant, with a power of two in the query and the
key's eight bits kept by every kernel, so scores are exact and grow, or fall, with the token."""
import pytest

from test_gpu_attn import DEV, Setup

pytestmark = pytest.mark.gpu

HEADS = [(16, 2, 256), (32, 8, 128), (32, 4, 64)]


def setup(Hq, Hkv, D, q_exp, k_exp, sign, form):
    # the largest score lies between 2^(x + 3.5) and 2^(x + 5.6), x = q_exp + k_exp
    import torch
    n = {"token": 1, "draft": 3, "chunk": 40, "prepared": -(-9 * 128 * Hkv // Hq)}[form]
    L = n + 2000

    def alive(s):
        key = sign * (1 + torch.arange(L, device=DEV) / L)
        s.k[:] = (key * 2.0 ** k_exp).bfloat16()[:, None, None]
    q = torch.full((n, Hq, D), 2.0 ** q_exp, device=DEV).bfloat16()
    q[:, 1::2] = 0.5  # rows beside them are ordinary ones
    return Setup(Hq, Hkv, D, 64, [n], [L], seed=3, q=q, alive=alive)


FORMS = ["token", "draft", "chunk", "prepared"]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("q_exp,k_exp", [(10, 5), (16, 0), (50, -33), (0, 17), (-20, 37)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("form", FORMS)
def test_the_largest_scores_in_range(Hq, Hkv, D, q_exp, k_exp, sign, form):
    s = setup(Hq, Hkv, D, q_exp, k_exp, sign, form)
    got, ref = s.forward(), s.reference()
    s.close_to(got[:, ::2], ref[:, ::2])
    if k_exp <= 5:  # (the ordinary rows' scores are in range)
        s.close_to(got[:, 1::2], ref[:, 1::2])


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("q_exp,k_exp", [(20, 5), (40, 0), (120, -20), (126, -60), (60, 40)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("form", FORMS)
def test_scores_beyond_the_range_read_nan(Hq, Hkv, D, q_exp, k_exp, sign, form):
    s = setup(Hq, Hkv, D, q_exp, k_exp, sign, form)
    got = s.forward()
    assert bool(got[:, ::2].isnan().all())
    if k_exp <= 5:  # (the ordinary rows' scores are in range)
        s.close_to(got[:, 1::2], s.reference()[:, 1::2])
