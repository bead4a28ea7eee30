"""Tokens whose values differ by more than fp32's exponents reach, zero values among them: each still
counts in the softmax sum with its own weight (bounds of test_gpu_attn.py, whose second term allows for
what is lost of the small values themselves)."""
import pytest

from test_gpu_attn import Setup

pytestmark = pytest.mark.gpu

HEADS = [(16, 2, 256), (32, 8, 128), (32, 4, 64)]


def n_rows(G, form):
    return {"token": 1, "draft": 3, "chunk": 40, "prepared": -(-9 * 128 // G)}[form]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("large,small", [(1e10, 0.0), (1e30, 0.0), (1e30, 1e-30), (1e20, 1e-20)])
@pytest.mark.parametrize("large_first", [False, True])
@pytest.mark.parametrize("form", ["token", "draft", "chunk", "prepared"])
def test_runs_of_large_and_small_values(Hq, Hkv, D, large, small, large_first, form):
    # runs that fill records, steps and a good part of a context; the larger half has the weight of
    # its tokens, so the outputs are near half of a mean of large values
    n = n_rows(Hq // Hkv, form)
    L = n + 900

    def alive(s):
        run = [16, 100, 300][n % 3]
        for i, at in enumerate(range(0, L, run)):
            s.v[at:at + run] *= large if (i % 2 == 0) == large_first else small
    s = Setup(Hq, Hkv, D, 64, [n], [L], seed=2, alive=alive)
    s.check(s.forward())


@pytest.mark.parametrize("form", ["token", "prepared"])
@pytest.mark.parametrize("constant", [False, True])
@pytest.mark.parametrize("large_first", [False, True])
def test_contexts_that_blocks_share(form, constant, large_first):
    # whole parts of a shared context hold nothing but zeros
    n = n_rows(8, form)
    L = 20000

    def alive(s):
        if constant:
            s.v.fill_(1.0)
        s.v *= 1e30
        half = slice(L // 3, L) if large_first else slice(0, 2 * L // 3)
        s.v[half] = 0.0
    s = Setup(16, 2, 256, 64, [n], [L], seed=3, alive=alive, q_gain=0.0 if constant else 1.5)
    s.check(s.forward())


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("form", ["token", "chunk", "prepared"])
def test_constant_values_of_either_sign_and_none(Hq, Hkv, D, form):
    n = n_rows(Hq // Hkv, form)

    def alive(s):
        s.v.fill_(1e30)
        s.v[::3] = -2.5e29
        s.v[100:200] = 0.0
    s = Setup(Hq, Hkv, D, 64, [n], [n + 900], seed=4, alive=alive)
    s.check(s.forward())
