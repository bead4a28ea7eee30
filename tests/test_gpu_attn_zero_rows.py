"""Query rows and keys of zeros, or so small that the units of their scores vanish in fp32: every score
is 0, and the output the mean of the values that the row sees (bounds of test_gpu_attn.py).  Contexts
end inside a step of 64 tokens and inside a record of 16, or with either."""
import pytest

from test_gpu_attn import DEV, Setup, gen, randn

pytestmark = pytest.mark.gpu

HEADS = [(16, 2, 256), (32, 8, 128), (32, 4, 64)]
ENDS = [1, 16, 48, 49, 64]


def queries(T, Hq, D, seed, tiny=None):
    """Ordinary rows with zero ones, or ones of size `tiny`, among them."""
    q = randn(gen(seed), T, Hq, D) * 1.5
    q[::3] *= tiny or 0.0
    q[:, ::5] *= tiny or 0.0
    return q.bfloat16()


def n_rows(G, form):
    return {"token": 1, "chunk": 40, "prepared": -(-9 * 128 // G)}[form]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("end", ENDS)
@pytest.mark.parametrize("form", ["token", "chunk", "prepared"])
def test_zero_queries_give_the_mean(Hq, Hkv, D, end, form):
    n = n_rows(Hq // Hkv, form)
    L = (n // 64 + 3) * 64 + end
    s = Setup(Hq, Hkv, D, 64, [n, n], [L, L + 64], seed=end, q=queries(2 * n, Hq, D, end))
    s.check(s.forward())


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("form", ["token", "chunk", "prepared"])
def test_zero_queries_over_zero_keys_give_the_mean(Hq, Hkv, D, form):
    import torch
    n = n_rows(Hq // Hkv, form)

    def alive(s):
        s.k.zero_()
    s = Setup(Hq, Hkv, D, 32, [n], [n + 100], seed=3, alive=alive,
              q=torch.zeros(n, Hq, D, dtype=torch.bfloat16, device=DEV))
    s.check(s.forward())


@pytest.mark.parametrize("form", ["token", "chunk", "prepared"])
@pytest.mark.parametrize("tiny", [1e-10, 1e-20, 1e-30, 1e-38])
def test_tiny_queries_give_the_mean(form, tiny):
    n = n_rows(8, form)
    s = Setup(16, 2, 256, 64, [n], [n + 177], seed=4, q=queries(n, 16, 256, 4, tiny))
    s.check(s.forward())


@pytest.mark.parametrize("form", ["token", "chunk", "prepared"])
@pytest.mark.parametrize("scale", [1e-12, 1e-30])
def test_tiny_softmax_scales_give_the_mean(form, scale):
    n = n_rows(8, form)
    s = Setup(16, 2, 256, 64, [n], [n + 177], seed=5, scale=scale, q=queries(n, 16, 256, 5))
    s.check(s.forward())
