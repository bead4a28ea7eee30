"""The same as test_gpu_attn_hidden_values.py for many query rows, where cached tokens are formed into
operands that all rows share: chunks, prompts (their contexts formed once, and by each block), windows and
wide trees.

Bound: the same.  An operand has f16's 11 bits where it is 2^-14 and more; below, its rounding is half a
spacing, 2^-25.  Operands are formed with a power of two that puts a bound b of a token's entries at 2^-6, or
at up to 2^5 less where the tokens of a record differ by no more.  b is below 8 times the token's
largest entry, so the rounding is at most 2^(-25 + 6 + 5 + 3) = 2^-11 of that: weighted means of them stay
within 2^-10 of the largest seen value, and keys' within what the bound has for scores.
"""
import pytest

from test_gpu_attn import DEV, randn, gen
from test_gpu_attn_hidden_values import HEADS, ancestors, check, plant
from test_gpu_attn_masked import View

pytestmark = pytest.mark.gpu

WAYS = [(2.0 ** e, False) for e in (5, 8, 9, 12, 24, 100)] + [(2.0 ** e, True) for e in (12, 60)]


def n_prepared(G):
    return -(-12 * 128 // G)


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("gain,keys", WAYS)
def test_chunks(Hq, Hkv, D, gain, keys):
    tokens = [310, 325]
    s = View(Hq, Hkv, D, 16, [40, 3], [340, 90], seed=1, alive=plant(tokens, gain, keys))
    check(s, s.forward(), without=tokens if keys else [])


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("gain,keys", WAYS)
def test_chunks_through_a_window(Hq, Hkv, D, gain, keys):
    # 7, 15: behind the first tokens, before every window; the others before some windows, behind others
    tokens = [7, 15, 885, 890, 960]
    s = View(Hq, Hkv, D, 32, [60, 2], [1000, 70], seed=2, alive=plant(tokens, gain, keys), window=60,
             sinks=5)
    check(s, s.forward(), without=tokens if keys else [])


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("gain,keys", WAYS)
@pytest.mark.parametrize("window", [0, 60])
def test_wide_trees(Hq, Hkv, D, gain, keys, window):
    # tokens 20 and 33 have siblings and no children
    c, n, leaves = 500, 50, (20, 33)
    parents = [-1]
    for i in range(1, n):
        parents.append(max(j for j in range(i) if j not in leaves))
    tokens = [c + j for j in leaves]
    s = View(Hq, Hkv, D, 16, [n, 3], [c + n, 203], seed=3, alive=plant(tokens, gain, keys),
             seen=[ancestors(parents), ancestors([-1, 0, 0])], window=window, sinks=3)
    check(s, s.forward(), without=tokens if keys else [])


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("gain,keys", WAYS)
@pytest.mark.parametrize("window", [0, 300])
def test_prompts_over_prepared_contexts(Hq, Hkv, D, gain, keys, window):
    import torch
    n = n_prepared(Hq // Hkv)
    L = n + 900
    tokens = [100, L - n // 2, L - 9] if window else [L - n // 2, L - 9]
    s = View(Hq, Hkv, D, 64, [n], [L], seed=4, alive=plant(tokens, gain, keys), window=window, sinks=5)
    got = s.forward()
    check(s, got, without=tokens if keys else [])
    # (rows that see the keys may read NaN)
    assert torch.equal(got.nan_to_num(nan=7.0), s.forward().nan_to_num(nan=7.0))


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("gain,keys", WAYS)
def test_prompts_whose_contexts_are_formed_by_each_block(Hq, Hkv, D, gain, keys):
    # long enough to ask whether contexts are formed first, too short for it
    n = {256: 129, 128: 321, 64: 65}[D]
    L = n + 350
    tokens = [L - n // 2, L - 9]
    s = View(Hq, Hkv, D, 32, [n], [L], seed=7, alive=plant(tokens, gain, keys))
    check(s, s.forward(), without=tokens if keys else [])


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("n", [40, None])
def test_every_token_of_another_size(Hq, Hkv, D, n):
    # keys and values whose sizes jump from token to token, some of them zero: scores stay ordinary, as the
    # large keys meet small parts of the queries
    import torch
    n = n or n_prepared(Hq // Hkv)
    L = n + 300
    g = gen(11)
    q = randn(g, n, Hq, D)
    q[..., ::2] *= 2.0 ** -20

    def alive(s):
        size = 2.0 ** (torch.arange(L, device=DEV) * 7 % 21)[:, None, None].double()
        k = s.k.double()
        k[..., ::2] *= size
        s.k = k.bfloat16()
        s.v[1::3] *= 2.0 ** -12
        s.v[2::3] = 0.0
    s = View(Hq, Hkv, D, 32, [n], [L], seed=6, alive=alive, q=q.bfloat16())
    check(s, s.forward())
