"""Tokens that a query does not see cost it nothing, whatever they hold: siblings in a tree, later drafts,
and tokens just outside a window or the first tokens, beside seen ones in the same 16-token record.

Bound: that of test_gpu_attn.py, |got - ref| <= 2^-8 |ref| + 2^-10 max|v|, with the largest value among
the tokens that the row sees (of its key/value head) only: a hidden token's weight is 0, so every rounding
that the bound counts is relative to a seen value.
"""
import pytest

from test_gpu_attn import DEV, gen, randn
from test_gpu_attn_masked import View

pytestmark = pytest.mark.gpu

HEADS = [(16, 2, 256), (32, 8, 128), (32, 4, 64)]
GAINS = [2.0 ** 12, 2.0 ** 24, 2.0 ** 100]  # of a hidden token's values
KEY_GAINS = [2.0 ** 12, 2.0 ** 60]          # of its keys


def plant(tokens, gain, keys):
    """Multiplies the rows of cached tokens (of the first request)."""
    def alive(s):
        x = s.k if keys else s.v
        more = randn(gen(9), len(tokens), s.Hkv, s.D) * gain
        x[tokens] = more.bfloat16()
    return alive


def check(s, got, without=()):
    """Rows against 64 bits, by the largest value that each sees; without: not those that see one of these
    tokens of the first request (whose scores are far beyond what the bound allows for)."""
    import torch
    ref = s.reference()
    _, v = s.cached()
    row = key = 0
    for b, (n, L) in enumerate(zip(s.new, s.kv)):
        if L == 0:
            assert not got[row:row + n].any()
            row += n
            continue
        sees = s.visible(b)
        top = v[key:key + L].abs().amax(-1)  # [tokens][heads]
        most = torch.where(sees[:, :, None], top[None], 0.0).amax(1)
        most = most.repeat_interleave(s.Hq // s.Hkv, 1)[:, :, None]
        err = (got[row:row + n].double() - ref[row:row + n]).abs()
        bad = ~(err <= 2.0 ** -8 * ref[row:row + n].abs() + 2.0 ** -10 * most)
        if b == 0 and len(without):
            bad = bad[~sees[:, without].any(1)]
            assert len(bad)
        assert not bad.any(), f"request {b}: {int(bad.sum())} of {bad.numel()}, {(err / most).max()}"
        row, key = row + n, key + L
    assert s.attn.device_error() == 0


def ancestors(parents):
    seen = []
    for i, p in enumerate(parents):
        seen.append((seen[p] if p >= 0 else set()) | {i})
    return seen


WAYS = [(gain, False) for gain in GAINS] + [(gain, True) for gain in KEY_GAINS]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("gain,keys", WAYS)
def test_single_tokens_through_a_window(Hq, Hkv, D, gain, keys):
    # the window begins at token 940, inside the record of 928 .. 943; the first tokens end at 5
    tokens = [7, 15, 930, 939]
    s = View(Hq, Hkv, D, 16, [1, 1], [1000, 300], seed=1, alive=plant(tokens, gain, keys), window=60,
             sinks=5)
    check(s, s.forward())
    check(s, s.forward(max_kv_len=1 << 20))


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("gain,keys", WAYS)
@pytest.mark.parametrize("window", [0, 60])
def test_small_trees(Hq, Hkv, D, gain, keys, window):
    # token 2 is a sibling of 1, and no other token's ancestor
    c = 500
    s = View(Hq, Hkv, D, 16, [4, 3], [c + 4, 203], seed=2, alive=plant([c + 2], gain, keys),
             seen=[ancestors([-1, 0, 0, 1]), ancestors([-1, 0, 0])], window=window, sinks=3)
    check(s, s.forward(), without=[c + 2] if keys else [])
    check(s, s.forward(max_kv_len=1 << 20), without=[c + 2] if keys else [])


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("gain,keys", WAYS)
def test_chains_of_drafts(Hq, Hkv, D, gain, keys):
    # the last draft is hidden from those before it
    L = 777
    s = View(Hq, Hkv, D, 16, [4, 2], [L, 90], seed=3, alive=plant([L - 1], gain, keys))
    check(s, s.forward(), without=[L - 1] if keys else [])
    check(s, s.forward(max_kv_len=1 << 20), without=[L - 1] if keys else [])


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_a_large_value_of_next_to_no_weight(Hq, Hkv, D):
    # seen, 2^-100 of the row's weight and less, and 2^60 times as large: what it adds is nothing
    import torch
    L, at = 400, [120, 391]
    q = torch.ones(1, Hq, D, device=DEV).bfloat16()

    def alive(s):
        s.k[at] = -200.0 / D ** 0.5
        s.v[at] = (randn(gen(9), len(at), s.Hkv, s.D) * 2.0 ** 60).bfloat16()
        s.k[[i for i in range(L) if i not in at]] *= 0.25
    s = View(Hq, Hkv, D, 16, [1], [L], seed=4, alive=alive, q=q)
    got, ref = s.forward().double(), s.reference()
    v = s.cached()[1]
    v[at] = 0.0
    assert bool(((got - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * v.abs().max()).all())


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("form", ["drafts", "chunk", "prompt"])
@pytest.mark.parametrize("zeros", [False, True])
def test_unseen_large_keys_beside_large_queries(Hq, Hkv, D, form, zeros):
    # ordinary scores of queries 2^40 times as large and keys as much smaller (or none at all beside it); the
    # last token's keys are so large that a query's unit times theirs leaves fp32
    import torch
    n = {"drafts": 4, "chunk": 40, "prompt": -(-12 * 128 * Hkv // Hq)}[form]
    L = n + 300
    q = (randn(gen(3), n, Hq, D) * 1.5 * 2.0 ** 40).bfloat16()

    def alive(s):
        s.k *= 2.0 ** -40
        if zeros:
            s.k[L - 50:L - 1] = 0.0
        plant([L - 1], 2.0 ** 110, True)(s)
    s = View(Hq, Hkv, D, 32, [n], [L], seed=8, alive=alive, q=q)
    check(s, s.forward(), without=[L - 1])
