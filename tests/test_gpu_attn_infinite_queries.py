"""Query rows with an entry that is not finite read NaN where they see a token, whatever the signs of the
keys, and zeros where they see none; the other rows are the definition's (bounds of
test_gpu_attn.py)."""
import math

import pytest

from test_gpu_attn import DEV, Setup, gen, randn

pytestmark = pytest.mark.gpu

HEADS = [(16, 2, 256), (32, 8, 128), (32, 4, 64)]


class Case(Setup):
    def cached(self):
        """As Setup's, with the definition's division: torch divides by a Python number through its
        reciprocal, which takes another step for one group in 300 of rows of one sign (their ranges
        often are 15 times a number halfway between two of bf16)."""
        import torch
        ks = []
        for x in (self.k, self.v):
            g = x.float().unflatten(-1, (-1, 64))
            lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
            step = ((hi - lo) / torch.full_like(hi, 15.0)).bfloat16().float()
            code = torch.where(step > 0, ((g - lo) / step).round(), 0.0).clamp(0, 15)
            ks.append((step.double() * code.double() + lo.double()).flatten(-2))
        return ks


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("entry", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("sign", [1, -1, 0])
@pytest.mark.parametrize("form", ["token", "draft", "chunk", "prepared"])
def test_rows_that_are_not_finite(Hq, Hkv, D, entry, sign, form):
    import torch
    n = {"token": 1, "draft": 3, "chunk": 40, "prepared": -(-9 * 128 * Hkv // Hq)}[form]
    L = [n, n + 500, max(1, n // 2)]  # the last one's first queries see nothing

    def alive(s):
        if sign:  # one sign in every channel: scores are all +inf or all -inf
            s.k.abs_()
            s.k.mul_(sign)
    q = randn(gen(1), 3 * n, Hq, D).bfloat16()
    q[:, 1, 7] = entry
    q[:, Hq - 1, D - 1] = entry
    s = Case(Hq, Hkv, D, 64, [n] * 3, L, seed=2, q=q, alive=alive)
    got = s.forward()
    bad = torch.zeros(Hq, dtype=torch.bool, device=DEV)
    bad[1] = bad[Hq - 1] = True
    sees = torch.ones(3 * n, dtype=torch.bool, device=DEV)
    sees[2 * n:2 * n + n - L[2]] = False
    assert bool(got[sees][:, bad].isnan().all())
    assert not bool(got[~sees].any())
    s.q = torch.where(bad[None, :, None], torch.zeros_like(q), q)
    s.close_to(got[:, ~bad], s.reference()[:, ~bad])
    assert s.attn.device_error() == 0
