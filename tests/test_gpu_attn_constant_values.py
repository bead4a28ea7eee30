"""Value rows whose groups are constant: their scales are 0 and the biases carry everything, at any size
that the cache holds (bounds of test_gpu_attn.py)."""
import pytest

from test_gpu_attn import Setup

pytestmark = pytest.mark.gpu

HEADS = [(16, 2, 256), (32, 8, 128), (32, 4, 64)]
LARGEST = 8.2e34  # below 2^116


def n_rows(G, form):
    return {"token": 1, "draft": 3, "chunk": 40, "prepared": -(-9 * 128 // G)}[form]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("size", [1e-30, 1.0, 1e10, -1e30, LARGEST])
@pytest.mark.parametrize("form", ["token", "draft", "chunk", "prepared"])
def test_constant_rows(Hq, Hkv, D, size, form):
    n = n_rows(Hq // Hkv, form)

    def alive(s):
        s.v.fill_(size)
    s = Setup(Hq, Hkv, D, 32, [n, n], [n, n + 700], seed=1, alive=alive)
    s.check(s.forward())
    s.check(s.forward(max_kv_len=1 << 17))


@pytest.mark.parametrize("form", ["token", "chunk"])
def test_constant_groups_beside_ordinary_ones(form):
    n = n_rows(8, form)

    def alive(s):
        s.v[:, :, :64] = 300.0
        s.v[:, :, 64:128] = -1e4
    s = Setup(16, 2, 256, 64, [n], [n + 900], seed=3, alive=alive)
    s.check(s.forward())
