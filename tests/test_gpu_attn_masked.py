"""Attention through a window with first tokens and of drafted trees (attn_kv4_forward_masked) against a
plain implementation in 64 bits, with the bounds of test_gpu_attn.py: the arithmetic is the same, only
fewer tokens are seen."""
import math
import random

import numpy as np
import pytest

import sparse_moe_02_gb300 as moe
from test_gpu_attn import DEV, HEADS, LENGTHS, Setup, gen, ints

pytestmark = pytest.mark.gpu


class View(Setup):
    """Requests whose queries see part of their context: a window with first tokens (window 0: none),
    and, with `seen` (for each request the set of drafted tokens that each token sees), a tree."""

    def __init__(self, *args, window=0, sinks=0, seen=None, words=None, **kw):
        super().__init__(*args, **kw)
        import torch
        self.window, self.sinks, self.seen, self.masks = window, sinks, seen, None
        if seen is not None:
            words = words or -(-max(self.new + [1]) // 32)
            bits = np.zeros((self.T, words), np.uint32)
            row = 0
            for tree in seen:
                for mine in tree:
                    for j in mine:
                        bits[row, j // 32] |= np.uint32(1 << j % 32)
                    row += 1
            self.masks = torch.from_numpy(bits.view(np.int32)).to(DEV)

    def visible(self, b):
        """[new tokens][cached tokens] of request b."""
        import torch
        n, L = self.new[b], self.kv[b]
        c = L - n
        t = torch.arange(L)
        if self.seen is None:
            pos = c + torch.arange(n)
            sees = t <= pos[:, None]
        else:
            pos = torch.tensor([c + max(len([j for j in m if j < n]) - 1, 0) for m in self.seen[b]],
                               dtype=torch.long)
            sees = (t < c).repeat(n, 1)
            for i, mine in enumerate(self.seen[b]):
                for j in mine:
                    if 0 <= c + j < L and j < n:
                        sees[i, c + j] = True
        if self.window:
            sees &= (t < self.sinks) | (t > pos[:, None] - self.window)
        return sees.to(DEV)

    def reference(self):
        import torch
        k, v = self.cached()
        out = torch.zeros(self.T, self.Hq, self.D, dtype=torch.float64, device=DEV)
        G = self.Hq // self.Hkv
        row = key = 0
        for b, (n, L) in enumerate(zip(self.new, self.kv)):
            if n and L:
                kk = k[key:key + L].repeat_interleave(G, 1)
                vv = v[key:key + L].repeat_interleave(G, 1)
                sees = self.visible(b)
                some = sees.any(-1)
                s = torch.einsum("ihd,thd->hit", self.q[row:row + n].double(), kk) * self.scale
                s.masked_fill_(~sees, -math.inf)
                s[:, ~some] = 0.0
                p = torch.softmax(s, -1) * some[None, :, None]
                # (tokens that are not seen count for nothing, whatever they hold)
                vv = vv.masked_fill(~sees.any(0)[:, None, None], 0.0)
                out[row:row + n] = torch.einsum("hit,thd->ihd", p, vv)
            row, key = row + n, key + L
        return out

    def forward(self, **kw):
        return super().forward(window=self.window, sinks=self.sinks, masks=self.masks, **kw)

    def give_back(self):
        """Takes away the pages that no query sees any token of."""
        for b in range(len(self.new)):
            if self.new[b] == 0 or self.kv[b] == 0:
                self.table[b] = 1 << 30
                continue
            any_row = self.visible(b).any(0)
            for p in range(-(-self.kv[b] // self.P)):
                if not bool(any_row[p * self.P:(p + 1) * self.P].any()):
                    self.table[b, p] = 1 << 30
        return self


def drafted(n, rng, branch=0.3):
    """What each token of a random tree of n tokens sees, its ancestors and itself."""
    seen = []
    for i in range(n):
        p = rng.randint(-1, i - 1) if rng.random() < branch else i - 1
        seen.append((seen[p] if p >= 0 else set()) | {i})
    return seen


WINDOWS = [(1, 0), (1, 3), (15, 0), (16, 16), (17, 1), (100, 4), (129, 100), (512, 0), (10 ** 6, 5)]


# ------------------------------------------------------------------------------------- windows

@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_one_token_through_a_window(Hq, Hkv, D, window, sinks):
    P = {256: 64, 128: 16, 64: 256}[D]
    s = View(Hq, Hkv, D, P, [1] * len(LENGTHS), LENGTHS, seed=D + window, window=window,
             sinks=sinks).give_back()
    got = s.forward()
    s.check(got)
    # the other kernel choices: a block per context, and the evenly cut launch
    s.check(s.forward(max_kv_len=0))
    s.check(s.forward(max_kv_len=1 << 20))


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 1), (16, 0), (40, 20), (900, 64)])
def test_several_tokens_through_a_window(Hq, Hkv, D, window, sinks):
    new = [2, 5, 1, 8, 3, 0, 7]
    kv = [2, 300, 1, 2000, 64, 90, 31]
    s = View(Hq, Hkv, D, 16, new, kv, seed=D, window=window, sinks=sinks).give_back()
    s.check(s.forward())


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("window,sinks,P", [(1, 0, 16), (20, 70, 128), (64, 0, 16), (65, 1, 64),
                                            (333, 16, 16), (2000, 200, 32)])
def test_prompts_and_chunks_through_a_window(Hq, Hkv, D, window, sinks, P):
    new = [130, 1, 257, 64, 0, 33]
    kv = [130, 700, 1000, 64, 77, 1500]
    s = View(Hq, Hkv, D, P, new, kv, seed=D + P, window=window, sinks=sinks).give_back()
    got = s.forward()
    s.check(got)
    import torch
    assert torch.equal(got, s.forward())


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 2, 256), (28, 4, 128), (32, 8, 128), (32, 4, 64),
                                      (8, 8, 64), (16, 1, 256)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 4), (700, 100), (1024, 0)])
def test_long_prompts_through_a_window(Hq, Hkv, D, window, sinks):
    # (long enough that contexts are formed into operands first, where they are read often enough)
    new, kv = [2100, 0, 1, 1030], [2100, 70, 1500, 2600]
    s = View(Hq, Hkv, D, 16, new, kv, seed=window + D, window=window, sinks=sinks).give_back()
    got = s.forward()
    s.check(got)
    import torch
    assert torch.equal(got, s.forward())


@pytest.mark.parametrize("new,kv", [([4], [2]), ([6, 1, 20], [0, 0, 3]), ([40], [10]),
                                    ([300], [100]), ([1200], [1000])])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 2), (64, 0)])
def test_queries_before_the_first_cached_token(new, kv, window, sinks):
    s = View(16, 2, 256, 16, new, kv, seed=5, window=window, sinks=sinks)
    got = s.forward()
    s.check(got)
    assert not got[:max(0, new[0] - kv[0])].any()


def test_a_window_wider_than_all_is_causal():
    import torch
    for new, kv in (([1, 3], [700, 90]), ([300, 1], [400, 33])):
        s = View(16, 2, 256, 16, new, kv, seed=6, window=1 << 30, sinks=1 << 30)
        got = s.forward()
        s.check(got)
        s.window = 0
        s.check(got, Setup.reference(s))
        s.check(s.forward(), Setup.reference(s))  # first tokens alone mean nothing
        s.sinks = 0
        assert torch.equal(s.forward(), Setup.forward(s))


@pytest.mark.parametrize("n", [1, 3, 50, 600])
def test_tokens_outside_the_view_may_hold_anything(n):
    import torch

    def alive(s):
        s.k[50, 1, 3] = math.nan   # behind the first tokens, before the window
        s.v[51, 0, 200] = math.inf
        s.v[52] = 3e4
        s.k[L - n - 10, 0, 0] = math.nan
    L = 1000
    s = View(16, 2, 256, 16, [n], [L], seed=11, alive=alive, window=60, sinks=50)
    got = s.forward()
    nan = got.isnan().any(-1)
    pos = L - n + torch.arange(n, device=DEV)
    # token 50 and the others are in the windows of queries up to 60 behind them only
    for t, heads in ((50, slice(8, 16)), (51, slice(0, 8)), (L - n - 10, slice(0, 8))):
        inside = (pos >= t) & (pos < t + 60)
        assert bool(nan[inside][:, heads].all())
    seen = torch.zeros(n, 16, dtype=torch.bool, device=DEV)
    for t, heads in ((50, slice(8, 16)), (51, slice(0, 8)), (L - n - 10, slice(0, 8))):
        seen[(pos >= t) & (pos < t + 60), heads] = True
    assert torch.equal(nan, seen)


# --------------------------------------------------------------------------------------- trees

@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (8, 0), (33, 17), (600, 4)])
def test_small_trees(Hq, Hkv, D, window, sinks):
    new = [2, 5, 1, 8, 3, 0, 7, 8]
    kv = [2, 300, 1, 2000, 64, 90, 31, 8]
    rng = random.Random(D)
    s = View(Hq, Hkv, D, 16, new, kv, seed=D, window=window, sinks=sinks,
             seen=[drafted(n, rng) for n in new]).give_back()
    got = s.forward()
    s.check(got)
    s.check(s.forward(max_kv_len=0))
    s.check(s.forward(max_kv_len=1 << 20))


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (256, 0), (300, 17)])
def test_wide_trees(Hq, Hkv, D, window, sinks):
    new = [33, 256, 1, 64, 65, 0, 127]
    kv = [33, 1000, 70, 64, 1500, 90, 400]
    rng = random.Random(D)
    s = View(Hq, Hkv, D, 32, new, kv, seed=D, window=window, sinks=sinks,
             seen=[drafted(n, rng) for n in new]).give_back()
    got = s.forward()
    s.check(got)
    import torch
    assert torch.equal(got, s.forward())


@pytest.mark.parametrize("n", [4, 32, 100, 256])
@pytest.mark.parametrize("c", [0, 1, 63, 200])
def test_any_mask(n, c):
    # rows without bits (with no context they see nothing), bits above and below their own, bits of
    # tokens that are not there, more words than needed
    rng = random.Random(n + c)
    seen = [{j for j in range(n) if rng.random() < 0.2} for _ in range(n)]
    seen[1] = set()
    seen[n - 1] = set()
    seen[2] = {2} | set(range(n, 256))
    new, kv = [n, 2], [n + c, 40]
    for Hq, Hkv, D in ((16, 2, 256), (1, 1, 64), (32, 8, 128)):
        s = View(Hq, Hkv, D, 16, new, kv, seed=n, seen=[seen, [{0}, {0, 1}]], words=8)
        got = s.forward()
        s.check(got)
        if c == 0:
            assert not got[1].any() and not got[n - 1].any()


def test_drafts_that_are_not_all_cached():
    # fewer cached tokens than drafted ones: those before the first row are not there
    rng = random.Random(1)
    for n, L in ((8, 3), (40, 10), (200, 65)):
        s = View(16, 2, 256, 16, [n], [L], seed=n, seen=[drafted(n, rng)])
        s.check(s.forward())


def test_chains_are_causal():
    for new, kv in (([3, 2], [500, 90]), ([100, 200], [400, 200])):
        s = View(16, 2, 256, 16, new, kv, seed=8,
                 seen=[[set(range(i + 1)) for i in range(n)] for n in new])
        got = s.forward()
        s.check(got, Setup.reference(s))


@pytest.mark.parametrize("n", [3, 100])
def test_a_poisoned_draft_reaches_its_descendants_only(n):
    import torch
    rng = random.Random(n)
    seen = drafted(n, rng, 0.6)

    def alive(s):
        s.v[200 + 1, 0, 7] = math.nan
    s = View(16, 2, 256, 16, [n], [200 + n], seed=n, alive=alive, seen=[seen])
    nan = s.forward().isnan()
    want = torch.tensor([1 in m for m in seen], device=DEV)
    assert torch.equal(nan.any(-1)[:, :8], want[:, None].expand(n, 8))
    assert not nan[:, 8:].any()


@pytest.mark.parametrize("n", [2, 60])
def test_infinite_and_nan_queries_stay_in_their_row(n):
    import torch
    g = gen(1)
    q = torch.randn(2 * n, 16, 256, generator=g, device=DEV).bfloat16()
    q[0, 3, 7] = math.nan
    q[1, 9, 0] = math.inf
    for kw in (dict(window=50, sinks=4),
               dict(seen=[[{i} for i in range(n)], [set() for _ in range(n)]])):
        s = View(16, 2, 256, 64, [n, n], [100, n], seed=12, q=q, **kw)
        if "seen" in kw:
            s.q = s.q.clone()
            s.q[n, 2, 2] = math.nan  # a row that sees nothing stays zero
        got = s.forward()
        bad = torch.zeros(2 * n, 16, dtype=torch.bool, device=DEV)
        bad[0, 3] = bad[1, 9] = True
        assert torch.equal(got.isnan().any(-1), bad)
        if "seen" in kw:
            assert not got[n:].any()


# --------------------------------------------------------------------------------- as it is used

@pytest.mark.parametrize("kw", [dict(window=70, sinks=5), dict(tree=True), dict(window=256, tree=True)])
def test_strided_rows_other_streams_graphs_and_rows_of_nobody(kw):
    import torch
    kw = dict(kw)
    rng = random.Random(4)
    for new, kv in (([1, 3, 2], [2000, 700, 17]), ([1, 3, 17, 200], [2000, 700, 17, 1000])):
        seen = [drafted(n, rng) for n in new] if kw.get("tree") else None
        s = View(32, 8, 128, 32, new, kv, seed=13, seen=seen, window=kw.get("window", 0),
                 sinks=kw.get("sinks", 0))
        want = s.forward()
        s.check(want)
        wide_q = torch.full((s.T + 2, 50 * 128), 9.0, dtype=torch.bfloat16, device=DEV)
        wide_o = torch.full((s.T + 4, 40 * 128), 7.0, dtype=torch.bfloat16, device=DEV)
        q = wide_q[:, 128:33 * 128].unflatten(1, (32, 128))
        q[:s.T].copy_(s.q)
        o = wide_o[1:s.T + 3, 256:34 * 128].unflatten(1, (32, 128))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        s.q = q
        if s.masks is not None:
            s.masks = torch.cat([s.masks, s.masks[:2]])
        s.forward(out=o, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(o[:s.T], want)
        wide_o[1:s.T + 1, 256:34 * 128] = 7.0
        assert bool((wide_o == 7.0).all())  # rows behind the last request and around the heads
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.forward(out=o)
        for _ in range(2):
            o.zero_()
            graph.replay()
            assert torch.equal(o[:s.T], want) and not o[s.T:].any()
        assert s.attn.device_error() == moe.MOE_OK


def test_pages_and_lengths_out_of_range_are_recorded_and_harmless():
    for new, kv in (([1, 1, 1], [300, 900, 64]), ([40, 1, 1], [300, 900, 64])):
        s = View(16, 2, 256, 64, new, kv, seed=16, window=200, sinks=70)
        ref = s.reference()
        keep = s.table.clone()
        n0 = new[0]
        for page in (s.n_pages, -1):
            s.table = keep.clone()
            s.table[1, 12] = page
            got = s.forward()
            assert s.attn.device_error() == moe.MOE_ERR_DEVICE
            s.close_to(got[:n0], ref[:n0])
            s.close_to(got[n0 + 1:], ref[n0 + 1:])
        s.table = keep
        for lens in ([kv[0], -5, 64], [kv[0], 1 << 30, 64]):
            s.kv_lens = ints(lens)
            s.forward()
            assert s.attn.device_error() == moe.MOE_ERR_DEVICE
        s.kv_lens = ints(kv)
        for offs in ([0, n0, n0 + 1, 1 << 20], [0, n0, -1, n0 + 2]):
            s.q_offsets = ints(offs)
            s.forward()
            assert s.attn.device_error() == moe.MOE_ERR_DEVICE
        s.q_offsets = ints([0, n0, n0 + 1, n0 + 2])
        s.check(s.forward(), ref)


def test_many_requests():
    rng = np.random.default_rng(3)
    B = 300
    new = rng.integers(0, 4, B).tolist()
    kv = [int(n + x) for n, x in zip(new, np.exp(rng.uniform(0, 7.5, B)))]
    r = random.Random(5)
    for kw in (dict(window=90, sinks=3), dict(seen=[drafted(n, r) for n in new])):
        s = View(8, 8, 64, 16, new, kv, seed=14, **kw).give_back()
        s.check(s.forward())


def test_a_cache_beyond_32_bit_offsets():
    n_pages = (10 << 30) // (64 * 2 * 288)
    for new in ([1, 1], [1, 90]):
        s = View(16, 2, 256, 64, new, [700, 100], seed=15, n_pages=n_pages,
                 first_page=n_pages - 20, window=80, sinks=65)
        assert s.cache.data.numel() > 5e9
        s.check(s.forward())
        s.attn.close()
        del s


@pytest.mark.parametrize("L,window,sinks", [(131071, 20000, 64), (100001, 1, 99999)])
def test_long_contexts_through_a_window(L, window, sinks):
    for new in ([1], [9]):
        s = View(16, 2, 256, 64, new, [L], seed=7, window=window, sinks=sinks)
        ref = s.reference()
        got = s.forward()
        s.check(got, ref)
        rel = ((got.double() - ref).square().sum() / ref.square().sum()).sqrt().item()
        assert rel < 2.0 ** -8, rel


@pytest.mark.parametrize("kw", [dict(window=40, sinks=3), dict(tree=True), dict(window=128, tree=True)])
@pytest.mark.parametrize("new,kv", [([1, 1, 2, 4], [0, 90, 0, 60]), ([30, 1, 100, 60], [0, 90, 0, 500])])
def test_refused_requests_read_as_zeros(kw, new, kv):
    kw = dict(kw)
    rng = random.Random(9)
    seen = [drafted(n, rng) for n in new] if kw.pop("tree", False) else None
    s = View(16, 2, 256, 16, new, kv, seed=18, seen=seen, **kw)
    s.table[0] = s.table[2] = -1
    got = s.forward()
    s.check(got)
    for b in (0, 2):
        first = sum(new[:b])
        assert not got[first:first + new[b]].any()


@pytest.mark.parametrize("window,sinks", [(300, 5), (0, 0)])
def test_two_objects_at_once_on_two_streams(window, sinks):
    import torch
    rng = random.Random(2)
    new, kv = [40, 3, 200], [700, 900, 1200]
    seen = None if window else [drafted(n, rng) for n in new]
    sides = [View(Hq, Hkv, D, 16, new, kv, seed=i, window=window, sinks=sinks, seen=seen)
             for i, (Hq, Hkv, D) in enumerate(((16, 2, 256), (32, 8, 128)))]
    want = [s.forward() for s in sides]
    streams = [torch.cuda.Stream() for _ in sides]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s, stream in zip(sides, streams):
            got.append(s.forward(stream=stream))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 2])
    for s in sides:
        assert s.attn.device_error() == moe.MOE_OK


def test_capacities_in_place_of_lengths():
    # bounds that are far above the lengths, as a captured step gives them
    rng = random.Random(3)
    new, kv = [3, 1, 2], [90, 200, 17]
    for kw in (dict(window=60, sinks=2), dict(seen=[drafted(n, rng) for n in new], words=8),
               dict(window=300, sinks=2, seen=[drafted(n, rng) for n in new], words=8)):
        s = View(16, 2, 256, 16, new, kv, seed=19, **kw)
        for q, k in ((3, 200), (4, 1 << 30), (256, 1 << 30)):
            if s.masks is not None or q < 256:
                s.check(s.forward(max_q_len=q, max_kv_len=k))


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 2, 256), (28, 4, 128), (32, 4, 64)])
@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("new,kv", [([1, 2], [300, 90]), ([70, 200], [700, 200]), ([1500], [1600])])
def test_output_rows_on_sixteen_bytes(Hq, Hkv, D, window, new, kv):
    # rows that start on 16 bytes but not on 32, as an odd number of eights in the stride gives them
    import torch
    s = View(Hq, Hkv, D, 16, new, kv, seed=20, window=window, sinks=3)
    want = s.forward()
    s.check(want)
    width = Hq * D
    for shift, more in ((8, 0), (0, 8), (8, 24)):
        wide = torch.full((s.T, width + 8 + shift + more), 3.0, dtype=torch.bfloat16, device=DEV)
        out = wide[:, shift:shift + width].unflatten(1, (Hq, D))
        s.forward(out=out)
        assert torch.equal(out, want)
        wide[:, shift:shift + width] = 3.0
        assert bool((wide == 3.0).all())
