"""Drafted trees around their attention: depths and masks (attn_tree_plan), the one-pass norm, rotation
and append (attn_qk_norm_rope_append), the acceptance (attn_kv4_accept), and all of them together.

Bounds: whole numbers and cached rows are equal (the definition's single fp32 operations); turned queries
as in test_gpu_attn.py."""
import math
import random

import numpy as np
import pytest

import sparse_moe_02_gb300 as moe
from test_gpu_attn import (DEV, HEADS, check_rope, code_reference, cos_sin_table, gen, ints, randn,
                           rope_reference)

pytestmark = pytest.mark.gpu


def tree(n, rng, branch=0.3):
    return [rng.randint(-1, i - 1) if rng.random() < branch else i - 1 for i in range(n)]


def tree_reference(parents, n, kv, words):
    """(positions, masks) of one request, token by token."""
    c, depth, rows = max(kv - n, 0), [], []
    for i, p in enumerate(parents):
        p = p if -1 <= p < i else -1
        depth.append(depth[p] + 1 if p >= 0 else 0)
        rows.append((rows[p] if p >= 0 else 0) | 1 << i)
    return [c + d for d in depth], [[r >> 32 * w & 0xffffffff for w in range(words)] for r in rows]


def run_tree_plan(attn, parents, offsets, kv, max_q, words=None, T=None):
    import torch
    masks = None
    if words is not None:
        masks = torch.full((T or len(parents), words), 7, dtype=torch.int32, device=DEV)
    pos, masks = attn.tree_plan(ints(parents), ints(offsets), ints(kv), max_q, masks=masks)
    return pos.tolist(), masks.cpu().numpy().view(np.uint32).tolist()


@pytest.mark.parametrize("new,words", [
    ([1], None), ([0, 1, 0], 1), ([26], None), ([32, 31, 33], None), ([64, 0, 7, 65, 1], None),
    ([256, 255, 1, 100], None), ([5, 9], 8), (list(range(70)), None), ([0, 0], 2),
])
def test_tree_plan(new, words):
    rng = random.Random(sum(new))
    kv = [n + rng.choice([0, 1, 5000]) for n in new]
    parents, pos, masks = [], [], []
    max_q = max(new + [1])
    w = words or -(-max_q // 32)
    for n, L in zip(new, kv):
        # chains, stars and what lies between
        t = tree(n, rng, rng.choice([0.0, 0.3, 1.0]))
        parents += t
        p, m = tree_reference(t, n, L, w)
        pos += p
        masks += m
    attn = moe.PagedAttention(16, 2, 256, 64, 1, len(new))
    offsets = np.concatenate([[0], np.cumsum(new)]).astype(int).tolist()
    got = run_tree_plan(attn, parents, offsets, kv, max_q, words)
    assert got == (pos, masks)
    assert attn.device_error() == moe.MOE_OK
    # rows behind the last request become 0
    got = run_tree_plan(attn, parents + [3, -1, 900], offsets, kv, max_q, words)
    assert got == (pos + [0] * 3, masks + [[0] * w] * 3)
    assert attn.device_error() == moe.MOE_OK
    attn.close()


def test_tree_plan_records_what_does_not_fit():
    attn = moe.PagedAttention(16, 2, 256, 64, 1, 4)
    got = run_tree_plan(attn, [-1, 1, 0, -2, 7], [0, 5], [105], 5)  # 1, -2 and 7 are no parents
    assert got == ([100, 100, 101, 100, 100], [[1], [2], [5], [8], [16]])
    assert attn.device_error() == moe.MOE_ERR_INVALID_ARG
    # refused requests (no cached tokens), and one longer than max_q_len, which is cut
    pos, masks = run_tree_plan(attn, [-1, 0, -1, 0, 1], [0, 2, 5], [0, 50], 2)
    assert pos[:4] == [0, 1, 48, 49] and masks[:4] == [[1], [3], [1], [3]]
    assert attn.device_error() == moe.MOE_ERR_DEVICE
    for offs in ([0, 1 << 20, 5], [-7, 3, 5], [3, 2, 1]):
        run_tree_plan(attn, [-1] * 5, offs, [9, 9], 5)
        assert attn.device_error() == moe.MOE_ERR_DEVICE
    # no requests: all rows are behind the last one
    pos, masks = run_tree_plan(attn, [-1] * 3, [0], [], 1)
    assert pos == [0] * 3 and masks == [[0]] * 3
    assert attn.device_error() == moe.MOE_OK
    attn.close()


# ---------------------------------------------------------------------- norm, rotation, append

def turned(x, w, eps, cos_sin, pos, inter):
    """The definition's single operations in fp32, rounded to bf16."""
    import torch
    y = x.float()
    if w is not None:
        D = y.shape[-1]
        total = y.double().square().sum(-1, keepdim=True).float()
        y = y * (total * (1.0 / D) + eps).sqrt().reciprocal() * w.float()
    if cos_sin is not None:
        r = cos_sin.shape[1]
        cs = cos_sin[pos.long()][:, None]
        cos, sin = cs[..., :r // 2], cs[..., r // 2:]
        a, b = (y[..., 0:r:2], y[..., 1:r:2]) if inter else (y[..., :r // 2], y[..., r // 2:r])
        u, v = a * cos - b * sin, b * cos + a * sin
        y = y.clone()
        if inter:
            y[..., 0:r:2], y[..., 1:r:2] = u, v
        else:
            y[..., :r // 2], y[..., r // 2:r] = u, v
    return y.bfloat16()


def plain_turn(x, cos_sin, pos, inter):
    """The rotation alone, in 64 bits."""
    import torch
    norm = x.double().square().mean(-1, keepdim=True).sqrt()
    one = torch.ones(x.shape[-1], device=DEV)
    return rope_reference(x, one, 0.0, cos_sin, pos, inter) * norm


@pytest.mark.parametrize("T,Hq,Hkv,D,P,rot,inter,normed,gain", [
    (1, 16, 2, 256, 64, 64, False, True, 3.0),
    (1, 1, 1, 64, 16, 16, True, True, 1.0),
    (37, 16, 2, 256, 16, 256, False, True, 1e-3),
    (37, 32, 8, 128, 32, 128, True, True, 1e3),
    (5, 8, 8, 64, 256, 64, False, False, 3.0),
    (333, 6, 2, 256, 64, 32, True, True, 1e-12),
    (1031, 16, 1, 128, 128, 48, False, True, 3.0),   # a rotated part that is no power of two
    (64, 28, 4, 128, 64, 0, False, True, 1e15),      # no rotation
    (64, 28, 4, 128, 64, 0, False, False, 3.0),      # neither: an append
    (3001, 32, 4, 64, 16, 32, False, True, 3.0),
    (4099, 16, 2, 256, 64, 64, True, False, 1e-30),
])
def test_one_pass_equals_the_definition(T, Hq, Hkv, D, P, rot, inter, normed, gain):
    import torch
    g = gen(T + D)
    n_pages = -(-T // P) + 3
    qkv = (randn(g, T, Hq + 2 * Hkv, D) * gain).bfloat16()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]  # strided rows
    k[0, 0, :64] = 0
    wq = wk = None
    if normed:
        wq, wk = ((1 + 0.3 * randn(g, D)).bfloat16() for _ in range(2))
    table = cos_sin_table(700, rot) if rot else None
    pos = torch.randint(0, 700, (T,), generator=g, device=DEV).int()
    slots = torch.randperm(n_pages * P, generator=g, device=DEV)[:T].int()
    if T > 1:
        slots[T - 1] = -1
    attn = moe.PagedAttention(Hq, Hkv, D, P, n_pages, 1)
    cache = attn.new_cache()
    cache.data.fill_(77)
    before = qkv.clone()
    got = attn.qk_norm_rope_append(q, k, v, pos if rot else None, slots, wq, wk, table, cache,
                                   eps=1e-5, interleaved=inter)
    assert torch.equal(qkv, before)
    check_rope(got, rope_reference(q, wq, 1e-5, table, pos, inter) if normed else
               plain_turn(q, table, pos, inter))
    # the same bytes as an append of the turned rows: codes and parameters, and nothing else touched
    other = attn.new_cache()
    other.data.fill_(77)
    attn.append(turned(k, wk, 1e-5, table, pos, inter), v, slots, other)
    assert torch.equal(cache.data, other.data)
    k2, v2 = attn.read(slots, cache)
    n = T - 1 if T > 1 else T
    for back, x in ((k2, turned(k, wk, 1e-5, table, pos, inter)), (v2, v)):
        want, _ = code_reference(x.float().cpu().numpy())
        assert np.array_equal(back.float().cpu().numpy()[:n], want[:n])
    # queries in place give the same bits and leave the rest of the rows alone
    attn.qk_norm_rope_append(q, k, v, pos if rot else None, slots, wq, wk, table, cache, eps=1e-5,
                             interleaved=inter, q_out=q)
    assert torch.equal(q, got) and torch.equal(qkv[:, Hq:], before[:, Hq:])
    assert torch.equal(cache.data, other.data)
    assert attn.device_error() == moe.MOE_OK
    attn.close()


def test_one_pass_of_rows_that_are_not_finite_and_bad_slots_and_positions():
    import torch
    attn = moe.PagedAttention(8, 4, 128, 16, 4, 1)
    cache = attn.new_cache()
    g = gen(1)
    q, k, v = (randn(g, 6, h, 128).bfloat16() for h in (8, 4, 4))
    k[1, 2, 5] = math.nan
    v[2, 3, 100] = math.inf
    k[3, 0, 0] = -math.inf
    k[4, 1] = 3e38     # squares beyond fp32: the norm makes zeros of it
    q[5, 1, 1] = math.nan
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    table = cos_sin_table(10, 64)
    slots = ints([3, 4, 5, 60, 7, 64])
    got = attn.qk_norm_rope_append(q, k, v, ints([0, 1, 2, 3, 10, -1]), slots, w, w, table, cache)
    assert attn.device_error() == moe.MOE_ERR_DEVICE  # positions 10 and -1, slot 64 of 64
    k2, v2 = attn.read(slots[:5], cache)
    assert attn.device_error() == moe.MOE_OK
    nan = torch.zeros(5, 4, dtype=torch.bool, device=DEV)
    nan[1, 2] = nan[2, 3] = nan[3, 0] = True
    assert torch.equal(k2.isnan().all(-1), nan) and torch.equal(k2.isnan().any(-1), nan)
    assert bool((v2[nan] == 0).all()) and not bool(v2.isnan().any())
    assert not k2[4, 1].any()
    bad = torch.zeros(6, 8, dtype=torch.bool, device=DEV)
    bad[5, 1] = True
    assert torch.equal(got.isnan().any(-1), bad)
    want = attn.qk_norm_rope_append(q, k, v, ints([0, 1, 2, 3, 0, 0]), ints([-1] * 6), w, w, table,
                                    cache)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(), want.nan_to_num())
    assert attn.device_error() == moe.MOE_OK
    attn.close()


# ---------------------------------------------------------------------------------- acceptance

def paths_of(lens, drafts, rng):
    return [sorted(rng.sample(range(n), m)) for m, n in zip(lens, drafts)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("P,lens,drafts", [
    (16, [0, 1, 3, 5, 2], [0, 1, 8, 5, 60]),
    (64, [12, 0, 40], [60, 9, 256]),
    (32, [256, 1], [256, 200]),
    (256, [100], [130]),
])
def test_accepted_rows_move(Hq, Hkv, D, P, lens, drafts):
    import torch
    rng = random.Random(P + D)
    ctx = [rng.choice([0, 1, P - 1, P, 5 * P + 3]) for _ in lens]
    paths = paths_of(lens, drafts, rng)
    pages = [-(-(c + n) // P) for c, n in zip(ctx, drafts)]
    n_pages, width = sum(pages) + 2, max(pages) + 1
    g = gen(D)
    ids = torch.randperm(n_pages, generator=g, device=DEV)
    table = torch.full((len(lens), width), 1 << 30, dtype=torch.int32, device=DEV)
    used = 0
    for b, n in enumerate(pages):
        table[b, :n] = ids[used:used + n].int()
        used += n
    attn = moe.PagedAttention(Hq, Hkv, D, P, n_pages, len(lens))
    cache = attn.new_cache()
    every = torch.arange(n_pages * P, device=DEV).int()
    k, v = (randn(g, n_pages * P, Hkv, D).bfloat16() for _ in range(2))
    k[::7, 0, 3] = math.nan  # marked rows move like others
    attn.append(k, v, every, cache)
    old = [t.clone() for t in attn.read(every, cache)]
    want = [t.clone() for t in old]
    for b, path in enumerate(paths):
        def slot(t):
            return int(table[b, t // P]) * P + t % P
        for i, at in enumerate(path):
            for t, o in zip(want, old):
                t[slot(ctx[b] + i)] = o[slot(ctx[b] + at)]
    pw = max(lens) + 1
    rows = ints([p + [-5] * (pw - len(p)) for p in paths])
    attn.accept(cache, table, ints(ctx), rows, ints(lens))
    assert attn.device_error() == moe.MOE_OK
    for t, w in zip(attn.read(every, cache), want):
        assert torch.equal(t.isnan(), w.isnan()) and torch.equal(t.nan_to_num(), w.nan_to_num())
    attn.close()


def test_accepted_rows_out_of_range_are_recorded():
    import torch
    P = 16
    attn = moe.PagedAttention(8, 4, 128, P, 4, 2)
    cache = attn.new_cache()
    every = torch.arange(4 * P, device=DEV).int()
    g = gen(2)
    attn.append(randn(g, 4 * P, 4, 128).bfloat16(), randn(g, 4 * P, 4, 128).bfloat16(), every, cache)
    keep = cache.data.clone()
    table = ints([[0, 1], [2, 3]])

    def accept(ctx, paths, lens, table=table):
        attn.accept(cache, table, ints(ctx), ints(paths), ints(lens))
        return attn.device_error()
    for lens in ([-1, 0], [3, 0]):  # a length out of range moves nothing
        assert accept([3, 3], [[1, 2], [1, 2]], lens) == moe.MOE_ERR_DEVICE
    assert accept([-1, 3], [[1, 2], [1, 2]], [2, 0]) == moe.MOE_ERR_DEVICE
    # rows outside the table or the cache, entries that are negative
    assert accept([31, 3], [[5, 2000], [0, 1]], [1, 0]) == moe.MOE_ERR_DEVICE
    assert accept([31, 1 << 30], [[5, 9], [1 << 30, 9]], [1, 1]) == moe.MOE_ERR_DEVICE
    assert accept([3, 3], [[-1, 2], [0, 0]], [1, 0]) == moe.MOE_ERR_DEVICE
    assert accept([3, 3], [[1, 2], [0, 0]], [2, 0], ints([[4, 1], [2, 3]])) == moe.MOE_ERR_DEVICE
    assert accept([3, 3], [[1, 2], [0, 0]], [2, 0], ints([[-1, 1], [2, 3]])) == moe.MOE_ERR_DEVICE
    assert torch.equal(cache.data, keep)
    # the other request's rows move all the same
    assert accept([31, 3], [[5, 2000], [1, 0]], [1, 1]) == moe.MOE_ERR_DEVICE
    k, v = attn.read(ints([2 * P + 3, 2 * P + 4]), cache)
    assert torch.equal(k[0], k[1]) and torch.equal(v[0], v[1])
    assert accept([3, 3], [[0, 1], [0, 1]], [2, 2]) == moe.MOE_OK  # rows that stay where they are
    attn.close()


# -------------------------------------------------------------------------------------- together

@pytest.mark.parametrize("Hq,Hkv,D,window,sinks", [(16, 2, 256, 0, 0), (16, 2, 256, 150, 4),
                                                   (32, 8, 128, 40, 0), (8, 8, 64, 0, 0)])
@pytest.mark.parametrize("drafts", [[3, 2, 4], [20, 37, 1]])
def test_steps_with_drafts_leave_the_cache_of_their_accepted_tokens(Hq, Hkv, D, window, sinks,
                                                                    drafts):
    """Prompts, a drafted step, the acceptance of a path of each tree, and a step of one token behind it:
    the cache and the outputs are those of the same tokens without the rejected ones.  Every output
    lies within 2^-8 |o| + 2^-10 max|v| of the formula over equal cached rows, values below 4."""
    import torch
    rng = random.Random(D + sum(drafts))
    P, B, prompts = 16, 3, [100, 1, 333]
    total = max(prompts) + max(drafts) + 2
    width = -(-total // P)
    attn = moe.PagedAttention(Hq, Hkv, D, P, B * width, B)
    g = gen(D)
    wq, wk = ((1 + 0.1 * randn(g, D)).bfloat16() for _ in range(2))
    turns = cos_sin_table(total, D // 4)

    class Run:
        def __init__(self):
            self.cache = attn.new_cache()
            self.table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
            order = torch.randperm(B * width, generator=gen(3), device=DEV)
            self.free, self.cursor = order.int(), ints([0])

        def step(self, rows, ctx, new, trees=None):
            x = torch.cat(rows)
            offs, kv, pos, slots, _ = attn.plan(self.table, ints(ctx), ints(new), self.free,
                                                self.cursor, T=x.shape[0], cursor_out=self.cursor)
            masks = None
            if trees is not None:
                pos, masks = attn.tree_plan(ints(sum(trees, [])), offs, kv, max(new), positions=pos)
            q = attn.qk_norm_rope_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pos, slots,
                                         wq, wk, turns, self.cache)
            out = attn.forward(q, self.cache, self.table, offs, kv, max(new), total, window=window,
                               sinks=sinks, masks=masks)
            return out.split(new)

        def rows(self, lens):
            at = [(self.table[b].long()[torch.arange(n, device=DEV) // P] * P
                   + torch.arange(n, device=DEV) % P).int() for b, n in enumerate(lens)]
            return attn.read(torch.cat(at), self.cache)

    def random_rows(lens):
        return [(randn(g, n, Hq + 2 * Hkv, D) * 0.5).clamp(-4, 4).bfloat16() for n in lens]

    first, drafted_rows, last = random_rows(prompts), random_rows(drafts), random_rows([1] * B)
    trees = [tree(n, rng) for n in drafts]
    paths = []
    for t in trees:
        node, path = rng.randrange(len(t)), []
        while node >= 0:
            path.insert(0, node)
            node = t[node]
        paths.append(path)
    lens = [len(p) for p in paths]

    a = Run()
    a.step(first, [0] * B, prompts)
    tree_out = a.step(drafted_rows, prompts, drafts, trees)
    attn.accept(a.cache, a.table, ints(prompts),
                ints([p + [0] * (max(lens) - len(p)) for p in paths]), ints(lens))
    after = [n + m for n, m in zip(prompts, lens)]
    # (the pages of the rejected tokens stay with their requests)
    a_last = a.step(last, after, [1] * B)

    b = Run()
    b.step(first, [0] * B, prompts)
    kept = [r[p] for r, p in zip(drafted_rows, paths)]
    kept_out = b.step(kept, prompts, lens)
    b_last = b.step(last, after, [1] * B)
    assert attn.device_error() == moe.MOE_OK

    ends = [n + 1 for n in after]
    for x, y in zip(a.rows(ends), b.rows(ends)):
        assert torch.equal(x, y)

    def near(x, y):
        bound = 2 * (2.0 ** -8 * y.double().abs() + 2.0 ** -10 * 4)
        assert bool(((x.double() - y.double()).abs() <= bound).all())
    for t, k, p in zip(tree_out, kept_out, paths):
        near(t[p], k)
        assert bool(k.any())
    for x, y in zip(a_last, b_last):
        near(x, y)
    attn.close()


def test_arguments_are_refused_on_the_host():
    attn = moe.PagedAttention(16, 2, 256, 64, 4, 1)
    cache = attn.new_cache()
    A = 0x100000  # never dereferenced: every call below fails in the argument checks
    h, c = attn.handle, cache.ptr
    OK, INV, UNS, ALI = (moe.MOE_OK, moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED,
                         moe.MOE_ERR_ALIGNMENT)

    def fwd(h=h, q=A, qs=4096, cache=c, table=A, width=4, qo=A, kv=A, B=1, T=1, mq=1, mk=1, w=8, s=1,
            m=A, mw=1, out=A, os=4096):
        return moe.attn_kv4_forward_masked(h, q, qs, cache, table, width, qo, kv, B, T, mq, mk, w, s,
                                           m, mw, out, os, None)
    assert fwd(T=0) == OK and fwd(B=0) == OK and fwd(h=None) == INV
    for name in ("q", "cache", "table", "qo", "kv", "out"):
        assert fwd(**{name: None}) == INV, name
        assert fwd(**{name: A + 2}) == ALI, name
    assert fwd(w=-1) == INV and fwd(s=-1) == INV and fwd(mw=0) == INV and fwd(mq=0) == INV
    assert fwd(w=(1 << 30) + 1) == UNS and fwd(s=(1 << 30) + 1) == UNS
    assert fwd(m=A + 2) == ALI
    assert fwd(mq=33) == UNS and fwd(mq=257, mw=9) == UNS and fwd(mw=9) == UNS
    assert fwd(mq=9) == UNS  # a window that could hide drafted tokens
    assert fwd(mq=9, w=0, T=0) == OK and fwd(mq=9, m=None, mw=0, T=0) == OK
    assert fwd(B=2) == UNS and fwd(T=(1 << 20) + 1) == UNS and fwd(B=-1) == INV and fwd(mk=-1) == INV
    assert fwd(qs=4000) == INV and fwd(os=4100) == ALI

    def plan(h=h, p=A, qo=A, kv=A, B=1, T=1, mq=1, pos=A, m=A, mw=1):
        return moe.attn_tree_plan(h, p, qo, kv, B, T, mq, pos, m, mw, None)
    assert plan(T=0) == OK and plan(h=None) == INV
    for name in ("p", "qo", "kv", "pos", "m"):
        assert plan(**{name: None}) == INV, name
        assert plan(**{name: A + 2}) == ALI, name
    assert plan(B=-1) == INV and plan(T=-1) == INV and plan(mq=0) == INV and plan(mw=0) == INV
    assert plan(B=2) == UNS and plan(T=(1 << 20) + 1) == UNS
    assert plan(mq=33) == UNS and plan(mq=257, mw=8) == UNS and plan(mw=9) == UNS

    def accept(h=h, cache=c, table=A, width=4, ctx=A, p=A, pw=1, n=A, B=1):
        return moe.attn_kv4_accept(h, cache, table, width, ctx, p, pw, n, B, None)
    assert accept(B=0) == OK and accept(pw=0) == OK and accept(h=None) == INV
    for name in ("cache", "table", "ctx", "p", "n"):
        assert accept(**{name: None}) == INV, name
        assert accept(**{name: A + 2}) == ALI, name
    assert accept(B=-1) == INV and accept(pw=-1) == INV and accept(width=-1) == INV
    assert accept(B=2) == UNS and accept(pw=(1 << 20) + 1) == UNS

    def rope(h=h, q=A, qs=4096, k=A, ks=512, v=A, vs=512, pos=A, slots=A, qw=A, kw=A, eps=1e-6, cs=A,
             n=4, rot=64, T=1, qo=A, qos=4096, cache=c):
        return moe.attn_qk_norm_rope_append(h, q, qs, k, ks, v, vs, pos, slots, qw, kw, eps, cs, n,
                                            rot, 0, T, qo, qos, cache, None)
    assert rope(T=0) == OK and rope(h=None) == INV
    for name in ("q", "k", "v", "pos", "slots", "qw", "kw", "cs", "qo", "cache"):
        assert rope(**{name: None}) == INV, name
        assert rope(**{name: A + 2}) == ALI, name
    assert rope(T=-1) == INV and rope(n=0) == INV and rope(rot=-16) == INV
    assert rope(eps=-1.0) == INV and rope(eps=math.nan) == INV
    assert rope(rot=40) == UNS and rope(rot=272) == UNS and rope(T=(1 << 20) + 1) == UNS
    assert rope(ks=504) == INV and rope(vs=516) == ALI and rope(qos=4104, q=A + 8) == ALI
    attn.close()


def test_a_step_with_drafts_as_one_graph():
    """Plan of the trees, one-pass append, attention and acceptance, captured once and replayed on other
    inputs in the same tensors."""
    import torch
    Hq, Hkv, D, P, B, n = 16, 2, 256, 16, 3, 6
    ctx = [40, 5, 90]
    width = 8
    attn = moe.PagedAttention(Hq, Hkv, D, P, B * width, B)
    cache = attn.new_cache()
    table = torch.randperm(B * width, generator=gen(1), device=DEV).int().view(B, width)
    slots = torch.cat([(table[b].long()[torch.arange(c, c + n, device=DEV) // P] * P
                        + torch.arange(c, c + n, device=DEV) % P).int() for b, c in enumerate(ctx)])
    every = torch.arange(B * width * P, device=DEV).int()
    g = gen(2)
    k0, v0 = (randn(g, len(every), Hkv, D).bfloat16() for _ in range(2))
    offs, kv = ints([0, n, 2 * n, 3 * n]), ints([c + n for c in ctx])
    w = (1 + 0.1 * randn(g, D)).bfloat16()
    turns = cos_sin_table(200, 64)
    x = torch.empty(B * n, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)
    parents, paths, lens = ints([0] * (B * n)), ints([[0] * n] * B), ints([0] * B)

    def step():
        pos, masks = attn.tree_plan(parents, offs, kv, n)
        q = attn.qk_norm_rope_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pos, slots, w, w,
                                     turns, cache)
        out = attn.forward(q, cache, table, offs, kv, n, 1000, window=64, sinks=2, masks=masks)
        attn.accept(cache, table, ints_ctx, paths, lens)
        return out

    ints_ctx = ints(ctx)

    def fill(seed):
        rng = random.Random(seed)
        trees = [tree(n, rng) for _ in range(B)]
        attn.append(k0, v0, every, cache)
        x.copy_(randn(gen(seed), *x.shape))
        parents.copy_(ints(sum(trees, [])))
        chosen = []
        for t in trees:
            node, path = rng.randrange(n), []
            while node >= 0:
                path.insert(0, node)
                node = t[node]
            chosen.append(path)
        paths.copy_(ints([p + [0] * (n - len(p)) for p in chosen]))
        lens.copy_(ints([len(p) for p in chosen]))

    fill(3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (4, 5, 6):
        fill(seed)
        want = step().clone()
        rows = cache.data.clone()
        fill(seed)
        graph.replay()
        assert torch.equal(out, want) and bool(want.any())
        assert torch.equal(cache.data, rows)
    assert attn.device_error() == moe.MOE_OK
    attn.close()


def test_an_entry_twice_and_a_path_that_falls_are_recorded():
    import torch
    attn = moe.PagedAttention(8, 4, 128, 16, 4, 1)
    cache = attn.new_cache()
    table = ints([[0, 1, 2, 3]])
    for path in ([1, 1, 2], [2, 1], [0, 3, 3]):
        attn.accept(cache, table, ints([5]), ints([path]), ints([len(path)]))
        assert attn.device_error() == moe.MOE_ERR_DEVICE
    attn.accept(cache, table, ints([5]), ints([[0, 1, 2]]), ints([0]))
    assert attn.device_error() == moe.MOE_OK
    # nothing to do: no requests, no tokens
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    attn.accept(cache, none.view(0, 4), none, none.view(0, 3), none)
    rows = torch.empty(0, 8, 128, dtype=torch.bfloat16, device=DEV)
    keys = rows[:, :4]
    got = attn.qk_norm_rope_append(rows, keys, keys, none, none, None, None, cos_sin_table(4, 16),
                                   cache)
    assert got.shape == (0, 8, 128)
    pos, masks = attn.tree_plan(none, ints([0, 0]), ints([3]), 1)
    assert pos.numel() == 0 and masks.shape == (0, 1)
    assert attn.device_error() == moe.MOE_OK
    attn.close()


def test_tree_plan_of_lengths_and_capacities_at_the_ends_of_their_type():
    import torch
    attn = moe.PagedAttention(16, 2, 256, 64, 1, 2)
    pos, masks = run_tree_plan(attn, [-1, 0, -1], [0, 2, 3], [-(1 << 31), -1], 2)
    assert pos == [0, 1, 0] and masks == [[1], [3], [1]]
    assert attn.device_error() == moe.MOE_ERR_DEVICE
    pos, masks = run_tree_plan(attn, [-1, 0, -1], [0, 2, 3], [(1 << 31) - 1, 1], 2)
    assert pos == [(1 << 31) - 3, (1 << 31) - 2, 0] and masks == [[1], [3], [1]]
    assert attn.device_error() == moe.MOE_OK
    # refused before masks of that width are made
    a = ints([-1]), ints([0, 1]), ints([1])
    held = torch.cuda.memory_reserved()
    for most in (257, (1 << 31) - 1):
        with pytest.raises(moe.MoeError):
            attn.tree_plan(*a, most)
    assert torch.cuda.memory_reserved() == held
    attn.close()
