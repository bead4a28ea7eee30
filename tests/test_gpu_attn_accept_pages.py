"""The acceptance that puts the pages of rejected tokens back on the free list (attn_kv4_accept_pages): whole
numbers, equal to a plain count; rows move as without; a captured step that runs on as many pages as it
needs; what the C entry refuses."""
import random

import pytest

import sparse_moe_02_gb300 as moe
from test_gpu_attn import DEV, gen, ints, randn

pytestmark = pytest.mark.gpu


def put_back(table, ctx, kv, lens, free, cursor, P):
    """The free list and the cursor behind the call."""
    back = []
    for b, (c, L, m) in enumerate(zip(ctx, kv, lens)):
        if L >= c:
            back += table[b][-(-(c + m) // P):-(-L // P)]
    return free[:cursor - len(back)] + back + free[cursor:], cursor - len(back)


def setup(B, P, most, seed, refused=0.1):
    """Requests behind a plan of `most` new tokens at most, and what is accepted of them."""
    rng = random.Random(seed)
    ctx = [rng.choice([0, 1, P - 1, P, 3 * P + 5]) for _ in range(B)]
    new = [rng.randint(0, most) for _ in range(B)]
    kv = [0 if rng.random() < refused else c + n for c, n in zip(ctx, new)]
    lens = [rng.choice([0, n, rng.randint(0, n)]) if L else 0 for n, L in zip(new, kv)]
    paths = [sorted(rng.sample(range(n), m)) for n, m in zip(new, lens)]
    pages = [-(-(c + n) // P) for c, n in zip(ctx, new)]
    n_pages, width = sum(pages) + 3, max(pages + [0]) + 1
    ids = list(range(n_pages))
    rng.shuffle(ids)
    table, used = [], 0
    for n in pages:
        table.append(ids[used:used + n] + [1 << 30] * (width - n))
        used += n
    free = [rng.randrange(n_pages) for _ in range(sum(pages))] + ids[used:]
    return ctx, kv, lens, paths, table, n_pages, free, sum(pages) + 1


def matrix(paths, width):
    return ints([p + [-5] * (width - len(p)) for p in paths]).view(len(paths), width)


@pytest.mark.parametrize("B,P,most,seed", [(1, 16, 40, 1), (1, 256, 9, 2), (7, 64, 60, 3),
                                           (64, 16, 33, 4), (300, 32, 100, 5), (1024, 16, 20, 6)])
def test_pages_go_back_and_rows_move(B, P, most, seed):
    import torch
    ctx, kv, lens, paths, table, n_pages, free, cursor = setup(B, P, most, seed)
    attn = moe.PagedAttention(2, 1, 64, P, n_pages, B)
    caches = [attn.new_cache() for _ in range(2)]
    every = torch.arange(n_pages * P, device=DEV).int()
    g = gen(seed)
    k, v = (randn(g, n_pages * P, 1, 64).bfloat16() for _ in range(2))
    for c in caches:
        attn.append(k, v, every, c)
    t, f, cur = ints(table), ints(free), ints([cursor])
    rows = matrix(paths, max(lens) + 1)
    args = (t, ints(ctx), rows, ints(lens))
    attn.accept(caches[0], *args)
    attn.accept(caches[1], *args, kv_lens=ints(kv), free_pages=f, cursor=cur)
    assert attn.device_error() == moe.MOE_OK
    assert torch.equal(caches[0].data, caches[1].data)
    assert (f.tolist(), cur.item()) == put_back(table, ctx, kv, lens, free, cursor, P)
    assert t.tolist() == table
    attn.close()


def test_everything_rejected_needs_no_paths():
    import torch
    P = 16
    attn = moe.PagedAttention(2, 1, 64, P, 8, 2)
    f, cur = ints([7, 7, 7, 7, 5]), ints([4])
    attn.accept(attn.new_cache(), ints([[0, 1, 2], [3, 4, 6]]), ints([10, 32]),
                torch.empty(2, 0, dtype=torch.int32, device=DEV), ints([0, 0]), kv_lens=ints([40, 33]),
                free_pages=f, cursor=cur)
    assert attn.device_error() == moe.MOE_OK
    assert f.tolist() == [7, 1, 2, 6, 5] and cur.item() == 1
    attn.close()


@pytest.mark.parametrize("change", [
    dict(cursor=1), dict(cursor=6), dict(cursor=-1), dict(cursor=1 << 30),  # no room, no such cursor
    dict(lens=[-1, 0]), dict(lens=[3, 0]), dict(ctx=[-1, 32]), dict(table=[[0, 8, 1], [3, 4, -6]]),
])
def test_what_makes_no_sense_is_recorded(change):
    P = 16
    attn = moe.PagedAttention(2, 1, 64, P, 8, 2)
    a = dict(cursor=4, lens=[0, 0], ctx=[10, 32], table=[[0, 1, 2], [3, 4, 6]])
    a.update(change)
    f, cur = ints([7, 7, 7, 7, 5]), ints([a["cursor"]])
    attn.accept(attn.new_cache(), ints(a["table"]), ints(a["ctx"]), ints([[0, 1], [0, 1]]),
                ints(a["lens"]), kv_lens=ints([40, 33]), free_pages=f, cursor=cur)
    assert attn.device_error() == moe.MOE_ERR_DEVICE
    want = ([7, 7, 7, 7, 5], a["cursor"])
    if "lens" in change or "ctx" in change:  # the other request's page goes back all the same
        want = ([7, 7, 7, 6, 5], 3)
    if "table" in change:  # a page that is there
        want = ([7, 7, 7, 1, 5], 3)
    assert (f.tolist(), cur.item()) == want
    attn.close()


def test_a_captured_step_runs_on_the_pages_that_it_needs():
    # contexts grow by what is accepted; every step drafts across pages, and the pool holds what the
    # longest step needs, no more
    import torch
    B, P, n, steps = 3, 16, 20, 40
    rng = random.Random(8)
    lens = [[rng.choice([0, 0, 1, 2]) for _ in range(B)] for _ in range(steps)]
    most = [sum(x) for x in zip(*lens)]
    n_pages = sum(-(-(m + n) // P) for m in most)
    attn = moe.PagedAttention(2, 1, 64, P, n_pages, B)
    cache = attn.new_cache()
    table = torch.full((B, -(-(max(most) + n) // P)), -1, dtype=torch.int32, device=DEV)
    free, cursor = torch.randperm(n_pages, device=DEV).int(), ints([0])
    ctx, new = ints([0] * B), ints([n] * B)
    paths, path_lens = ints([[0, 1]] * B), ints([0] * B)
    k = randn(gen(3), B * n, 1, 64).bfloat16()

    def step():
        _, kv, _, slots, _ = attn.plan(table, ctx, new, free, cursor, T=B * n, cursor_out=cursor)
        attn.append(k, k, slots, cache)
        attn.accept(cache, table, ctx, paths, path_lens, kv_lens=kv, free_pages=free, cursor=cursor)
        ctx.add_(path_lens)

    def reset():
        ctx.zero_(), cursor.zero_(), path_lens.zero_()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    reset()
    free.copy_(torch.randperm(n_pages, device=DEV).int())
    for i in range(steps):
        path_lens.copy_(ints(lens[i]))
        graph.replay()
        assert attn.device_error() == moe.MOE_OK, i
        held = [table[b, :-(-int(c) // P)].tolist() for b, c in enumerate(ctx.tolist())]
        pages = sum(held, []) + free[cursor.item():].tolist()
        assert sorted(pages) == list(range(n_pages)), i
    assert ctx.tolist() == most
    attn.close()


def test_refusals():
    h = moe.PagedAttention(2, 1, 64, 16, 8, 2)
    A = 0x100000  # never dereferenced
    INV, ALI, UNS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_ALIGNMENT, moe.MOE_ERR_UNSUPPORTED

    def accept(cache=A, table=A, width=4, ctx=A, p=A, pw=1, n=A, B=1, kv=A, free=A, n_free=9, cur=A):
        return moe.attn_kv4_accept_pages(h.handle, cache, table, width, ctx, p, pw, n, B, kv, free,
                                         n_free, cur, None)
    assert accept(B=0) == moe.MOE_OK
    for name in ("cache", "table", "ctx", "p", "n", "kv", "free", "cur"):
        assert accept(**{name: None}) == INV, name
        assert accept(**{name: A + 2}) == ALI, name
    assert accept(B=-1) == INV and accept(pw=-1) == INV and accept(width=-1) == INV
    assert accept(n_free=-1) == INV
    assert accept(B=3) == UNS and accept(pw=(1 << 20) + 1) == UNS
    h.close()
