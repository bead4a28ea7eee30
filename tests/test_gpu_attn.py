"""GPU parity of the attention step (include/attn.h) against plain implementations in 64 bits.

Bounds, from the arithmetic:
  plan, cached codes: whole numbers and the definition's fp32 operations: equal.
  norm and rotation: fp32 with one bf16 rounding: |got - ref| <= 2^-8 |ref| + 2^-16 max|ref| (half a
    bf16 ulp is 2^-9 |ref|; a rotated pair that cancels keeps the fp32 error of its parts).
  attention: one bf16 rounding of the output (2^-9 |ref|), values and weights whose f16 roundings
    are 2^-12 of a part no larger than twice the largest cached value, scores within 2^-13:
    |got - ref| <= 2^-8 |ref| + 2^-10 max|v|.
"""
import math

import numpy as np
import pytest

import sparse_moe_02_gb300 as moe

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    yield
    torch.cuda.synchronize()


def ints(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def gen(seed):
    import torch
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    import torch
    return torch.randn(*shape, generator=g, device=DEV)


# ---------------------------------------------------------------------------------------- plan

def plan_reference(table, ctx, new, free, cursor, T, P):
    """Request by request, token by token."""
    table = table.copy()
    W = table.shape[1]
    offs, kv, pos, slots = [0], [], [0] * T, [-1] * T
    wanted, taken, status, total = 0, 0, moe.MOE_OK, 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        ok = 0 <= c <= 1 << 30 and 0 <= n <= 1 << 30
        c = c if 0 <= c <= 1 << 30 else 0
        n = min(max(n, 0), 1 << 30)
        first = total
        total += n
        offs.append(min(total, T))
        before, after = -(-c // P), -(-(c + n) // P)
        refused = False
        if not ok or total > T or after > W:
            refused, status = True, max(status, moe.MOE_ERR_INVALID_ARG)
        else:
            need = after - before
            wanted += need
            if need and wanted > len(free) - cursor:
                refused, status = True, max(status, moe.MOE_ERR_NO_MEMORY)
            elif need:
                table[b, before:after] = free[cursor + wanted - need:cursor + wanted]
                taken = wanted
        kv.append(0 if refused else c + n)
        for i in range(min(first, T), min(total, T)):
            p = c + i - first
            pos[i] = p
            if not refused:
                slots[i] = table[b, p // P] * P + p % P
    return table, offs, kv, pos, slots, cursor + taken, status


def run_plan(attn, table, ctx, new, free, cursor, T, in_place=False):
    t, cur = ints(table), ints([cursor])
    q, kv, pos, slots, cur2 = attn.plan(t, ints(ctx), ints(new), ints(free), cur, T=T,
                                        cursor_out=cur if in_place else None)
    err = attn.device_error()
    if not in_place:
        assert cur.item() == cursor
    return (t.cpu().numpy(), q.tolist(), kv.tolist(), pos.tolist(), slots.tolist(), cur2.item(),
            err)


def check_plan(got, want):
    assert np.array_equal(got[0], want[0])
    for g, w, what in zip(got[1:], want[1:], ("offsets", "kv", "positions", "slots", "cursor",
                                              "status")):
        assert g == w, what


@pytest.mark.parametrize("B,P,q_max,ctx_max,spare,seed", [
    (1, 64, 1, 0, 0, 1),       # the very first token
    (1, 16, 1, 16, 0, 2),      # a page exactly full
    (64, 64, 1, 8192, 3, 3),
    (7, 32, 0, 100, 0, 4),     # no new tokens at all
    (33, 16, 40, 300, -5, 5),  # the list runs out
    (513, 128, 9, 2000, 0, 6),  # more requests than threads
    (40, 256, 700, 5000, -1, 7),
    (3, 16, 5000, 0, 0, 8),    # several blocks, ragged
])
def test_plan(B, P, q_max, ctx_max, spare, seed):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, ctx_max + 1, B).tolist()
    new = rng.integers(0, q_max + 1, B).tolist()
    ctx[0], new[0] = ctx_max, q_max
    held = [-(-c // P) for c in ctx]
    fresh = sum(-(-(c + n) // P) - h for c, n, h in zip(ctx, new, held))
    W = max(-(-(c + n) // P) for c, n in zip(ctx, new)) + 1
    ids = rng.permutation(sum(held) + fresh + 8)
    table = np.full((B, W), -1, np.int32)
    used = 0
    for b in range(B):
        table[b, :held[b]] = ids[used:used + held[b]]
        used += held[b]
    free = ids[used:used + max(0, 2 + fresh + spare)].tolist()
    T = sum(new) + (5 if seed % 2 else 0)
    attn = moe.PagedAttention(16, 2, 256, P, len(ids), B)
    want = plan_reference(table, ctx, new, free, 2, T, P)
    check_plan(run_plan(attn, table, ctx, new, free, 2, T), want)
    # the same again, the cursor written in place
    check_plan(run_plan(attn, table, ctx, new, free, 2, T, in_place=True), want)
    attn.close()


def test_plan_refuses_what_does_not_fit():
    P, W = 16, 3
    attn = moe.PagedAttention(16, 2, 256, P, 100, 8)
    table = np.arange(24, dtype=np.int32).reshape(8, W)
    #       ok  negative  too many pages  negative  ok   too long     needs no page, list empty
    ctx = [0, -3, 40, 5, 16, 5, 17, 0]
    new = [3, 2, 20, -1, 16, (1 << 30) + 1, 3, 0]
    free = [50, 51]
    want = plan_reference(table, ctx, new, free, 0, 40, P)
    assert want[6] == moe.MOE_ERR_INVALID_ARG
    check_plan(run_plan(attn, table, ctx, new, free, 0, 40), want)
    # tokens that end behind T; a cursor behind the list and before it
    want = plan_reference(table, [0, 0], [3, 9], free, 0, 8, P)
    check_plan(run_plan(attn, table[:2], [0, 0], [3, 9], free, 0, 8),
               (want[0][:2],) + want[1:])
    for cursor in (2, 9, -4):
        got = run_plan(attn, table[:2], [0, 5], [3, 1], free, cursor, 4)
        assert got[2] == [0, 6] and got[4] == [-1] * 3 + [table[1, 0] * P + 5]
        assert got[5] == cursor and got[6] == moe.MOE_ERR_NO_MEMORY
        assert np.array_equal(got[0], table[:2])
    # no requests, no tokens
    got = run_plan(attn, np.zeros((0, 4), np.int32), [], [], free, 1, 3)
    assert got[1:] == ([0], [], [0] * 3, [-1] * 3, 1, moe.MOE_OK)
    got = run_plan(attn, table, ctx, new, free, 0, 0)
    assert got[1] == [0] * 9
    attn.close()


# ----------------------------------------------------------------------- norm and rotation

def rope_reference(x, w, eps, cos_sin, pos, inter):
    import torch
    y = x.double()
    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    if cos_sin is None:
        return y
    r = cos_sin.shape[1]
    cs = cos_sin.double()[pos.long()][:, None]
    cos, sin = cs[..., :r // 2], cs[..., r // 2:]
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if inter else (y[..., :r // 2], y[..., r // 2:r])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = y.clone()
    if inter:
        y[..., 0:r:2], y[..., 1:r:2] = u, v
    else:
        y[..., :r // 2], y[..., r // 2:r] = u, v
    return y


def check_rope(got, ref):
    err = (got.double() - ref).abs()
    bound = 2.0 ** -8 * ref.abs() + 2.0 ** -16 * ref.abs().max()
    assert bool((err <= bound).all()), f"max error {err.max().item()}"


def cos_sin_table(n, r):
    import torch
    inv = 1e6 ** (-torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / r)
    ang = torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,fused", [
    (1, 16, 2, 256, 64, False, True),
    (1, 1, 1, 64, 16, True, False),
    (37, 16, 2, 256, 256, False, True),
    (37, 32, 8, 128, 128, True, True),
    (5, 8, 8, 64, 64, False, False),
    (333, 6, 2, 256, 32, True, True),
    (1031, 16, 1, 128, 48, False, True),   # a rotated part that is no power of two
    (64, 28, 4, 128, 0, False, True),      # no rotation
    (3001, 32, 4, 64, 32, False, True),    # several heads per group of lanes
])
def test_norm_and_rotation(T, Hq, Hkv, D, rot, inter, fused):
    import torch
    g = gen(T + D)
    qkv = (randn(g, T, (Hq + 2 * Hkv) * D) * 3).bfloat16()
    q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    k = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    q[0, 0] = 0  # a head of zeros stays zero
    wq, wk = (1 + 0.3 * randn(g, D)).bfloat16(), (1 + 0.3 * randn(g, D)).bfloat16()
    table = cos_sin_table(700, rot) if rot else None
    pos = torch.randint(0, 700, (T,), generator=g, device=DEV).int()
    attn = moe.PagedAttention(Hq, Hkv, D, 64, 1, 1)
    before = qkv.clone()
    qo, ko = attn.qk_norm_rope(q, k, pos, wq, wk, table, eps=1e-5, interleaved=inter)
    assert torch.equal(qkv, before)
    check_rope(qo, rope_reference(q, wq, 1e-5, table, pos, inter))
    check_rope(ko, rope_reference(k, wk, 1e-5, table, pos, inter))
    assert bool((qo[0, 0] == 0).all())
    # in place gives the same bits and leaves the values between the rows alone
    attn.qk_norm_rope(q, k, pos, wq, wk, table, eps=1e-5, interleaved=inter, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    if fused:
        assert torch.equal(qkv[:, (Hq + Hkv) * D:], before[:, (Hq + Hkv) * D:])
    assert attn.device_error() == moe.MOE_OK
    attn.close()


def test_rotation_beyond_the_table_is_recorded():
    import torch
    g = gen(3)
    q, k = randn(g, 3, 4, 128).bfloat16(), randn(g, 3, 2, 128).bfloat16()
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    attn = moe.PagedAttention(4, 2, 128, 64, 1, 1)
    table = cos_sin_table(10, 64)
    got = attn.qk_norm_rope(q, k, ints([-1, 4, 10]), w, w, table)
    assert attn.device_error() == moe.MOE_ERR_DEVICE
    want = attn.qk_norm_rope(q, k, ints([0, 4, 0]), w, w, table)
    assert attn.device_error() == moe.MOE_OK
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    attn.close()


# ------------------------------------------------------------------------------- cached rows

def code_reference(x):
    """The definition in numpy fp32: (values read back, codes), rows [..., D] of fp32 holding
    bf16 values, all finite."""
    x = x.astype(np.float32)
    g = x.reshape(x.shape[:-1] + (-1, 64))
    lo, hi = g.min(-1, keepdims=True), g.max(-1, keepdims=True)
    step = to_bf16((hi - lo) / np.float32(15))
    with np.errstate(divide="ignore", invalid="ignore"):
        code = np.where(step > 0, np.rint((g - lo) / step), np.float32(0))
    code = np.clip(code, 0, 15).astype(np.float32)
    return to_bf16((step * code + lo).reshape(x.shape)), code.reshape(x.shape)


def to_bf16(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).bfloat16().float().numpy()


@pytest.mark.parametrize("T,Hq,Hkv,D,P,scale", [
    (1, 16, 2, 256, 64, 1.0),
    (7, 8, 8, 64, 16, 1e-3),
    (100, 32, 8, 128, 32, 30.0),
    (1000, 16, 1, 128, 256, 1e-30),
    (777, 6, 2, 256, 16, 1e30),
    (4097, 16, 2, 256, 128, 1.0),
])
def test_cached_rows_equal_the_definition(T, Hq, Hkv, D, P, scale):
    import torch
    g = gen(T)
    n_pages = -(-T // P) + 3
    attn = moe.PagedAttention(Hq, Hkv, D, P, n_pages, 1)
    cache = attn.new_cache()
    cache.data.fill_(77)
    kv = (randn(g, T, 2, Hkv, D) * scale).bfloat16()
    kv[0, 0, 0, :64] = 3.0            # a constant group: step 0
    kv[0, 1, 0, :64] = 0.0
    kv[T // 2, 0, 0, 1] = 1e-40       # beside subnormal and large entries
    kv[T // 2, 1, 0, 2] = 100.0 * scale
    k, v = kv[:, 0], kv[:, 1]         # strided rows
    slots = torch.randperm(n_pages * P, generator=g, device=DEV)[:T].int()
    slots[T - 1] = -1 if T > 1 else slots[T - 1]
    attn.append(k, v, slots, cache)
    k2, v2 = attn.read(slots, cache)
    assert attn.device_error() == moe.MOE_OK
    n = T - 1 if T > 1 else T
    for got, x in ((k2, k), (v2, v)):
        want, code = code_reference(x.float().cpu().numpy())
        assert np.array_equal(got.float().cpu().numpy()[:n], want[:n])
        assert T == 1 or not got[n].any()  # the skipped slot reads as zeros
        if T > 6:
            assert set(np.unique(code)) == set(range(16))
    # the documented layout: word j of group g at (j ^ f(s)) * (D / 64) + g, lowest nibble first
    s = int(slots[0])
    f = ((s & 3) << 1) ^ (s & 4)
    record = cache.data[s // P, Hkv - 1, s % P // 16]
    words = record[s % 16 * D // 2:][:D // 2].cpu().numpy().view(np.uint32)
    _, code = code_reference(k[0, Hkv - 1].float().cpu().numpy())
    for j in range(8):
        for grp in range(D // 64):
            w = int(words[(j ^ f) * (D // 64) + grp])
            assert [(w >> (4 * e)) & 15 for e in range(8)] == \
                code[64 * grp + 8 * j:64 * grp + 8 * j + 8].astype(int).tolist()
    # rows that no slot names are left alone
    rest = torch.ones(n_pages * P, dtype=torch.bool, device=DEV)
    rest[slots[:n].long()] = False
    codes = cache.data[..., 10 * D:].unflatten(-1, (16, D // 2))  # of the values
    flat = codes.flatten(2, 3).transpose(1, 2).reshape(n_pages * P, -1)
    assert bool((flat[rest] == 77).all())
    attn.close()


def test_rows_that_are_not_finite_read_as_nan_and_bad_slots_are_recorded():
    import torch
    attn = moe.PagedAttention(8, 4, 128, 16, 4, 1)
    cache = attn.new_cache()
    k, v = randn(gen(1), 5, 4, 128).bfloat16(), randn(gen(2), 5, 4, 128).bfloat16()
    k[1, 2, 5] = math.nan
    v[2, 3, 100] = math.inf
    k[3, 0, 0], k[3, 0, 1] = 3e38, -3e38  # a range beyond fp32
    slots = ints([3, 4, 5, 60, 64])
    attn.append(k, v, slots, cache)
    assert attn.device_error() == moe.MOE_ERR_DEVICE  # slot 64 of 64
    k2, v2 = attn.read(slots, cache)
    assert attn.device_error() == moe.MOE_ERR_DEVICE
    nan = torch.zeros(5, 4, dtype=torch.bool, device=DEV)
    nan[1, 2] = nan[2, 3] = nan[3, 0] = True
    assert torch.equal(k2.isnan().all(-1), nan) and torch.equal(k2.isnan().any(-1), nan)
    assert bool((v2[nan] == 0).all()) and not bool(v2.isnan().any())
    assert not k2[4].any() and not v2[4].any()
    attn.close()


# --------------------------------------------------------------------------------- attention

class Setup:
    """Requests with random contexts in randomly placed pages; what was not written is NaN."""

    def __init__(self, Hq, Hkv, D, P, new, kv, seed, scale=0.0, v_gain=0.5, q_gain=1.5, q=None,
                 first_page=0, n_pages=None, alive=None):
        import torch
        g = gen(seed)
        self.Hq, self.Hkv, self.D, self.P, self.new, self.kv = Hq, Hkv, D, P, new, kv
        B, pages = len(new), [-(-n // P) for n in kv]
        self.n_pages = n_pages or first_page + sum(pages) + 2
        self.width = max(pages + [0]) + 1
        self.scale = scale or D ** -0.5
        self.attn = moe.PagedAttention(Hq, Hkv, D, P, self.n_pages, max(B, 1), scale=scale)
        self.cache = self.attn.new_cache()
        self.cache.data.fill_(255)
        ids = first_page + torch.randperm(self.n_pages - first_page, generator=g, device=DEV)
        self.table = torch.full((B, self.width), 1 << 30, dtype=torch.int32, device=DEV)
        slots, used = [], 0
        for b in range(B):
            mine = ids[used:used + pages[b]]
            used += pages[b]
            self.table[b, :pages[b]] = mine.int()
            at = torch.arange(kv[b], device=DEV)
            slots.append(mine[at // P] * P + at % P if kv[b] else at)
        self.slots = torch.cat(slots).int()
        n = sum(kv)
        k = (randn(g, n, Hkv, D) * (0.5 + torch.rand(Hkv, D, generator=g, device=DEV)))
        v = randn(g, n, Hkv, D) * v_gain
        self.k, self.v = k.bfloat16(), v.bfloat16()
        if alive:
            alive(self)
        if n:
            self.attn.append(self.k, self.v, self.slots, self.cache)
        self.T = sum(new)
        self.q = (randn(g, self.T, Hq, D) * q_gain).bfloat16() if q is None else q
        self.q_offsets = ints(np.concatenate([[0], np.cumsum(new)]).astype(int).tolist())
        self.kv_lens = ints(kv)

    def forward(self, **kw):
        a = dict(max_q_len=max(self.new + [1]), max_kv_len=max(self.kv + [0]))
        a.update(kw)
        return self.attn.forward(self.q, self.cache, self.table, self.q_offsets, self.kv_lens, **a)

    def cached(self):
        """What the cache holds, per the definition, in fp64."""
        import torch
        ks = []
        for x in (self.k, self.v):
            g = x.float().unflatten(-1, (-1, 64))
            lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
            step = ((hi - lo) / 15.0).bfloat16().float()
            code = torch.where(step > 0, ((g - lo) / step).round(), 0.0).clamp(0, 15)
            ks.append((step.double() * code.double() + lo.double()).flatten(-2))
        return ks

    def reference(self):
        import torch
        k, v = self.cached()
        out = torch.zeros(self.T, self.Hq, self.D, dtype=torch.float64, device=DEV)
        G = self.Hq // self.Hkv
        row = key = 0
        for n, L in zip(self.new, self.kv):
            kk = k[key:key + L].repeat_interleave(G, 1)
            vv = v[key:key + L].repeat_interleave(G, 1)
            if n and L:
                s = torch.einsum("ihd,thd->hit", self.q[row:row + n].double(), kk) * self.scale
                pos = L - n + torch.arange(n, device=DEV)
                s.masked_fill_(torch.arange(L, device=DEV) > pos[:, None], -math.inf)
                p = torch.softmax(s, -1)
                p[:, pos < 0] = 0.0
                p = torch.where(p.isnan() & (pos < 0)[None, :, None], 0.0, p)
                out[row:row + n] = torch.einsum("hit,thd->ihd", p, vv)
            row, key = row + n, key + L
        return out

    def close_to(self, got, ref):
        vmax = self.v.double().abs().max() if self.v.numel() else 0.0
        err = (got.double() - ref).abs()
        bad = ~(err <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * vmax)
        assert not bool(bad.any()), (f"{int(bad.sum())} of {bad.numel()} outputs out of bound, "
                                     f"max error {err.max().item()}, max |v| {float(vmax)}")

    def check(self, got, ref=None):
        self.close_to(got, self.reference() if ref is None else ref)
        assert self.attn.device_error() == moe.MOE_OK


HEADS = [(16, 2, 256), (32, 8, 128), (28, 4, 128), (16, 1, 128), (8, 8, 64), (6, 2, 256),
         (32, 4, 64), (16, 1, 256), (1, 1, 64)]
LENGTHS = [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 500, 513, 0]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("P", [16, 64, 256])
def test_one_token_over_ragged_contexts(Hq, Hkv, D, P):
    s = Setup(Hq, Hkv, D, P, [1] * len(LENGTHS), LENGTHS, seed=D + P)
    got = s.forward()
    s.check(got)
    # the other kernel choices: short contexts in one block each, and the evenly cut launch
    s.check(s.forward(max_kv_len=0))
    s.check(s.forward(max_kv_len=1 << 20))


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_several_tokens_are_causal(Hq, Hkv, D):
    new = [2, 5, 1, 8, 3, 0, 7]
    kv = [2, 300, 1, 2000, 64, 90, 31]
    s = Setup(Hq, Hkv, D, 32, new, kv, seed=D)
    s.check(s.forward())


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("P", [16, 128])
def test_prompts_and_chunks(Hq, Hkv, D, P):
    new = [130, 1, 257, 64, 0, 33]
    kv = [130, 700, 1000, 64, 77, 1500]
    s = Setup(Hq, Hkv, D, P, new, kv, seed=D + P)
    s.check(s.forward())


@pytest.mark.parametrize("Hq,Hkv,D,n,L", [(16, 2, 256, 1500, 1500), (28, 4, 128, 700, 5000),
                                          (8, 8, 64, 1111, 1234)])
def test_long_prompts(Hq, Hkv, D, n, L):
    s = Setup(Hq, Hkv, D, 64, [n], [L], seed=n)
    s.check(s.forward())


def test_queries_that_see_nothing_give_zero():
    # fewer cached tokens than queries: the first queries sit before the context's start
    for new, kv in (([4], [2]), ([6, 1, 20], [0, 0, 3]), ([40], [10])):
        s = Setup(16, 2, 256, 16, new, kv, seed=5)
        got = s.forward()
        s.check(got)
        assert not got[:max(0, new[0] - kv[0])].any()


@pytest.mark.parametrize("L", [20000, 131071])
@pytest.mark.parametrize("q_gain", [0.0, 1.5, 40.0])
def test_long_contexts(L, q_gain):
    # uniform weights (every token counts alike), ordinary ones, and weights of a single token;
    # the mean of L values is small beside them, so the bound follows the output's size
    s = Setup(16, 2, 256, 64, [1], [L], seed=7, q_gain=q_gain)
    ref = s.reference()
    got = s.forward()
    s.check(got, ref)
    rel = ((got.double() - ref).square().sum() / ref.square().sum()).sqrt().item()
    assert rel < 2.0 ** -8, rel


@pytest.mark.parametrize("v_gain", [1e-20, 1e-4, 3e3, 1e30])
@pytest.mark.parametrize("n", [1, 40])
def test_values_of_any_size(v_gain, n):
    s = Setup(16, 2, 256, 32, [n, n], [300, 900], seed=9, v_gain=v_gain)
    s.check(s.forward())


@pytest.mark.parametrize("n", [1, 40])
def test_values_of_mixed_sizes(n):
    # groups and tokens whose scales lie 40 binary orders apart: each group keeps its own accuracy
    def alive(s):
        s.v[:, :, 64:128] *= 2.0 ** -20
        s.v[::3] *= 2.0 ** -20
        s.k[:, :, :64] *= 2.0 ** -12
    s = Setup(16, 2, 256, 32, [n], [800], seed=10, alive=alive)
    got, ref = s.forward(), s.reference()
    for g in range(4):
        part = slice(64 * g, 64 * g + 64)
        top = s.v[:, :, part].double().abs().max()
        err = (got[..., part].double() - ref[..., part]).abs()
        # decode kernels keep 2^-12 of each token's values, prompts 2^-19 of a tile's largest
        floor = 2.0 ** -10 * top + (2.0 ** -17 * s.v.double().abs().max() if n > 1 else 0)
        assert bool((err <= 2.0 ** -8 * ref[..., part].abs() + floor).all())


@pytest.mark.parametrize("n", [1, 3, 50])
def test_a_poisoned_token_reaches_exactly_the_queries_that_see_it(n):
    import torch

    def alive(s):
        s.k[120, 1, 3] = math.nan
        s.v[118, 0, 200] = math.inf
    s = Setup(16, 2, 256, 16, [n], [121], seed=11, alive=alive)
    got = s.forward()
    pos = 121 - n + torch.arange(n, device=DEV)
    nan = got.isnan()
    assert torch.equal(nan.any(-1), nan.all(-1))
    nan = nan.any(-1)
    assert torch.equal(nan[:, :8], (pos >= 118)[:, None].expand(n, 8))
    assert torch.equal(nan[:, 8:], (pos >= 120)[:, None].expand(n, 8))


@pytest.mark.parametrize("n", [1, 40])
def test_infinite_and_nan_queries_stay_in_their_row(n):
    import torch
    q = (randn(gen(1), 2 * n, 16, 256)).bfloat16()
    q[0, 3, 7] = math.nan
    q[1, 9, 0] = math.inf
    s = Setup(16, 2, 256, 64, [n, n], [100, 200], seed=12, q=q)
    got = s.forward()
    bad = torch.zeros(2 * n, 16, dtype=torch.bool, device=DEV)
    bad[0, 3] = bad[1, 9] = True
    assert torch.equal(got.isnan().any(-1), bad)
    s.q = torch.where(bad[..., None], torch.zeros_like(q), q)
    want = s.forward()
    assert torch.equal(got[~bad], want[~bad])


def test_strided_rows_other_streams_and_the_same_bits_again():
    import torch
    new, kv = [1, 3, 17, 200], [2000, 700, 17, 1000]
    s = Setup(32, 8, 128, 32, new, kv, seed=13)
    want = s.forward()
    s.check(want)
    assert torch.equal(want, s.forward())
    wide_q = torch.full((s.T, 50 * 128), 9.0, dtype=torch.bfloat16, device=DEV)
    wide_o = torch.full((s.T + 2, 40 * 128), 7.0, dtype=torch.bfloat16, device=DEV)
    q = wide_q[:, 128:33 * 128].unflatten(1, (32, 128))
    q.copy_(s.q)
    o = wide_o[1:s.T + 1, 256:34 * 128].unflatten(1, (32, 128))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.q = q
    s.forward(out=o, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, want)
    wide_o[1:s.T + 1, 256:34 * 128] = 7.0
    assert bool((wide_o == 7.0).all())


def test_many_requests_and_rows_of_nobody():
    import torch
    rng = np.random.default_rng(3)
    B = 300  # more requests than a block has threads
    new = rng.integers(0, 3, B).tolist()
    kv = [int(n + x) for n, x in zip(new, np.exp(rng.uniform(0, 7.5, B)))]
    s = Setup(8, 8, 64, 16, new, kv, seed=14)
    extra = torch.cat([s.q, s.q[:3]])
    out = torch.full_like(extra, 5.0)
    s.q = extra
    s.forward(out=out)
    assert bool((out[s.T:] == 5.0).all())
    s.q = extra[:s.T]
    s.check(out[:s.T])


def test_a_cache_beyond_32_bit_offsets():
    # the last pages of a cache whose arrays pass 4 GiB
    n_pages = (10 << 30) // (64 * 2 * 288)
    for new in ([1, 1], [1, 90]):
        s = Setup(16, 2, 256, 64, new, [700, 100], seed=15, n_pages=n_pages,
                  first_page=n_pages - 20)
        assert s.cache.data.numel() > 5e9
        s.check(s.forward())
        s.attn.close()
        del s


def test_pages_and_lengths_out_of_range_are_recorded_and_harmless():
    import torch
    for new, kv in (([1, 1, 1], [300, 900, 64]), ([40, 1, 1], [300, 900, 64])):
        s = Setup(16, 2, 256, 64, new, kv, seed=16)
        want = s.forward()
        assert s.attn.device_error() == moe.MOE_OK
        keep = s.table.clone()
        s.table[1, 3] = s.n_pages
        got = s.forward()
        assert s.attn.device_error() == moe.MOE_ERR_DEVICE
        # (the batch as a whole decides where contexts are cut, so the bits of the other
        # requests may change with it, within the bound)
        n0, ref = new[0], s.reference()
        s.close_to(got[:n0], ref[:n0])
        s.close_to(got[n0 + 1:], ref[n0 + 1:])
        s.table[1, 3] = -1
        s.forward()
        assert s.attn.device_error() == moe.MOE_ERR_DEVICE
        s.table = keep
        s.kv_lens = ints([kv[0], -5, 64])
        got = s.forward()
        assert s.attn.device_error() == moe.MOE_ERR_DEVICE
        s.close_to(got[:n0], ref[:n0])
        assert not got[n0].any()
        s.kv_lens = ints([kv[0], 1 << 30, 64])  # longer than the table
        s.forward()
        assert s.attn.device_error() == moe.MOE_ERR_DEVICE
        s.kv_lens = ints(kv)
        s.q_offsets = ints([0, n0, n0 + 1, 1 << 20])
        s.forward()
        assert s.attn.device_error() == moe.MOE_ERR_DEVICE
        s.q_offsets = ints([0, n0, -1, n0 + 2])
        s.forward()
        assert s.attn.device_error() == moe.MOE_ERR_DEVICE
        s.q_offsets = ints([0, n0, n0 + 1, n0 + 2])
        assert torch.equal(s.forward(), want)
        assert s.attn.device_error() == moe.MOE_OK


def test_arguments_are_refused_on_the_host():
    import torch
    s = Setup(16, 2, 256, 64, [1], [100], seed=17)
    A = 0x100000  # never dereferenced: every call below fails in the argument checks
    h, c = s.attn.handle, s.cache.ptr
    OK, INV, UNS, ALI = (moe.MOE_OK, moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED,
                         moe.MOE_ERR_ALIGNMENT)

    def fwd(q=A, qs=4096, cache=c, table=A, width=4, qo=A, kv=A, B=1, T=1, mq=1, mk=1, out=A,
            os=4096):
        return moe.attn_kv4_forward(h, q, qs, cache, table, width, qo, kv, B, T, mq, mk, out, os,
                                    None)
    assert fwd(T=0) == OK and fwd(B=0) == OK
    assert fwd(q=None) == INV and fwd(out=None) == INV and fwd(cache=None) == INV
    assert fwd(qo=None) == INV and fwd(kv=None) == INV and fwd(table=None) == INV
    assert fwd(B=-1) == INV and fwd(T=-1) == INV and fwd(mq=0) == INV and fwd(mk=-1) == INV
    assert fwd(qs=4000) == INV and fwd(os=4088) == INV
    assert fwd(B=2) == UNS and fwd(T=(1 << 20) + 1) == UNS
    assert fwd(q=A + 8) == ALI and fwd(out=A + 2) == ALI and fwd(qs=4100) == ALI
    assert fwd(table=A + 2) == ALI and fwd(qo=A + 1) == ALI and fwd(kv=A + 2) == ALI
    assert fwd(cache=A + 64) == ALI

    def rope(q=A, qs=4096, k=A, ks=512, pos=A, qw=A, kw=A, eps=1e-6, cs=A, n=4, rot=64, T=1,
             qo=A, qos=4096, ko=A, kos=512):
        return moe.attn_qk_norm_rope(h, q, qs, k, ks, pos, qw, kw, eps, cs, n, rot, 0, T, qo, qos,
                                     ko, kos, None)
    assert rope(T=0) == OK
    for name in ("q", "k", "pos", "qw", "kw", "cs", "qo", "ko"):
        assert rope(**{name: None}) == INV, name
    assert rope(T=-1) == INV and rope(n=0) == INV and rope(rot=-16) == INV
    assert rope(eps=-1.0) == INV and rope(eps=math.nan) == INV
    assert rope(rot=40) == UNS and rope(rot=272) == UNS and rope(T=(1 << 20) + 1) == UNS
    assert rope(ks=504) == INV and rope(kos=516) == ALI and rope(q=A + 4) == ALI
    assert rope(cs=A + 4) == ALI and rope(pos=A + 2) == ALI and rope(kw=A + 8) == ALI

    def rows(fn, k=A, ks=512, v=A, vs=512, slots=A, T=1, cache=c):
        if fn == "append":
            return moe.attn_kv4_append(h, k, ks, v, vs, slots, T, cache, None)
        return moe.attn_kv4_read(h, cache, slots, T, k, ks, v, vs, None)
    for fn in ("append", "read"):
        assert rows(fn, T=0) == OK and rows(fn, T=-1) == INV
        for name in ("k", "v", "slots", "cache"):
            assert rows(fn, **{name: None}) == INV, name
        assert rows(fn, ks=511) == INV and rows(fn, vs=516) == ALI
        assert rows(fn, k=A + 8) == ALI and rows(fn, slots=A + 2) == ALI

    def plan(table=A, w=4, ctx=A, new=A, B=1, free=A, nf=1, cur=A, T=1, qo=A, kv=A, pos=A,
             slots=A, co=A):
        return moe.attn_plan(h, table, w, ctx, new, B, free, nf, cur, T, qo, kv, pos, slots, co,
                             None)
    for name in ("table", "ctx", "new", "free", "cur", "qo", "kv", "pos", "slots", "co"):
        assert plan(**{name: None}) == INV, name
        assert plan(**{name: A + 2}) == ALI, name
    assert plan(B=-1) == INV and plan(T=-1) == INV and plan(w=-1) == INV and plan(nf=-1) == INV
    assert plan(B=2) == UNS and plan(T=(1 << 20) + 1) == UNS

    # the class: types, shapes, devices and strides
    with pytest.raises(moe.MoeError):
        s.attn.forward(s.q.float(), s.cache, s.table, s.q_offsets, s.kv_lens, 1, 100)
    with pytest.raises(moe.MoeError):
        s.attn.forward(s.q[:, :8], s.cache, s.table, s.q_offsets, s.kv_lens, 1, 100)
    with pytest.raises(moe.MoeError):
        s.attn.forward(s.q, s.cache, s.table, s.q_offsets.long(), s.kv_lens, 1, 100)
    with pytest.raises(moe.MoeError):
        s.attn.forward(s.q, s.cache, s.table, s.q_offsets.cpu(), s.kv_lens, 1, 100)
    with pytest.raises(moe.MoeError):
        s.attn.append(s.k, s.v[:-1], s.slots, s.cache)
    with pytest.raises(moe.MoeError):
        s.attn.append(s.k.transpose(1, 2).contiguous().transpose(1, 2), s.v, s.slots, s.cache)
    with pytest.raises(moe.MoeError):
        s.attn.plan(s.table, s.kv_lens, s.kv_lens, s.slots, ints([0]))
    torch.cuda.synchronize()
    s.check(s.forward())
