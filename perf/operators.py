"""The attention step of serving over a paged 4-bit key/value cache, as measured work.

Four operators, in the order in which a serving step runs them: the step's block tables and slot
maps ("plan"), the norm and rotation of the query and key heads ("rotate"), the quantisation of
keys and values into cached pages and their read-back ("append"), and the attention of the new
tokens over the cache ("attention").  `run` computes each in plain torch operations (own = False)
or through the package (own = True), from the same state.
"""
import math
import random

import torch

own = False

DEV = "cuda"
GROUP = 64  # channels that share one scale and one bias


# ------------------------------------------------------------------------------------- cases

# (query heads, key/value heads, head size)
HEADS = [(16, 2, 256), (16, 2, 256), (32, 8, 128), (28, 4, 128), (16, 1, 128), (8, 8, 64),
         (6, 2, 256), (32, 4, 64)]


def listed():
    return [
        # a serving step of 64 requests with one new token each
        dict(name="plan_tokens", op="plan", B=64, q_min=1, q_max=1, ctx_min=0, ctx_max=8192,
             page=64, mix=1, short=0),
        # a step that admits many prompts at once, small pages, more pages wanted than are free
        dict(name="plan_prompts", op="plan", B=301, q_min=0, q_max=400, ctx_min=0, ctx_max=32768,
             page=16, mix=2, short=40),
        # one new token of one request: latency
        dict(name="rotate_token", op="rotate", T=1, Hq=16, Hkv=2, D=256, rot=64, inter=False,
             pos_max=131072),
        # a prompt's queries and keys, all channels rotated in neighbouring pairs
        dict(name="rotate_prompt", op="rotate", T=16381, Hq=32, Hkv=8, D=128, rot=128, inter=True,
             pos_max=32768),
        # one new token of each of 48 requests
        dict(name="append_tokens", op="append", T=48, Hq=16, Hkv=2, D=256, page=64),
        # a prompt's keys and values
        dict(name="append_prompt", op="append", T=32768, Hq=16, Hkv=2, D=256, page=64),
        # one request, one new token, a short context: latency
        dict(name="attend_token", op="attention", B=1, Hq=16, Hkv=2, D=256, page=64, q_min=1,
             q_max=1, ctx_min=256, ctx_max=256, mix=1, refused=0),
        # a serving batch of ragged contexts, one new token each, two requests without pages
        dict(name="attend_batch", op="attention", B=48, Hq=16, Hkv=2, D=256, page=64, q_min=1,
             q_max=1, ctx_min=0, ctx_max=16384, mix=2, refused=2),
        # one request at the longest context
        dict(name="attend_long", op="attention", B=1, Hq=16, Hkv=2, D=256, page=64, q_min=1,
             q_max=1, ctx_min=131071, ctx_max=131071, mix=3, refused=0),
        # drafted tokens verified at once, small pages, four query heads to a key/value head
        dict(name="attend_drafts", op="attention", B=8, Hq=32, Hkv=8, D=128, page=16, q_min=2,
             q_max=5, ctx_min=500, ctx_max=8000, mix=4, refused=0),
        # a first prompt of 4096 tokens
        dict(name="attend_prompt", op="attention", B=1, Hq=16, Hkv=2, D=256, page=64, q_min=4096,
             q_max=4096, ctx_min=0, ctx_max=0, mix=5, refused=0),
        # chunks of several prompts beside requests that decode, ragged contexts
        dict(name="attend_chunks", op="attention", B=7, Hq=28, Hkv=4, D=128, page=32, q_min=1,
             q_max=1500, ctx_min=0, ctx_max=20000, mix=6, refused=1),
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _size_ok(case):
    widths = [v for v in case.values() if not isinstance(v, (str, bool))]
    if "D" in case:
        widths += [case["Hq"] * case["D"], (case["Hq"] + 2 * case["Hkv"]) * case["D"]]
    return 3 * 1024 not in widths


def draw(rng):
    top = {k: max(work(c)[k] for c in listed()) for k in ("bytes", "flops")}
    while True:
        Hq, Hkv, D = rng.choice(HEADS)
        heads = dict(Hq=Hq, Hkv=Hkv, D=D)
        kind = rng.choice(["plan", "rotate", "append", "attention", "attention", "attention"])
        if kind == "plan":
            one = rng.random() < 0.4
            case = dict(op="plan", B=_log(rng, 1, 301), q_min=1 if one else 0,
                        q_max=1 if one else _log(rng, 2, 400), ctx_min=0,
                        ctx_max=_log(rng, 64, 32768), page=rng.choice([16, 32, 64, 128, 256]),
                        mix=rng.randrange(1 << 20), short=rng.choice([0, 0, 1, 40]))
        elif kind == "rotate":
            rot = rng.choice([r for r in (16, 32, 64, 128, 256) if r <= D])
            case = dict(op="rotate", T=_log(rng, 1, 16381), rot=rot, inter=rng.random() < 0.5,
                        pos_max=rng.choice([4096, 32768, 131072]), **heads)
        elif kind == "append":
            case = dict(op="append", T=_log(rng, 1, 32768),
                        page=rng.choice([16, 32, 64, 128, 256]), **heads)
        else:
            form = rng.choice(["tokens", "drafts", "chunks"])
            B = {"tokens": _log(rng, 1, 64), "drafts": _log(rng, 1, 16),
                 "chunks": _log(rng, 1, 8)}[form]
            q_max = {"tokens": 1, "drafts": rng.randint(2, 8),
                     "chunks": _log(rng, 9, 4096)}[form]
            ctx_max = _log(rng, 1, 131071 if B == 1 else 32768)
            case = dict(op="attention", B=B, page=rng.choice([16, 32, 64, 128, 256]), q_min=1,
                        q_max=q_max, ctx_min=0, ctx_max=ctx_max, mix=rng.randrange(1 << 20),
                        refused=rng.choice([0, 0, 1]) if B > 1 else 0, **heads)
        w = work(case)
        # (a rotation's positions are rows of its table, which holds pos_max of them)
        if _size_ok(case) and all(w[k] <= top[k] for k in top) \
                and case.get("T", 0) <= case.get("pos_max", math.inf):
            return case


def _lengths(case):
    """(new tokens, cached tokens) of each request: one spread of lengths for each mix, ragged,
    drawn over their logarithm, with the longest of each among them."""
    rng = random.Random(case["mix"] * 7919 + case["B"])
    new, ctx = [], []
    for i in range(case["B"]):
        new.append(_log(rng, case["q_min"] + 1, case["q_max"] + 1) - 1 if i else case["q_max"])
        ctx.append(_log(rng, case["ctx_min"] + 1, case["ctx_max"] + 1) - 1 if i
                   else case["ctx_max"])
    return new, ctx


def _row_bytes(case):
    """Bytes of one cached key (or value) row of one head: codes, scales, biases."""
    return case["D"] // 2 + 4 * (case["D"] // GROUP)


def work(case):
    if case["op"] == "plan":
        new, ctx = _lengths(case)
        fresh = sum(-(-(c + n) // case["page"]) - -(-c // case["page"]) for n, c in zip(new, ctx))
        # lengths in, offsets and lengths out, the new table entries, a position and a slot a token
        return {"bytes": 4 * (4 * case["B"] + 2 * fresh + 2 * sum(new)), "flops": 0}
    T = case.get("T")
    if case["op"] == "rotate":
        n = (case["Hq"] + case["Hkv"]) * case["D"]
        # heads in and out, the rotations and positions of the tokens; a square, two scalings a
        # channel and three operations a rotated channel
        return {"bytes": T * (4 * n + 4 * case["rot"] + 4) + 4 * case["D"],
                "flops": T * (4 * n + 3 * (case["Hq"] + case["Hkv"]) * case["rot"])}
    if case["op"] == "append":
        n = 2 * case["Hkv"]
        # rows in, rows into the cache, rows out of it, rows back; about six operations a channel
        return {"bytes": T * n * (4 * case["D"] + 2 * _row_bytes(case)) + 4 * T,
                "flops": T * n * 8 * case["D"]}
    new, ctx = _lengths(case)
    kept = list(zip(new, ctx))[case["refused"]:]
    pairs = sum(n * c + n * (n + 1) // 2 for n, c in kept)
    rows = sum(n + c for n, c in kept if n)
    # queries in, outputs out, every visible cached row once; two products over the head size
    return {"bytes": 4 * sum(new) * case["Hq"] * case["D"]
                     + 2 * rows * case["Hkv"] * _row_bytes(case),
            "flops": 4 * case["D"] * case["Hq"] * pairs}


# ------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _keys_values(g, T, Hkv, D):
    """Keys as they leave the norm (a few channels much larger than the rest) and values."""
    gain = 0.5 + torch.rand(Hkv, D, generator=g, device=DEV)
    gain[:, ::61] *= 4.0
    k = (_randn(g, T, Hkv, D) * gain).bfloat16()
    v = (_randn(g, T, Hkv, D) * 0.5).bfloat16()
    return k, v


def _plan_inputs(case, seed):
    g = _gen(seed)
    new, ctx = _lengths(case)
    page, B = case["page"], case["B"]
    width = max(-(-(c + n) // page) for n, c in zip(new, ctx)) + 1
    held = [-(-c // page) for c in ctx]
    fresh = [-(-(c + n) // page) - h for n, c, h in zip(new, ctx, held)]
    n_pages = sum(held) + sum(fresh) + 8
    ids = torch.randperm(n_pages, generator=g, device=DEV).int()
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    cols = torch.arange(width, device=DEV)
    has = cols[None, :] < torch.tensor(held, device=DEV)[:, None]
    table[has] = ids[:sum(held)]
    first = 3  # entries of the free list that earlier steps took
    free = ids[sum(held):]
    free = torch.cat([free[-first:], free])[:first + max(1, sum(fresh) - case["short"])]
    return dict(new=torch.tensor(new, dtype=torch.int32, device=DEV),
                ctx=torch.tensor(ctx, dtype=torch.int32, device=DEV), table=table,
                free=free.contiguous(),
                cursor=torch.tensor([first], dtype=torch.int32, device=DEV), T=sum(new),
                n_pages=n_pages, width=width)


def _rotate_inputs(case, seed):
    g = _gen(seed)
    T, Hq, Hkv, D, rot = (case[n] for n in ("T", "Hq", "Hkv", "D", "rot"))
    qkv = (_randn(g, T, (Hq + 2 * Hkv) * D) * 1.5).bfloat16()
    wq = (1.0 + 0.2 * _randn(g, D)).bfloat16()
    wk = (1.0 + 0.2 * _randn(g, D)).bfloat16()
    start = int(torch.randint(0, max(1, case["pos_max"] - T), (1,), generator=g, device=DEV))
    positions = torch.arange(start, start + T, device=DEV, dtype=torch.int32)
    inv = 1.0e6 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    angle = torch.arange(case["pos_max"], device=DEV, dtype=torch.float64)[:, None] * inv
    table = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
    return dict(qkv=qkv, wq=wq, wk=wk, positions=positions, table=table, eps=1e-6)


def _quantise(x):
    """Codes and bf16 (scale, bias) of rows x [..., D] in groups of 64 channels, in 32 bits."""
    xg = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = xg.amin(-1), xg.amax(-1)
    scale = ((hi - lo) / 15.0).bfloat16()
    s = scale.float().unsqueeze(-1)
    code = torch.where(s > 0, ((xg - lo.unsqueeze(-1)) / s).round(), torch.zeros_like(xg))
    return code.clamp(0, 15).to(torch.uint8).flatten(-2), scale, lo.bfloat16()


def _append_inputs(case, seed):
    g = _gen(seed)
    T, Hkv, D, page = (case[n] for n in ("T", "Hkv", "D", "page"))
    n_pages = -(-T // page) + 5
    k, v = _keys_values(g, T, Hkv, D)
    fused = torch.empty(T, 2 * Hkv * D, dtype=torch.bfloat16, device=DEV)
    fused[:, Hkv * D:] = v.flatten(1)  # the values as a projection's output holds them
    ids = torch.randperm(n_pages, generator=g, device=DEV)
    at = torch.arange(3, 3 + T, device=DEV)  # from inside a page on
    slots = (ids[at // page] * page + at % page).int()
    return dict(k=k, v=fused[:, Hkv * D:].unflatten(1, (Hkv, D)), slots=slots, n_pages=n_pages)


def _attention_inputs(case, seed):
    g = _gen(seed)
    Hq, Hkv, D, page, B = (case[n] for n in ("Hq", "Hkv", "D", "page", "B"))
    new, ctx = _lengths(case)
    kv = [0 if b < case["refused"] else n + c for b, (n, c) in enumerate(zip(new, ctx))]
    q = (_randn(g, sum(new), Hq, D) * 1.5).bfloat16()
    pages = [-(-n // page) for n in kv]
    n_pages = sum(pages) + 3
    width = max(max(pages), 1) + 1
    ids = torch.randperm(n_pages, generator=g, device=DEV)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    slots, used = [], 0
    for b in range(B):
        mine = ids[used:used + pages[b]]
        used += pages[b]
        table[b, :pages[b]] = mine.int()
        at = torch.arange(kv[b], device=DEV)
        if kv[b]:
            slots.append(mine[at // page] * page + at % page)
    slots = torch.cat(slots).int() if slots else torch.empty(0, dtype=torch.int32, device=DEV)
    k, v = _keys_values(g, sum(kv), Hkv, D)
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    return dict(q=q, k=k, v=v, slots=slots, table=table, new=new, kv=kv, n_pages=n_pages,
                width=width, q_offsets=torch.tensor(offsets, dtype=torch.int32, device=DEV),
                kv_lens=torch.tensor(kv, dtype=torch.int32, device=DEV))


_INPUTS = {"plan": _plan_inputs, "rotate": _rotate_inputs, "append": _append_inputs,
           "attention": _attention_inputs}


def _pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).contiguous()


def _unpack(packed):
    return torch.stack([packed & 15, packed >> 4], -1).flatten(-2)


def prepare(case, seed):
    s = dict(_INPUTS[case["op"]](case, seed), case=case)
    op = case["op"]
    if own:
        import sparse_moe_02_gb300 as moe
        s["attn"] = moe.PagedAttention(case.get("Hq", 16), case.get("Hkv", 2), case.get("D", 256),
                                       case.get("page", 64), s.get("n_pages", 1),
                                       max_requests=case.get("B", 1))
    if op == "plan":
        T, B = s["T"], case["B"]
        s["out"] = dict(q_offsets=torch.empty(B + 1, dtype=torch.int32, device=DEV),
                        kv_lens=torch.empty(B, dtype=torch.int32, device=DEV),
                        positions=torch.empty(T, dtype=torch.int32, device=DEV),
                        slots=torch.empty(T, dtype=torch.int32, device=DEV),
                        cursor=torch.empty(1, dtype=torch.int32, device=DEV))
    elif op == "rotate":
        T, Hq, Hkv, D = (case[n] for n in ("T", "Hq", "Hkv", "D"))
        s["q"] = s["qkv"][:, :Hq * D].unflatten(1, (Hq, D))
        s["k"] = s["qkv"][:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["k_out"] = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV)
    else:
        rows, Hkv, D = s["n_pages"] * case["page"], case["Hkv"], case["D"]
        if own:
            s["cache"] = s["attn"].new_cache()
        else:  # what was never written reads as NaN
            s["codes"] = torch.full((2, rows, Hkv, D // 2), 255, dtype=torch.uint8, device=DEV)
            s["scale"] = torch.full((2, rows, Hkv, D // GROUP), math.nan, dtype=torch.bfloat16,
                                    device=DEV)
            s["bias"] = s["scale"].clone()
        if op == "append":
            s["k_out"] = torch.empty(case["T"], Hkv, D, dtype=torch.bfloat16, device=DEV)
            s["v_out"] = torch.empty_like(s["k_out"])
        else:
            s["out"] = torch.empty_like(s["q"])
            if own:
                s["attn"].append(s["k"], s["v"], s["slots"], s["cache"])
            else:
                _plain_write(s)
            del s["k"], s["v"]
    return s


# ---------------------------------------------------------------------------------- plain forms

def _plain_plan(s):
    case, T = s["case"], s["T"]
    page = case["page"]
    new, ctx, table, free = s["new"].long(), s["ctx"].long(), s["table"], s["free"].long()
    before = (ctx + page - 1) // page
    after = (ctx + new + page - 1) // page
    ends = new.cumsum(0)
    bad = (after > table.shape[1]) | (ends > T)
    need = torch.where(bad, 0, after - before)
    end = need.cumsum(0)
    cursor = s["cursor"].long()
    refused = bad | ((need > 0) & (end > free.numel() - cursor))
    cols = torch.arange(table.shape[1], device=DEV)[None, :]
    j = cols - before[:, None]
    fill = (j >= 0) & (j < need[:, None]) & ~refused[:, None]
    take = (cursor + (end - need)[:, None] + j).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fill, free[take], table.long()))
    q_offsets = torch.cat([ends.new_zeros(1), ends]).clamp(max=T)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(q_offsets[1:].contiguous(), t, right=True)
    pos = ctx[b] + t - q_offsets[b]
    slot = table[b, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    o = s["out"]
    o["q_offsets"].copy_(q_offsets)
    o["kv_lens"].copy_(torch.where(refused, 0, ctx + new))
    o["positions"].copy_(pos)
    o["slots"].copy_(torch.where(refused[b], -1, slot))
    o["cursor"].copy_(cursor + torch.where(refused | (need == 0), 0, end).max())
    return [table, o["q_offsets"], o["kv_lens"], o["positions"], o["slots"], o["cursor"]]


def _plain_norm_rotate(x, w, cos, sin, rot, inter, eps):
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + eps) * w.float()
    head, tail = y[..., :rot], y[..., rot:]
    if inter:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([head, tail], -1)


def _plain_rotate(s):
    case = s["case"]
    rot = case["rot"]
    cs = s["table"][s["positions"].long()].unsqueeze(1)
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    for x, w, out in ((s["q"], s["wq"], s["q_out"]), (s["k"], s["wk"], s["k_out"])):
        out.copy_(_plain_norm_rotate(x, w, cos, sin, rot, case["inter"], s["eps"]))
    return [s["q_out"], s["k_out"]]


def _plain_write(s):
    at = s["slots"].long()
    for i, x in enumerate((s["k"], s["v"])):
        codes, scale, bias = _quantise(x)
        s["codes"][i, at] = _pack(codes)
        s["scale"][i, at] = scale
        s["bias"][i, at] = bias


def _plain_read(s, i, at):
    codes = _unpack(s["codes"][i, at]).float().unflatten(-1, (-1, GROUP))
    return (codes * s["scale"][i, at].float().unsqueeze(-1)
            + s["bias"][i, at].float().unsqueeze(-1)).flatten(-2)


def _plain_append(s):
    _plain_write(s)
    at = s["slots"].long()
    s["k_out"].copy_(_plain_read(s, 0, at))
    s["v_out"].copy_(_plain_read(s, 1, at))
    return [s["k_out"], s["v_out"]]


def _plain_attention(s):
    case = s["case"]
    Hq, Hkv, D, page = (case[n] for n in ("Hq", "Hkv", "D", "page"))
    G, out, first = Hq // Hkv, s["out"], 0
    for b, (n, L) in enumerate(zip(s["new"], s["kv"])):
        if n and not L:
            out[first:first + n] = 0
        elif n:
            at = torch.arange(L, device=DEV)
            at = s["table"][b].long()[at // page] * page + at % page
            k = _plain_read(s, 0, at).permute(1, 2, 0)            # [Hkv, D, L]
            v = _plain_read(s, 1, at).permute(1, 0, 2)            # [Hkv, L, D]
            rows = max(1, (1 << 29) // (Hq * L))                  # tokens at a time
            for i in range(0, n, rows):
                m = min(rows, n - i)
                x = s["q"][first + i:first + i + m].float().unflatten(1, (Hkv, G))
                x = x.permute(1, 0, 2, 3).reshape(Hkv, m * G, D)
                score = (x @ k) * D ** -0.5
                if n > 1:
                    pos = L - n + i + torch.arange(m, device=DEV).repeat_interleave(G)
                    score.masked_fill_(torch.arange(L, device=DEV) > pos[:, None], -math.inf)
                p = (score - score.amax(-1, keepdim=True)).exp()
                y = (p @ v) / p.sum(-1, keepdim=True)
                out[first + i:first + i + m] = y.view(Hkv, m, G, D).transpose(0, 1).flatten(1, 2)
        first += n
    return out


_PLAIN = {"plan": _plain_plan, "rotate": _plain_rotate, "append": _plain_append,
          "attention": _plain_attention}


# -------------------------------------------------------------------------------- the framework

def _own(s):
    case, attn = s["case"], s["attn"]
    op = case["op"]
    if op == "plan":
        o = s["out"]
        attn.plan(s["table"], s["ctx"], s["new"], s["free"], s["cursor"], o["q_offsets"],
                  o["kv_lens"], o["positions"], o["slots"], o["cursor"])
        return [s["table"], o["q_offsets"], o["kv_lens"], o["positions"], o["slots"], o["cursor"]]
    if op == "rotate":
        attn.qk_norm_rope(s["q"], s["k"], s["positions"], s["wq"], s["wk"], s["table"],
                          eps=s["eps"], interleaved=case["inter"], q_out=s["q_out"],
                          k_out=s["k_out"])
        return [s["q_out"], s["k_out"]]
    if op == "append":
        attn.append(s["k"], s["v"], s["slots"], s["cache"])
        attn.read(s["slots"], s["cache"], k_out=s["k_out"], v_out=s["v_out"])
        return [s["k_out"], s["v_out"]]
    return attn.forward(s["q"], s["cache"], s["table"], s["q_offsets"], s["kv_lens"],
                        max_q_len=max(s["new"]), max_kv_len=max(s["kv"]), out=s["out"])


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------- in 64 bits

def _exact_rotate(case, seed):
    s = _rotate_inputs(case, seed)
    Hq, Hkv, D, rot = (case[n] for n in ("Hq", "Hkv", "D", "rot"))
    x = s["qkv"].double().view(case["T"], -1, D)
    inv = 1.0e6 ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float64) * 2 / rot)
    turn = torch.polar(torch.ones(case["T"], rot // 2, dtype=torch.float64, device=DEV),
                       s["positions"].double()[:, None] * inv)
    outs = []
    for part, w in ((x[:, :Hq], s["wq"]), (x[:, Hq:Hq + Hkv], s["wk"])):
        norm = torch.linalg.vector_norm(part, dim=-1, keepdim=True)
        y = part / torch.sqrt(norm ** 2 / D + s["eps"]) * w.double()
        if case["inter"]:
            z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * turn[:, None]
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        else:
            z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn[:, None]
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        outs.append(y)
    return outs


def _exact_cached(x):
    """What the cache holds of rows x, as 64-bit values: 16 levels from each group's smallest
    value on, a bf16 step apart."""
    g = x.double().reshape(*x.shape[:-1], -1, GROUP)
    low = g.min(-1, keepdim=True).values
    step = ((g.max(-1, keepdim=True).values - low) / 15).bfloat16().double()
    level = torch.nan_to_num((g - low) / step, nan=0.0).round().clamp(max=15)
    return (low + step * level).reshape(x.shape)


def _exact_attention(case, seed):
    s = _attention_inputs(case, seed)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    k, v = _exact_cached(s["k"]), _exact_cached(s["v"])
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    row, key = 0, 0
    for n, L in zip(s["new"], s["kv"]):
        for h in range(Hq if n and L else 0):
            kh, vh = k[key:key + L, h // G], v[key:key + L, h // G]
            score = s["q"][row:row + n, h].double() @ kh.T / math.sqrt(D)
            score += torch.full_like(score, -math.inf).triu(L - n + 1) if n > 1 else 0
            out[row:row + n, h] = torch.softmax(score, -1) @ vh
        row, key = row + n, key + L
    return out


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    if case["op"] == "rotate":
        return _exact_rotate(case, seed)
    if case["op"] == "append":
        s = _append_inputs(case, seed)
        return [_exact_cached(s["k"]), _exact_cached(s["v"])]
    return _exact_attention(case, seed)
