"""What serving with drafted tokens and window layers adds to the attention step, as measured work.

Five operators over the paged 4-bit key/value cache: the norm, rotation and quantisation of a step's
rows in one pass ("append"), attention through a sliding window with a few first tokens that stay
visible ("window"), attention of a tree of drafted tokens ("tree"), the tree's depths and ancestor
masks ("plan") and the move of the accepted tokens' cached rows to where they belong ("accept").
`run` computes each in plain torch operations (own = False) or through the package (own = True),
from the same state.
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
        # one new token of each of 48 requests: latency
        dict(name="append_tokens", op="append", T=48, Hq=16, Hkv=2, D=256, rot=64, inter=False,
             normed=True, pos_max=131072, page=64),
        # a prompt's rows, all channels rotated in neighbouring pairs, small pages
        dict(name="append_prompt", op="append", T=16381, Hq=32, Hkv=8, D=128, rot=128, inter=True,
             normed=True, pos_max=32768, page=16),
        # a serving batch on a window layer: one new token each, ragged contexts behind the window
        dict(name="window_tokens", op="window", B=48, Hq=16, Hkv=2, D=256, page=64, q_min=1,
             q_max=1, ctx_min=0, ctx_max=32768, mix=2, window=2048, sinks=4),
        # a first prompt of 8192 tokens on a window layer
        dict(name="window_prompt", op="window", B=1, Hq=16, Hkv=2, D=256, page=64, q_min=8192,
             q_max=8192, ctx_min=0, ctx_max=0, mix=5, window=1024, sinks=16),
        # chunks of several prompts beside requests that decode, an odd window, no first tokens
        dict(name="window_chunks", op="window", B=7, Hq=28, Hkv=4, D=128, page=32, q_min=1,
             q_max=1500, ctx_min=0, ctx_max=20000, mix=6, window=777, sinks=0),
        # small trees, verified at once: few query rows
        dict(name="tree_few", op="tree", B=8, Hq=32, Hkv=8, D=128, page=16, q_min=2, q_max=8,
             ctx_min=500, ctx_max=8000, mix=4, window=0, sinks=0),
        # a batch of wide trees over long ragged contexts
        dict(name="tree_batch", op="tree", B=16, Hq=16, Hkv=2, D=256, page=64, q_min=20, q_max=60,
             ctx_min=0, ctx_max=16384, mix=8, window=0, sinks=0),
        # trees on a window layer
        dict(name="tree_window", op="tree", B=32, Hq=16, Hkv=2, D=256, page=64, q_min=8, q_max=31,
             ctx_min=0, ctx_max=16384, mix=9, window=1024, sinks=4),
        # one request's tree: latency
        dict(name="plan_one", op="plan", B=1, q_min=26, q_max=26, ctx_min=700, ctx_max=700, mix=1),
        # the trees of a large batch
        dict(name="plan_batch", op="plan", B=256, q_min=1, q_max=64, ctx_min=0, ctx_max=32768,
             mix=2),
        # acceptance in a small batch: latency
        dict(name="accept_few", op="accept", B=8, Hq=32, Hkv=8, D=128, page=16, q_min=2, q_max=8,
             ctx_min=500, ctx_max=8000, mix=4),
        # acceptance in a large batch of wide trees
        dict(name="accept_batch", op="accept", B=64, Hq=16, Hkv=2, D=256, page=64, q_min=20,
             q_max=60, ctx_min=0, ctx_max=8192, mix=7),
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    top = {k: max(work(c)[k] for c in listed()) for k in ("bytes", "flops")}
    while True:
        Hq, Hkv, D = rng.choice(HEADS)
        heads = dict(Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128, 256]))
        op = rng.choice(["append", "window", "window", "window", "tree", "tree", "tree", "plan",
                         "accept"])
        mix = rng.randrange(1 << 20)
        if op == "append":
            rot = rng.choice([r for r in (16, 32, 64, 128, 256) if r <= D])
            case = dict(op=op, T=_log(rng, 1, 16381), rot=rot, inter=rng.random() < 0.5,
                        normed=rng.random() < 0.7, pos_max=rng.choice([32768, 131072]), **heads)
        elif op == "window":
            form = rng.choice(["tokens", "drafts", "chunks"])
            B = {"tokens": _log(rng, 1, 64), "drafts": _log(rng, 1, 16),
                 "chunks": _log(rng, 1, 8)}[form]
            q_max = {"tokens": 1, "drafts": rng.randint(2, 8),
                     "chunks": _log(rng, 9, 8192)}[form]
            case = dict(op=op, B=B, q_min=1, q_max=q_max, ctx_min=0, ctx_max=_log(rng, 1, 32768),
                        mix=mix, window=_log(rng, 1, 8192),
                        sinks=rng.choice([0, 0, 1, 4, 16, 100]), **heads)
        elif op == "tree":
            q_max = _log(rng, 1, 128)
            windowed = rng.random() < 0.4
            case = dict(op=op, B=_log(rng, 1, 32), q_min=rng.randint(1, q_max), q_max=q_max,
                        ctx_min=0, ctx_max=_log(rng, 1, 32768), mix=mix,
                        window=_log(rng, q_max, 8192) if windowed else 0,
                        sinks=rng.choice([0, 4, 100]) if windowed else 0, **heads)
        else:
            q_max = _log(rng, 1, 128)
            case = dict(op=op, B=_log(rng, 1, 256 if op == "plan" else 64),
                        q_min=rng.randint(1, q_max), q_max=q_max, ctx_min=0,
                        ctx_max=_log(rng, 1, 32768 if op == "plan" else 8192), mix=mix)
            if op == "accept":
                case.update(heads)
        w = work(case)
        if all(w[k] <= top[k] for k in top):
            return case


def _lengths(case):
    """(new tokens, cached tokens before them) of each request: one spread of lengths for each mix,
    ragged, drawn over their logarithm, with the longest of each among them."""
    rng = random.Random(case["mix"] * 7919 + case["B"])
    new, ctx = [], []
    for i in range(case["B"]):
        new.append(_log(rng, case["q_min"] + 1, case["q_max"] + 1) - 1 if i else case["q_max"])
        ctx.append(_log(rng, case["ctx_min"] + 1, case["ctx_max"] + 1) - 1 if i
                   else case["ctx_max"])
    return new, ctx


def _parents(case, seed):
    """Drafted trees, chain by chain: a token mostly follows the one before it, else it begins a
    branch behind an earlier one or (-1) behind the context."""
    rng = random.Random(seed * 65537 + case["mix"])
    trees = []
    for n in _lengths(case)[0]:
        tree = []
        for i in range(n):
            tree.append(i - 1 if rng.random() < 0.7 else rng.randint(-1, i - 1))
        trees.append(tree)
    return trees


def _depths(tree):
    deep = []
    for p in tree:
        deep.append(deep[p] + 1 if p >= 0 else 0)
    return deep


def _accepted(case):
    """Accepted tokens of each request, ascending: the start of the first chain, then a branch
    whose tokens were drafted behind that chain."""
    rng = random.Random(case["mix"] * 31 + 7)
    paths = []
    for n in _lengths(case)[0]:
        size = rng.randint(0, min(n, 12))
        chain = rng.randint(0, size)
        late = n - size
        chain = max(chain, size - late)
        paths.append(list(range(chain)) + sorted(rng.sample(range(size, n), size - chain)))
    return paths


def _row_bytes(case):
    """Bytes of one cached key (or value) row of one head: codes, scales, biases."""
    return case["D"] // 2 + 4 * (case["D"] // GROUP)


def _sum_upto(lo, hi):
    """lo + (lo + 1) + ... + hi"""
    return (lo + hi) * (hi - lo + 1) // 2 if hi >= lo else 0


def _pairs(n, c, window, sinks):
    """(query, token) pairs of n causal tokens behind c cached ones, and the tokens any of them
    sees."""
    if not window:
        return _sum_upto(c + 1, c + n), c + n
    far = min(max(window + sinks - c, 0), n)  # queries that still see everything
    return (_sum_upto(c + 1, c + far) + (n - far) * (window + sinks),
            min(c + n, sinks + window + n - 1))


def work(case):
    op = case["op"]
    if op == "append":
        T, kv = case["T"], 2 * case["Hkv"]
        # heads in, queries out, rows into the cache and back out of it, rotations, a position and a
        # slot a token; a square, two scalings and three rotations a channel, about eight operations
        # a cached channel
        n = (case["Hq"] + kv) * case["D"]
        return {"bytes": T * (2 * n + 2 * case["Hq"] * case["D"] + 2 * kv * _row_bytes(case)
                              + 2 * kv * case["D"] + 4 * case["rot"] + 8),
                "flops": T * (7 * n + 8 * kv * case["D"])}
    new, ctx = _lengths(case)
    if op == "plan":
        # parents, offsets and lengths in, a position and a mask of 32-bit words a token out
        words = -(-case["q_max"] // 32)
        return {"bytes": 4 * (sum(new) * (2 + words) + 2 * case["B"]), "flops": 0}
    if op == "accept":
        # accepted rows out of the cache, into it, out of it again and out as bf16
        rows = sum(len(p) for p in _accepted(case)) * 2 * case["Hkv"]
        return {"bytes": rows * (3 * _row_bytes(case) + 2 * case["D"]) + 8 * case["B"] + 4 * rows,
                "flops": 0}
    pairs = rows = 0
    for tree, n, c in zip(_parents(case, 1) if op == "tree" else new, new, ctx):
        if op == "window":
            p, r = _pairs(n, c, case["window"], case["sinks"])
        elif not case["window"]:
            p, r = n * c + sum(d + 1 for d in _depths(tree)), c + n
        else:
            p, r = 0, 0
            for d in _depths(tree):
                p += min(c + d + 1, case["window"] + min(case["sinks"], c))
            r = min(c + n, case["sinks"] + case["window"] + n - 1)
        pairs, rows = pairs + p, rows + r
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


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _keys_values(g, T, Hkv, D):
    """Keys as they leave the norm (a few channels much larger than the rest) and values."""
    gain = 0.5 + torch.rand(Hkv, D, generator=g, device=DEV)
    gain[:, ::61] *= 4.0
    k = (_randn(g, T, Hkv, D) * gain).bfloat16()
    v = (_randn(g, T, Hkv, D) * 0.5).bfloat16()
    return k, v


def _append_inputs(case, seed):
    g = _gen(seed)
    T, Hq, Hkv, D, rot, page = (case[n] for n in ("T", "Hq", "Hkv", "D", "rot", "page"))
    qkv = (_randn(g, T, Hq + 2 * Hkv, D) * 1.5).bfloat16()  # a fused projection's rows
    wq = (1.0 + 0.2 * _randn(g, D)).bfloat16()
    wk = (1.0 + 0.2 * _randn(g, D)).bfloat16()
    start = int(torch.randint(0, case["pos_max"] - T, (1,), generator=g, device=DEV))
    positions = torch.arange(start, start + T, device=DEV, dtype=torch.int32)
    inv = 1.0e6 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    angle = torch.arange(case["pos_max"], device=DEV, dtype=torch.float64)[:, None] * inv
    table = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
    n_pages = -(-T // page) + 5
    ids = torch.randperm(n_pages, generator=g, device=DEV)
    at = torch.arange(3, 3 + T, device=DEV)  # from inside a page on
    slots = (ids[at // page] * page + at % page).int()
    return dict(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], positions=positions,
                wq=wq if case["normed"] else None, wk=wk if case["normed"] else None, table=table,
                eps=1e-6, slots=slots, n_pages=n_pages)


def _pages(case, g, kv):
    """Requests of kv cached tokens in randomly placed pages: their table, and the slots of all
    cached tokens request by request."""
    page = case["page"]
    held = [-(-n // page) for n in kv]
    n_pages, width = sum(held) + 3, max(held + [1]) + 1
    ids = torch.randperm(n_pages, generator=g, device=DEV)
    table = torch.full((len(kv), width), -1, dtype=torch.int32, device=DEV)
    slots, used = [], 0
    for b, n in enumerate(kv):
        mine = ids[used:used + held[b]]
        used += held[b]
        table[b, :held[b]] = mine.int()
        at = torch.arange(n, device=DEV)
        slots.append(mine[at // page] * page + at % page if n else at)
    return table, slots, n_pages


def _offsets(new):
    total = [0]
    for n in new:
        total.append(total[-1] + n)
    return total


def _masks(trees, words):
    """A row of 32-bit words for each drafted token: bit j for itself and each ancestor j."""
    rows = []
    for tree in trees:
        own_rows = []
        for i, p in enumerate(tree):
            own_rows.append((own_rows[p] if p >= 0 else 0) | 1 << i)
        rows += own_rows
    flat = [(r >> 32 * w) & 0xffffffff for r in rows for w in range(words)]
    return torch.tensor(flat, dtype=torch.int64).to(torch.int32).view(-1, words).to(DEV)


def _attention_inputs(case, seed):
    g = _gen(seed)
    Hq, Hkv, D = (case[n] for n in ("Hq", "Hkv", "D"))
    new, ctx = _lengths(case)
    kv = [n + c for n, c in zip(new, ctx)]
    q = (_randn(g, sum(new), Hq, D) * 1.5).bfloat16()
    table, slots, n_pages = _pages(case, g, kv)
    k, v = _keys_values(g, sum(kv), Hkv, D)
    masks = None
    if case["op"] == "tree":
        masks = _masks(_parents(case, seed), -(-case["q_max"] // 32))
    return dict(q=q, k=k, v=v, slots=torch.cat(slots).int(), table=table, new=new, kv=kv,
                n_pages=n_pages, masks=masks, q_offsets=_ints(_offsets(new)), kv_lens=_ints(kv))


def _plan_inputs(case, seed):
    new, ctx = _lengths(case)
    parents = [p for tree in _parents(case, seed) for p in tree]
    return dict(parents=_ints(parents), new=new, q_offsets=_ints(_offsets(new)),
                kv_lens=_ints([n + c for n, c in zip(new, ctx)]),
                words=-(-case["q_max"] // 32), n_pages=1)


def _accept_inputs(case, seed):
    g = _gen(seed)
    new, ctx = _lengths(case)
    table, slots, n_pages = _pages(case, g, [n + c for n, c in zip(new, ctx)])
    paths = _accepted(case)
    width = max(len(p) for p in paths) or 1
    k, v = _keys_values(g, sum(new), case["Hkv"], case["D"])
    return dict(k=k, v=v, slots=torch.cat([s[c:] for s, c in zip(slots, ctx)]).int(), table=table,
                ctx=_ints(ctx), paths=_ints([p + [-1] * (width - len(p)) for p in paths]),
                path_lens=_ints([len(p) for p in paths]), n_pages=n_pages,
                kept=torch.cat([s[c:c + len(p)] for s, c, p in zip(slots, ctx, paths)]).int())


_INPUTS = {"append": _append_inputs, "window": _attention_inputs, "tree": _attention_inputs,
           "plan": _plan_inputs, "accept": _accept_inputs}


def _quantise(x):
    """Codes and bf16 (scale, bias) of rows x [..., D] in groups of 64 channels, in 32 bits."""
    xg = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = xg.amin(-1), xg.amax(-1)
    scale = ((hi - lo) / 15.0).bfloat16()
    s = scale.float().unsqueeze(-1)
    code = torch.where(s > 0, ((xg - lo.unsqueeze(-1)) / s).round(), torch.zeros_like(xg))
    return code.clamp(0, 15).to(torch.uint8).flatten(-2), scale, lo.bfloat16()


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
                                       case.get("page", 64), s["n_pages"],
                                       max_requests=case.get("B", 1))
    if op == "plan":
        T = len(s["parents"])
        s["positions"] = torch.empty(T, dtype=torch.int32, device=DEV)
        s["masks"] = torch.empty(T, s["words"], dtype=torch.int32, device=DEV)
        return s
    rows, Hkv, D = s["n_pages"] * case["page"], case["Hkv"], case["D"]
    if own:
        s["cache"] = s["attn"].new_cache()
    else:  # what was never written reads as NaN
        s["codes"] = torch.full((2, rows, Hkv, D // 2), 255, dtype=torch.uint8, device=DEV)
        s["scale"] = torch.full((2, rows, Hkv, D // GROUP), math.nan, dtype=torch.bfloat16,
                                device=DEV)
        s["bias"] = s["scale"].clone()
    if op in ("append", "accept"):
        n = case["T"] if op == "append" else len(s["kept"])
        s["k_out"] = torch.empty(n, Hkv, D, dtype=torch.bfloat16, device=DEV)
        s["v_out"] = torch.empty_like(s["k_out"])
    if op != "accept":
        s["out"] = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=DEV)
    if op != "append":
        if own:
            s["attn"].append(s["k"], s["v"], s["slots"], s["cache"])
        else:
            _plain_write(s, s["k"], s["v"])
        del s["k"], s["v"]
    return s


# ---------------------------------------------------------------------------------- plain forms

def _plain_write(s, k, v):
    at = s["slots"].long()
    for i, x in enumerate((k, v)):
        codes, scale, bias = _quantise(x)
        s["codes"][i, at] = _pack(codes)
        s["scale"][i, at] = scale
        s["bias"][i, at] = bias


def _plain_read(s, i, at):
    codes = _unpack(s["codes"][i, at]).float().unflatten(-1, (-1, GROUP))
    return (codes * s["scale"][i, at].float().unsqueeze(-1)
            + s["bias"][i, at].float().unsqueeze(-1)).flatten(-2)


def _plain_norm_rotate(x, w, cos, sin, rot, inter, eps):
    """Norm (where there are weights) and rotation, rounded to bf16.  The squares' sum is taken in
    64 bits: codes next to a border follow its last bit."""
    y = x.float()
    if w is not None:
        mean = y.double().square().sum(-1, keepdim=True).float() / y.shape[-1]
        y = y * (mean + eps).sqrt().reciprocal() * w.float()
    head, tail = y[..., :rot], y[..., rot:]
    if inter:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([head, tail], -1).bfloat16()


def _plain_append(s):
    case, at = s["case"], s["slots"].long()
    cs = s["table"][s["positions"].long()].unsqueeze(1)
    how = (cs[..., :case["rot"] // 2], cs[..., case["rot"] // 2:], case["rot"], case["inter"],
           s["eps"])
    s["out"].copy_(_plain_norm_rotate(s["q"], s["wq"], *how))
    _plain_write(s, _plain_norm_rotate(s["k"], s["wk"], *how), s["v"])
    s["k_out"].copy_(_plain_read(s, 0, at))
    s["v_out"].copy_(_plain_read(s, 1, at))
    return [s["out"], s["k_out"], s["v_out"]]


def _plain_attention(s):
    case = s["case"]
    Hq, Hkv, D, page = (case[n] for n in ("Hq", "Hkv", "D", "page"))
    G, out, first = Hq // Hkv, s["out"], 0
    window, sinks = case["window"], case["sinks"]
    for b, (n, L) in enumerate(zip(s["new"], s["kv"])):
        c = L - n
        if s["masks"] is not None:
            bits = s["masks"][first:first + n]
            bits = (bits.unsqueeze(-1) >> torch.arange(32, device=DEV)) & 1
            bits = bits.flatten(1)[:, :n].bool()  # [token][drafted token]
        step = n if s["masks"] is not None else max(1, (1 << 27) // (Hq * min(L, 2 * window)))
        for i in range(0, n, step):
            m = min(step, n - i)
            # the tokens that any of these rows sees
            end = L if s["masks"] is not None else c + i + m
            lo = max(0, c + i + 1 - window) if window else 0
            t = torch.arange(end, device=DEV)
            if lo > sinks:
                t = torch.cat([t[:sinks], t[lo:]])
            at = s["table"][b].long()[t // page] * page + t % page
            k = _plain_read(s, 0, at).permute(1, 2, 0)            # [Hkv, D, tokens]
            v = _plain_read(s, 1, at).permute(1, 0, 2)            # [Hkv, tokens, D]
            x = s["q"][first + i:first + i + m].float().unflatten(1, (Hkv, G))
            x = x.permute(1, 0, 2, 3).reshape(Hkv, m * G, D)
            score = (x @ k) * D ** -0.5
            if s["masks"] is None:
                pos = c + i + torch.arange(m, device=DEV)[:, None]
                hidden = t > pos
            else:
                pos = c - 1 + bits.sum(-1, keepdim=True)
                hidden = (t >= c) & ~bits[:, (t - c).clamp(min=0)]
            if window:
                hidden = hidden | ((t >= sinks) & (t <= pos - window))
            score.masked_fill_(hidden.repeat_interleave(G, 0), -math.inf)
            p = (score - score.amax(-1, keepdim=True)).exp()
            y = (p @ v) / p.sum(-1, keepdim=True)
            out[first + i:first + i + m] = y.view(Hkv, m, G, D).transpose(0, 1).flatten(1, 2)
        first += n
    return out


def _plain_plan(s):
    off, kv, parents = s["q_offsets"].long(), s["kv_lens"].long(), s["parents"].long()
    T, words = parents.numel(), s["words"]
    B, N = kv.numel(), 32 * words
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(off[1:].contiguous(), t, right=True)
    i = t - off[b]
    # reach[b, i, j]: j is i itself or an ancestor; each product doubles the steps taken
    reach = torch.zeros(B, N, N, device=DEV)
    reach[b, i, i] = 1.0
    has = (parents >= 0).float()
    reach[b, i, parents.clamp(min=0)] = torch.maximum(reach[b, i, parents.clamp(min=0)], has)
    for _ in range(max(1, (N - 1).bit_length())):
        reach = (reach @ reach > 0).float()
    rows = reach[b, i].long()
    s["positions"].copy_((kv - off.diff())[b] + rows.sum(-1) - 1)
    s["masks"].copy_((rows.view(T, words, 32) << torch.arange(32, device=DEV)).sum(-1))
    return [s["positions"], s["masks"]]


def _plain_accept(s):
    page, table = s["case"]["page"], s["table"].long()
    width = s["paths"].shape[1]
    j = torch.arange(width, device=DEV).expand(s["paths"].shape)
    b, i = (j < s["path_lens"][:, None]).nonzero(as_tuple=True)
    c = s["ctx"].long()[b]
    src, dst = c + s["paths"].long()[b, i], c + i
    src, dst = (table[b, x // page] * page + x % page for x in (src, dst))
    for part in (s["codes"], s["scale"], s["bias"]):
        part[:, dst] = part[:, src]
    at = s["kept"].long()
    s["k_out"].copy_(_plain_read(s, 0, at))
    s["v_out"].copy_(_plain_read(s, 1, at))
    return [s["k_out"], s["v_out"]]


_PLAIN = {"append": _plain_append, "window": _plain_attention, "tree": _plain_attention,
          "plan": _plain_plan, "accept": _plain_accept}


# -------------------------------------------------------------------------------- the framework

def _own(s):
    case, attn = s["case"], s["attn"]
    op = case["op"]
    if op == "append":
        attn.qk_norm_rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["wq"],
                                 s["wk"], s["table"], s["cache"], eps=s["eps"],
                                 interleaved=case["inter"], q_out=s["out"])
        attn.read(s["slots"], s["cache"], k_out=s["k_out"], v_out=s["v_out"])
        return [s["out"], s["k_out"], s["v_out"]]
    if op == "plan":
        return list(attn.tree_plan(s["parents"], s["q_offsets"], s["kv_lens"],
                                   max_q_len=max(s["new"]), positions=s["positions"],
                                   masks=s["masks"]))
    if op == "accept":
        attn.accept(s["cache"], s["table"], s["ctx"], s["paths"], s["path_lens"])
        attn.read(s["kept"], s["cache"], k_out=s["k_out"], v_out=s["v_out"])
        return [s["k_out"], s["v_out"]]
    return attn.forward(s["q"], s["cache"], s["table"], s["q_offsets"], s["kv_lens"],
                        max_q_len=max(s["new"]), max_kv_len=max(s["kv"]), out=s["out"],
                        window=case["window"], sinks=case["sinks"], masks=s["masks"])


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------- in 64 bits

def _exact_cached(x):
    """What the cache holds of rows x, as 64-bit values: 16 levels from each group's smallest
    value on, a bf16 step apart."""
    g = x.double().reshape(*x.shape[:-1], -1, GROUP)
    low = g.min(-1, keepdim=True).values
    step = ((g.max(-1, keepdim=True).values - low) / 15).bfloat16().double()
    level = torch.nan_to_num((g - low) / step, nan=0.0).round().clamp(max=15)
    return (low + step * level).reshape(x.shape)


def _exact_append(case, seed):
    s = _append_inputs(case, seed)
    D, rot = case["D"], case["rot"]
    inv = 1.0e6 ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float64) * 2 / rot)
    turn = torch.polar(torch.ones(case["T"], rot // 2, dtype=torch.float64, device=DEV),
                       s["positions"].double()[:, None] * inv)
    outs = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = x.double()
        if w is not None:
            norm = torch.linalg.vector_norm(y, dim=-1, keepdim=True)
            y = y / torch.sqrt(norm ** 2 / D + s["eps"]) * w.double()
        y = y.clone()
        if case["inter"]:
            z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * turn[:, None]
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        else:
            z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn[:, None]
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        outs.append(y)
    return [outs[0], _exact_cached(outs[1].bfloat16()), _exact_cached(s["v"])]


def _exact_attention(case, seed):
    s = _attention_inputs(case, seed)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G, window, sinks = Hq // Hkv, case["window"], case["sinks"]
    trees = _parents(case, seed) if case["op"] == "tree" else None
    k, v = _exact_cached(s["k"]), _exact_cached(s["v"])
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    row = key = 0
    for b, (n, L) in enumerate(zip(s["new"], s["kv"])):
        c = L - n
        sees = torch.ones(n, L, dtype=torch.bool)
        where = list(range(c, L))
        if trees:
            sees[:, c:] = False
            for i, p in enumerate(trees[b]):
                if p >= 0:
                    sees[i, c:] = sees[p, c:]
                sees[i, c + i] = True
            where = [c + d for d in _depths(trees[b])]
        else:
            sees = sees.tril(c)
        if window:
            t = torch.arange(L)
            sees &= (t < sinks) | (t > torch.tensor(where)[:, None] - window)
        bias = torch.zeros(n, L, dtype=torch.float64, device=DEV)
        bias[~sees.to(DEV)] = -math.inf
        for h in range(Hq):
            kh, vh = k[key:key + L, h // G], v[key:key + L, h // G]
            score = s["q"][row:row + n, h].double() @ kh.T / math.sqrt(D) + bias
            out[row:row + n, h] = torch.softmax(score, -1) @ vh
        row, key = row + n, key + L
    return out


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    if case["op"] == "append":
        return _exact_append(case, seed)
    if case["op"] == "accept":
        s = _accept_inputs(case, seed)
        first, rows = 0, []
        for n, path in zip(_lengths(case)[0], _accepted(case)):
            rows += [first + p for p in path]
            first += n
        return [_exact_cached(x[rows]) for x in (s["k"], s["v"])]
    return _exact_attention(case, seed)
