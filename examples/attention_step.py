"""Serving one full-attention layer of the hybrid model with its MoE FFN, from prompts to tokens.

A batch of requests with ragged prompts runs through the layer: one step for the prompts, then a
step per generated token, the latter as one CUDA graph that is replayed.  Each step is

    plan -> projections -> norm, rotation and append to the 4-bit cache -> attention
         -> output projection -> MoE FFN

The layer's shapes are those of the model (16 query heads over 2 key/value heads of 256 channels,
hidden size 2048, 256 experts of which 8 are taken); weights and inputs are random.  A token's next
input is the layer's output, normalised.  At the end each request's rows are run once more as one
prompt over a fresh cache, which has to give the outputs that the steps gave.

    python examples/attention_step.py [--tokens N] [--small]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_moe_02_gb300 as moe  # noqa: E402

HQ, HKV, D, PAGE, ROTARY = 16, 2, 256, 64, 64


def unit_rows(x, eps=1e-6):
    """Rows of mean square 1 (the norm before the layer, without weights)."""
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + eps)).to(torch.bfloat16)


def angles(n_positions, rotary, base=1e7):
    """[n_positions][rotary] fp32: the cosines of a position's angles, then their sines."""
    inv = base ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)
    a = torch.arange(n_positions, dtype=torch.float64)[:, None] * inv
    return torch.cat((a.cos(), a.sin()), 1).float().cuda()


class Layer:
    """Attention and FFN of one layer, with its cache and block tables for a batch of requests."""

    def __init__(self, hidden, inner, requests, tokens_per_request, max_tokens, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)

        def randn(*shape, gain):
            return (torch.randn(*shape, generator=g, device="cuda") * gain).to(torch.bfloat16)

        self.width = -(-tokens_per_request // PAGE)  # pages of a request
        n_pages = requests * self.width
        self.w_qkv = randn(hidden, (HQ + 2 * HKV) * D, gain=hidden ** -0.5)
        self.w_out = randn(HQ * D, hidden, gain=(HQ * D) ** -0.5)
        self.q_weight = 1 + randn(D, gain=0.1)
        self.k_weight = 1 + randn(D, gain=0.1)
        self.cos_sin = angles(tokens_per_request, ROTARY)
        self.attention = moe.PagedAttention(HQ, HKV, D, PAGE, n_pages, max_requests=requests)
        shapes = dict(w_router=(256, hidden), w_gate=(256, inner, hidden),
                      w_up=(256, inner, hidden), w_down=(256, hidden, inner),
                      ws_gate=(inner, hidden), ws_up=(inner, hidden), ws_down=(hidden, inner))
        self.ffn = moe.MoeLayer({k: randn(*s, gain=s[-1] ** -0.5) for k, s in shapes.items()},
                                max_tokens)
        # pages are handed out in a mixed order, as they are once requests have come and gone
        order = torch.randperm(n_pages, generator=g, device="cuda")
        self.free = order.to(torch.int32)
        self.max_kv = tokens_per_request
        self.reset(requests)

    def reset(self, requests):
        """An empty cache for a batch of requests."""
        self.cache = self.attention.new_cache()
        self.table = torch.full((requests, self.width), -1, dtype=torch.int32, device="cuda")
        self.cursor = torch.zeros(1, dtype=torch.int32, device="cuda")

    def attend(self, qkv, ctx_lens, new_lens, max_new):
        """Attention of projected rows [T][Hq + 2 Hkv][D]; extends the cache by them."""
        offsets, kv_lens, positions, slots, _ = self.attention.plan(
            self.table, ctx_lens, new_lens, self.free, self.cursor, T=qkv.shape[0],
            cursor_out=self.cursor)
        q = self.attention.qk_norm_rope_append(qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:],
                                               positions, slots, self.q_weight, self.k_weight,
                                               self.cos_sin, self.cache)
        return self.attention.forward(q, self.cache, self.table, offsets, kv_lens, max_new,
                                      self.max_kv)

    def step(self, x, ctx_lens, new_lens, max_new):
        """One step for rows x [T][hidden]; returns (outputs, projected rows, attention rows)."""
        qkv = (unit_rows(x) @ self.w_qkv).view(-1, HQ + 2 * HKV, D)
        o = self.attend(qkv, ctx_lens, new_lens, max_new)
        x = x + o.view(-1, HQ * D) @ self.w_out
        return x + self.ffn.forward(unit_rows(x)), qkv, o

    def check(self):
        assert self.attention.device_error() == moe.MOE_OK
        assert self.ffn.device_error() == moe.MOE_OK

    def close(self):
        self.attention.close()
        self.ffn.close()


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def run(prompts, tokens, hidden=2048, inner=512, report=print):
    """Prompts of the given lengths, then `tokens` single-token steps; returns the attention rows of
    all steps and of the replay, [request] -> [tokens][Hq][D] each, and the microseconds of a
    single-token step."""
    B, total = len(prompts), sum(prompts)
    layer = Layer(hidden, inner, B, max(prompts) + tokens, max(total, B))
    x = torch.randn(total, hidden, device="cuda",
                    generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    ctx, new = ints([0] * B), ints(prompts)
    y, qkv, o = layer.step(x, ctx, new, max(prompts))
    rows_qkv, rows_o = [list(t.split(prompts)) for t in (qkv, o)]
    last = torch.tensor(prompts).cumsum(0) - 1
    x1 = unit_rows(y[last.cuda()])  # every request's next input
    ctx.copy_(new)
    new.fill_(1)

    def token():
        y1, qkv1, o1 = layer.step(x1, ctx, new, 1)
        x1.copy_(unit_rows(y1))
        ctx.add_(new)
        return qkv1, o1

    def keep(rows):
        for b in range(B):
            rows_qkv[b] = torch.cat((rows_qkv[b], rows[0][b:b + 1]))
            rows_o[b] = torch.cat((rows_o[b], rows[1][b:b + 1]))

    # the first token warms the libraries up on a side stream, the others replay one graph
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        keep(token())
    torch.cuda.current_stream().wait_stream(side)
    us = float("nan")
    if tokens > 1:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rows = token()
        marks = []
        for _ in range(tokens - 1):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            graph.replay()
            b.record()
            marks.append((a, b))
            keep(rows)
        torch.cuda.synchronize()
        us = sorted(1e3 * a.elapsed_time(b) for a, b in marks)[len(marks) // 2]
    layer.check()

    layer.reset(B)
    lens = [n + tokens for n in prompts]
    replay = []
    for b in range(0, B):  # request by request: every row in one prompt
        only = [n if i == b else 0 for i, n in enumerate(lens)]
        replay.append(layer.attend(rows_qkv[b], ints([0] * B), ints(only), lens[b]))
    layer.check()
    worst = max((s.float() - r.float()).abs().max().item() for s, r in zip(rows_o, replay))
    report(f"{B} requests, prompts {prompts}, {tokens} tokens each: a single-token step of the "
           f"layer takes {us:.0f} us (one graph)")
    report(f"steps against one prompt: largest difference {worst:.2e} of outputs up to "
           f"{max(r.float().abs().max().item() for r in replay):.2f}")
    layer.close()
    return rows_o, replay, us


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--tokens", type=int, default=32, help="tokens generated for each request")
    p.add_argument("--small", action="store_true", help="hidden size 512 and inner size 128")
    a = p.parse_args()
    size = dict(hidden=512, inner=128) if a.small else {}
    run([1000, 1, 257, 4096], max(1, a.tokens), **size)


if __name__ == "__main__":
    main()
