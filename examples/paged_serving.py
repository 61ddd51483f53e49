"""One decoder layer of a served MoE model over a paged INT8 KV cache.

A batch of requests with prompts of different lengths is served as a scheduler
would: prompts come in chunks of at most `chunk` tokens, beside the single
tokens of requests that already answer, in one call per step; requests leave,
and their pages serve others. Each step runs

    plan     block tables, slots and positions from the lengths (paged_kv_plan)
    norm + QKV projection (rmsnorm_linear), K and V into their slots
             (paged_kv_write), attention over the pages (attention_paged),
             output projection (linear), residual
    norm, router logits, the gate (moe_gate), the expert FFN (moe_ffn), residual

with random weights. Run it on a GB300:

    python examples/paged_serving.py [--steps N]

It prints what each step served, and at the end how far the answers of a request
are from serving it alone, prompt in one piece.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_gemm_gb300 as w8  # noqa: E402

D = 128


class Layer:
    """The weights of one layer: INT8 projections and experts, BF16 norms, an
    FP32 router with a balance bias and expert groups."""

    def __init__(self, hidden=512, q_heads=8, kv_heads=2, experts=16, topk=4, inner=256, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std=0.02):
            return torch.randn(*shape, generator=g, device="cuda") * std

        self.hidden, self.q_heads, self.kv_heads, self.topk = hidden, q_heads, kv_heads, topk
        self.norm1, self.norm2 = (1 + normal(2, hidden, std=0.1)).to(torch.bfloat16)
        self.qkv = w8.quant_weight(normal((q_heads + 2 * kv_heads) * D, hidden))
        self.out = w8.quant_weight(normal(hidden, q_heads * D))
        self.router = normal(experts, hidden)
        self.balance = normal(experts)
        up = [w8.quant_weight(normal(2 * inner, hidden)) for _ in range(experts)]
        down = [w8.quant_weight(normal(hidden, inner)) for _ in range(experts)]
        self.up = [torch.stack(t) for t in zip(*up)]
        self.down = [torch.stack(t) for t in zip(*down)]

    def __call__(self, x, cache, plan):
        """x [T, hidden] BF16: the new tokens of all requests, packed."""
        cu_new, kv_lens, slots, _ = plan
        T, hq, hkv = x.shape[0], self.q_heads, self.kv_heads
        qkv = w8.rmsnorm_linear(x, self.norm1, 1e-6, *self.qkv).view(T, hq + 2 * hkv, D)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        w8.paged_kv_write(k, v, slots, cache.k, cache.v, k_scale=cache.ks, v_scale=cache.vs)
        a = w8.attention_paged(q, cache.k, cache.v, cache.table, kv_lens, cu_new,
                               1 / math.sqrt(D), k_scale=cache.ks, v_scale=cache.vs)
        x = x + w8.linear(a.view(T, hq * D), *self.out)
        y = w8.rmsnorm(x, self.norm2, 1e-6)
        ids, weights = w8.moe_gate(y.float() @ self.router.T, self.topk, scoring="sigmoid",
                                   bias=self.balance, n_group=4, topk_group=2)
        return x + w8.moe_ffn(y, ids, weights, *self.up, *self.down)


class Cache:
    """The pages of one layer, and the block tables of up to `requests` requests."""

    def __init__(self, layer, requests, pages, page=16, longest=1024):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.page = page
        self.k = torch.zeros(pages, layer.kv_heads, page, D, dtype=torch.int8, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.ks = torch.zeros(pages, layer.kv_heads, page, device="cuda")
        self.vs = torch.zeros_like(self.ks)
        self.table = torch.full((requests, -(-longest // page)), -1, **i32)
        self.lens = torch.zeros(requests, **i32)
        self.free = torch.arange(pages, **i32)
        self.n_free = torch.full((1,), pages, **i32)

    def plan(self, target, n_tokens):
        return w8.paged_kv_plan(self.table, self.lens,
                                torch.tensor(target, dtype=torch.int32, device="cuda"), self.free,
                                self.n_free, self.page, n_tokens)


def serve(layer, streams, arrive, chunk=128, pages=256, steps=None, say=None):
    """Serves streams[b] [n_b, hidden], the hidden states of request b's tokens
    (its prompt, then one per step), of which arrive[b] are its prompt. Returns
    the layer's outputs of every request."""
    B = len(streams)
    cache = Cache(layer, B, pages)
    held = [0] * B
    outs = [[] for _ in range(B)]
    step = 0
    while any(held[b] < len(streams[b]) for b in range(B)) and (steps is None or step < steps):
        target = []
        for b in range(B):
            if held[b] >= len(streams[b]):
                target.append(0)                                    # done: it leaves
            elif held[b] < arrive[b]:
                target.append(min(held[b] + chunk, arrive[b]))      # a piece of its prompt
            else:
                target.append(held[b] + 1)
        grows = [b for b in range(B) if target[b] > held[b] and held[b] < len(streams[b])]
        new = [target[b] - held[b] if b in grows else 0 for b in range(B)]
        x = torch.cat([streams[b][held[b]:target[b]] for b in grows])
        plan = cache.plan(target, len(x))
        y = layer(x, cache, plan)
        served = plan[1].tolist()          # (a scheduler reads this to learn who was refused)
        at = 0
        for b in grows:
            if served[b] == target[b]:
                outs[b].append(y[at:at + new[b]])
                held[b] = target[b]
            at += new[b]
        if say:
            say(f"step {step}: {len(x)} new tokens of {len(grows)} requests, "
                f"{int(cache.n_free)} pages free")
        step += 1
    return [torch.cat(o) if o else None for o in outs]


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=None)
    args = ap.parse_args(argv)
    layer = Layer()
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts, answers = [300, 17, 128, 1, 75], [9, 30, 4, 12, 20]
    streams = [torch.randn(p + a, layer.hidden, generator=g, device="cuda").to(torch.bfloat16)
               for p, a in zip(prompts, answers)]
    together = serve(layer, streams, prompts, steps=args.steps, say=print)
    worst = 0.0
    for b, s in enumerate(streams):
        if together[b] is None or len(together[b]) < len(s):
            continue
        alone = serve(layer, [s], [prompts[b]], chunk=len(s))[0]
        err = (together[b].float() - alone.float()).norm() / alone.float().norm()
        worst = max(worst, float(err))
    assert w8.device_error() == 0
    print(f"largest relative difference to serving a request alone: {worst:.2e}")
    return worst


if __name__ == "__main__":
    main()
