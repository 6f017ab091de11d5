"""A decode loop of one sparse transformer block: a cache that keeps the entries which received the most attention,
and a mixture of experts.  It runs the hard selections together as a serving program would:

    prompt:  keys and values of all tokens, attention of the last tokens over them with accounts, first eviction
    a step:  append -> cache_attend (adds to the accounts) -> cache_evict -> route -> plan -> dispatch -> experts -> combine

Weights are random; only shapes and data flow are those of a model.

    python examples/sparse_decode.py
"""
import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import sparse_selection_primitive_amd as L  # noqa: E402


@dataclass
class Shape:
    batch: int = 4
    prompt: int = 600
    window: int = 16     # last prompt tokens whose attention makes the first accounts
    budget: int = 256    # entries a key head keeps
    width: int = 512
    heads: int = 8
    kv_heads: int = 2
    head_width: int = 64
    experts: int = 32
    k: int = 4
    sinks: int = 4
    recent: int = 32


class Block:
    """Weights of the block, and the experts' load balance."""

    def __init__(self, s, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") / shape[-2] ** 0.5).bfloat16()

        self.s = s
        self.q, self.o = w(s.width, s.heads * s.head_width), w(s.heads * s.head_width, s.width)
        self.kv = w(s.width, 2 * s.kv_heads * s.head_width)
        self.router = w(s.width, s.experts)
        self.up, self.down = w(s.experts, s.width, 2 * s.width), w(s.experts, 2 * s.width, s.width)
        self.bias = torch.zeros(s.experts, device="cuda")

    def keys_values(self, x):
        """x [batch, tokens, width] -> keys, values [batch, kv_heads, tokens, head_width]"""
        b, t, _ = x.shape
        kv = (x @ self.kv).view(b, t, 2, self.s.kv_heads, self.s.head_width)
        return kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)

    def queries(self, x):
        return (x @ self.q).view(x.shape[0], x.shape[1], self.s.heads, self.s.head_width)

    def mixture(self, x):
        """x [tokens, width]: every token through its k experts."""
        s = self.s
        weights, chosen = L.route(x @ self.router, s.k, self.bias, score="sigmoid", groups=4, top_groups=2)
        offsets, slot, _ = L.dispatch_plan(chosen, s.experts)
        xs = L.dispatch(x, slot, offsets)
        bounds = offsets.tolist()
        ys = torch.cat([torch.relu(xs[a:b] @ self.up[e]) @ self.down[e]
                        for e, (a, b) in enumerate(zip(bounds, bounds[1:])) if b > a])
        load = (offsets[1:] - offsets[:-1]).float()
        self.bias += 1e-3 * torch.sign(load.mean() - load)  # busy experts become less likely
        return L.combine(ys, weights, slot, offsets)


class BudgetedCache:
    """Keys, values, accounts and positions of every sequence and key head."""

    def __init__(self, s, capacity):
        shape = (s.batch, s.kv_heads, capacity)
        self.s = s
        self.k = torch.zeros(*shape, s.head_width, dtype=torch.bfloat16, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.account = torch.zeros(shape, device="cuda")
        self.positions = torch.zeros(shape, dtype=torch.int32, device="cuda")
        self.lengths = torch.zeros(s.batch, dtype=torch.int32, device="cuda")
        self.next_position = torch.zeros_like(self.lengths)

    def append(self, k, v):
        b, h, t, _ = k.shape
        at = self.lengths.long()[:, None] + torch.arange(t, device="cuda")
        batch = torch.arange(b, device="cuda")[:, None]
        self.k[batch, :, at] = k.transpose(1, 2)
        self.v[batch, :, at] = v.transpose(1, 2)
        self.account[batch, :, at] = 0.0
        where = self.next_position[:, None] + torch.arange(t, device="cuda", dtype=torch.int32)
        self.positions[batch, :, at] = where[:, :, None].expand(b, t, h)
        self.lengths = self.lengths + t
        self.next_position = self.next_position + t

    def attend(self, q):
        return L.cache_attend(q, self.k, self.v, self.lengths, self.account)

    def evict(self, budget):
        kept, self.lengths = L.cache_evict(self.k, self.v, self.account, self.positions, self.lengths, budget,
                                           next_position=self.next_position, sinks=self.s.sinks, recent=self.s.recent)
        return kept


def prefill(block, x):
    """The prompt x [batch, tokens, width] into two caches: a long one for the first accounts, and the budgeted one
    that the decode steps use (budget + 1 entries: one over leaves at every step)."""
    s = block.s
    k, v = block.keys_values(x)
    long = BudgetedCache(s, x.shape[1])
    long.append(k, v)
    long.attend(block.queries(x[:, -s.window:]))
    long.evict(min(s.budget, x.shape[1]))
    cache = BudgetedCache(s, s.budget + 1)
    m = min(s.budget, x.shape[1])
    for name in ("k", "v", "account", "positions"):
        getattr(cache, name)[:, :, :m] = getattr(long, name)[:, :, :m]
    cache.lengths, cache.next_position = long.lengths, long.next_position
    return cache


def step(block, cache, x):
    """One token of every sequence: x [batch, width] -> [batch, width]"""
    s = block.s
    x = x[:, None]
    cache.append(*block.keys_values(x))
    out = cache.attend(block.queries(x)).view(x.shape[0], s.heads * s.head_width)
    cache.evict(s.budget)
    x = x[:, 0] + out @ block.o
    return x + block.mixture(x)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--seed", type=int, default=0)
    a = p.parse_args(argv)
    s = Shape()
    block = Block(s, a.seed)
    g = torch.Generator(device="cuda").manual_seed(a.seed + 1)
    with torch.no_grad():
        cache = prefill(block, torch.randn(s.batch, s.prompt, s.width, generator=g, device="cuda").bfloat16())
        x = torch.randn(s.batch, s.width, generator=g, device="cuda").bfloat16()
        for _ in range(a.steps):
            y = step(block, cache, x)
            x = (y.float() / y.float().pow(2).mean(1, keepdim=True).sqrt()).bfloat16()
    old = (cache.next_position[:, None, None] - cache.positions[:, :, :s.budget]).float()
    print(f"{a.steps} steps, {s.batch} sequences: {int(cache.next_position[0])} tokens seen, "
          f"{int(cache.lengths[0])} entries kept, oldest {int(old.max())} tokens back, median {int(old.median())}; "
          f"experts' bias {float(block.bias.min()):+.3f} .. {float(block.bias.max()):+.3f}")
    return cache, x


if __name__ == "__main__":
    main()
