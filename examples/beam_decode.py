"""A beam search through one sparse transformer block: caches that keep the entries which received the most attention, a
mixture of experts, and beams that fork, end and are dropped.  It runs the operators together as a serving program
would, without a copy to the host in a step:

    prompt:  as in sparse_decode.py, one cache a search, then one a beam
    a step:  append -> cache_attend -> cache_evict -> route -> plan -> dispatch -> expert_product twice -> combine
             -> logits -> beam_select -> cache_reorder

Weights are random; only shapes and data flow are those of a model.

    python examples/beam_decode.py
"""
import argparse
import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from sparse_decode import Block, BudgetedCache, Shape, prefill  # noqa: E402

import sparse_selection_primitive_amd as L  # noqa: E402


class Model(Block):
    """The block with an embedding that also reads the tokens back."""

    def __init__(self, s, vocab, seed=0):
        super().__init__(s, seed)
        g = torch.Generator(device="cuda").manual_seed(seed + 100)
        self.vocab = vocab
        self.embedding = torch.randn(vocab, s.width, generator=g, device="cuda").bfloat16()

    def mixture(self, x):
        """x [tokens, width]: every token through its k experts, by ragged products."""
        s = self.s
        weights, chosen = L.route(x @ self.router, s.k, self.bias, score="sigmoid", groups=4, top_groups=2)
        offsets, slot, _ = L.dispatch_plan(chosen, s.experts)
        hidden = torch.relu(L.expert_product(L.dispatch(x, slot, offsets), self.up, offsets))
        return L.combine(L.expert_product(hidden, self.down, offsets), weights, slot, offsets)

    def logits(self, x):
        x = x.float()
        x = (x / x.pow(2).mean(1, keepdim=True).sqrt()).bfloat16()
        return x @ self.embedding.t() * (4.0 / self.s.width ** 0.5)


class Search:
    """The state of `batch` searches of `beams` beams each."""

    def __init__(self, model, prompt, beams, end_token=2):
        """prompt [batch, tokens] of token numbers; its last token is the first step's input"""
        s, batch = model.s, prompt.shape[0]
        one = prefill(model, model.embedding[prompt[:, :-1]])
        self.model, self.beams, self.end_token = model, beams, end_token
        self.cache = BudgetedCache(dataclasses.replace(s, batch=batch * beams), s.budget + 1)
        for name in ("k", "v", "account", "positions", "lengths", "next_position"):
            setattr(self.cache, name, getattr(one, name).repeat_interleave(beams, 0))
        # one beam of each search lives, the others are still the same
        self.scores = torch.full((batch, beams), -torch.inf, device="cuda")
        self.scores[:, 0] = 0.0
        self.ended = torch.zeros(batch, beams, dtype=torch.bool, device="cuda")
        self.tokens = prompt[:, -1:].repeat_interleave(beams, 1).view(batch, beams, 1)

    def step(self):
        """All beams by one token; returns the logits and whom each beam continues."""
        model, cache, s = self.model, self.cache, self.model.s
        batch, beams = self.scores.shape
        x = model.embedding[self.tokens[:, :, -1].flatten()]
        cache.append(*model.keys_values(x[:, None]))
        out = cache.attend(model.queries(x[:, None])).view(batch * beams, s.heads * s.head_width)
        cache.evict(s.budget)
        x = x + out @ model.o
        x = x + model.mixture(x)
        logits = model.logits(x).view(batch, beams, model.vocab)
        self.scores, parents, tokens = L.beam_select(logits, self.scores, beams, ended=self.ended,
                                                     end_token=self.end_token)
        cache.lengths = L.cache_reorder(cache.k, cache.v, parents, cache.lengths, cache.account, cache.positions)
        # places without a continuation keep a dead beam: its score is -inf
        at = parents.clamp(min=0).long()
        cache.next_position = cache.next_position.view(batch, beams).gather(1, at).flatten()
        self.ended = self.ended.gather(1, at) | (tokens == self.end_token)
        self.tokens = torch.cat([self.tokens.gather(1, at[:, :, None].expand_as(self.tokens)),
                                 tokens.clamp(min=0).long()[:, :, None]], 2)
        return logits, parents


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--beams", type=int, default=4)
    p.add_argument("--seed", type=int, default=0)
    a = p.parse_args(argv)
    model = Model(Shape(), vocab=8000, seed=a.seed)
    g = torch.Generator(device="cuda").manual_seed(a.seed + 1)
    with torch.no_grad():
        search = Search(model, torch.randint(3, model.vocab, (model.s.batch, model.s.prompt), generator=g, device="cuda"),
                        a.beams)
        for _ in range(a.steps):
            search.step()
    print(f"{a.steps} steps, {model.s.batch} searches of {a.beams} beams: best scores "
          f"{[round(x, 2) for x in search.scores[:, 0].tolist()]}, {int(search.ended.sum())} beams ended, "
          f"{int(search.cache.lengths[0])} entries kept")
    return search


if __name__ == "__main__":
    main()
