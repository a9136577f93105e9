"""Beam-search decoding of a small state-space language model with random 4-bit weights: packed
prompts of different lengths, then one token of every beam a step.

    python examples/state_space_decode.py [--dim 512 --layers 4 --requests 3 --beams 4 --tokens 16]

Every layer runs on the library's sequence operators (depthwise_pointwise_convolution_amd.sequence);
torch adds the embedding, the residuals and their normalisation.  `--check` runs every finished beam
again as one prompt and compares the score it was given.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from depthwise_pointwise_convolution_amd.sequence import (BeamSearch, Q4Linear,  # noqa: E402
                                                          StateSpaceBlock)


class Model:
    def __init__(self, dim, layers, vocab, slots, N=16, W=4, group=64, dtype=torch.bfloat16, seed=0,
                 device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std=1.0):
            return torch.randn(*shape, device=device, generator=g) * std

        def linear(C, K):
            return Q4Linear.from_weight(normal(K, C, std=C ** -0.5).to(dtype), group=group)

        inner, rank = 2 * dim, max(8, dim // 16 // 8 * 8)
        self.vocab, self.dtype = vocab, dtype
        self.embed = normal(vocab, dim).to(dtype)
        self.blocks = []
        for _ in range(layers):
            step = torch.exp(torch.rand(inner, device=device, generator=g) * math.log(100) + math.log(1e-3))
            self.blocks.append(StateSpaceBlock(
                linear(dim, 2 * inner), normal(inner, W, std=0.5).to(dtype), normal(inner, std=0.1),
                linear(inner, rank + 2 * N), linear(rank, inner), step + torch.log(-torch.expm1(-step)),
                -torch.arange(1, N + 1, device=device).float().repeat(inner, 1),
                torch.ones(inner, device=device), linear(inner, dim), slots))
        self.head = linear(dim, vocab)

    def pools(self):
        return [p for b in self.blocks for p in (b.window, b.state)]

    @staticmethod
    def _norm(x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)

    def _run(self, tokens, mix):
        x = self.embed[tokens.long()]
        for b in self.blocks:
            x = x + mix(b, self._norm(x))
        return self._norm(x)

    def prompt(self, tokens, cu, slots, carry=None):
        """Logits after the last token of each packed prompt."""
        x = self._run(tokens, lambda b, v: b.prompt(v, cu, slots, carry))
        return self.head(x[(cu[1:] - 1).long()])

    def all_logits(self, tokens, cu, slots):
        return self.head(self._run(tokens, lambda b, v: b.prompt(v, cu, slots)))

    def step(self, tokens, slots):
        return self.head(self._run(tokens, lambda b, v: b.step(v, slots)))


def decode(model, prompts, beams, tokens, eos=-1):
    """The best beams' tokens [requests, beams, tokens] and scores."""
    dev, R = model.embed.device, len(prompts)
    cu = torch.tensor([0] + [len(p) for p in prompts], device=dev).cumsum(0).to(torch.int32)
    # beam j of request r lives in slot r*beams + j; the prompts run in the first beams' slots
    slots = torch.arange(R * beams, dtype=torch.int32, device=dev)
    search = BeamSearch(R, beams, model.vocab, slots, eos)
    first = model.prompt(torch.cat(prompts), cu, slots[::beams].contiguous())
    logits = first.repeat_interleave(beams, 0)
    history = torch.zeros(R * beams, 0, dtype=torch.int64, device=dev)
    base = torch.arange(R, device=dev).repeat_interleave(beams) * beams
    for t in range(tokens):
        parent, token = search.advance(logits, model.pools())
        history = torch.cat([history[base + parent.long()], token.long()[:, None]], 1)
        if t + 1 < tokens:
            logits = model.step(token, search.slots)
    return history.reshape(R, beams, tokens), search.scores.reshape(R, beams)


def rescore(model, prompt, beam):
    """The score of one beam's tokens, from one prompt run over all of them."""
    dev = model.embed.device
    whole = torch.cat([prompt, beam.to(prompt.dtype)])
    cu = torch.tensor([0, len(whole)], dtype=torch.int32, device=dev)
    logp = torch.log_softmax(model.all_logits(whole, cu, torch.zeros(1, dtype=torch.int32, device=dev)).double(), -1)
    at = torch.arange(len(prompt) - 1, len(whole) - 1, device=dev)
    return float(logp[at, beam].sum())


def main(argv=None):
    ap = argparse.ArgumentParser()
    for name, v in (("dim", 512), ("layers", 4), ("vocab", 4000), ("requests", 3), ("beams", 4), ("tokens", 16),
                    ("seed", 0)):
        ap.add_argument("--" + name, type=int, default=v)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    model = Model(a.dim, a.layers, a.vocab, a.requests * a.beams, seed=a.seed)
    g = torch.Generator().manual_seed(a.seed)
    prompts = [torch.randint(0, a.vocab, (int(n),), generator=g).cuda()
               for n in torch.randint(1, 60, (a.requests,), generator=g)]
    history, scores = decode(model, prompts, a.beams, a.tokens)
    for r in range(a.requests):
        print(f"request {r} ({len(prompts[r])} tokens): score {float(scores[r, 0]):.3f}, "
              f"tokens {history[r, 0, :8].tolist()}...")
    if a.check:
        worst = max(abs(rescore(model, prompts[r], history[r, j]) - float(scores[r, j]))
                    for r in range(a.requests) for j in range(a.beams))
        print(f"largest difference of a beam's score from its tokens' in one prompt run: {worst:.4f}")
        return worst
    return 0.0


if __name__ == "__main__":
    main()
