"""Decoding with drafted tokens: a model of one block drafts tokens, a deeper one verifies a request's
drafts in one pass, and both move their states on over those that stand.  Random 4-bit weights.

    python examples/draft_decode.py [--dim 512 --layers 4 --requests 3 --drafts 4 --tokens 32]

Every layer runs on the library's sequence operators (depthwise_pointwise_convolution_amd.sequence);
torch adds the embedding, the residuals and their normalisation.  `--check` decodes once more with drafts
that never stand and counts the tokens that differ: with temperature 0, the default, and up to 15 drafts
they only change how many passes it takes.  (A pass then has at most 16 rows of a request, which the delta
rule takes token by token wherever they are cut.  More go in chunks, whose results differ by roundings, and
with them a token may whose logits are nearly another's.)
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from depthwise_pointwise_convolution_amd.sequence import (DeltaRuleBlock, DraftVerifier,  # noqa: E402
                                                          MX4Linear)


class Model:
    """Blocks with the states of `slots` requests, and a second set of slots that verifications write to."""

    def __init__(self, dim, layers, vocab, slots, heads=4, D=64, W=4, dtype=torch.bfloat16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std=1.0):
            return torch.randn(*shape, device=device, generator=g) * std

        def linear(C, K):
            return MX4Linear.from_weight(normal(K, C, std=C ** -0.5).to(dtype))

        self.vocab, self.slots = vocab, slots
        # (the embeddings are the seed's that both models share: what they say of a token is alike)
        self.embed = torch.randn(vocab, dim, device=device,
                                 generator=torch.Generator(device=device).manual_seed(0)).to(dtype)
        inner, Hk = heads * D, heads // 2
        self.blocks = [DeltaRuleBlock(
            linear(dim, 2 * Hk * D + 2 * inner + 2 * heads), normal(2 * Hk * D + inner, W, std=0.5).to(dtype),
            normal(2 * Hk * D + inner, std=0.1), -torch.exp(normal(heads)), normal(heads) - 2,
            torch.ones(D, device=device), linear(inner, dim), Hk, D, D, 2 * slots) for _ in range(layers)]
        self.head = MX4Linear.from_weight(self.embed)

    @staticmethod
    def _norm(x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)

    def rows(self, tokens, cu, slots, carry=None):
        """What the head reads, for every row."""
        x = self.embed[tokens.long()]
        for b in self.blocks:
            x = x + b.prompt(self._norm(x), cu, slots, carry)
        return self._norm(x)

    def step(self, tokens, slots):
        x = self.embed[tokens.long()]
        for b in self.blocks:
            x = x + b.step(self._norm(x), slots)
        return self.head(self._norm(x))

    def set_aside(self):
        """The states again in the second set of slots."""
        for b in self.blocks:
            for p in (b.window, b.state):
                p[self.slots:] = p[:self.slots]


def drafts_of(model, last, drafts):
    """(tokens [requests, drafts], their logits): each the likeliest behind the one before, in the spare slots."""
    spare = torch.arange(model.slots, 2 * model.slots, dtype=torch.int32, device=last.device)
    model.set_aside()
    tokens, rows = [], []
    for _ in range(drafts):
        logits = model.step(last, spare)
        last = logits.float().argmax(-1).to(torch.int32)
        tokens.append(last)
        rows.append(logits)
    return torch.stack(tokens, 1), rows


def decode(target, prompts, drafts, tokens, propose, follow=None, temperature=0.0):
    """(at least `tokens` tokens of each prompt's request, passes of the target).  propose(last tokens,
    tokens so far) gives drafts [requests, drafts]; `follow` are models whose states keep up."""
    dev, R = target.embed.device, len(prompts)
    models = [target] + list(follow or [])
    cu = torch.tensor([0] + [len(p) - 1 for p in prompts], device=dev).cumsum(0).to(torch.int32)
    slots = torch.arange(R, dtype=torch.int32, device=dev)
    spare = slots + target.slots
    for m in models:  # all but the last token, which opens the first pass
        m.rows(torch.cat([p[:-1] for p in prompts]), cu, slots)
    last = torch.stack([p[-1] for p in prompts]).to(torch.int32)
    verify = DraftVerifier(R, drafts, target.vocab, temperature)
    whole = torch.arange(0, R * (drafts + 1) + 1, drafts + 1, dtype=torch.int32, device=dev)
    ones = torch.ones(2 * R, dtype=torch.int32, device=dev)
    out, passes = [[] for _ in range(R)], 0
    while min(len(o) for o in out) < tokens:
        proposed = propose(last, out)
        rows = torch.cat([last[:, None], proposed], 1).reshape(-1)
        target.set_aside()
        logits = target.head(target.rows(rows, whole, spare, ones[:R]))
        accepted, following = verify(logits, proposed)
        kept, kept_slots = verify.kept(accepted, slots)
        for m in models:
            m.rows(rows, kept, kept_slots, ones)
        for r in range(R):
            n = int(accepted[r])
            out[r] += proposed[r, :n].tolist() + [int(following[r])]
        last = following
        passes += 1
    return [o[:tokens] for o in out], passes


def main(argv=None):
    ap = argparse.ArgumentParser()
    for name, v in (("dim", 512), ("layers", 4), ("vocab", 4000), ("requests", 3), ("drafts", 4), ("tokens", 32),
                    ("seed", 0)):
        ap.add_argument("--" + name, type=int, default=v)
    ap.add_argument("--temperature", type=float, default=0.0)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    if a.check and a.drafts > 15:
        ap.error("--check needs at most 15 drafts: longer passes round their sums otherwise")
    torch.manual_seed(a.seed)
    g = torch.Generator().manual_seed(a.seed)
    prompts = [torch.randint(0, a.vocab, (int(n),), generator=g).cuda()
               for n in torch.randint(1, 60, (a.requests,), generator=g)]
    target, draft = (Model(a.dim, n, a.vocab, a.requests, seed=a.seed) for n in (a.layers, 1))
    tokens, passes = decode(target, prompts, a.drafts, a.tokens,
                            lambda last, out: drafts_of(draft, last, a.drafts)[0], [draft], a.temperature)
    for r in range(a.requests):
        print(f"request {r} ({len(prompts[r])} tokens): {tokens[r][:8]}...")
    print(f"{a.tokens} tokens of each request in {passes} passes")
    if a.check:
        target = Model(a.dim, a.layers, a.vocab, a.requests, seed=a.seed)
        alone, _ = decode(target, prompts, a.drafts, a.tokens,
                          lambda last, out: torch.full((a.requests, a.drafts), -1, dtype=torch.int32, device="cuda"),
                          temperature=a.temperature)
        differ = sum(x != y for t, u in zip(tokens, alone) for x, y in zip(t, u))
        print(f"tokens that differ from those without drafts: {differ}")
        return differ
    return 0


if __name__ == "__main__":
    main()
