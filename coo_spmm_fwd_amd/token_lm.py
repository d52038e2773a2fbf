"""A small next-token model trained with the library's operators: embedding, two truly sparse layers,
cross entropy over the vocabulary, clipping, and a restructure of the sparse layers now and then.  GELU,
the residual sum and Adam are torch's.

    python -m coo_spmm_fwd_amd.token_lm [--steps 200] [--vocab 2000] [--width 256]

The text is synthetic (each token mostly decides the next), so the loss has to fall from about
log(vocab) towards the entropy of that rule.
"""
from __future__ import annotations

import argparse
import math

import torch

from .sparse_linear import SparseLinear
from .token_ops import clip_grad_norm, embedding, linear_cross_entropy


class TokenModel(torch.nn.Module):
    """logits = head (x + down gelu(up x)), x = sqrt(width) E[id]; `up` and `down` keep a share of
    `density` of their weights."""

    def __init__(self, vocab: int, width: int, density: float = 0.1, seed: int = 0):
        super().__init__()
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.scale = math.sqrt(width)
        self.embed = torch.nn.Parameter(rand(vocab, width) / width)
        self.head = torch.nn.Parameter(rand(vocab, width) / width)
        self.up, self.down = self._sparse(4 * width, width, density, g), self._sparse(width, 4 * width, density, g)

    @staticmethod
    def _sparse(out, in_, density, g):
        nnz = max(1, round(density * out * in_))
        at = torch.randperm(out * in_, generator=g, device="cuda")[:nnz]
        vals = torch.randn(nnz, generator=g, device="cuda") / math.sqrt(density * in_)
        return SparseLinear((at // in_).int(), (at % in_).int(), vals, out, in_)

    def forward(self, ids, targets):
        x = embedding(ids, self.embed, self.scale)
        h = x + self.down(torch.nn.functional.gelu(self.up(x)))
        return linear_cross_entropy(h, self.head, targets)


def text(n: int, vocab: int, seed: int):
    """n tokens of a chain: the next token is a fixed function of the last, or (one in ten) any."""
    g = torch.Generator().manual_seed(1)
    rule = torch.randperm(vocab, generator=g)
    g = torch.Generator().manual_seed(seed)
    jump, any_ = torch.rand(n, generator=g) < 0.1, torch.randint(0, vocab, (n,), generator=g)
    out = [int(any_[0])]
    for i in range(1, n):
        out.append(int(any_[i]) if jump[i] else int(rule[out[-1]]))
    return torch.tensor(out)


def train(steps: int = 200, vocab: int = 2000, width: int = 256, tokens: int = 512, lr: float = 0.02,
          restructure_every: int = 50, log=print):
    """The losses of `steps` steps (read back at the end; each line of the log reads one)."""
    model = TokenModel(vocab, width)
    params = list(model.parameters())
    opt = torch.optim.Adam(params, lr=lr)
    data = text(tokens * 16 + 1, vocab, seed=2).cuda()
    losses = []
    for step in range(steps):
        at = step % 16 * tokens
        ids, targets = data[at:at + tokens], data[at + 1:at + tokens + 1].clone()
        targets[::64] = -100  # tokens that are not learnt from
        loss = model(ids, targets)
        opt.zero_grad()
        loss.backward()
        clip_grad_norm(params, 1.0)
        opt.step()
        losses.append(loss.detach())
        if restructure_every and (step + 1) % restructure_every == 0:
            for k, layer in enumerate((model.up, model.down)):
                layer.restructure(layer.nnz // 20, seed=k, step=step)
                opt.state.pop(layer.values, None)  # the entries changed: so did what their moments were of
        if log and (step + 1) % 50 == 0:
            log(f"step {step + 1}: loss {float(loss.detach()):.4f}")
    return torch.stack(losses).tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--vocab", type=int, default=2000)
    ap.add_argument("--width", type=int, default=256)
    a = ap.parse_args()
    losses = train(a.steps, a.vocab, a.width)
    print(f"loss {losses[0]:.4f} (log vocab {math.log(a.vocab):.4f}) -> {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
